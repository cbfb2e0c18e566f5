"""Refusals of the cache in 8 bits: every call here fails on the host before anything is
launched (no GPU needed)."""
import ctypes

import pytest

import block_sparse_attention_token_gb300 as sp

FAKE = 1 << 20   # aligned, never-dereferenced addresses, far apart
GAP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_token_gb300 import build
    build.build()
    return sp.lib()


def cache(**kw):
    args = dict(blocks=10, heads=2, d=64, bt=64)
    args.update(kw)
    return sp.CacheShape(**args)


def at(i):
    return FAKE + i * GAP


BAD_CACHES = [
    (dict(cache=None), sp.INVALID_ARG), (dict(cache=cache(blocks=0)), sp.SHAPE), (dict(cache=cache(heads=-1)), sp.SHAPE),
    (dict(cache=cache(d=96)), sp.UNSUPPORTED), (dict(cache=cache(bt=32)), sp.UNSUPPORTED),
    (dict(cache=cache(heads=65536)), sp.UNSUPPORTED), (dict(cache=cache(blocks=1 << 25)), sp.UNSUPPORTED),
    (dict(status=FAKE + 4), sp.ALIGN),
]


def extend(lib, cache=cache(), B=3, max_blocks=4, ln=at(0), add=at(1), free=at(2), n_free=5, used=None, table=at(3),
           len_out=at(4), start=at(5), slots=at(6), tokens=9, used_out=None, status=None):
    return lib.sparsp_cache_extend(None if cache is None else ctypes.byref(cache), B, max_blocks, ln, add, free, n_free, used,
                                   table, len_out, start, slots, tokens, used_out, status, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(B=0), sp.SHAPE), (dict(B=16385), sp.UNSUPPORTED), (dict(max_blocks=0), sp.SHAPE),
    (dict(max_blocks=1 << 25), sp.UNSUPPORTED), (dict(tokens=-1), sp.SHAPE), (dict(tokens=1 << 31), sp.UNSUPPORTED),
    (dict(n_free=-1), sp.SHAPE), (dict(ln=None), sp.INVALID_ARG), (dict(add=None), sp.INVALID_ARG),
    (dict(free=None), sp.INVALID_ARG), (dict(free=FAKE + 2), sp.ALIGN), (dict(table=None), sp.INVALID_ARG), (dict(len_out=None), sp.INVALID_ARG),
    (dict(start=None), sp.INVALID_ARG), (dict(slots=None), sp.INVALID_ARG), (dict(slots=FAKE + 4), sp.ALIGN),
    (dict(used=FAKE + 4), sp.ALIGN), (dict(used_out=FAKE + 8), sp.ALIGN), (dict(table=FAKE + 4), sp.ALIGN),
    (dict(len_out=at(1)), sp.INVALID_ARG), (dict(B=100, len_out=at(0) + 64), sp.INVALID_ARG), (dict(start=at(0)), sp.INVALID_ARG), (dict(start=at(4)), sp.INVALID_ARG),
    (dict(slots=at(3)), sp.INVALID_ARG), (dict(B=7, slots=at(5) + 16), sp.INVALID_ARG), (dict(used_out=at(1)), sp.INVALID_ARG),
    (dict(table=at(2)), sp.INVALID_ARG), (dict(used=at(7), used_out=at(7), len_out=at(7)), sp.INVALID_ARG),
    (dict(used=at(7), used_out=at(8), start=at(7)), sp.INVALID_ARG),
])
def test_extend_refuses(lib, kw, code):
    assert extend(lib, **kw) == code


def write(lib, cache=cache(), dtype=sp.BF16, k=at(0), ks=0, kh=0, v=at(1), vs=0, vh=0, slots=at(2), tokens=5, kc=at(3),
          ksc=at(4), vc=at(5), vsc=at(6), status=None):
    return lib.sparsp_cache_write(None if cache is None else ctypes.byref(cache), dtype, k, ks, kh, v, vs, vh, slots, tokens,
                                  kc, ksc, vc, vsc, status, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(dtype=5), sp.UNSUPPORTED), (dict(tokens=-1), sp.SHAPE), (dict(tokens=1 << 31), sp.UNSUPPORTED),
    (dict(k=None), sp.INVALID_ARG), (dict(v=None), sp.INVALID_ARG), (dict(slots=None), sp.INVALID_ARG),
    (dict(kc=None), sp.INVALID_ARG), (dict(ksc=None), sp.INVALID_ARG), (dict(vc=None), sp.INVALID_ARG),
    (dict(vsc=None), sp.INVALID_ARG), (dict(kc=FAKE + 8), sp.ALIGN), (dict(k=FAKE + 8), sp.ALIGN),
    (dict(ks=60), sp.SHAPE), (dict(ks=-128), sp.SHAPE), (dict(kh=63), sp.SHAPE), (dict(vh=1 << 41), sp.SHAPE),
    (dict(vs=132), sp.ALIGN), (dict(kh=68), sp.ALIGN), (dict(vc=at(3)), sp.INVALID_ARG), (dict(vsc=at(4)), sp.INVALID_ARG),
])
def test_write_refuses(lib, kw, code):
    assert write(lib, **kw) == code


def attn(lib, cache=cache(), B=3, H=4, q=at(0), qs=0, start=at(1), tokens=5, max_add=2, ln=at(2), table=at(3),
         max_blocks=4, kc=at(4), ksc=at(5), vc=at(6), vsc=at(7), row_ptr=None, col_idx=None, col_cap=0, scale=0.0,
         flags=0, o=at(8), lse=at(9), ws=at(10), ws_bytes=1 << 40, status=None):
    return lib.sparsp_attn_cache_fwd(None if cache is None else ctypes.byref(cache), B, H, q, qs, start, tokens, max_add,
                                     ln, table, max_blocks, kc, ksc, vc, vsc, row_ptr, col_idx, col_cap, scale, flags, o,
                                     lse, ws, ws_bytes, status, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + [
    (dict(B=0), sp.SHAPE), (dict(B=16385), sp.UNSUPPORTED), (dict(H=3), sp.SHAPE), (dict(H=0), sp.SHAPE),
    (dict(max_add=0), sp.SHAPE), (dict(max_add=1 << 30), sp.UNSUPPORTED), (dict(tokens=-1), sp.SHAPE),
    (dict(tokens=1 << 30), sp.UNSUPPORTED), (dict(max_blocks=0), sp.SHAPE),
    (dict(qs=128), sp.SHAPE), (dict(qs=260), sp.ALIGN), (dict(qs=-256), sp.SHAPE), (dict(q=None), sp.INVALID_ARG),
    (dict(o=None), sp.INVALID_ARG), (dict(lse=None), sp.INVALID_ARG), (dict(start=None), sp.INVALID_ARG),
    (dict(ln=None), sp.INVALID_ARG), (dict(table=None), sp.INVALID_ARG), (dict(kc=None), sp.INVALID_ARG),
    (dict(vsc=FAKE + 4), sp.ALIGN), (dict(row_ptr=at(11)), sp.INVALID_ARG), (dict(col_idx=at(11)), sp.INVALID_ARG),
    (dict(row_ptr=at(11) + 4, col_idx=at(12)), sp.ALIGN), (dict(row_ptr=at(11), col_idx=at(12), col_cap=-1), sp.INVALID_ARG),
    (dict(scale=float("nan")), sp.INVALID_ARG), (dict(scale=float("inf")), sp.INVALID_ARG), (dict(flags=2), sp.INVALID_ARG),
    (dict(ws=None), sp.INVALID_ARG), (dict(ws_bytes=100), sp.WORKSPACE), (dict(o=at(0)), sp.INVALID_ARG),
    (dict(o=at(0) + 512), sp.INVALID_ARG), (dict(qs=1024, o=at(0) + 8192), sp.INVALID_ARG),
    (dict(lse=at(0) + 256), sp.INVALID_ARG), (dict(o=at(5), lse=at(5) + 64), sp.INVALID_ARG),
    (dict(tokens=0, q=None, o=None, lse=None), sp.OK),     # nothing to do, nothing launched
])
def test_attn_refuses(lib, kw, code):
    assert attn(lib, **kw) == code


def test_workspace(lib):
    size = lambda c=cache(), B=3, H=4, tokens=5, max_add=2, mb=4: lib.sparsp_attn_cache_workspace_size(
        ctypes.byref(c), B, H, tokens, max_add, mb)
    n = size()
    assert n > 0 and size(c=cache(d=128)) > n and size(max_add=100) >= n
    assert size(H=3) == 0 and size(max_add=0) == 0 and size(c=cache(d=32)) == 0
    assert attn(lib, ws_bytes=n - 1) == sp.WORKSPACE
    assert n == size(B=1000, tokens=900, mb=1000)          # it does not grow with the lengths


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    pool = sp.block_pool(3, 2, 64, 64, device="cpu")
    assert pool.k.dtype is torch.float8_e4m3fn and tuple(pool.k.shape) == (3, 2, 64, 64)
    x, n = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: sp.cache_write(pool, x, x, n), lambda: sp.cache_extend(pool.shape, n, n, n, n.view(4, 1), 4),
                 lambda: sp.attn_cache_fwd(pool, x.bfloat16(), n, n, n.view(4, 1), 1)):
        with pytest.raises((ValueError, AssertionError, RuntimeError)):
            call()                                         # not on a CUDA device
