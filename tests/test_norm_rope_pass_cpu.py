"""Refusals of norm and rotation in one pass: every call here fails on the host before
anything is launched (no GPU needed)."""
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


def shape(**kw):
    args = dict(B=1, H=2, T=4, Y=16, X=16, d=64, ta=4, tb=4, tc=4, dtype=sp.BF16)
    args.update(kw)
    return sp.make_shape(**args)


def axes(cols=(24, 20, 20), extent=(4, 16, 16), half=0):
    return sp.RopeAxes((ctypes.c_int32 * 3)(*cols), (ctypes.c_int32 * 3)(*extent), half)


def part(n, heads=2, **kw):
    at = FAKE + 8 * n * GAP
    t = sp.NormRope(heads, at, 0, at + GAP, 0, None, None, at + 2 * GAP, 0, None, None, None)
    for name, v in kw.items():
        setattr(t, name, v)
    return t


def call(lib, name="fwd", s=None, flags=0, eps=1e-6, rope=None, table=FAKE - 4096, pos=None, q=None, k=None, no_q=False,
         ws=FAKE + 40 * GAP, ws_bytes=1 << 30, status=None):
    rope = rope or axes()
    q, args = q or part(0), []
    if name == "bwd":
        args = [ws, ws_bytes]
    return getattr(lib, "sparsp_norm_rope_" + name)(
        ctypes.byref(s or shape()), flags, eps, ctypes.byref(rope), table, pos, None if no_q else ctypes.byref(q),
        None if k is None else ctypes.byref(k), *args, status, None)


@pytest.mark.parametrize("name", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), sp.INVALID_ARG), (dict(no_q=True), sp.INVALID_ARG),
    (dict(eps=-1.0), sp.INVALID_ARG), (dict(eps=float("nan")), sp.INVALID_ARG), (dict(eps=float("inf")), sp.INVALID_ARG),
    (dict(rope=axes(cols=(24, 21, 19))), sp.SHAPE), (dict(rope=axes(cols=(30, 20, 20))), sp.SHAPE),
    (dict(rope=axes(cols=(20, 20, 20), half=1)), sp.SHAPE), (dict(rope=axes(extent=(3, 16, 16))), sp.SHAPE),
    (dict(table=None), sp.INVALID_ARG), (dict(pos=FAKE + 4), sp.ALIGN), (dict(status=FAKE + 4), sp.ALIGN),
    (dict(q=part(0, heads=3)), sp.SHAPE), (dict(k=part(1, heads=0)), sp.SHAPE), (dict(k=part(1, heads=-1)), sp.SHAPE),
    (dict(k=part(1, heads=70000)), sp.UNSUPPORTED),
    (dict(q=part(0, x=None)), sp.INVALID_ARG), (dict(q=part(0, out=None)), sp.INVALID_ARG),
    (dict(k=part(1, x=FAKE + 8)), sp.ALIGN), (dict(k=part(1, w=FAKE + 8)), sp.ALIGN),
    (dict(q=part(0, x_stride=64)), sp.SHAPE), (dict(q=part(0, x_stride=132)), sp.ALIGN),
    (dict(q=part(0, out_stride=-128)), sp.SHAPE), (dict(k=part(1, out_stride=1 << 61)), sp.SHAPE),
    (dict(q=part(0, x_stride=1 << 31)), sp.UNSUPPORTED),
    (dict(q=part(0, out=FAKE)), sp.INVALID_ARG),                                      # in place
    (dict(k=part(1, out=FAKE + 1024)), sp.INVALID_ARG),                               # k's result over q
    (dict(k=part(1, out=FAKE + 2 * GAP)), sp.INVALID_ARG),                            # both results in one place
    (dict(k=part(1, out=FAKE + 2 * GAP + 128, out_stride=512), q=part(0, out_stride=512)), sp.INVALID_ARG),
    (dict(k=part(1, out=FAKE + 2 * GAP + 256, out_stride=256), q=part(0, out_stride=512)), sp.INVALID_ARG),
    (dict(s=shape(d=96)), sp.UNSUPPORTED), (dict(s=shape(T=0)), sp.SHAPE), (dict(s=shape(dtype=7)), sp.UNSUPPORTED),
    (dict(s=shape(T=1 << 16, Y=1 << 14, X=16), rope=axes(cols=(0, 0, 0))), sp.UNSUPPORTED),   # 2^34 tokens
    (dict(s=shape(ta=3), flags=2), sp.SHAPE), (dict(s=shape(T=5), flags=2), sp.SHAPE),  # tile order wants tiles
])
def test_refuses(lib, name, kw, code):
    assert call(lib, name, **kw) == code


def test_backward_refuses(lib):
    assert call(lib, "bwd", q=part(0, dy=None)) == sp.INVALID_ARG
    assert call(lib, "bwd", q=part(0, dy=FAKE + GAP + 2)) == sp.ALIGN
    assert call(lib, "bwd", q=part(0, out=FAKE + GAP)) == sp.INVALID_ARG               # over the gradient read
    assert call(lib, "bwd", q=part(0, dw=FAKE + 4)) == sp.ALIGN
    dw = part(0, dw=FAKE + 60 * GAP)
    assert call(lib, "bwd", q=dw, ws=None) == sp.INVALID_ARG
    s = shape()
    n = lib.sparsp_norm_rope_workspace_size(ctypes.byref(s), 0)
    assert n > 0 and call(lib, "bwd", q=dw, ws_bytes=n - 1) == sp.WORKSPACE
    assert lib.sparsp_norm_rope_workspace_size(ctypes.byref(s), 2) > n
    assert lib.sparsp_norm_rope_workspace_size(ctypes.byref(s), -1) == 0
    assert lib.sparsp_norm_rope_workspace_size(ctypes.byref(shape(d=32)), 0) == 0


def test_forward_refuses_means(lib):
    assert call(lib, q=part(0, means=FAKE + 4)) == sp.ALIGN
    assert call(lib, s=shape(T=5), q=part(0, means=FAKE + 60 * GAP), rope=axes(extent=(5, 16, 16))) == sp.SHAPE


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    s = shape()
    x = torch.zeros(1, s.N, s.H, s.d, dtype=torch.bfloat16)
    table = sp.RopeTable(axes(), torch.zeros(64))
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        sp.norm_rope_fwd(s, table, x)                        # not on a CUDA device
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        sp.norm_rope_fwd(s, table, x[0])
