"""Refusals of the token norm and the rotary positions: every call here fails on
the host before anything is launched (no GPU needed)."""
import ctypes

import pytest

import block_sparse_attention_token_gb300 as sp

FAKE = 1 << 20   # an aligned, never-dereferenced address
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


def fwd(lib, s, flags=0, x=FAKE, xs=0, w=None, b=None, eps=1e-6, y=FAKE + GAP, mean=None, rstd=None):
    return lib.sparsp_norm_fwd(ctypes.byref(s), flags, x, xs, w, b, eps, y, mean, rstd, None)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), sp.INVALID_ARG),
    (dict(x=None), sp.INVALID_ARG), (dict(y=None), sp.INVALID_ARG),
    (dict(x=FAKE + 8), sp.ALIGN), (dict(w=FAKE + 4), sp.ALIGN), (dict(rstd=FAKE + 2), sp.ALIGN),
    (dict(eps=-1.0), sp.INVALID_ARG), (dict(eps=float("nan")), sp.INVALID_ARG), (dict(eps=float("inf")), sp.INVALID_ARG),
    (dict(xs=127), sp.SHAPE), (dict(xs=-128), sp.SHAPE), (dict(xs=132), sp.ALIGN), (dict(xs=1 << 60), sp.SHAPE),
    (dict(y=FAKE), sp.INVALID_ARG), (dict(y=FAKE + 1024), sp.INVALID_ARG),
    (dict(xs=384, y=FAKE + 256), sp.INVALID_ARG),   # between the tokens of a wider tensor
])
def test_norm_forward_refuses(lib, kw, code):
    assert fwd(lib, shape(), **kw) == code


def test_norm_row_limit(lib):
    wide = shape(H=129, d=128)
    assert fwd(lib, wide) == sp.UNSUPPORTED
    assert lib.sparsp_norm_workspace_size(ctypes.byref(wide), 0) == 0
    assert lib.sparsp_norm_workspace_size(ctypes.byref(wide), sp.NORM_HEAD) > 0
    assert lib.sparsp_norm_workspace_size(ctypes.byref(shape(T=5)), 0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), sp.INVALID_ARG), (dict(mean=None), sp.INVALID_ARG), (dict(rstd=None), sp.INVALID_ARG),
    (dict(dx=None), sp.INVALID_ARG), (dict(ws=None), sp.INVALID_ARG), (dict(ws_bytes=64), sp.WORKSPACE),
    (dict(dx=FAKE), sp.INVALID_ARG), (dict(dx=FAKE + GAP), sp.INVALID_ARG),
    (dict(xs=64), sp.SHAPE), (dict(dxs=130), sp.ALIGN), (dict(flags=8), sp.INVALID_ARG),
])
def test_norm_backward_refuses(lib, kw, code):
    a = dict(flags=0, dy=FAKE, x=FAKE + GAP, xs=0, w=None, mean=FAKE + 2 * GAP, rstd=FAKE + 3 * GAP, dx=FAKE + 4 * GAP,
             dxs=0, dw=FAKE + 5 * GAP, db=None, ws=FAKE + 6 * GAP, ws_bytes=1 << 30)
    a.update(kw)
    assert lib.sparsp_norm_bwd(ctypes.byref(shape()), a["flags"], a["dy"], a["x"], a["xs"], a["w"], a["mean"],
                               a["rstd"], a["dx"], a["dxs"], a["dw"], a["db"], a["ws"], a["ws_bytes"], None) == code


def axes(cols=(24, 20, 20), extent=(4, 16, 16), half=0):
    return sp.RopeAxes((ctypes.c_int32 * 3)(*cols), (ctypes.c_int32 * 3)(*extent), half)


@pytest.mark.parametrize("kw,code", [
    (dict(cols=(24, 21, 19)), sp.SHAPE), (dict(cols=(-2, 20, 20)), sp.SHAPE), (dict(cols=(30, 20, 20)), sp.SHAPE),
    (dict(cols=(20, 20, 20), half=1), sp.SHAPE),          # halves pair the whole head
    (dict(extent=(3, 16, 16)), sp.SHAPE), (dict(extent=(0, 16, 16)), sp.SHAPE),
    (dict(inp=None), sp.INVALID_ARG), (dict(out=FAKE), sp.INVALID_ARG), (dict(table=None), sp.INVALID_ARG),
    (dict(pos=FAKE + 4), sp.ALIGN), (dict(means=FAKE + 4), sp.ALIGN), (dict(flags=8), sp.INVALID_ARG),
    (dict(in_stride=120), sp.SHAPE), (dict(out_stride=129), sp.ALIGN), (dict(out=FAKE + 16), sp.INVALID_ARG),
])
def test_rope_refuses(lib, kw, code):
    a = dict(cols=(24, 20, 20), extent=(4, 16, 16), half=0, table=FAKE + 2 * GAP, pos=None, inp=FAKE, in_stride=0,
             out=FAKE + GAP, out_stride=0, flags=0, means=None)
    a.update(kw)
    r = axes(a["cols"], a["extent"], a["half"])
    assert lib.sparsp_rope(ctypes.byref(shape()), ctypes.byref(r), a["table"], a["pos"], a["inp"], a["in_stride"],
                           a["out"], a["out_stride"], a["flags"], a["means"], None, None) == code


def test_rope_table_refuses(lib):
    d3 = ctypes.c_double * 3
    ok = axes()
    n = lib.sparsp_rope_table_size(ctypes.byref(ok))
    assert n == 8 * (4 * 12 + 16 * 10 + 16 * 10)
    assert lib.sparsp_rope_table_size(ctypes.byref(axes(cols=(3, 0, 0)))) == 0

    def call(theta=1e4, off=(0, 0, 0), scale=(1, 1, 1), table=FAKE, nbytes=n):
        return lib.sparsp_rope_table(ctypes.byref(ok), theta, ctypes.byref(d3(*off)), ctypes.byref(d3(*scale)), table,
                                     nbytes, None)
    assert call(nbytes=n - 1) == sp.WORKSPACE
    assert call(theta=0.0) == sp.INVALID_ARG and call(theta=float("nan")) == sp.INVALID_ARG
    assert call(off=(0, float("inf"), 0)) == sp.INVALID_ARG and call(scale=(float("nan"), 1, 1)) == sp.INVALID_ARG
    assert call(table=None) == sp.INVALID_ARG


def test_binding_checks_tensors():
    """The binding refuses wrong tensors before the library sees an address."""
    torch = pytest.importorskip("torch")
    s = shape()
    x = torch.zeros(1, s.N, s.H, s.d, dtype=torch.bfloat16)
    with pytest.raises((ValueError, AssertionError, RuntimeError)):
        sp.norm_fwd(s, x)                                   # not on a CUDA device
    with pytest.raises(ValueError):
        sp.rope_table(s, (24, 20, 22))
    with pytest.raises(ValueError):
        sp.rope_table(s, (20, 20, 20), half=True)
