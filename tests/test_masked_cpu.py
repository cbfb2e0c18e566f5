"""Refusals of token masks and masked, capped attention: every call here fails on the
host before anything is launched (no GPU needed)."""
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


def test_plan(lib):
    s = shape()
    n = lib.sparsp_mask_plan_size(ctypes.byref(s))
    assert n >= 3 * 4 * s.N + 3 * 8 * s.nb
    assert lib.sparsp_mask_plan_size(ctypes.byref(shape(T=5))) == 0

    def call(pos=FAKE, lo=FAKE, hi=FAKE, plan=FAKE + GAP, nbytes=n, sh=s):
        return lib.sparsp_mask_plan(ctypes.byref(sh), pos, lo, hi, plan, nbytes, None)
    for name in ("pos", "lo", "hi", "plan"):
        assert call(**{name: None}) == sp.INVALID_ARG
        assert call(**{name: FAKE + 4}) == sp.ALIGN
    assert call(nbytes=n - 1) == sp.WORKSPACE
    assert call(sh=shape(d=96)) == sp.UNSUPPORTED
    assert lib.sparsp_mask_scores(ctypes.byref(s), None, FAKE, None) == sp.INVALID_ARG
    assert lib.sparsp_mask_scores(ctypes.byref(s), FAKE, FAKE + 8, None) == sp.ALIGN


BIG = 1 << 40


def fwd(lib, s=None, scale=0.0, cap=0.0, plan=None, ws=FAKE, ws_bytes=BIG, flags=0, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, row_ptr=FAKE, col_idx=FAKE, o=FAKE, lse=FAKE, status=None)
    a.update(kw)
    return lib.sparsp_attn_masked_fwd(ctypes.byref(s or shape()), a["q"], a["k"], a["v"], a["row_ptr"], a["col_idx"],
                                      scale, cap, plan, a["o"], a["lse"], ws, ws_bytes, flags, None, a["status"], None)


def bwd(lib, s=None, scale=0.0, cap=0.0, plan=None, ws=FAKE, ws_bytes=BIG, flags=0, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, row_ptr=FAKE, col_idx=FAKE, o=FAKE, lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE)
    a.update(kw)
    return lib.sparsp_attn_masked_bwd(ctypes.byref(s or shape()), a["q"], a["k"], a["v"], a["o"], a["lse"], a["dout"],
                                      a["row_ptr"], a["col_idx"], scale, cap, plan, a["dq"], a["dk"], a["dv"], ws,
                                      ws_bytes, flags, None, None, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(cap=-1.0), sp.INVALID_ARG), (dict(cap=float("nan")), sp.INVALID_ARG), (dict(cap=float("inf")), sp.INVALID_ARG),
    (dict(cap=2.0 ** -21), sp.INVALID_ARG), (dict(cap=2.0 ** 21), sp.INVALID_ARG),
    (dict(cap=1e6, scale=1e-38), sp.INVALID_ARG),                 # scale / cap underflows
    (dict(scale=float("nan")), sp.INVALID_ARG), (dict(scale=float("inf")), sp.INVALID_ARG),
    (dict(flags=1 << 9), sp.INVALID_ARG),
    (dict(q=None), sp.INVALID_ARG), (dict(k=FAKE + 8), sp.ALIGN), (dict(lse=None), sp.INVALID_ARG),
    (dict(plan=FAKE + 4), sp.ALIGN), (dict(ws=None), sp.INVALID_ARG), (dict(ws_bytes=1024), sp.WORKSPACE),
    (dict(flags=sp.KERNEL_PORTABLE), sp.UNSUPPORTED),
    (dict(flags=sp.KERNEL_PORTABLE, cap=3.0), sp.UNSUPPORTED),
    (dict(s=shape(dtype=sp.F32)), sp.UNSUPPORTED),
    (dict(s=shape(T=5)), sp.SHAPE), (dict(s=shape(d=32)), sp.UNSUPPORTED),
])
def test_attention_refuses(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_backward_reads_block_order(lib):
    assert bwd(lib, flags=sp.IN_RASTER) == sp.UNSUPPORTED


def test_workspace_covers_the_masked_csr(lib):
    s = shape()
    for backward in (0, 1):
        plain = lib.sparsp_attn_workspace_size(ctypes.byref(s), backward)
        masked = lib.sparsp_attn_masked_workspace_size(ctypes.byref(s), backward)
        assert masked >= plain + 4 * s.rows * s.nb
        call = bwd if backward else fwd
        assert call(lib, ws_bytes=masked - 1) == sp.WORKSPACE
    assert lib.sparsp_attn_masked_workspace_size(ctypes.byref(shape(B=0)), 0) == 0


def test_binding_refuses_another_shapes_plan():
    torch = pytest.importorskip("torch")
    s, other = shape(), shape(T=8)
    plan = sp.MaskPlan(sp._mask_dims(s), torch.zeros(16, dtype=torch.uint8))
    assert sp._plan_ptr(shape(H=7, d=128), plan) == plan.plan.data_ptr()   # any heads and head size
    with pytest.raises(ValueError):
        sp._plan_ptr(other, plan)
    assert sp._plan_ptr(s, None) is None


def test_the_binding_refuses_other_devices_and_types(lib):
    """Every tensor of the calls is checked before the library sees it: a table, a plan, indices, a workspace or a
    status word on another device than the current one."""
    import torch
    cpu = {"device": "cpu"}
    with pytest.raises(ValueError, match="ws"):
        sp._space(torch.empty(64, dtype=torch.uint8), 0)
    with pytest.raises(ValueError, match="col_idx"):
        sp._buffer("col_idx", torch.empty(4, dtype=torch.int64, **cpu), torch.int32, -1)
    with pytest.raises(ValueError, match="col_idx"):
        sp._buffer("col_idx", torch.empty(4, dtype=torch.int32, **cpu), torch.int32, 0)
    with pytest.raises(ValueError, match="col_idx"):
        sp._buffer("col_idx", torch.empty(4, 4, dtype=torch.int32, **cpu).t()[:2], torch.int32, -1)
    with pytest.raises(ValueError, match="col_idx"):
        sp._buffer("col_idx", None, torch.int32, 0)
    assert sp._buffer("status", None, torch.int32, 0, True) is None
    assert sp._buffer("status", FAKE, torch.int32, 0, True) == FAKE
    with pytest.raises(ValueError, match="expected"):
        sp._want("w", "text", (4,), torch.float32, 0)
