"""Tensors that are not one contiguous piece are refused where only an address is handed on (no GPU needed)."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp


def shape():
    return sp.make_shape(1, 2, 4, 16, 16, 64, 4, 4, 4, sp.BF16)


def qkv(s):
    return torch.zeros(s.B, s.N, 3, s.H, s.d, dtype=torch.bfloat16)


@pytest.mark.parametrize("call", [sp.reorder, sp.reorder_pool, sp.pool_means])
def test_reorders_refuse_slices(call):
    s = shape()
    for bad in (qkv(s)[:, :, 2], torch.zeros(s.B, s.N, s.H, s.d), torch.zeros(s.B, s.N - 1, s.H, s.d).bfloat16(), None):
        with pytest.raises(ValueError, match="x: expected a contiguous"):
            call(s, bad)
    if call is not sp.pool_means:
        with pytest.raises(ValueError, match="out: expected a contiguous"):
            call(s, torch.zeros(s.B, s.N, s.H, s.d).bfloat16(), qkv(s)[:, :, 0])


def pipeline(**kw):
    """A Pipeline as far as its checks of arguments need it (no device memory)."""
    p = sp.Pipeline.__new__(sp.Pipeline)
    p.shape, p.norm, p.rope, p.raster_in = shape(), None, None, False
    for name, value in kw.items():
        setattr(p, name, value)
    return p


@pytest.mark.parametrize("raster_in", [False, True])
def test_pipeline_refuses_a_slice_for_v(raster_in):
    p = pipeline(raster_in=raster_in, norm=sp.QKNorm())
    q, k, v = qkv(p.shape).unbind(2)
    with pytest.raises(ValueError, match="v: expected a contiguous"):
        p.forward(q, k, v)
    with pytest.raises(ValueError, match="out: expected a contiguous"):
        p.forward(q, k, v.contiguous(), out=v)


@pytest.mark.parametrize("norm,rope,refused", [(None, None, ("dq", "dk", "dv")), (sp.QKNorm(), None, ("dv",)),
                                               (None, object(), ("dv",))])
def test_pipeline_refuses_slices_for_gradients(norm, rope, refused):
    p = pipeline(norm=norm, rope=rope)
    whole = torch.zeros(1, p.shape.N, 2, 64, dtype=torch.bfloat16)
    piece = qkv(p.shape)[:, :, 0]
    with pytest.raises(ValueError, match="dout: expected a contiguous"):
        p.backward(piece)
    for i, name in enumerate(("dq", "dk", "dv")):
        if name in refused:
            outs = [whole] * 3
            outs[i] = piece
            with pytest.raises(ValueError, match=f"{name}: expected a contiguous"):
                p.backward(whole, outs=outs)
