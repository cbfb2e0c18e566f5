"""Pipeline with norm and rotation in one pass: the same bits as the public calls in a row, in every
way of running it, and the kernel counts it states."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_launches import kernels
from tests.test_gpu_layer import SHAPES, setting

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def one_pass(norm):
    return sp.QKNorm(norm.q_weight, norm.k_weight, norm.q_bias, norm.k_bias, norm.eps, norm.rms, True, True)


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("rms,flags", [(False, 0), (True, 0), (True, sp.KERNEL_PORTABLE)])
def test_is_the_calls_in_a_row(dims, rms, flags):
    s, q, k, v, do, norm, tab, m, _ = setting(dims, rms, True, 0.0)
    raster_out = flags == 0
    pipe = sp.Pipeline(s, "mean", 0.6, 2, 2, backward=True, norm=one_pass(norm), rope=tab, flags=flags)
    o, lse = pipe.forward(q, k, v)
    dq, dk, dv = pipe.backward(do)
    assert int(pipe.status) == 0
    means = [torch.empty(s.B, s.H, s.nb, s.d, device="cuda") for _ in range(2)]
    qb, kb = sp.norm_rope_fwd(s, tab, q, k, norm.q_weight, norm.k_weight, norm.q_bias, norm.k_bias, norm.eps, rms,
                              q_means=means[0], k_means=means[1])
    vb = sp.reorder(s, v)
    rp, ci = sp.select(s, sp.block_scores_pooled(s, *means), 0.6, 2)
    aflags = flags | (sp.OUT_RASTER if raster_out else 0)
    o2, lse2 = sp.attn_fwd(s, qb, kb, vb, rp, ci, flags=aflags)
    g = sp.attn_bwd(s, qb, kb, vb, o2, lse2, sp.reorder(s, do), rp, ci, flags=aflags)
    want = sp.norm_rope_bwd(s, tab, g[0], g[1], q, k, norm.q_weight, norm.k_weight, norm.eps, rms,
                            in_blocked=not raster_out)
    if not raster_out:
        o2, g = sp.reorder(s, o2, inverse=True), (None, None, sp.reorder(s, g[2], inverse=True))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1]) and torch.equal(dv, g[2])
    for i, name in enumerate("qk"):
        assert torch.equal(pipe.norm_grads[name + "_weight"], want[2][i])
        assert rms or torch.equal(pipe.norm_grads[name + "_bias"], want[3][i])
    graph = pipe.capture(q, k, v, dout=do)
    for _ in range(2):
        outs = graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, (o2, lse2, dq, dk, dv)))


@pytest.mark.parametrize("kw", [{}, dict(mask=True, cap=9.0), dict(raster_inputs=True), dict(flags=sp.KERNEL_PORTABLE),
                                dict(fused_estimation=False)])
def test_counts_and_ways(kw):
    s, q, k, v, do, norm, tab, m, _ = setting(SHAPES[0], True, True, 0.0)
    kw = dict(kw)
    if kw.pop("mask", False):
        kw["mask"] = sp.mask_plan(s, *m)
    back = not kw.get("raster_inputs")
    pipe = sp.Pipeline(s, "mean", 0.9, 2, 2, backward=back, norm=one_pass(norm), rope=tab, overlap_demand=False, **kw)
    assert kernels(lambda: pipe.forward(q, k, v)) == pipe.kernels_per_forward()
    o, lse = pipe.forward(q, k, v)
    assert torch.isfinite(o.float()).all() and float(o.float().abs().max()) > 0
    if back:
        assert kernels(lambda: pipe.backward(do)) == pipe.kernels_per_backward()
        assert all(torch.isfinite(x.float()).all() for x in pipe.backward(do))
    assert int(pipe.status) == 0


def test_refuses():
    s, q, k, v, do, norm, tab, m, _ = setting(SHAPES[0], True, True, 0.0)
    with pytest.raises(ValueError):
        sp.Pipeline(s, "mean", 0.9, 2, 2, norm=one_pass(norm))                       # no rotation
    token = sp.QKNorm(rms=True, one_pass=True)
    with pytest.raises(ValueError):
        sp.Pipeline(s, "mean", 0.9, 2, 2, norm=token, rope=tab)                      # a norm per token
