"""Pipeline with a part of a layer (norm or rotation alone, both, neither) in each of its ways through the step: the same
bits as the public calls in a row, forward and backward, the weights' gradients among them."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_layer import SHAPES, setting
from tests.test_gpu_masked import csr, gen, inputs, masks

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

PARTS = [(True, False), (False, True), (True, True), (False, False)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def before_attention(s, x, norm, w, b, tab):
    """(statistics, turned raster x, its tile order, its tile means) of Q or K by the public calls."""
    mu = rs = None
    if norm is not None:
        x, mu, rs = sp.norm_fwd(s, x, w, b, norm.eps, norm.rms, norm.per_head)
    means = torch.empty(s.B, s.H, s.nb, s.d, device="cuda")
    if tab is not None:
        return (mu, rs), sp.rope(s, tab, x, out_blocked=False), sp.rope(s, tab, x, means=means), means
    blocked, means = sp.reorder_pool(s, x.contiguous())
    return (mu, rs), x, blocked, means


def after_attention(s, g, blocked, x, norm, w, stat, tab):
    """(gradient, weight's, bias') of Q or K from attention's gradient g (tile order where `blocked`)."""
    if tab is not None:
        g = sp.rope(s, tab, g, inverse=True, in_blocked=blocked, out_blocked=False)
    elif blocked:
        g = sp.reorder(s, g, inverse=True)
    return (g, None, None) if norm is None else sp.norm_bwd(s, g, x, w, *stat, norm.rms, norm.per_head)


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("norm_on,rope_on", PARTS)
@pytest.mark.parametrize("way", ["fused", "not fused", "raster", "portable"])
@pytest.mark.parametrize("rms,per_head", [(False, False), (True, True)])
def test_parts_are_the_calls_in_a_row(dims, norm_on, rope_on, way, rms, per_head):
    s, q, k, v, do, norm, tab, m, _ = setting(dims, rms, per_head, 0.0, 61)
    norm, tab = norm if norm_on else None, tab if rope_on else None
    if norm is None and tab is None:
        q, k = q.contiguous(), k.contiguous()
    portable, raster = way == "portable", way == "raster"
    plan = None if portable else sp.mask_plan(s, *m)
    flags = sp.KERNEL_PORTABLE if portable else 0
    pipe = sp.Pipeline(s, "mean", 0.6, 2, 2, norm=norm, rope=tab, mask=plan, flags=flags, backward=not raster,
                       raster_inputs=raster, fused_estimation=way != "not fused")
    o, lse = pipe.forward(q, k, v)
    nq, nk = norm or sp.QKNorm(), norm or sp.QKNorm()
    sq, rq, bq, mq = before_attention(s, q, norm, nq.q_weight, nq.q_bias, tab)
    sk, rk, bk, mk = before_attention(s, k, norm, nk.k_weight, nk.k_bias, tab)
    vb = sp.reorder(s, v)
    if raster:
        mq, mk = sp.pool_means(s, rq) if tab is None else mq, sp.pool_means(s, rk) if tab is None else mk
    scores = sp.block_scores(s, bq, bk) if way == "not fused" else sp.block_scores_pooled(s, mq, mk)
    if plan is not None:
        scores = sp.mask_scores(s, plan, scores)
    rp, ci = sp.select(s, scores, 0.6, 2)
    if portable:
        ob, lse2 = sp.attn_fwd(s, bq, bk, vb, rp, ci, flags=flags)
        o2 = sp.reorder(s, ob, inverse=True)
    else:
        o2, lse2 = sp.attn_masked_fwd(s, bq, bk, vb, rp, ci, mask=plan, flags=sp.OUT_RASTER)
    assert int(pipe.status) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if raster:
        return
    dob = sp.reorder(s, do)
    if portable:
        g = sp.attn_bwd(s, bq, bk, vb, ob, lse2, dob, rp, ci, flags=flags)
        dv2 = sp.reorder(s, g[2], inverse=True)
    else:
        g = sp.attn_masked_bwd(s, bq, bk, vb, o2, lse2, dob, rp, ci, mask=plan, flags=sp.OUT_RASTER)
        dv2 = g[2]
    want = [after_attention(s, g[0], portable, q, norm, nq.q_weight, sq, tab),
            after_attention(s, g[1], portable, k, norm, nk.k_weight, sk, tab)]
    wide = torch.full((2, s.B, s.N, 2, s.H, s.d), 7.0, device="cuda").bfloat16()
    for outs in (None, (wide[0][:, :, 1], wide[1][:, :, 0], torch.empty_like(v))):   # and into slices of wider tensors
        if outs is not None and norm is None and tab is None:
            continue
        dq, dk, dv = pipe.backward(do, outs=outs)
        assert torch.equal(dv, dv2)
        for got, (dx, dw, db), name in ((dq, want[0], "q"), (dk, want[1], "k")):
            assert torch.equal(got, dx)
            if norm is not None:
                assert torch.equal(pipe.norm_grads[name + "_weight"], dw)
                assert rms or torch.equal(pipe.norm_grads[name + "_bias"], db)
    assert (wide[0][:, :, 0] == 7).all() and (wide[1][:, :, 1] == 7).all()


def test_backward_on_a_given_stream():
    """The stream argument of the backward calls: the gradients of the current stream."""
    s = sp.make_shape(1, 2, 6, 16, 24, 64, 2, 8, 8, "bf16")
    g = gen(62)
    q, k, v, do = inputs(s, g)
    rp, ci, _ = csr(s, 0.6, g)
    plan = sp.mask_plan(s, *masks(s, "docs", g))
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, mask=plan)
    x = torch.randn(s.B, s.N, s.H, s.d, generator=g, device="cuda").bfloat16()
    y, mu, rs = sp.norm_fwd(s, x)
    tab = sp.rope_table(s, (24, 20, 20))

    def calls(stream=None):
        return (*sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=12.0, mask=plan, stream=stream),
                *sp.norm_bwd(s, y, x, None, mu, rs, stream=stream),
                sp.rope(s, tab, x, inverse=True, out_blocked=False, stream=stream),
                *sp.mask_csr(s, plan, rp, ci, stream=stream)[:1])
    want = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
