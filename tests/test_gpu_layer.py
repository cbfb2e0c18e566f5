"""Token norm, rotary positions, masked selection and masked, capped attention run
together by Pipeline, as a layer of a video DiT uses them: the same bits as the public
calls in a row, and the values and gradients of the float64 formulas."""
import math

import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_masked import csr, gen, masks, to_blocked, to_raster   # noqa: F401
from tests.test_gpu_norm_rope import angles, grid_pos, turn

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

SHAPES = [(1, 2, 6, 16, 24, 128, 2, 8, 8), (2, 3, 4, 16, 12, 64, 4, 4, 4)]
COLS = {64: (24, 20, 20), 128: (44, 42, 42)}


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def setting(dims, rms, per_head, cap, seed=21):
    s = sp.make_shape(*dims, "bf16")
    g = gen(seed)
    x = [torch.randn(s.B, s.N, 3, s.H, s.d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    q, k, v = x[0].unbind(2)
    v = v.contiguous()
    do = x[1][:, :, 0].contiguous()
    cols = s.d if per_head else s.H * s.d
    rand = lambda scale, base: base + scale * torch.randn(cols, generator=g, device="cuda")
    norm = sp.QKNorm(rand(0.2, 1.0), rand(0.2, 1.0), None if rms else rand(0.1, 0.0), None if rms else rand(0.1, 0.0),
                     rms=rms, per_head=per_head)
    tab = sp.rope_table(s, COLS[s.d], 100.0)
    plan_in = masks(s, "docs", g)
    return s, q, k, v, do, norm, tab, plan_in, cap


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("rms,per_head,cap", [(False, False, 0.0), (True, True, 15.0)])
def test_pipeline_is_the_calls_in_a_row(dims, rms, per_head, cap):
    s, q, k, v, do, norm, tab, m, cap = setting(dims, rms, per_head, cap)
    plan = sp.mask_plan(s, *m)
    pipe = sp.Pipeline(s, "mean", 0.6, 2, 2, backward=True, norm=norm, rope=tab, mask=plan, cap=cap)
    o, lse = pipe.forward(q, k, v)
    dq, dk, dv = pipe.backward(do)
    assert int(pipe.status) == 0
    means = [torch.empty(s.B, s.H, s.nb, s.d, device="cuda") for _ in range(2)]
    stats, blocked = [], []
    for x, w, b, mean in ((q, norm.q_weight, norm.q_bias, means[0]), (k, norm.k_weight, norm.k_bias, means[1])):
        y, mu, rs = sp.norm_fwd(s, x, w, b, norm.eps, rms, per_head)
        stats.append((mu, rs))
        blocked.append(sp.rope(s, tab, y, means=mean))
    vb = sp.reorder(s, v)
    scores = sp.mask_scores(s, plan, sp.block_scores_pooled(s, *means))
    rp, ci = sp.select(s, scores, 0.6, 2)
    o2, lse2 = sp.attn_masked_fwd(s, *blocked, vb, rp, ci, cap=cap, mask=plan, flags=sp.OUT_RASTER)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = sp.attn_masked_bwd(s, *blocked, vb, o2, lse2, sp.reorder(s, do), rp, ci, cap=cap, mask=plan,
                           flags=sp.OUT_RASTER)
    assert torch.equal(dv, g[2])
    for x, gx, w, (mu, rs), got, name in ((q, g[0], norm.q_weight, stats[0], dq, "q"),
                                          (k, g[1], norm.k_weight, stats[1], dk, "k")):
        up = sp.rope(s, tab, gx, inverse=True, out_blocked=False)
        dx, dw, db = sp.norm_bwd(s, up, x, w, mu, rs, rms, per_head)
        assert torch.equal(dx, got) and torch.equal(dw, pipe.norm_grads[name + "_weight"])
        assert rms or torch.equal(db, pipe.norm_grads[name + "_bias"])
    # and as one CUDA graph, on a second set of values
    graph = pipe.capture(q, k, v, dout=do)
    for _ in range(2):
        outs = graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, (o2, lse2, dq, dk, dv)))


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("rms,per_head,cap", [(False, True, 10.0), (True, False, 0.0)])
def test_layer_values_and_gradients(dims, rms, per_head, cap):
    """Against float64 autograd over the pairs that the layer selected. Between the inputs and a result lie at most
    eight roundings to bf16 (norm, rotation, P or dS, O, the gradients of attention, rotation and norm, and the
    result), each at most 2^-8 of the values it rounds: 8 2^-8 of the result's 2-norm bounds the error."""
    s, q, k, v, do, norm, tab, m, cap = setting(dims, rms, per_head, cap, 22)
    plan = sp.mask_plan(s, *m)
    pipe = sp.Pipeline(s, "mean", 0.7, 2, 2, backward=True, norm=norm, rope=tab, mask=plan, cap=cap)
    o, lse = pipe.forward(q, k, v)
    grads = pipe.backward(do)
    leaves = [t.double().requires_grad_() for t in (q, k, v, norm.q_weight, norm.k_weight)]
    phi = angles(s, COLS[s.d], 100.0, (0,) * 3, (1,) * 3, grid_pos(s))
    turned = []
    for x, w, b in zip(leaves[:2], leaves[3:], (norm.q_bias, norm.k_bias)):
        rows = x if per_head else x.flatten(2)
        c = rows if rms else rows - rows.mean(-1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + norm.eps) * w
        y = y if b is None else y + b.double()
        turned.append(to_blocked(s, turn_grad(y.view(x.shape), phi)).transpose(1, 2))
    vb = to_blocked(s, leaves[2]).transpose(1, 2)
    rp, ci = (t.long() for t in pipe.csr)
    chosen = torch.zeros(s.rows, s.nb, dtype=torch.bool, device="cuda")
    chosen[torch.repeat_interleave(torch.arange(s.rows, device="cuda"), rp[1:] - rp[:-1]), ci[: int(rp[-1])]] = True
    pos, lo, hi = (to_blocked(s, t).long() for t in m)
    see = (lo[:, :, None] <= pos[:, None]) & (pos[:, None] < hi[:, :, None])
    pick = chosen.view(s.B, s.H, s.nb, s.nb).repeat_interleave(s.Bt, 2).repeat_interleave(s.Bt, 3) & see[:, None]
    t = turned[0] @ turned[1].transpose(-1, -2) / math.sqrt(s.d)
    t = cap * torch.tanh(t / cap) if cap > 0 else t
    dead = ~pick.any(-1, keepdim=True)
    p = torch.softmax(t.masked_fill(~pick, -1e300), -1).masked_fill(~pick | dead, 0.0)
    out = to_raster(s, p @ vb)
    (out * do.double()).sum().backward()
    pairs = [("O", o, out), ("dV", grads[2], leaves[2].grad), ("dQ", grads[0], leaves[0].grad),
             ("dK", grads[1], leaves[1].grad), ("dWq", pipe.norm_grads["q_weight"], leaves[3].grad),
             ("dWk", pipe.norm_grads["k_weight"], leaves[4].grad)]
    for name, got, ref in pairs:
        err = float((got.double() - ref.detach()).norm() / ref.detach().norm())
        assert err <= 8 * 2.0 ** -8, (name, err)


def turn_grad(x, phi):
    """The rotation of adjacent pairs in float64, differentiable."""
    c, sn = phi.cos()[:, :, None], phi.sin()[:, :, None]
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)


@pytest.mark.parametrize("norm_on,rope_on,raster", [(True, False, True), (False, True, True), (True, True, True),
                                                   (True, False, False), (False, True, False)])
def test_partial_layers(norm_on, rope_on, raster):
    """Norm or rotation alone, and the forward without a reorder pass: the values of the reordered form."""
    s, q, k, v, do, norm, tab, m, _ = setting(SHAPES[0], False, False, 0.0, 23)
    q, k = q.contiguous(), k.contiguous()
    kw = dict(norm=norm if norm_on else None, rope=tab if rope_on else None, mask=sp.mask_plan(s, *m))
    want = sp.Pipeline(s, "mean", 0.6, 2, 2, **kw).forward(q, k, v)
    got = sp.Pipeline(s, "mean", 0.6, 2, 2, raster_inputs=raster, fused_estimation=True, **kw).forward(q, k, v)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if not raster:
        back = sp.Pipeline(s, "mean", 0.6, 2, 2, backward=True, **kw)
        back.forward(q, k, v)
        one = [t.clone() for t in back.backward(do)]
        assert all(torch.isfinite(t).all() for t in one)


def test_portable_and_fp32_shapes():
    """Norm and rotation also serve the kernels that write block order; mask and cap are refused there."""
    s, q, k, v, do, norm, tab, m, _ = setting(SHAPES[0], False, False, 0.0, 24)
    kw = dict(norm=norm, rope=tab, backward=True)
    fast, slow = sp.Pipeline(s, "mean", 0.6, 2, 2, **kw), sp.Pipeline(s, "mean", 0.6, 2, 2, flags=sp.KERNEL_PORTABLE, **kw)
    outs = []
    for pipe in (fast, slow):
        o, _ = pipe.forward(q, k, v)
        outs.append([t.clone() for t in (o, *pipe.backward(do), pipe.norm_grads["q_weight"])])
    for a, b in zip(*outs):   # two bf16 kernels of one formula: six roundings apart each
        assert float((a.double() - b.double()).norm() / b.double().norm()) <= 12 * 2.0 ** -8
    plan = sp.mask_plan(s, *m)
    for bad in (dict(mask=plan), dict(cap=5.0)):
        with pytest.raises(ValueError):
            sp.Pipeline(s, "mean", 0.6, 2, 2, flags=sp.KERNEL_PORTABLE, **bad)
    f = sp.make_shape(1, 2, 4, 16, 16, 64, 4, 4, 4, "f32")
    x = [torch.randn(1, f.N, 2, 64, generator=gen(25), device="cuda") for _ in range(3)]
    o, lse = sp.Pipeline(f, "mean", 0.6, 2, 2, norm=sp.QKNorm(rms=True), rope=sp.rope_table(f, (24, 20, 20))).forward(*x)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


def test_host_pipeline_with_a_norm():
    """The host pipeline keeps a training step's q and k until the norm's backward has read them."""
    s, q, k, v, do, norm, tab, m, _ = setting(SHAPES[0], True, False, 0.0, 26)
    pipe = sp.Pipeline(s, "mean", 0.6, 2, 2, backward=True, norm=norm, rope=tab, mask=sp.mask_plan(s, *m))
    host = sp.HostPipeline(pipe)
    steps = []
    for i in range(4):
        ins = [(t.contiguous() * (1 + 0.25 * i)).cpu().pin_memory() for t in (q, k, v, do)]
        outs = [torch.empty_like(ins[0]).pin_memory() for _ in range(4)]
        steps.append((ins, outs))
    for ins, outs in steps:
        host.train_step(*ins, *outs)
    host.synchronize()
    torch.cuda.synchronize()
    for ins, outs in steps:
        dev = [t.cuda() for t in ins]
        want = [t.clone() for t in (pipe.forward(*dev[:3])[0], *pipe.backward(dev[3]))]
        assert all(torch.equal(a.cuda(), b) for a, b in zip(outs, want))


def test_mask_builders():
    s = sp.make_shape(2, 1, 4, 8, 8, 64, 1, 8, 8, "bf16")
    ids = torch.arange(s.N, device="cuda").expand(2, s.N).clone() // 100 - 1
    pos, lo, hi = sp.document_mask(s, ids.int())
    see = (lo[:, :, None] <= pos[:, None]) & (pos[:, None] < hi[:, :, None])
    want = (ids[:, :, None] == ids[:, None]) & (ids >= 0)[:, :, None]
    assert torch.equal(see, want)
    t = torch.arange(s.N, device="cuda") // 64
    for prefix, window in ((0, None), (2, None), (9, None), (0, 2)):
        pos, lo, hi = sp.frame_mask(s, prefix, window)
        see = (lo[0, :, None] <= pos[0, None]) & (pos[0, None] < hi[0, :, None])
        want = (t[None] <= t[:, None]) | (t[None] < prefix)
        if window:
            want &= t[None] > t[:, None] - window
        assert torch.equal(see, want)
    with pytest.raises(ValueError):
        sp.frame_mask(s, 1, 2)
