"""Token masks and score caps in block-sparse attention, forward and backward,
against dense float64 attention of the same pairs.

Tolerances. A rounding to bf16 is off by at most 2^-8 relative. The kernels
round P (and dS) once to bf16 before the second product, and the result once:
  O  : 2^-8 sum p|v| + 2^-8 |O|                       dV: the same with P^T, |dO|
  dK : 2^-8 scale sum |dS||q| + 2^-8 |dK|             dQ: 2^-16 in place of the first 2^-8 (dS in two bf16 parts)
fp32 arithmetic adds an exponent error e_y = (d + 16) 2^-24 scale |q||k| (a dot
product of d terms; the scale, the subtraction of the maximum) + 2^-20 cap (the
cap from an exponential and a reciprocal, each good to 2 units in the last
place, or from a polynomial; the backward's is good to 2.3e-6 of 0.54 cap), which changes P by 2 e_y + 2^-20 relative (the sum's own error beside
it), and, in dP - D, (2 d + 16) 2^-24 (|dO||v| + |dO||O|), |.| the norms."""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_token_gb300 as sp

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

U16, U32 = 2.0 ** -8, 2.0 ** -24

# B, H, T, Y, X, d, ta, tb, tc: every kernel (64- and 128-token blocks, d = 64 and 128), one block, odd block counts
SHAPES = [
    (1, 2, 4, 16, 12, 64, 4, 4, 4),
    (2, 2, 3, 8, 24, 64, 1, 8, 8),
    (1, 2, 6, 16, 24, 64, 2, 8, 8),
    (1, 2, 5, 8, 24, 128, 1, 8, 8),
    (2, 3, 6, 8, 24, 128, 2, 8, 8),
    (1, 1, 8, 4, 4, 128, 8, 4, 4),
    (1, 1, 4, 4, 4, 64, 4, 4, 4),
]
I32 = torch.iinfo(torch.int32)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def to_blocked(s, x):
    """Raster [B, N, ...] -> tile order."""
    rest = x.shape[2:]
    v = x.reshape(s.B, s.T // s.ta, s.ta, s.Y // s.tb, s.tb, s.X // s.tc, s.tc, *rest)
    k = tuple(range(7, 7 + len(rest)))
    return v.permute(0, 1, 3, 5, 2, 4, 6, *k).reshape(s.B, s.N, *rest)


def to_raster(s, x):
    """[B, H, N, d] tile order -> raster [B, N, H, d]."""
    v = x.reshape(s.B, s.H, s.T // s.ta, s.Y // s.tb, s.X // s.tc, s.ta, s.tb, s.tc, s.d)
    return v.permute(0, 2, 5, 3, 6, 4, 7, 1, 8).reshape(s.B, s.N, s.H, s.d).contiguous()


def masks(s, kind, g):
    n = torch.arange(s.N, device="cuda").expand(s.B, s.N)
    frame = n // (s.Y * s.X)
    if kind == "docs":       # documents with borders inside blocks, padding at the end of the last batch element
        ids = (n * 3 + 5) // s.N
        pad = (n >= s.N - s.N // 7) & (torch.arange(s.B, device="cuda")[:, None] == s.B - 1)
        pos = torch.where(pad, -1, ids)
        lo, hi = torch.where(pad, 0, ids), torch.where(pad, 0, ids + 1)
    elif kind == "frames":   # causal in frames with a prefix of two
        pos, lo, hi = frame, torch.zeros_like(frame), torch.clamp(frame + 1, min=2)
    elif kind == "random":   # any intervals, some empty, some reversed, some of the whole range
        pos = torch.randint(-50, 50, (s.B, s.N), generator=g, device="cuda")
        lo = torch.randint(-60, 40, (s.B, s.N), generator=g, device="cuda")
        hi = lo + torch.randint(-10, 60, (s.B, s.N), generator=g, device="cuda")
        pos[:, ::17], pos[:, 3::29] = I32.max, I32.min
        lo[:, 5::11], hi[:, 5::11] = I32.min, I32.max
    elif kind == "nothing":
        pos, lo, hi = torch.zeros_like(n), torch.ones_like(n), torch.ones_like(n)
    else:                    # everything
        pos, lo, hi = frame, torch.full_like(n, I32.min), torch.full_like(n, I32.max)
    return tuple(t.int().contiguous() for t in (pos, lo, hi))


def csr(s, density, g, empty=True):
    chosen = torch.rand(s.B * s.H, s.nb, s.nb, generator=g, device="cuda") < density
    chosen[:, :, 0] |= ~chosen.any(-1)
    if empty and s.nb > 2:
        chosen[:, 1] = False      # a row without blocks
        chosen[:, 2] = True       # and one with all
    rp = torch.zeros(s.rows + 1, dtype=torch.int32, device="cuda")
    rp[1:] = chosen.view(-1, s.nb).sum(1).cumsum(0)
    ci = chosen.view(-1, s.nb).nonzero()[:, 1].int()
    return rp, torch.cat([ci, ci.new_zeros(4)]), chosen


def inputs(s, g, spread=1.0):
    q, k, v, do = (torch.randn(s.B, s.H, s.N, s.d, generator=g, device="cuda") for _ in range(4))
    return (q * spread).bfloat16(), (k * spread).bfloat16(), v.bfloat16(), do.bfloat16()


def reference(s, q, k, v, chosen, mask, scale, cap):
    """Scores, pairs that count, P, O and LSE in float64."""
    pos, lo, hi = (to_blocked(s, t).long() for t in mask)
    see = (lo[:, :, None] <= pos[:, None]) & (pos[:, None] < hi[:, :, None])
    pick = chosen.view(s.B, s.H, s.nb, s.nb).repeat_interleave(s.Bt, 2).repeat_interleave(s.Bt, 3) & see[:, None]
    t = scale * q.double() @ k.double().transpose(-1, -2)
    slope = torch.ones_like(t)
    if cap > 0:
        slope = 1 - torch.tanh(t / cap) ** 2
        t = cap * torch.tanh(t / cap)
    t = t.masked_fill(~pick, -math.inf)
    lse = torch.logsumexp(t, -1)
    p = torch.exp(t - lse[..., None]).masked_fill(~pick, 0.0)
    return t, pick, slope, p, p @ v.double(), lse


def exp_error(s, q, k, scale, cap):
    return ((s.d + 16) * U32 * scale * q.double().norm(dim=-1).amax() * k.double().norm(dim=-1).amax()
            + 2.0 ** -20 * cap)


def close(got, ref, tol, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of tol"


def check_forward(s, o, lse, ref, q, k, v, scale, cap):
    _, pick, _, p, O, L = ref
    rel = 2 * exp_error(s, q, k, scale, cap) + 2.0 ** -20
    mass = p @ v.double().abs()
    close(o, O, (U16 + rel) * mass * (1 + U16) + U16 * O.abs() + 1e-30, "O")
    dead = ~pick.any(-1)
    assert torch.isneginf(lse[dead]).all() and (o[dead] == 0).all()
    close(lse[~dead], L[~dead], rel + 4 * U32 * L[~dead].abs(), "LSE")


def check_backward(s, grads, ref, lse, o, do, q, k, v, scale, cap, plain=False):
    t, pick, slope, _, _, _ = ref
    dead = ~pick.any(-1, keepdim=True)
    p = torch.exp(t - lse.double()[..., None].masked_fill(dead, 0.0)).masked_fill(~pick, 0.0)
    d64 = do.double()
    delta = (d64 * o.double()).sum(-1, keepdim=True)
    dp = d64 @ v.double().transpose(-1, -2)
    ds = p * (dp - delta) * slope
    rel = 2 * exp_error(s, q, k, scale, cap) + 2.0 ** -20 * (1 + cap)
    norms = d64.norm(dim=-1, keepdim=True) * (v.double().norm(dim=-1).amax() + o.double().norm(dim=-1, keepdim=True))
    e_ds = rel * ds.abs() + p * (2 * s.d + 16) * U32 * norms + 2.0 ** -20 * p * (dp - delta).abs()
    two = e_ds + (U16 if plain else U16 ** 2) * ds.abs()   # plain: neither mask nor cap, dS in one part
    e_ds = e_ds + U16 * ds.abs()
    T = (lambda x: x.transpose(-1, -2))
    for name, got, ref_, tol in (
            ("dQ", grads[0], scale * ds @ k.double(), scale * two @ k.double().abs()),
            ("dK", grads[1], scale * T(ds) @ q.double(), scale * T(e_ds) @ q.double().abs()),
            ("dV", grads[2], T(p) @ d64, (U16 + rel) * T(p) @ d64.abs())):
        close(got, ref_, tol * (1 + U16) + U16 * ref_.abs() + 1e-30, name)


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("kind", ["docs", "frames", "random", "all", "nothing", None])
@pytest.mark.parametrize("cap", [0.0, 2.0, 40.0, 60.0])
def test_forward_and_backward(dims, kind, cap):
    s = sp.make_shape(*dims, "bf16")
    g = gen(11)
    q, k, v, do = inputs(s, g)
    rp, ci, chosen = csr(s, 0.6, g)
    mask = masks(s, kind or "all", g)
    plan = sp.mask_plan(s, *mask) if kind else None
    scale = 0.3                      # scores of a few units: well beyond the smaller cap
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, scale, cap, plan, status=st)
    ref = reference(s, q, k, v, chosen, mask, scale, cap)
    check_forward(s, o, lse, ref, q, k, v, scale, cap)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, scale, cap, plan, status=st)
    check_backward(s, grads, ref, lse, o, do, q, k, v, scale, cap, plain=kind is None and cap == 0)
    assert int(st) == 0


@pytest.mark.parametrize("dims", SHAPES[:5])
def test_gradients_are_the_derivative(dims):
    """The formula's gradients against central differences of the float64 forward."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(12)
    q, k, v, do = inputs(s, g)
    rp, ci, chosen = csr(s, 0.6, g)
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    scale, cap = 0.2, 4.0
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, scale, cap, plan)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, scale, cap, plan)
    base = [x.double() for x in (q, k, v)]
    for which in range(3):
        along = torch.randn(base[which].shape, generator=g, device="cuda").double()
        step, vals = 1e-4, []
        for sign in (1, -1):
            args = list(base)
            args[which] = base[which] + sign * step * along
            vals.append(float((reference(s, *args, chosen, mask, scale, cap)[4] * do.double()).sum()))
        diff = (vals[0] - vals[1]) / (2 * step)
        got = float((grads[which].double() * along).sum())
        # each gradient entry is off by at most a few 2^-8 of its terms; the signs of `along` are independent, so
        # the sum is off by sqrt(n) of that with room to spare (5 deviations)
        tol = 5 * 4 * U16 * float((grads[which].double() * along).norm()) + 5e-3
        assert abs(diff - got) <= tol, (which, diff, got, tol)


@pytest.mark.parametrize("dims", SHAPES[:5])
def test_without_mask_and_cap_the_plain_bits(dims):
    s = sp.make_shape(*dims, "bf16")
    g = gen(13)
    q, k, v, do = inputs(s, g)
    rp, ci, chosen = csr(s, 0.5, g)
    o, lse = sp.attn_fwd(s, q, k, v, rp, ci)
    grads = sp.attn_bwd(s, q, k, v, o, lse, do, rp, ci)
    o2, lse2 = sp.attn_masked_fwd(s, q, k, v, rp, ci)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(grads, sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci)))
    # a mask that hides nothing: the forward rounds exp(y) to bf16 against another reference than the plain one, so
    # each is within the bounds of the exact value that check_forward states, not equal to the other; in the
    # backward from one (O, LSE) dK and dV are the same arithmetic and the same bits, dQ has dS in two parts
    mask = masks(s, "all", g)
    plan = sp.mask_plan(s, *mask)
    scale = s.d ** -0.5
    ref = reference(s, q, k, v, chosen, mask, scale, 0.0)
    check_forward(s, o, lse, ref, q, k, v, scale, 0.0)
    check_forward(s, *sp.attn_masked_fwd(s, q, k, v, rp, ci, mask=plan), ref, q, k, v, scale, 0.0)
    got = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, mask=plan)
    assert torch.equal(grads[1], got[1]) and torch.equal(grads[2], got[2])
    check_backward(s, got, ref, lse, o, do, q, k, v, scale, 0.0)


@pytest.mark.parametrize("dims", SHAPES[:5])
@pytest.mark.parametrize("cap", [0.0, 10.0, 100.0])
def test_layouts_grid_and_order(dims, cap):
    """Raster inputs and outputs, the flat order, capped grids, repeated calls: the same bits."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(14)
    q, k, v, do = inputs(s, g)
    rp, ci, _ = csr(s, 0.6, g)
    plan = sp.mask_plan(s, *masks(s, "docs", g))
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=cap, mask=plan)
    for flags in (0, sp.SCHED_FLAT, sp.GRID_CAP(1), sp.GRID_CAP(7), sp.BWD_SPLIT_KV):
        o2, lse2 = sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan, flags=flags)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        got = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=cap, mask=plan, flags=flags)
        assert all(torch.equal(a, b) for a, b in zip(grads, got))
    ro, rl = sp.attn_masked_fwd(s, *(to_raster(s, x) for x in (q, k, v)), rp, ci, cap=cap, mask=plan,
                                flags=sp.OUT_RASTER | sp.IN_RASTER)
    assert torch.equal(ro, to_raster(s, o)) and torch.equal(rl, lse)
    got = sp.attn_masked_bwd(s, q, k, v, ro, lse, do, rp, ci, cap=cap, mask=plan, flags=sp.OUT_RASTER)
    assert all(torch.equal(to_raster(s, a), b) for a, b in zip(grads, got))


@pytest.mark.parametrize("dims", SHAPES[:5])
@pytest.mark.parametrize("cap", [0.0, 8.0, 50.0, 300.0])
def test_extreme_scores(dims, cap):
    """Scores of hundreds (the softmax is one key; the cap saturates) and of zero."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(15)
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    rp, ci, chosen = csr(s, 0.7, g)
    for spread in (8.0, 3.0, 0.0):
        q, k, v, do = inputs(s, g, spread)
        if spread == 3.0:                 # a few query blocks only, all of one sign: the others stay in range
            q[:, :, s.Bt:] *= 0.05
            k, v = k.abs(), v * 1e30
            q[:, :, : s.Bt] = -q[:, :, : s.Bt].abs()
        o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, 1.0, cap, plan)
        ref = reference(s, q, k, v, chosen, mask, 1.0, cap)
        check_forward(s, o, lse, ref, q, k, v, 1.0, cap)
        grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, 1.0, cap, plan)
        check_backward(s, grads, ref, lse, o, do, q, k, v, 1.0, cap)


@pytest.mark.parametrize("dims", SHAPES[:5])
@pytest.mark.parametrize("cap", [0.0, 18.0, 20.0, 21.0, 50.0, 200.0])
def test_scores_all_low_and_small_values(dims, cap):
    """Every score of some rows is at -cap (or far below zero), of others at +cap, and the values are small or large:
    the probabilities keep their precision whatever the reference of the exponentials."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(31)
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    rp, ci, chosen = csr(s, 0.7, g)
    q, k, v, do = inputs(s, g)
    k = k.abs()
    q[:, :, 1::3], q[:, :, 2::3] = -q[:, :, 1::3].abs(), q[:, :, 2::3].abs()
    for small in (1e-9, 1e9):
        o, lse = sp.attn_masked_fwd(s, q, k, (v * small).bfloat16(), rp, ci, 1.0, cap, plan)
        v_ = (v * small).bfloat16()
        ref = reference(s, q, k, v_, chosen, mask, 1.0, cap)
        check_forward(s, o, lse, ref, q, k, v_, 1.0, cap)
        grads = sp.attn_masked_bwd(s, q, k, v_, o, lse, do, rp, ci, 1.0, cap, plan)
        check_backward(s, grads, ref, lse, o, do, q, k, v_, 1.0, cap)


@pytest.mark.parametrize("dims", SHAPES[:5])
@pytest.mark.parametrize("cap", [2048.0, 2.0 ** 20])
@pytest.mark.parametrize("level", [8.0, 600.0])
def test_large_caps_keep_the_scores(dims, cap, level):
    """Under a cap that scores do not come near, they lose no more than the products' own rounding: here all of them
    are about `level` with differences of a few units, in the range of the kernel without a maximum and out of it. The
    cap adds to the exponent's error 2^-20 of the largest score, a polynomial's relative error, not 2^-20 of the cap."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(32)
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    rp, ci, chosen = csr(s, 0.7, g)
    q, k, v, do = inputs(s, g)
    q, k = q * 0.25, k * 0.25
    q[..., 0], k[..., 0] = math.sqrt(level), math.sqrt(level)
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, 1.0, cap, plan)
    ref = reference(s, q, k, v, chosen, mask, 1.0, cap)
    top = 2.0 * level                         # in place of the cap: exp_error's cap term
    assert float(ref[0].masked_fill(~ref[1], 0.0).abs().amax()) < top
    e = exp_error(s, q, k, 1.0, top)
    rel = 2 * e + 2.0 ** -20
    close(o, ref[4], (U16 + rel) * (ref[3] @ v.double().abs()) * (1 + U16) + U16 * ref[4].abs() + 1e-30, "O")
    live = ref[1].any(-1)
    close(lse[live], ref[5][live], rel + 4 * U32 * ref[5][live].abs(), "LSE")
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, 1.0, cap, plan)
    check_backward(s, grads, ref, lse, o, do, q, k, v, 1.0, top)


def test_masked_keys_do_not_reach_the_scores():
    """A key that nobody sees may hold any finite values: the largest bf16 changes nothing."""
    s = sp.make_shape(1, 2, 6, 16, 24, 64, 2, 8, 8, "bf16")
    g = gen(16)
    q, k, v, do = inputs(s, g)
    rp, ci, _ = csr(s, 0.7, g)
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    dead = to_blocked(s, mask[0])[0] < 0
    assert dead.any()
    first = sp.attn_masked_fwd(s, q, k, v, rp, ci, mask=plan)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, dead], v2[:, :, dead] = 1e4, -1e4
    second = sp.attn_masked_fwd(s, q, k2, v2, rp, ci, mask=plan)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    g1 = sp.attn_masked_bwd(s, q, k, v, *first, do, rp, ci, mask=plan)
    g2 = sp.attn_masked_bwd(s, q, k2, v2, *first, do, rp, ci, mask=plan)
    assert all(torch.equal(a, b) for a, b in zip(g1, g2))
    assert (g1[1][:, :, dead] == 0).all() and (g1[2][:, :, dead] == 0).all()


@pytest.mark.parametrize("dims", SHAPES[:5])
@pytest.mark.parametrize("kind,cap", [("docs", 0.0), ("frames", 9.0), (None, 9.0)])
@pytest.mark.parametrize("how", ["index", "length", "twice"])
def test_malformed_rows_count_as_empty(dims, kind, cap, how):
    s = sp.make_shape(*dims, "bf16")
    g = gen(17)
    q, k, v, do = inputs(s, g)
    rp, ci, chosen = csr(s, 0.7, g)
    mask = masks(s, kind or "all", g)
    plan = sp.mask_plan(s, *mask) if kind else None
    rp, ci, chosen = rp.clone(), ci.clone(), chosen.clone()
    if how == "index":
        ci[int(rp[2])] = s.nb             # row 2 (every block): its first index out of range
        bad = 2
    elif how == "twice":
        if s.Bt != 64:
            pytest.skip("128-token blocks attend to a block as often as it is listed")
        ci[int(rp[2])] = ci[int(rp[2]) + 1]
        bad = 2
    else:
        rp[2] = rp[3] + 1                 # row 2 ends before it begins; row 1 (empty) then holds row 2 and a block more
        bad = 2
        row1 = ci[int(rp[1]):int(rp[2])].long()
        chosen[0, 1] = False
        if int(rp[2] - rp[1]) <= s.nb and row1.unique().numel() == row1.numel():
            chosen[0, 1, row1] = True
        elif int(rp[2] - rp[1]) <= s.nb and s.Bt != 64:
            pytest.skip("row 1 lists a block twice here")
    chosen[0, bad] = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = s.d ** -0.5
    o, lse = (torch.full_like(q, 7.0), torch.full((s.B, s.H, s.N), 7.0, device="cuda"))
    sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan, status=st, o=o, lse=lse)
    assert int(st) == sp.DATA
    ref = reference(s, q, k, v, chosen, mask, scale, cap)
    check_forward(s, o, lse, ref, q, k, v, scale, cap)
    st.zero_()                            # the backward reports it; its gradients are not defined then
    sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=cap, mask=plan, status=st)
    assert int(st) == sp.DATA


@pytest.mark.parametrize("dims", SHAPES[:6])
@pytest.mark.parametrize("kind", ["docs", "frames", "random", "nothing"])
def test_mask_scores(dims, kind):
    """Exactly the block pairs with a query interval hull that misses every key position are masked, and no pair
    that holds a visible token pair is."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(18)
    mask = masks(s, kind, g)
    plan = sp.mask_plan(s, *mask)
    scores = torch.randn(s.B, s.H, s.nb, s.nb, generator=g, device="cuda")
    got = sp.mask_scores(s, plan, scores.clone())
    pos, lo, hi = (to_blocked(s, t).long().view(s.B, s.nb, s.Bt) for t in mask)
    see = (lo.view(s.B, -1, 1) <= pos.view(s.B, 1, -1)) & (pos.view(s.B, 1, -1) < hi.view(s.B, -1, 1))
    see = see.view(s.B, s.nb, s.Bt, s.nb, s.Bt).any(4).any(2)
    live = hi > lo
    hull_lo = torch.where(live, lo, I32.max).amin(-1)
    hull_hi = torch.where(live, hi, I32.min).amax(-1)
    keep = (pos.amax(-1)[:, None] >= hull_lo[..., None]) & (pos.amin(-1)[:, None] < hull_hi[..., None])
    assert (keep | ~see).all()
    want = torch.where(keep[:, None], scores, torch.full_like(scores, sp.MASKED_SCORE))
    assert torch.equal(got, want)
    rp, ci = sp.select(s, got, 0.9, 1)
    chosen = torch.zeros(s.rows, s.nb, dtype=torch.bool, device="cuda")
    n = int(rp[-1])
    rows = torch.repeat_interleave(torch.arange(s.rows, device="cuda"), (rp[1:] - rp[:-1]).long())
    chosen[rows, ci[:n].long()] = True
    k4 = keep[:, None].expand(s.B, s.H, s.nb, s.nb).reshape(-1, s.nb)
    some = k4.any(-1)
    assert (k4 | ~chosen)[some].all()      # no masked pair is picked while a row has others


# nb = 4,096 blocks: 262,144 tokens in 64-token blocks, 524,288 in 128-token ones (d = 64: rows of 64 MB and more)
@pytest.mark.parametrize("dims", [(1, 1, 64, 64, 64, 64, 1, 8, 8), (1, 1, 64, 128, 64, 128, 2, 8, 8),
                                  (1, 1, 64, 128, 64, 64, 2, 8, 8)])
@pytest.mark.parametrize("cap", [0.0, 12.0])
def test_longest_sequences(dims, cap):
    """The largest number of blocks, on query and key blocks at both ends, at document borders and in between."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(20)
    q, k, v, do = inputs(s, g)
    nb, bt = s.nb, s.Bt
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    # per row: the block itself, its neighbours and a few far ones; the same few are then in many lists
    far = torch.randint(0, nb, (64,), generator=g, device="cuda")
    own = torch.arange(nb, device="cuda")[:, None]
    cols = torch.cat([own, (own + 1) % nb, (own * 7 + 13) % nb, far[torch.arange(nb, device="cuda")[:, None] % 64],
                      far[(own // 64) % 64]], 1)
    chosen = torch.zeros(nb, nb, dtype=torch.bool, device="cuda").scatter_(1, cols, True)
    rp = torch.zeros(nb + 1, dtype=torch.int32, device="cuda")
    rp[1:] = chosen.sum(1).cumsum(0)
    ci = chosen.nonzero()[:, 1].int()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = s.d ** -0.5
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, scale, cap, plan, status=st)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, scale, cap, plan, status=st)
    assert int(st) == 0
    pos, lo, hi = (to_blocked(s, t)[0].view(nb, bt).long() for t in mask)
    qb, kb, vb, ob, dob = (x.view(nb, bt, s.d).double() for x in (q, k, v, o, do))
    lb = lse.view(nb, bt).double()

    def pair(i, j):      # rows of blocks i against the keys of blocks j, in float64
        t = scale * qb[i].flatten(0, 1) @ kb[j].flatten(0, 1).T
        see = (lo[i].view(-1, 1) <= pos[j].view(1, -1)) & (pos[j].view(1, -1) < hi[i].view(-1, 1))
        slope = 1.0
        if cap > 0:
            slope = 1 - torch.tanh(t / cap) ** 2
            t = cap * torch.tanh(t / cap)
        return t, see, slope

    e = exp_error(s, q[:, :, :4096], k[:, :, :4096], scale, cap) * 2
    rel = 2 * e + 2.0 ** -20 * (1 + cap)
    for i in (0, 1, nb // 3, nb // 2 + 5, nb - 600, nb - 1):
        j = chosen[i].nonzero()[:, 0]
        t, see, slope = pair(torch.tensor([i], device="cuda"), j)
        t = t.masked_fill(~see, -math.inf)
        L = torch.logsumexp(t, -1)
        dead = ~see.any(-1)
        p = torch.exp(t - L[:, None]).masked_fill(~see, 0.0)
        O, mass = p @ vb[j].flatten(0, 1), p @ vb[j].flatten(0, 1).abs()
        close(ob[i], O, (U16 + rel) * mass * (1 + U16) + U16 * O.abs() + 1e-30, f"O {i}")
        assert torch.isneginf(lb[i][dead]).all()
        close(lb[i][~dead], L[~dead], rel + 4 * U32 * L[~dead].abs(), f"LSE {i}")
        p = torch.exp(t - lb[i].masked_fill(dead, 0.0)[:, None]).masked_fill(~see, 0.0)
        dp = dob[i] @ vb[j].flatten(0, 1).T
        ds = p * (dp - (dob[i] * ob[i]).sum(-1, keepdim=True)) * slope
        dq = scale * ds @ kb[j].flatten(0, 1)
        tol = (U16 ** 2 + rel + 2.0 ** -12) * scale * ds.abs() @ kb[j].flatten(0, 1).abs()   # 2^-12: dP - D in fp32
        close(grads[0].view(nb, bt, s.d)[i], dq, tol * (1 + U16) + U16 * dq.abs() + 1e-6, f"dQ {i}")
    for j in (0, int(far[0]), nb // 3, nb - 1):
        i = chosen[:, j].nonzero()[:, 0]
        t, see, slope = pair(i, torch.tensor([j], device="cuda"))
        Li = lb[i].flatten()[:, None]
        p = torch.exp(t - torch.where(torch.isinf(Li), 0.0, Li)).masked_fill(~see, 0.0)
        d_i = dob[i].flatten(0, 1)
        dv = p.T @ d_i
        close(grads[2].view(nb, bt, s.d)[j], dv, (U16 + rel) * (p.T @ d_i.abs()) * (1 + U16) + U16 * dv.abs() + 1e-30,
              f"dV {j}")
        ds = p * (d_i @ vb[j].T - (d_i * ob[i].flatten(0, 1)).sum(-1, keepdim=True)) * slope
        dk = scale * ds.T @ qb[i].flatten(0, 1)
        tol = (U16 + rel + 2.0 ** -12) * scale * ds.abs().T @ qb[i].flatten(0, 1).abs()
        close(grads[1].view(nb, bt, s.d)[j], dk, tol * (1 + U16) + U16 * dk.abs() + 1e-6, f"dK {j}")


@pytest.mark.parametrize("dims", [(1, 64, 4, 32, 32, 64, 4, 4, 4), (2, 40, 4, 16, 24, 64, 2, 8, 8),
                                  (1, 40, 5, 8, 24, 128, 1, 8, 8)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_many_heads(dims, cap):
    """More items than the threads that order them (2,048 pairs), odd pairs and several batch elements: heads in every
    place against 64 bits; one CTA that takes all items in turn gives the same bits."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(33)
    q, k, v, do = inputs(s, g)
    rp, ci, chosen = csr(s, 0.5, g)
    mask = masks(s, "docs", g)
    plan = sp.mask_plan(s, *mask)
    scale = sp.default_scale(s.d)
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=cap, mask=plan)
    one = sp.make_shape(1, 1, *dims[2:], "bf16")
    for b, h in [(0, 0), (s.B - 1, s.H - 1), (s.B - 1, s.H // 2)]:
        r = b * s.H + h
        q1, k1, v1, do1, o1, *g1 = (t[b:b + 1, h:h + 1] for t in (q, k, v, do, o, *grads))
        lse1 = lse[b:b + 1, h:h + 1]
        ref = reference(one, q1, k1, v1, chosen[r:r + 1], tuple(t[b:b + 1] for t in mask), scale, cap)
        check_forward(one, o1, lse1, ref, q1, k1, v1, scale, cap)
        check_backward(one, g1, ref, lse1, o1, do1, q1, k1, v1, scale, cap)
    for got, want in zip(sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan, flags=sp.GRID_CAP(1)), (o, lse)):
        assert torch.equal(got, want)
    for got, want in zip(sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=cap, mask=plan, flags=sp.GRID_CAP(1)),
                         grads):
        assert torch.equal(got, want)


def test_given_stream_and_a_workspace_in_turn():
    """The stream argument (outputs and workspace made by the call), and one workspace for two captured steps that
    run in turn."""
    s = sp.make_shape(1, 2, 6, 16, 24, 64, 2, 8, 8, "bf16")
    g = gen(27)
    q, k, v, do = inputs(s, g)
    rp, ci, _ = csr(s, 0.6, g)
    plan = sp.mask_plan(s, *masks(s, "docs", g))
    args = (s, q, k, v, rp, ci)
    want = [[t.clone() for t in sp.attn_masked_fwd(*args, cap=cap, mask=plan)] for cap in (0.0, 80.0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sp.attn_masked_fwd(*args, mask=plan, stream=side)
    grads = sp.attn_masked_bwd(s, q, k, v, *got, do, rp, ci, mask=plan, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    assert all(torch.isfinite(t).all() for t in grads)
    ws = torch.empty(sp.attn_masked_workspace_size(s), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for cap in (0.0, 80.0):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sp.attn_masked_fwd(*args, cap=cap, mask=plan, ws=ws))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_other_stream_and_two_captured_graphs():
    """A call on a side stream, and two captured steps with workspaces of their own replayed in turn, give the same
    bits as eager calls; a captured step follows its inputs."""
    s = sp.make_shape(1, 2, 6, 16, 24, 128, 2, 8, 8, "bf16")
    g = gen(19)
    q, k, v, do = inputs(s, g)
    rp, ci, _ = csr(s, 0.6, g)
    plans = [sp.mask_plan(s, *masks(s, kind, g)) for kind in ("docs", "frames")]

    def step(i, ws):
        o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=(0.0, 6.0)[i], mask=plans[i], ws=ws)
        return (o, lse, *sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=(0.0, 6.0)[i], mask=plans[i], ws=ws))

    wss = [torch.empty(sp.attn_masked_workspace_size(s, True), dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = [[t.clone() for t in step(i, wss[i])] for i in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(0, wss[0])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(i, wss[i]))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    q.mul_(0.5)
    want = step(1, wss[1])
    want = [t.clone() for t in want]
    graphs[1].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[1], want))
