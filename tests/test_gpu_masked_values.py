"""Masked and capped attention on values at the ends of their range: NaN and infinite inputs in keys and queries that
count, sums that leave fp32's range, values so small or large that products do, in each range of the cap (none, up to
20, where no score leaves the kernel's range, and beyond). Tolerances are those of test_gpu_masked."""
import math

import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_masked import (U16, U32, check_backward, check_forward, close, csr, exp_error, gen, inputs, masks,
                                   reference, to_blocked)

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

# 128-token blocks with d = 128, and pairs of 64-token blocks with both head sizes
DIMS = [(1, 2, 6, 16, 24, 128, 2, 8, 8), (2, 2, 4, 16, 12, 64, 4, 4, 4), (1, 2, 5, 8, 24, 128, 1, 8, 8)]
CAPS = [0.0, 10.0, 50.0, 300.0]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def setting(dims, seed, kind="docs"):
    s = sp.make_shape(*dims, "bf16")
    g = gen(seed)
    mask = masks(s, kind, g)
    rp, ci, chosen = csr(s, 0.6, g)
    return s, g, mask, sp.mask_plan(s, *mask), rp, ci, chosen


def check_beside(o, lse, ref, bad, v, rel, what):
    """Rows in `bad` have neither a finite value nor a finite LSE; all others are those of the reference."""
    assert (~torch.isfinite(o[bad])).all() and (~torch.isfinite(lse[bad])).all(), what
    _, pick, _, p, O, L = ref
    live, dead = pick.any(-1) & ~bad, ~pick.any(-1)
    mass = (p[:, :, :, :].nan_to_num(0.0) @ v.double().abs())[live]
    close(o[live], O[live], (U16 + rel) * mass * (1 + U16) + U16 * O[live].abs() + 1e-30, what + " O")
    close(lse[live], L[live], rel + 4 * U32 * L[live].abs(), what + " LSE")
    assert (o[dead] == 0).all() and torch.isneginf(lse[dead]).all()


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cap", CAPS)
def test_nan_in_a_key_and_in_a_query(dims, cap):
    """A row that sees a NaN score has NaN in O and in LSE, not a plausible LSE of its other keys; the others are as
    they would be."""
    s, g, mask, plan, rp, ci, chosen = setting(dims, 41)
    q, k, v, _ = inputs(s, g)
    scale = s.d ** -0.5
    rel = 2 * exp_error(s, q, k, scale, cap) + 2.0 ** -20
    for t, at in ((k, 5), (k, s.N // 2 + 70), (q, s.N // 3)):
        q2, k2 = q.clone(), k.clone()
        (q2 if t is q else k2)[:, :, at, 3] = math.nan
        o, lse = sp.attn_masked_fwd(s, q2, k2, v, rp, ci, scale, cap, plan)
        ref = reference(s, q2, k2, v, chosen, mask, scale, cap)
        bad = (ref[0].isnan() & ref[1]).any(-1)
        assert bad.any() and not bad.all()
        assert o[bad].isnan().all() and lse[bad].isnan().all()
        check_beside(o, lse, ref, bad, v, rel, f"NaN at {at}")


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cap", [0.0, 60.0, 1000.0])
@pytest.mark.parametrize("large", [2.0 ** 50, 2.0 ** 70])
def test_products_beyond_fp32(dims, cap, large):
    """Scores of about 45 with sums inside the range of the kernel without a maximum (its probabilities reach 2^65),
    and values of both signs so large that the products leave fp32: every row is done again, none is NaN."""
    s, g, mask, plan, rp, ci, chosen = setting(dims, 42)
    q, k, v, _ = inputs(s, g, 0.05)
    level = math.sqrt(58.0 if cap == 60.0 else 45.0)      # 60 tanh(58 / 60) is 44.8
    q[..., 0], k[..., 0] = level, level
    v = (v * large).bfloat16()
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, 1.0, cap, plan)
    ref = reference(s, q, k, v, chosen, mask, 1.0, cap)
    top = ref[5][torch.isfinite(ref[5])]
    assert 40 < float(top.min()) and float(top.max()) < 55.4      # 2^80 is 55.45
    check_forward(s, o, lse, ref, q, k, v, 1.0, cap)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cap", [0.0, 60.0])
@pytest.mark.parametrize("small", [2.0 ** -60, 2.0 ** -80, 2.0 ** -95])
def test_products_below_fp32(dims, cap, small):
    """Scores of about -35 with sums inside the range of the kernel without a maximum, and values so small that the
    products (2^-50 and less times the value) leave fp32: O is good to its own roundings all the same."""
    s, g, mask, plan, rp, ci, chosen = setting(dims, 43)
    q, k, v, _ = inputs(s, g, 0.05)
    level = math.sqrt(35.0 if cap == 0 else 39.0)
    q[..., 0], k[..., 0] = -level, level
    v = (v * small).bfloat16()
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, 1.0, cap, plan)
    ref = reference(s, q, k, v, chosen, mask, 1.0, cap)
    seen = ref[5][torch.isfinite(ref[5])]
    assert -41.5 < float(seen.min()) and float(seen.max()) < -14.0     # 2^-60 is -41.6
    check_forward(s, o, lse, ref, q, k, v, 1.0, cap)
    rel = 2 * exp_error(s, q, k, 1.0, cap) + 2.0 ** -20
    close(o, ref[4], (U16 + rel) * (ref[3] @ v.double().abs()) * (1 + U16) + U16 * ref[4].abs(), "O without a floor")


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("scale,cap", [(3.27e6, 200.0), (3.27e6, 1000.0), (1e30, 2.0 ** 20), (2.0 ** -30, 2.0 ** -18)])
def test_scales_far_from_the_cap(dims, scale, cap):
    """scale / cap at the border where the polynomial's folded coefficients leave fp32 and beyond, queries small or
    large in turn, keys of which each 32 hold two far below (their chunk takes another form of the cap, and the row's
    sum stays in range) and keys that are all zeros: a score of 0 stays 0."""
    s, g, mask, plan, rp, ci, chosen = setting(dims, 44)
    q, k, v, do = inputs(s, g)
    q = (q * (0.3 / scale)).bfloat16()
    q[..., 0], k[:, :, 5::16, 0] = 1 / scale, -150.0
    k[:, :, : s.Bt] = 0
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, scale, cap, plan)
    ref = reference(s, q, k, v, chosen, mask, scale, cap)
    check_forward(s, o, lse, ref, q, k, v, scale, cap)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, scale, cap, plan)
    check_backward(s, grads, ref, lse, o, do, q, k, v, scale, cap)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cap", CAPS)
def test_largest_values_that_nobody_sees(dims, cap):
    """The largest bf16 in tokens that see nothing and that nobody sees (padding): their scores and dO V^T overflow, and
    no result of the other tokens changes beyond its bounds (the form that a cap takes goes by the largest score
    beside them); the gradients of the padding are zero."""
    s, g, mask, plan, rp, ci, chosen = setting(dims, 45)
    q, k, v, do = inputs(s, g)
    scale = s.d ** -0.5
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, scale, cap, plan)
    ref = reference(s, q, k, v, chosen, mask, scale, cap)
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, scale, cap, plan)
    pad = to_blocked(s, mask[0]) < 0
    assert pad.any()
    at = pad[:, None].expand(s.B, s.H, s.N)
    largest = torch.finfo(torch.bfloat16).max
    for i in range(4):
        x = [t.clone() for t in (q, k, v, do)]
        x[i][at] = largest * torch.randn(int(at.sum()), s.d, generator=g, device="cuda").sign().bfloat16()
        o2, lse2 = sp.attn_masked_fwd(s, *x[:3], rp, ci, scale, cap, plan)
        check_forward(s, o2, lse2, ref, q, k, v, scale, cap)
        got = sp.attn_masked_bwd(s, *x[:3], o, lse, x[3], rp, ci, scale, cap, plan)
        check_backward(s, got, ref, lse, o, do, q, k, v, scale, cap)
        for t in got:
            assert (t[at] == 0).all()
        if cap == 0:
            assert torch.equal(o2, o) and torch.equal(lse2, lse)
            assert all(torch.equal(a, b) for a, b in zip(got, grads))


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cap", CAPS)
def test_infinite_scores(dims, cap):
    """An infinite value in a key: scores of both signs of infinity by the queries' signs. A cap bounds them, +-cap as
    the formula has it, also where a row sees nothing but -inf; without one a row that sees +inf is not finite,
    and -inf is a weight of zero."""
    s, g, mask, plan, rp, ci, chosen = setting(dims, 46)
    q, k, v, _ = inputs(s, g)
    scale = s.d ** -0.5
    rel = 2 * exp_error(s, q, k, scale, cap) + 2.0 ** -20
    q[..., 7] = torch.where(q[..., 7] < 0, -1.0, 1.0).bfloat16()
    for at in (slice(5, 6), slice(0, s.N)):
        k2 = k.clone()
        k2[:, :, at, 7] = math.inf
        o, lse = sp.attn_masked_fwd(s, q, k2, v, rp, ci, scale, cap, plan)
        ref = reference(s, q, k2, v, chosen, mask, scale, cap)
        t, pick = ref[0], ref[1]
        if cap > 0:
            assert torch.isfinite(t[pick]).all()
            check_beside(o, lse, ref, torch.zeros_like(pick[..., 0]), v, rel, "capped")
            continue
        bad = (torch.isposinf(t) & pick).any(-1)
        none = pick.any(-1) & (torch.isneginf(t) | ~pick).all(-1)     # nothing but -inf: LSE = -inf, O is not defined
        assert bad.any() and torch.isneginf(lse[none]).all()
        live = ref[1].any(-1) & ~none
        p = torch.where(bad[..., None], 0.0, ref[3])
        ref = (t, pick & live[..., None], ref[2], p, torch.where(live[..., None], p @ v.double(), 0.0), ref[5])
        check_beside(torch.where(none[..., None], 0.0, o.float()), lse, ref, bad, v, rel, "uncapped")


@pytest.mark.parametrize("cap", CAPS)
def test_infinity_in_a_value(cap):
    """An infinite value is infinite (or NaN) in its column of O for the rows that see its key, and nothing else: LSE
    and the other columns are as they would be. (128-token blocks: a pair's other block has weights of zero there.)"""
    s, g, mask, plan, rp, ci, chosen = setting(DIMS[0], 47, "all")
    q, k, v, _ = inputs(s, g)
    scale = s.d ** -0.5
    ref = reference(s, q, k, v, chosen, mask, scale, cap)
    v2 = v.clone()
    v2[:, :, 5, 9] = math.inf
    o, lse = sp.attn_masked_fwd(s, q, k, v2, rp, ci, scale, cap, plan)
    sees = ref[1][..., 5]
    assert sees.any() and not torch.isfinite(o[..., 9][sees]).any()
    o = o.clone()
    o[..., 9] = torch.where(sees, ref[4][..., 9].bfloat16(), o[..., 9])
    check_forward(s, o, lse, ref, q, k, v, scale, cap)
