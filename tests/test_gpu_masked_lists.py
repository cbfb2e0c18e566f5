"""The block lists of a masked step: what augmentation, balancing, placement and the KV demand do with pairs of blocks
that see nothing of each other."""
import numpy as np
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from oracle import sparsp_oracle as orc
from tests.gpu_helpers import compare_augmented, host
from tests.test_gpu_masked import check_backward, check_forward, csr, gen, inputs, masks, reference, to_blocked

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

DIMS = [(1, 4, 6, 16, 24, 128, 2, 8, 8), (2, 3, 4, 16, 12, 64, 4, 4, 4)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def padded(s):
    """Documents, and padding from the middle of the last batch element on: whole blocks that see nothing. Returns the
    mask and which block pairs see something by the plan's ranges [B, nb, nb]."""
    pos, lo, hi = (t.clone() for t in masks(s, "docs", None))
    for t, v in ((pos, -1), (lo, 0), (hi, 0)):
        t.view(s.B, s.T, s.Y, s.X)[-1, :, :, s.X // 2:] = v
    p, l, h = (to_blocked(s, t).long().view(s.B, s.nb, s.Bt) for t in (pos, lo, hi))
    far = 1 << 40
    l, h = torch.where(h > l, l, far).amin(-1), torch.where(h > l, h, -far).amax(-1)
    return (pos, lo, hi), (p.amax(-1)[:, None] >= l[..., None]) & (p.amin(-1)[:, None] < h[..., None])


def chosen_of(s, rp, ci):
    out = torch.zeros(s.rows, s.nb, dtype=torch.bool, device="cuda")
    rows = torch.repeat_interleave(torch.arange(s.rows, device="cuda"), (rp[1:] - rp[:-1]).long())
    out[rows, ci[: int(rp[-1])].long()] = True
    return out.view(s.B, s.H, s.nb, s.nb)


def csr_of(chosen):
    flat = chosen.reshape(-1, chosen.shape[-1])
    rp = torch.zeros(flat.shape[0] + 1, dtype=torch.int32, device="cuda")
    rp[1:] = flat.sum(1).cumsum(0)
    return rp, torch.cat([flat.nonzero()[:, 1].int(), rp.new_zeros(4)])


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("P", [2, 3])
def test_augment_leaves_masked_pairs(dims, P):
    """No pair of blocks that see nothing of each other is added, whatever its row's masses, and the slack goes to the
    best of the others."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(51)
    mask, meet = padded(s)
    plan = sp.mask_plan(s, *mask)
    assert not meet.any(-1).all()
    S = sp.mask_scores(s, plan, torch.randn(s.B, s.H, s.nb, s.nb, generator=g, device="cuda"))
    density = torch.linspace(0.1, 0.9, s.H, device="cuda").view(1, -1, 1, 1)
    chosen = torch.rand(S.shape, generator=g, device="cuda") < density
    rp, ci = csr_of(chosen & meet[:, None])
    hr = (torch.arange(s.H) * P // s.H).int().expand(s.B, s.H).contiguous().cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rp2, ci2, added = sp.augment(s, P, S, rp, ci, hr, status=st)
    assert int(st) == 0 and int(added.sum()) > 0
    assert (meet[:, None] | ~chosen_of(s, rp2, ci2)).all()
    S_ = host(S).reshape(-1, s.nb)
    ref = orc.augment(S_, host(rp), host(ci), s.B, s.H, s.nb, host(hr), P)
    assert host(added).tolist() == ref.added.tolist()
    V = np.where(S_ == orc.MASKED_SCORE, np.float32(0), orc.block_values(S_))
    compare_augmented(host(rp2), host(ci2), ref, host(rp), host(ci), V, host(hr), s.B, s.H, s.nb, P)


@pytest.mark.parametrize("dims", DIMS)
def test_mask_csr(dims):
    """The rows' pairs that see something, in their order; a malformed row is empty and reported; attention on these
    lists gives the bits of its own compaction."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(52)
    mask, meet = padded(s)
    plan = sp.mask_plan(s, *mask)
    chosen = torch.rand(s.B, s.H, s.nb, s.nb, generator=g, device="cuda") < 0.6
    rp, ci = csr_of(chosen)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rp2, ci2 = sp.mask_csr(s, plan, rp, ci, status=st)
    want = csr_of(chosen & meet[:, None])
    n = int(rp2[-1])
    assert int(st) == 0 and torch.equal(rp2, want[0]) and torch.equal(ci2[:n], want[1][:n])
    # rows keep their own order
    back = torch.cat([ci[int(a):int(b)].flip(0) for a, b in zip(rp[:-1], rp[1:])] + [ci[-4:]])
    rp3, ci3 = sp.mask_csr(s, plan, rp, back)
    assert torch.equal(rp3, rp2)
    assert torch.equal(ci3[:n], torch.cat([ci2[int(a):int(b)].flip(0) for a, b in zip(rp2[:-1], rp2[1:])]))
    q, k, v = (torch.randn(s.B, s.H, s.N, s.d, generator=g, device="cuda").bfloat16() for _ in range(3))
    one = sp.attn_masked_fwd(s, q, k, v, rp2, ci2, mask=plan, flags=sp.LISTS_SEEN)
    two = sp.attn_masked_fwd(s, q, k, v, rp2, ci2, mask=plan)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    grads = [sp.attn_masked_bwd(s, q, k, v, *one, v, rp2, ci2, mask=plan, flags=f) for f in (0, sp.LISTS_SEEN)]
    assert all(torch.equal(a, b) for a, b in zip(*grads))
    if sp.attn_masked_compacts(s):
        two = sp.attn_masked_fwd(s, q, k, v, rp, ci, mask=plan)
        assert all(torch.equal(a, b) for a, b in zip(one, two))
    # malformed: an index out of range in row 3; row 5 longer than it may be, and row 4 if it then ends before it begins
    bad = ci.clone()
    bad[int(rp[3])] = s.nb
    long = rp.clone()
    long[5] = int(rp[6]) - s.nb - 1
    if int(long[5]) < 0:
        long[5] = 0
    size = long[1:] - long[:-1]
    for r, c, rows in ((rp, bad, [3]), (long, ci, ((size < 0) | (size > s.nb)).nonzero()[:, 0].tolist())):
        assert rows
        st.zero_()
        rp4, ci4 = sp.mask_csr(s, plan, r, c, status=st)
        assert int(st) == sp.DATA
        for x in rows:
            assert int(rp4[x]) == int(rp4[x + 1])
        assert int(rp4[3] - rp4[2]) == int(rp2[3] - rp2[2])


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("augmented", [False, True])
def test_pipeline_counts_pairs_that_see_something(dims, augmented):
    """Padding tiles, whose rows select as if all scores were equal, and a floor above what some rows see: neither the
    heads' costs, nor augmentation, nor the demand of a partition holds a block for a query block that sees nothing
    of it, and attention gives the same values."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(53)
    mask, meet = padded(s)
    plan = sp.mask_plan(s, *mask)
    q, k, v, do = (torch.randn(s.B, s.N, s.H, s.d, generator=g, device="cuda").bfloat16() for _ in range(4))
    P, floor = 3, int(meet.sum(-1).amax())
    kw = dict(migrations=2, augment=True) if augmented else {}
    pipe = sp.Pipeline(s, "mean", 0.7, floor, P, mask=plan, backward=True, **kw)
    o, lse = (t.clone() for t in pipe.forward(q, k, v))
    grads = [t.clone() for t in pipe.backward(do)]
    assert int(pipe.status) == 0
    picked = chosen_of(s, pipe.row_ptr, pipe.col_idx)
    assert (picked & ~meet[:, None]).any()          # the selection itself has such pairs
    lists = picked & meet[:, None]
    if augmented:
        assert host(pipe.balance.loads)[:, 0].sum(-1).tolist() == lists.flatten(1).sum(1).tolist()
        final = chosen_of(s, *pipe.csr)
        assert (meet[:, None] | ~final).all() and (final | ~lists).all()
        assert int(pipe.added.sum()) == int(final.sum()) - int(lists.sum())
        lists = final
    edges = [r * s.nb // P for r in range(P + 1)]
    want = torch.stack([lists[:, :, a:b].any(2) for a, b in zip(edges, edges[1:])], 2).view(-1, s.nb)
    dem = pipe.demand
    n = int(dem.dem_ptr[-1])
    got = torch.zeros_like(want)
    got[torch.repeat_interleave(torch.arange(want.shape[0], device="cuda"),
                                (dem.dem_ptr[1:] - dem.dem_ptr[:-1]).long()), dem.dem_idx[:n].long()] = True
    assert torch.equal(got, want) and n == int(want.sum())
    rows = got.nonzero()
    kb = sp.reorder(s, k).view(s.B * s.H, s.nb, s.Bt, s.d)
    assert torch.equal(dem.kg[:n], kb[rows[:, 0] // P, rows[:, 1]])
    # the same values as attention on the selection (with what was added) under the mask
    rp, ci = csr_of(lists)
    ins = [sp.reorder(s, x) for x in (q, k, v, do)]
    o2, lse2 = sp.attn_masked_fwd(s, *ins[:3], rp, ci, mask=plan, flags=sp.OUT_RASTER)
    seen = torch.isfinite(lse2)
    assert torch.equal(seen, torch.isfinite(lse))
    # the order of the sums alone differs: fp32 in LSE, a rounding of P and of the result (P, dS and the result) each
    apart = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())
    assert torch.allclose(lse[seen], lse2[seen], rtol=0, atol=2e-6) and apart(o, o2) < 2.0 ** -8
    g2 = sp.attn_masked_bwd(s, *ins[:3], o2, lse2, ins[3], rp, ci, mask=plan, flags=sp.OUT_RASTER)
    assert all(apart(a, b) < 2.0 ** -7 for a, b in zip(grads, g2))
    # placement takes the same lists
    if not augmented:
        placed = sp.Pipeline(s, "mean", 0.7, floor, P, mask=plan, placement=True)
        placed.forward(q, k, v)
        assert torch.equal(placed.owner, sp.placement(s, P, rp, ci))


@pytest.mark.parametrize("dims", [(2, 2, 6, 16, 24, 64, 2, 8, 8), (2, 1, 32, 48, 48, 64, 4, 4, 4)])
def test_transpose_leaves_out_rows_that_are_too_long(dims):
    """A row that claims more entries than there are blocks (all of them readable here) is reported and not read: its
    head's other rows and the other heads come out as without it."""
    s = sp.make_shape(*dims, "bf16")
    g = gen(54)
    chosen = torch.rand(s.B, s.H, s.nb, s.nb, generator=g, device="cuda") < (0.5 if s.nb < 100 else 0.02)
    chosen[..., 0] = True
    rp, ci = csr_of(chosen)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cp, ri = sp.csr_transpose(s, rp, ci, status=st)
    assert int(st) == 0 and torch.equal(chosen_of(s, cp, ri).transpose(-1, -2), chosen)
    n, last = int(rp[-1]), s.rows - 1
    long = rp.clone()
    long[last] = n - s.nb - 1          # the last row of the last head is now too long, the row before it ends too early
    ci = torch.cat([ci, ci])
    size = long[1:] - long[:-1]
    gone = (size < 0) | (size > s.nb)
    assert gone[last]
    want = chosen.view(s.rows, s.nb) & ~gone[:, None]
    for r in (~gone & (long[1:] != rp[1:])).nonzero()[:, 0].tolist():      # a row cut short keeps its first entries
        want[r, ci[int(long[r + 1]):int(rp[r + 1])].long()] = False
    cp, ri = sp.csr_transpose(s, long, ci, status=st)
    assert int(st) == sp.DATA
    cp_, ri_, want_ = cp.tolist(), ri.cpu(), want.view(s.B * s.H, s.nb, s.nb).cpu()
    for c in range(s.rows):
        h, j = divmod(c, s.nb)
        rows = want_[h, :, j].nonzero()[:, 0]
        assert torch.equal(ri_[cp_[c]:cp_[c] + len(rows)].long(), rows), (h, j)


@pytest.mark.parametrize("dims", [(1, 64, 4, 32, 32, 64, 4, 4, 4), (1, 40, 4, 32, 32, 128, 2, 8, 8)])
@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_malformed_rows_where_attention_compacts(dims, cap):
    """Shapes whose lists masked attention compacts itself: malformed rows are reported and count as empty, the others
    give the values of the formula, and the same bits as their own compaction handed in."""
    s, one = sp.make_shape(*dims, "bf16"), sp.make_shape(1, 1, *dims[2:], "bf16")
    assert sp.attn_masked_compacts(s) and sp.attn_masked_compacts(s, True) and not sp.attn_masked_compacts(one)
    g = gen(55)
    q, k, v, do = inputs(s, g)
    rp, ci, chosen = csr(s, 0.5, g)
    mask, meet = padded(s)
    plan = sp.mask_plan(s, *mask)
    ci, chosen = ci.clone(), chosen.clone()
    rows = [2, 5 * s.nb + 2, (s.H - 1) * s.nb + 2]       # rows that list every block
    for r, j in zip(rows, (s.nb, -1, 1 << 30)):
        ci[int(rp[r]) + 1] = j
        chosen[r // s.nb, r % s.nb] = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = sp.attn_masked_fwd(s, q, k, v, rp, ci, cap=cap, mask=plan, status=st)
    assert int(st) == sp.DATA
    st.zero_()
    grads = sp.attn_masked_bwd(s, q, k, v, o, lse, do, rp, ci, cap=cap, mask=plan, status=st)
    assert int(st) == sp.DATA
    scale = sp.default_scale(s.d)
    for h in (0, 5, s.H // 2, s.H - 1):
        q1, k1, v1, do1, o1, *g1 = (t[:, h:h + 1] for t in (q, k, v, do, o, *grads))
        ref = reference(one, q1, k1, v1, chosen[h:h + 1], mask, scale, cap)
        check_forward(one, o1, lse[:, h:h + 1], ref, q1, k1, v1, scale, cap)
        check_backward(one, g1, ref, lse[:, h:h + 1], o1, do1, q1, k1, v1, scale, cap)
    rp2, ci2 = sp.mask_csr(s, plan, rp, ci)
    o2, lse2 = sp.attn_masked_fwd(s, q, k, v, rp2, ci2, cap=cap, mask=plan, flags=sp.LISTS_SEEN)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
