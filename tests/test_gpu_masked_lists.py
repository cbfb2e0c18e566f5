"""The block lists of a masked step: what augmentation, balancing, placement and the KV demand do with pairs of blocks
that see nothing of each other."""
import numpy as np
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from oracle import sparsp_oracle as orc
from tests.gpu_helpers import compare_augmented, host
from tests.test_gpu_masked import gen, masks, to_blocked

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
    chosen = (torch.rand(S.shape, generator=g, device="cuda") < torch.linspace(0.1, 0.9, s.H, device="cuda").view(1, -1, 1, 1))
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
