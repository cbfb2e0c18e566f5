"""A step of generation as README writes it: positions, norm and rotation, tables and slots, the write and attention,
captured once and replayed with other requests' tokens, against the same step run eagerly and against float64."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_cache import attn_ref, built, fresh_pool, gen, i32, values, word  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]
B, H, HEADS, D, BT, TOKENS, WIDTH = 3, 4, 2, 64, 64, 90, 6
POSITIONS = WIDTH * BT


class Step:
    """State of the requests, and one step over it, length and place in the list updated in place."""

    def __init__(self):
        g = gen(5)
        self.pool = fresh_pool(B * WIDTH, HEADS, D, BT)
        self.free = torch.randperm(B * WIDTH, generator=g, device="cuda").int()
        self.table = torch.full((B, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.length, self.used, self.add, self.status = i32([0] * B), word(), i32([0] * B), word()
        self.x = torch.zeros(1, TOKENS, H + 2 * HEADS, D, device="cuda", dtype=torch.bfloat16)
        self.pos = torch.zeros(1, TOKENS, 3, dtype=torch.int32, device="cuda")
        self.shape = sp.make_shape(1, H, TOKENS, 1, 1, D, 1, 1, 1, "bf16")
        self.rope = sp.rope_table(self.shape, (D, 0, 0), extent=(POSITIONS, 1, 1))
        self.w = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]

    def run(self):
        held, x = self.length.clone(), self.x
        _, start, slots, _ = sp.cache_extend(self.pool.shape, self.length, self.add, self.free, self.table, TOKENS,
                                             used=self.used, len_out=self.length, used_out=self.used, status=self.status)
        i = torch.arange(TOKENS, dtype=torch.int32, device="cuda")
        b = (torch.searchsorted(start, i, right=True) - 1).clamp_(max=len(held) - 1)
        self.pos[0, :, 0] = (held[b] + i - start[b]).clamp_(max=POSITIONS - 1)
        q, k = sp.norm_rope_fwd(self.shape, self.rope, x[:, :, :H], x[:, :, H:H + HEADS], *self.w, rms=True, pos=self.pos,
                                out_blocked=False, status=self.status)
        sp.cache_write(self.pool, k[0], x[0, :, H + HEADS:], slots, status=self.status)
        o, lse = sp.attn_cache_fwd(self.pool, q[0], start, self.length, self.table, TOKENS, status=self.status)
        return o, lse, q[0], slots


def test_captured_step():
    one, two, g = Step(), Step(), gen(6)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two.run()                                    # nothing is new; what the calls keep is made
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = two.run()
    total = [0] * B
    for add in ([60, 1, 29], [1, 1, 1], [0, 70, 20], [5, 0, 64], [1, 0, 0], [0, 0, 0], [1, 40, 3]):
        x = torch.randn(one.x.shape, generator=g, device="cuda").bfloat16()
        for s in (one, two):
            s.x.copy_(x)
            s.add.copy_(i32(add))
        ref = one.run()
        graph.replay()
        n = sum(add)
        assert int(one.status) == 0 and int(two.status) == 0
        total = [t + a for t, a in zip(total, add)]
        assert one.length.tolist() == total == two.length.tolist() and int(one.used) == int(two.used)
        assert torch.equal(ref[3], out[3])
        for a, b in zip(ref[:3], out[:3]):
            assert torch.equal(a[:n], b[:n])
        at = 0
        place = torch.cat([torch.arange(t - a, t, device="cuda") for t, a in zip(total, add)])
        assert torch.equal(one.pos[0, :n, 0], place.int())
        for b, (a, t) in enumerate(zip(add, total)):
            if a == 0:
                continue
            page = two.table[b, : -(-t // BT)].long()
            keys = tuple((values(c)[page] * s.double()[page][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :t]
                         for c, s in ((two.pool.k, two.pool.k_scale), (two.pool.v, two.pool.v_scale)))
            O, L, to, tl = attn_ref(out[2][at: at + a], [keys], [a], [t], D ** -0.5, True, BT)
            assert ((out[0][at: at + a].double() - O).abs() <= to).all()
            assert ((out[1][at: at + a].double() - L).abs() <= tl).all()
            at += a
