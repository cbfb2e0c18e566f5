"""Steps in which the blocks run out: requests that wait, and the rows of the others, through tables, write and
attention; then the same requests once blocks are free."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_cache import attn_ref, built, fresh_pool, gen, i32, values, word  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]


@pytest.mark.parametrize("add,free", [([3, 70, 5, 64], 2), ([1, 1, 1, 1], 0), ([40, 1, 200, 2], 4), ([64, 65, 1, 0], 0)])
@pytest.mark.parametrize("short", ["blocks", "slots"])
def test_requests_that_wait(add, free, short):
    """The others' rows are what they are alone; what a waiting request holds stays as it is, and it goes on when it
    is brought again."""
    heads, d, bt, H = 2, 64, 64, 4
    held = [60, 64, 100, 0]
    most = [h + a for h, a in zip(held, add)]
    g, pool = gen(3), fresh_pool(40, heads, d, bt)
    order = torch.randperm(40, generator=g, device="cuda").int()
    table, length, used = torch.full((4, 8), -1, **dict(dtype=torch.int32, device="cuda")), i32([0] * 4), word()
    rows = [tuple(torch.randn(m, n, d, generator=g, device="cuda").bfloat16() for n in (H, heads, heads)) for m in most]

    def step(add, at, tokens, n_free):
        """A step that brings add[b] tokens of request b from at[b] on; (slots, start, o, lse, status)."""
        status = word()
        new = [torch.cat([r[i][a: a + n] for r, n, a in zip(rows, add, at)]) for i in range(3)]
        _, start, slots, _ = sp.cache_extend(pool.shape, length, i32(add), order[:n_free], table, tokens, used=used,
                                             len_out=length, used_out=used, status=status)
        pad = [torch.cat([t, t.new_zeros(max(0, tokens - t.shape[0]), *t.shape[1:])])[:tokens] for t in new]
        sp.cache_write(pool, pad[1], pad[2], slots)
        o, lse = sp.attn_cache_fwd(pool, pad[0], start, length, table, max(max(add), 1))
        return slots, start.tolist(), o, lse, int(status), pad[0]

    step(held, [0] * 4, sum(held), 40)
    first = int(used)
    before = [t.clone() for t in (table, length)]
    tokens = sum(add) if short == "blocks" else max(1, sum(add) - add[3] - (add[2] + 1) // 2)
    slots, start, o, lse, status, q = step(add, held, tokens, first + free if short == "blocks" else 40)
    now, waits = length.tolist(), [h + a > int(n) for h, a, n in zip(held, add, length.tolist())]
    assert any(waits) and status == sp.CAPACITY
    again = [a if w else 0 for a, w in zip(add, waits)]

    def check(b, n, total, o, lse, q):
        page = table[b, : -(-total // bt)].long()
        keys = tuple((values(c)[page] * s.double()[page][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :total]
                     for c, s in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)))
        O, L, to, tl = attn_ref(q, [keys], [n], [total], d ** -0.5, True, bt)
        assert ((o.double() - O).abs() <= to).all() and ((lse.double() - L).abs() <= tl).all()

    for b in range(4):
        s0, s1 = start[b], min(start[b + 1], tokens)
        if waits[b]:
            assert now[b] == held[b] and (slots[s0:s1] == -1).all() and torch.equal(table[b], before[0][b])
        elif add[b]:
            assert now[b] == most[b] and (slots[s0:s1] >= 0).all()
            check(b, add[b], most[b], o[s0:s1], lse[s0:s1], q[s0:s1])
    # brought again, with blocks for all
    slots, start, o, lse, status, q = step(again, held, sum(again), 40)
    assert status == 0 and (slots >= 0).all() and length.tolist() == most
    for b in range(4):
        if again[b]:
            check(b, add[b], most[b], *(t[start[b]: start[b + 1]] for t in (o, lse, q)))
    assert int(used) == sum(-(-m // bt) for m in most)
