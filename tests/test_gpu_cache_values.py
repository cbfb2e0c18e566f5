"""Attention over the cache in 8 bits at the ends of its range: zero queries and keys, values
whose scales are tiny or lie far apart, queries near the end of bf16; against float64.

Tolerances are those of test_gpu_cache.attn_ref. `far` adds what a score in base 2 that carries the logarithm of a
scale of V (up to LOG2 in magnitude) may be off by: its fp32 roundings, 2^-24 of LOG2 each, four of them at most."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp
from tests.test_gpu_cache import attn_ref, built, filled, gen, i32, values, word  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

LOG2 = 160   # a score here and log2 of a scale


def held(pool, table, lengths):
    """Per request the float64 keys and values [heads, n, d] that the pool's codes and scales stand for."""
    out = []
    for b, n in enumerate(lengths):
        page = table[b, : -(-n // pool.shape.bt)].long()
        out.append(tuple((values(c)[page] * s.double()[page][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
                         for c, s in ((pool.k, pool.k_scale), (pool.v, pool.v_scale))))
    return out


def queries(add, H, d, seed=11):
    return torch.randn(sum(add), H, d, generator=gen(seed), device="cuda")


def check(pool, table, lengths, add, q, causal=True, scale=None):
    bt, d = pool.shape.bt, pool.shape.d
    q, scale = q.bfloat16(), d ** -0.5 if scale is None else scale
    status = word()
    o, lse = sp.attn_cache_fwd(pool, q, i32([0] + add).cumsum(0).int(), i32(lengths), table, max(add), scale, causal=causal,
                               status=status)
    assert int(status) == 0
    O, L, to, tl = attn_ref(q, held(pool, table, lengths), add, lengths, scale, causal, bt)
    far = 4 * LOG2 * 2.0 ** -24
    to, tl = to + 2 * far * O.abs(), tl + far
    bad = ~((o.double() - O).abs() <= to)
    assert not bad.any(), f"O: {int(bad.sum())} off, {int(torch.isnan(o).sum())} NaN"
    bad = ~((lse.double() - L).abs() <= tl)
    assert not bad.any(), f"LSE: {int(bad.sum())} off, worst {float(torch.nan_to_num((lse.double() - L).abs(), 9e9).max())}"
    return o, lse


ROWS = [[2, 3], [9, 70], [70, 129], [129, 3]]    # of one request, times two: few and many rows in each kernel


def clear(pool, table, b, j, which):
    """Block j of request b becomes what the write of zeros leaves."""
    n, heads, d = pool.shape.bt, pool.shape.heads, pool.shape.d
    keep = {"k": (pool.v, pool.v_scale), "v": (pool.k, pool.k_scale)}[which]
    page = int(table[b, j])
    was = [t[page].clone() for t in (keep[0].view(torch.uint8), keep[1])]
    zero = torch.zeros(n, heads, d, device="cuda")
    sp.cache_write(pool, zero, zero.clone(), page * n + torch.arange(n, **dict(dtype=torch.int32, device="cuda")))
    keep[0].view(torch.uint8)[page], keep[1][page] = was


@pytest.mark.parametrize("add", ROWS)
@pytest.mark.parametrize("d,bt", [(64, 128), (128, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_zero_queries_and_zero_keys(add, d, bt, causal):
    """Every score of such a row is 0: the mean of what it sees, also where a mask or a request's end cuts a block."""
    lengths = [200, 333]
    pool, table, _ = filled(lengths, 2, d, bt)
    for b in range(2):
        clear(pool, table, b, 0, "k")
        clear(pool, table, b, -(-lengths[b] // bt) - 1, "k")     # the last one, filled in part
    q = queries(add, 4, d)
    q[::2] = 0.0
    check(pool, table, lengths, add, q, causal)


@pytest.mark.parametrize("add", ROWS)
@pytest.mark.parametrize("ks", [0.0, 2.0 ** -126, 2.0 ** -149])
def test_scales_of_keys_without_size(add, ks):
    lengths = [200, 333]
    pool, table, _ = filled(lengths, 2, 64, 64)
    pool.k_scale[table[0, 1]] = pool.k_scale[table[1, 5]] = ks
    q = queries(add, 4, 64)
    q[1::2] = 0.0
    check(pool, table, lengths, add, q)


@pytest.mark.parametrize("add", ROWS)
def test_hidden_block_with_a_scale_of_nan(add):
    """A causal row does not see the last block; what its scale of K is says nothing there."""
    lengths = [200, 333]
    pool, table, _ = filled(lengths, 2, 64, 64)
    q = queries(add, 4, 64).bfloat16()
    start, ln = i32([0] + add).cumsum(0).int(), i32(lengths)
    clean = sp.attn_cache_fwd(pool, q, start, ln, table, max(add))
    pool.k_scale[table[1, 5]] = float("nan")         # tokens 320 .. 332
    o, lse = sp.attn_cache_fwd(pool, q, start, ln, table, max(add))
    pos = torch.cat([torch.arange(n - a, n, device="cuda") for n, a in zip(lengths, add)])
    sees = (pos >= 320) & (torch.arange(sum(add), device="cuda") >= add[0])
    assert torch.isnan(o[sees]).all() and torch.isnan(lse[sees]).all()
    assert torch.equal(o[~sees], clean[0][~sees]) and torch.equal(lse[~sees], clean[1][~sees])


@pytest.mark.parametrize("add", ROWS)
@pytest.mark.parametrize("d", [64, 128])
def test_queries_near_the_end_of_bf16(add, d):
    """Queries of up to 3.3e38 and keys so small that the scores are ordinary."""
    lengths = [200, 333]
    pool, table, _ = filled(lengths, 2, d, 64)
    q = queries(add, 4, d).bfloat16().float()
    q *= 2.0 ** 125 / q.abs().amax()
    pool.k_scale.mul_(2.0 ** -122)
    o, _ = check(pool, table, lengths, add, q)
    assert torch.isfinite(o.float()).all()


# ------------------------------------------------------------------- scales of V

@pytest.mark.parametrize("add", ROWS)
@pytest.mark.parametrize("d,bt", [(64, 128), (128, 64)])
@pytest.mark.parametrize("exponent", [-120, -100, 60, 100])
def test_scales_of_values_all_alike(add, d, bt, exponent):
    lengths = [200, 333]
    pool, table, _ = filled(lengths, 2, d, bt)
    pool.v_scale.copy_(torch.full_like(pool.v_scale, 2.0 ** exponent))
    check(pool, table, lengths, add, queries(add, 4, d))


@pytest.mark.parametrize("add", ROWS)
@pytest.mark.parametrize("d,bt", [(64, 128), (128, 64)])
@pytest.mark.parametrize("exponents", [(-100, 0), (-100, 20), (-120, 100), (-100, 1, -40, 30)])
@pytest.mark.parametrize("seed", [0, 1])
def test_scales_of_values_far_apart(add, d, bt, exponents, seed):
    """Keys in a block of tiny values weigh as much as others, whatever order the scales come in."""
    lengths = [700, 1111]
    pool, table, _ = filled(lengths, 2, d, bt)
    pick = torch.randint(0, len(exponents), pool.v_scale.shape, generator=gen(seed), device="cuda")
    pool.v_scale.copy_(torch.exp2(torch.tensor(exponents, device="cuda").float()[pick]))
    check(pool, table, lengths, add, queries(add, 4, d))


@pytest.mark.parametrize("add", ROWS)
@pytest.mark.parametrize("which", ["zero", "tiny"])
def test_heavy_keys_with_values_of_no_size(add, which):
    """The keys that hold nearly all of the weight have values of 0, or of 2^-100."""
    lengths = [700, 1111]
    pool, table, _ = filled(lengths, 2, 64, 64)
    for b, j in ((0, 3), (0, 10), (1, 0), (1, 8)):
        page = int(table[b, j])
        if which == "zero":
            clear(pool, table, b, j, "v")
        else:
            pool.v_scale[page] = 2.0 ** -100
        pool.k_scale[page] *= 8.0
    check(pool, table, lengths, add, 2.0 * queries(add, 4, 64))


@pytest.mark.parametrize("add", [1, 40])
@pytest.mark.parametrize("low", [True, False])
def test_many_keys_without_values(add, low):
    """2^17 and more keys of zero values: the sum of the weights is what it is without values. With `low`, the scores
    rise by less than what moves a row's reference, after the first keys."""
    n, d, bt = (1 << 17) + 4000, 64, 128
    blocks = -(-n // bt)
    pool, table = sp.block_pool(blocks, 1, d, bt), i32([list(range(blocks))])
    k = torch.zeros(n, 1, d, device="cuda")
    if low:
        k[512:, 0, 0] = 1.0
    sp.cache_write(pool, k, torch.zeros_like(k), torch.arange(n, dtype=torch.int32, device="cuda"))
    q = torch.zeros(add, 1, d, device="cuda")
    q[:, 0, 0] = 20.0                                # 20 / 8 * log2(e) = 3.6 < 4
    o, lse = sp.attn_cache_fwd(pool, q.bfloat16(), i32([0, add]), i32([n]), table, add, causal=False)
    assert (o == 0).all()
    want = torch.full((add, 1), 2.5 if low else 0.0, dtype=torch.float64, device="cuda")
    want += torch.log(torch.tensor(n - 512 + 512 * torch.exp(torch.tensor(-2.5)).item() if low else float(n), dtype=torch.float64))
    # fp32 sums of at most 2^13 additions in a row (n keys of 64 lanes or more), 2^-24 each, and the far tolerance
    assert ((lse.double() - want).abs() <= 2.0 ** -11 + 4 * LOG2 * 2.0 ** -24).all(), lse.flatten()[:4]


@pytest.mark.parametrize("add", [1, 40])
@pytest.mark.parametrize("B", [1, 3])
def test_far_scales_over_many_parts(add, B):
    """A request that many CTAs share, each with scales of its own."""
    lengths = [30000 + 77 * b for b in range(B)]
    pool, table, _ = filled(lengths, 1, 64, 64)
    e = torch.randint(0, 5, pool.v_scale.shape, generator=gen(5), device="cuda")
    pool.v_scale.copy_(torch.exp2(torch.tensor([-120., -100., -30., 0., 40.], device="cuda")[e]))
    check(pool, table, lengths, [add] * B, queries([add] * B, 2, 64))
