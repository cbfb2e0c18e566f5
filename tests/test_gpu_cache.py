"""The cache of keys and values in 8 bits: tables and slots, the write, and attention,
against plain forms (integers exact, values in float64).

Tolerances. Codes and scales are exact: a scale is a power of two, so a code is one
rounding of the value. Attention, with y the base-e scores and p = exp(y - max):
the products of the scores are exact, their fp32 sums (at most 128 terms, rounded or cut)
are off by at most d 2^-23 sum |q k| scale, a score's scaling and exponential by a few 2^-22
of |y| + 1: `delta` in a weight's relative error. A weight is rounded to 11 bits (2^-11) or
lost below 2^-35 of its row's largest; with more than 32 rows of a request to a key head, queries lose what
is below 2^-18 of their row's largest value (`split`: d of them); sums over keys are fp32 with at most 2^-24 per key
in a row of additions, LONG keys at most here. The result is rounded to bf16 (2^-8)."""
import pytest
import torch

import block_sparse_attention_token_gb300 as sp

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, **I32)


def word():
    return torch.zeros(1, **I32)


# ------------------------------------------------------------------- tables and slots

def extend_ref(shape, length, add, free, table, tokens, used=0):
    """Request by request."""
    bt, width = shape.bt, len(table[0])
    table, out, start, slots, status, waiting = [list(r) for r in table], [], [0], [], 0, False
    for b, (h, a) in enumerate(zip(length, add)):
        if h < 0 or a < 0 or h + a > width * bt:
            status = status or sp.DATA
            out.append(h)
            start.append(start[-1])
            continue
        have, want = -(-h // bt), -(-(h + a) // bt)
        fits = start[-1] + a <= tokens
        waiting = waiting or used + want - have > len(free)
        refused = not fits or waiting and want > have
        if refused:
            status = status or sp.CAPACITY
        else:
            for j in range(have, want):
                good = 0 <= free[used] < shape.blocks
                status = status if good else status or sp.DATA
                table[b][j] = free[used] if good else -1
                used += 1
        for p in range(h, h + a):
            if len(slots) < tokens:
                page = -1 if refused else table[b][p // bt]
                good = 0 <= page < shape.blocks
                status = status if good or refused else status or sp.DATA
                slots.append(page * bt + p % bt if good else -1)
        out.append(h if refused else h + a)
        start.append(start[-1] + a)
    return table, out, start, slots + [-1] * (tokens - len(slots)), used, status


def extend_case(B, bt, most, new, seed, slack=3, zero=0.2):
    import random
    rng = random.Random(seed)
    length = [rng.choice([0, bt, bt - 1, rng.randint(0, most)]) for _ in range(B)]
    add = [0 if rng.random() < zero else rng.randint(0, new) for _ in range(B)]
    width = max(1, max(-(-(h + a) // bt) for h, a in zip(length, add)))
    have = [-(-h // bt) for h in length]
    need = sum(-(-(h + a) // bt) for h, a in zip(length, add)) - sum(have)
    blocks = sum(have) + need + slack
    order = list(range(blocks))
    rng.shuffle(order)
    table = [[order.pop() for _ in range(n)] + [-7] * (width - n) for n in have]
    return sp.CacheShape(blocks, 2, 64, bt), length, add, order, table, sum(add)


def check_extend(shape, length, add, free, table, tokens, used=0, in_place=False):
    ref = extend_ref(shape, length, add, free, table, tokens, used)
    t, status, ln = i32(table), word(), i32(length)
    u = i32([used]) if used or in_place else None
    got = sp.cache_extend(shape, ln, i32(add), i32(free), t, tokens, used=u, len_out=ln if in_place else None,
                          used_out=u if in_place else None, status=status)
    names = ("table", "length", "start", "slots", "used", "status")
    for name, g, r in zip(names, (t, got[0], got[1], got[2], got[3][0], status[0]), ref):
        assert g.tolist() == r, name
    if in_place:
        assert got[0] is ln and got[3] is u
    return t, got


@pytest.mark.parametrize("B,bt,most,new", [(1, 64, 0, 1), (1, 64, 1000, 5000), (3, 128, 300, 1), (64, 64, 4096, 1),
                                           (33, 64, 500, 777), (1024, 64, 100, 9), (1025, 128, 300, 40), (4096, 64, 300, 127),
                                           (16384, 64, 70, 3)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend(B, bt, most, new, in_place):
    check_extend(*extend_case(B, bt, most, new, B + bt), in_place=in_place)


def test_extend_from_the_middle_of_a_list():
    shape, length, add, free, table, tokens = extend_case(20, 64, 300, 200, 5)
    whole, t = i32([5, 6, 7] + free), i32(table)
    out = sp.cache_extend(shape, i32(length), i32(add), whole[3:], t, tokens)
    ref = extend_ref(shape, length, add, free, table, tokens)
    assert t.tolist() == ref[0] and out[2].tolist() == ref[3] and int(out[3]) == ref[4]


def test_extend_with_too_little_room():
    shape, length, add, free, table, tokens = extend_case(200, 64, 300, 200, 5)
    check_extend(shape, length, add, free[: len(free) // 3], table, tokens)          # too few blocks
    check_extend(shape, length, add, [], table, tokens)                              # none at all
    check_extend(shape, length, add, free, table, tokens, used=len(free))            # all of them used
    check_extend(shape, length, add, free, table, tokens, used=len(free) // 2, in_place=True)
    check_extend(shape, length, add, free, table, tokens // 2 + 1)                   # too few slots
    check_extend(shape, length, add, free, table, 0)
    check_extend(shape, length, add, free, table, tokens + 70)                       # slots to spare


def test_extend_with_bad_data():
    shape, length, add, free, table, tokens = extend_case(50, 64, 300, 200, 6)
    for at, bad_len, bad_add in ((3, -1, 4), (7, 10, -2), (9, len(table[0]) * 64, 1), (11, 2 ** 31 - 1, 2 ** 31 - 1)):
        ln, ad = list(length), list(add)
        ln[at], ad[at] = bad_len, bad_add
        check_extend(shape, ln, ad, free, table, tokens)
    check_extend(shape, length, add, [f if i % 3 else shape.blocks for i, f in enumerate(free)], table, tokens)
    check_extend(shape, length, add, [f if i % 3 else -1 for i, f in enumerate(free)], table, tokens)
    bad = [[-7 if j == 0 else p for j, p in enumerate(r)] for r in table]            # blocks that are half filled
    check_extend(shape, length, add, free, bad, tokens)
    status, used = word(), i32([len(free) + 1])                                      # a place past the list
    out = sp.cache_extend(shape, i32(length), i32(add), i32(free), i32(table), tokens, used=used, status=status)
    assert int(status) == sp.DATA
    ref = extend_ref(shape, length, add, free, table, tokens, len(free))
    assert out[0].tolist() == ref[1] and out[2].tolist() == ref[3]


# ------------------------------------------------------------------- the write

def scale_ref(most):
    """Smallest power of two, at least 2^-100, with most <= 448 scale (float64)."""
    s = torch.full_like(most, 2.0 ** -100)
    for _ in range(230):
        s = torch.where(448 * s < most, 2 * s, s)
    return s


def round_e4m3(x):
    """Nearest e4m3 value of float64 x, ties to even, |x| <= 448."""
    m, e = torch.frexp(x)
    step = torch.exp2(torch.clamp(e - 1, min=-6) - 3.0)
    return torch.round(x / step) * step


def values(codes):
    return codes.view(torch.uint8).view(torch.float8_e4m3fn).double()


def fresh_pool(blocks, heads, d, bt, seed=3):
    """A pool full of what earlier requests left, NaN codes among it."""
    pool = sp.block_pool(blocks, heads, d, bt)
    g = gen(seed)
    for codes, scales in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
        codes.view(torch.uint8).copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda").to(torch.uint8))
        scales.copy_(torch.exp2(torch.randint(-9, -3, scales.shape, generator=g, device="cuda").float()))
    return pool


def write_ref(pool, x, slots, part):
    """(codes as values, scales) after the write, by the definition."""
    codes = values(pool.k if part == 0 else pool.v)
    scales = (pool.k_scale if part == 0 else pool.v_scale).double()
    bt, i, n, slots = pool.shape.bt, 0, len(slots), list(slots)
    x = x.double()
    while i < n:
        if slots[i] < 0 or slots[i] >= pool.shape.blocks * bt:
            i += 1
            continue
        j = i + 1
        while j < n and slots[j] == slots[j - 1] + 1 and slots[j] % bt:
            j += 1
        block, off = slots[i] // bt, slots[i] % bt
        new = x[i:j].transpose(0, 1)
        most = torch.where(new.abs() < float("inf"), new.abs(), 0.0).amax((1, 2))
        s = scale_ref(most)
        if off:
            s = torch.maximum(s, scales[block])
            codes[block, :, :off] = round_e4m3(codes[block, :, :off] * (scales[block] / s)[:, None, None])
        held = round_e4m3(new / s[:, None, None])
        codes[block, :, off:off + j - i] = torch.where(new.abs() < float("inf"), held, float("nan"))
        scales[block] = s
        i = j
    return codes, scales


def same_values(got, ref, what):
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    assert torch.equal(got.nan_to_num(7.0), ref.nan_to_num(7.0)), what


def runs(pool, pieces, seed=0):
    """Slots of runs (offset, count), each in a block of its own."""
    order = torch.randperm(pool.shape.blocks, generator=gen(seed), device="cuda").tolist()
    out = []
    for off, count in pieces:
        block = order.pop()
        out += [block * pool.shape.bt + off + i for i in range(count)]
    return out


@pytest.mark.parametrize("d,bt", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,layout", [(1, "own"), (3, "packed"), (5, "tiles")])
def test_write(d, bt, dtype, heads, layout):
    pool = fresh_pool(40, heads, d, bt)
    pieces = [(0, bt), (0, 1), (bt - 1, 1), (5, 17), (0, bt - 1), (bt // 2, bt // 2), (1, 3)] + [(i, 1) for i in range(20)]
    slots = runs(pool, pieces)
    slots[bt + 1: bt + 1] = [-1, -5]
    n, g = len(slots), gen(1)
    spread = torch.exp2(torch.randint(-12, 6, (n, 1, 1), generator=g, device="cuda").float())
    make = lambda: torch.randn(n, heads, d, generator=g, device="cuda") * spread
    if layout == "packed":
        wide = torch.cat([make() for _ in range(3)], 1).to(dtype)
        k, v = wide[:, heads:2 * heads], wide[:, 2 * heads:]
    elif layout == "tiles":
        k, v = (make().to(dtype).transpose(0, 1).contiguous().transpose(0, 1) for _ in range(2))
    else:
        k, v = make().to(dtype), make().to(dtype)
    k[3] = 0.0                       # within a run
    k[bt] = 0.0                      # a run of zeros
    refs = write_ref(pool, k, slots, 0), write_ref(pool, v, slots, 1)
    status = word()
    for _ in range(2):               # the second call finds the scales as they are and changes nothing
        sp.cache_write(pool, k, v, i32(slots), status=status)
        assert int(status) == 0
        for (codes, scales), got, gs, what in zip(refs, (pool.k, pool.v), (pool.k_scale, pool.v_scale), "kv"):
            assert torch.equal(gs.double(), scales), what + " scales"
            same_values(values(got), codes, what)


def test_write_far_values():
    """The ends of the range, values at the borders of a scale and ties."""
    pool = fresh_pool(8, 1, 64, 64)
    x = torch.zeros(8, 1, 64, device="cuda")
    x[0, 0, :4] = torch.tensor([3e38, -1e30, 1.0, 1e38])
    x[1, 0, :3] = torch.tensor([1e-38, 1e-45, -3e-39])
    x[2, 0, :3] = torch.tensor([448.0, 232.0, -1.0625])       # scale 1, ties
    x[3, 0, :3] = torch.tensor([448.0001, 2.0 ** -9, 2.0 ** -10])
    x[4, 0, :5] = torch.tensor([1.75, 2.0 ** -17, 2.0 ** -18, 3 * 2.0 ** -18, 5 * 2.0 ** -18])   # scale 2^-8: subnormals
    x[5, 0, :2] = torch.tensor([float("nan"), 3.0])
    x[6, 0, :3] = torch.tensor([float("inf"), -float("inf"), 0.5])
    slots = runs(pool, [(0, 1)] * 8)
    ref, status = write_ref(pool, x, slots, 0), word()
    sp.cache_write(pool, x, x.clone(), i32(slots), status=status)
    assert int(status) == sp.DATA
    assert torch.equal(pool.k_scale.double(), ref[1])
    same_values(values(pool.k), ref[0], "k")


def test_write_refuses_slots_outside_and_scales_that_are_none():
    pool = fresh_pool(4, 2, 64, 64)
    before = pool.k.view(torch.uint8).clone()
    x = torch.randn(5, 2, 64, device="cuda")
    status = word()
    sp.cache_write(pool, x, x.clone(), i32([4 * 64, 4 * 64 + 1, 2 ** 31 - 1, -1, -2 ** 31]), status=status)
    assert int(status) == sp.DATA and torch.equal(pool.k.view(torch.uint8), before)
    status.zero_()
    pool.k_scale[1, 0], pool.k_scale[1, 1] = float("nan"), 0.0
    sp.cache_write(pool, x[:2], x[:2].clone(), i32([64 + 10, 64 + 11]), status=status)
    assert int(status) == sp.DATA
    assert torch.equal(pool.k.view(torch.uint8)[1, :, :10], before[1, :, :10])     # left as they were
    assert torch.equal(pool.k_scale[1].double(), scale_ref(x[:2].double().abs().amax((0, 2))))
    sp.cache_write(pool, x[:0], x[:0].clone(), i32([]))                              # nothing to do


# ------------------------------------------------------------------- attention

LONG = 70000


def filled(lengths, heads, d, bt, seed=4, spare=2):
    """A pool in which request b holds lengths[b] tokens; everything else is rubbish, NaN codes
    among it. Returns pool, table, and per request float64 keys and values [heads, n, d]."""
    each = [-(-n // bt) for n in lengths]
    pool = fresh_pool(sum(each) + spare, heads, d, bt, seed)
    g = gen(seed + 1)
    order = torch.randperm(pool.shape.blocks, generator=g, device="cuda").int()
    table = torch.full((len(lengths), max(1, max(each))), 12345678, **I32)
    at, keys = 0, []
    for b, (n, m) in enumerate(zip(lengths, each)):
        page = order[at: at + m]
        table[b, :m] = page
        at += m
        slots = (page.long()[:, None] * bt + torch.arange(bt, device="cuda")).flatten()[:n].int()
        k = torch.randn(n, heads, d, generator=g, device="cuda") * (1 + 2 * torch.rand(n, 1, 1, generator=g, device="cuda"))
        v = torch.randn(n, heads, d, generator=g, device="cuda") + 0.5
        sp.cache_write(pool, k, v, slots)
        pick = lambda c, s: (values(c)[page.long()] * s.double()[page.long()][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
        keys.append((pick(pool.k, pool.k_scale), pick(pool.v, pool.v_scale)))
    return pool, table, keys


def attn_ref(q, keys, add, lengths, scale, causal, bt, chosen=None):
    """O, LSE and their tolerances, request by request."""
    n_all, H, d = q.shape
    O, tol_o = (torch.zeros(n_all, H, d, dtype=torch.float64, device="cuda") for _ in range(2))
    L, tol_l = (torch.zeros(n_all, H, dtype=torch.float64, device="cuda") for _ in range(2))
    at = 0
    for b, (n, total) in enumerate(zip(add, lengths)):
        k, v = keys[b]
        G = H // k.shape[0]
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        qb = q[at: at + n].double().transpose(0, 1)
        y = qb @ k.transpose(1, 2) * scale
        mag = (qb.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale) if total else torch.zeros(H, n, 1, device="cuda")
        pos = torch.arange(total, device="cuda")
        see = torch.ones(H, n, total, dtype=torch.bool, device="cuda")
        if causal:
            see &= pos <= total - n + torch.arange(n, device="cuda")[:, None]
        if chosen is not None:
            see &= chosen[b].repeat_interleave(bt, 1)[:, :total].repeat_interleave(G, 0)[:, None]
        y = y.masked_fill(~see, -float("inf"))
        top = y.amax(-1, keepdim=True) if total else torch.full((H, n, 1), -float("inf"), dtype=torch.float64, device="cuda")
        top = torch.where(torch.isinf(top), 0.0, top)
        p = torch.exp(y - top)
        l = p.sum(-1, keepdim=True)
        safe = torch.where(l > 0, l, 1.0)
        delta = d * 2.0 ** -23 * mag + 2.0 ** -19 * (1 + mag)
        if n * G > 32 and total:
            split = qb.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax(-1)[:, None, None] * 2.0 ** -18
            delta = delta + split * abs(scale)
        spread = (p @ v.abs()) / safe
        o = p @ v / safe
        lost = total * 2.0 ** -35 * (v.abs().amax() if total else 0.0)
        O[at: at + n] = o.transpose(0, 1)
        L[at: at + n] = (top + torch.log(l)).squeeze(-1).T
        tol_o[at: at + n] = (2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * delta + total * 2.0 ** -24) * spread * 1.01 + lost).transpose(0, 1)
        tol_l[at: at + n] = (delta + total * 2.0 ** -24 + 2.0 ** -20 * (1 + top.abs())).squeeze(-1).T
        at += n
    return O, L, tol_o, tol_l


def csr(chosen):
    counts = torch.cat([c.sum(1) for c in chosen])
    row_ptr = torch.zeros(counts.numel() + 1, **I32)
    row_ptr[1:] = counts.cumsum(0)
    col = torch.cat([c.nonzero()[:, 1] for c in chosen]).int()
    return row_ptr, torch.cat([col, i32([99] * 4)])


def check_attn(lengths, add, heads, group, d, bt, causal, density=None, seed=7, behind=3, q_scale=1.0, grow=1):
    pool, table, keys = filled(lengths, heads, d, bt, seed)
    g, H, n = gen(seed + 2), heads * group, sum(add)
    wide = (torch.randn(n + behind, H + 2 * heads, d, generator=g, device="cuda") * q_scale).bfloat16()
    q = wide[:, :H]
    start, ln = i32([0] + add).cumsum(0).int(), i32(lengths)
    chosen = row_ptr = col = None
    if density is not None:
        chosen = [torch.rand(heads, -(-t // bt), generator=g, device="cuda") < density for t in lengths]
        row_ptr, col = csr(chosen)
    o = torch.full((n + behind, H, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((n + behind, H), 7.0, device="cuda")
    status = word()
    args = dict(causal=causal, row_ptr=row_ptr, col_idx=col, status=status)
    sp.attn_cache_fwd(pool, q, start, ln, table, max(1, max(add)) * grow, o=o, lse=lse, **args)
    assert int(status) == 0
    O, L, to, tl = attn_ref(q[:n], keys, add, lengths, d ** -0.5, causal, bt, chosen)
    assert (o[n:] == 7.0).all() and (lse[n:] == 7.0).all()          # rows behind the last request
    err = (o[:n].double() - O).abs()
    assert (err <= to).all(), f"O: {int((~(err <= to)).sum())} off, worst {float((err / to).max()):.2f} of tol"
    none = torch.isinf(L)
    assert torch.equal(torch.isinf(lse[:n]), none) and (lse[:n][none] < 0).all() and (o[:n][none] == 0).all()
    assert ((lse[:n].double() - L).abs()[~none] <= tl[~none]).all(), "LSE"
    again = sp.attn_cache_fwd(pool, q, start, ln, table, max(1, max(add)) * grow, **args)
    assert torch.equal(again[0][:n], o[:n]) and torch.equal(again[1][:n], lse[:n])
    return pool, table, start, ln, q


@pytest.mark.parametrize("d,bt", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 8)])
def test_attn_single_tokens(d, bt, heads, group):
    check_attn([1, 2, 63, 64, 65, 127, 128, 129, 200, 1000, 16, 17], [1] * 12, heads, group, d, bt, True)


@pytest.mark.parametrize("d,bt", [(64, 128), (128, 64)])
@pytest.mark.parametrize("heads,group,add", [(2, 1, [1, 0, 5, 2, 8]), (1, 4, [3, 2, 0, 1, 4]), (2, 3, [5, 5, 1, 0, 2]),
                                             (1, 2, [20, 1, 33, 7, 0])])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("density", [None, 0.4])
def test_attn_few_tokens(d, bt, heads, group, add, causal, density):
    check_attn([5, 77, 300, 129, 640], add, heads, group, d, bt, causal, density)


@pytest.mark.parametrize("d", [64, 128])
def test_attn_one_long_request(d):
    """One item spans every CTA; a few keys carry most of the weight."""
    check_attn([LONG - 5], [1], 1, 1, d, 64, True, q_scale=3.0)
    check_attn([LONG // 2 + 3], [3], 2, 1, d, 128, True, q_scale=0.3)


def test_attn_many_requests():
    import random
    rng = random.Random(3)
    lengths = [rng.randint(1, 150) for _ in range(700)]
    check_attn(lengths, [rng.randint(0, 1) for _ in lengths], 1, 1, 64, 64, True)


def test_attn_no_keys():
    """Requests without tokens, rows before the first token, empty lists."""
    check_attn([0, 3, 0, 70], [2, 5, 0, 1], 2, 2, 64, 64, True)      # 5 rows of 3 tokens: two see nothing
    check_attn([0, 0], [1, 3], 1, 1, 128, 128, False)
    check_attn([130, 64], [1, 2], 2, 1, 64, 64, True, density=0.0)


@pytest.mark.parametrize("d,bt", [(64, 64), (128, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_attn_whole_frames(d, bt, causal):
    check_attn([700, 1, 450], [300, 1, 129], 2, 1, d, bt, causal)
    check_attn([513], [513], 1, 3, d, bt, causal)
    check_attn([513], [200], 3, 1, d, bt, causal, density=0.5)


@pytest.mark.parametrize("add", [[2, 1], [90, 1], [33, 128]])
@pytest.mark.parametrize("d,bt", [(128, 64), (64, 128)])
def test_attn_wide_scales(add, d, bt):
    """Values whose scales lie far apart from block to block, rows of large and tiny queries."""
    heads, lengths = 2, [260, 128]
    pool, table, _ = filled(lengths, heads, d, bt)
    g = gen(11)
    for s in (pool.k_scale, pool.v_scale):
        s.mul_(torch.exp2(torch.randint(-20, 3, s.shape, generator=g, device="cuda").float()) * 1.37)
    keys = []
    for b, n in enumerate(lengths):
        page = table[b, : -(-n // bt)].long()
        keys.append(tuple((values(c)[page] * s.double()[page][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
                          for c, s in ((pool.k, pool.k_scale), (pool.v, pool.v_scale))))
    q = torch.randn(sum(add), 4, d, generator=g, device="cuda")
    q[0] *= 1e-6
    q[1] *= 50.0
    q[2, 0] = 0.0
    q[2, 1, ::2] *= 2.0 ** -16      # half the columns far below the others
    q = q.bfloat16()
    o, lse = sp.attn_cache_fwd(pool, q, i32([0] + add).cumsum(0).int(), i32(lengths), table, max(add))
    O, L, to, tl = attn_ref(q, keys, add, lengths, d ** -0.5, True, bt)
    assert ((o.double() - O).abs() <= to).all() and ((lse.double() - L).abs() <= tl).all()


@pytest.mark.parametrize("add", [[1, 2, 1], [1, 80, 1], [90, 5, 33]])
def test_attn_not_finite(add):
    """NaN and infinities in a row's own query, or in a key that it sees, give NaN there and only there."""
    lengths, n = [100, 90, 100], sum(add)
    pool, table, start, ln, q = check_attn(lengths, add, 1, 4, 64, 64, True)
    clean, lc = sp.attn_cache_fwd(pool, q, start, ln, table, max(add))
    bad = q.clone()
    bad[1, 2, 5], bad[2, 0, 7], bad[n - 1, 3, 0] = float("nan"), float("inf"), -float("inf")
    o, lse = sp.attn_cache_fwd(pool, bad, start, ln, table, max(add))
    hit = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
    hit[1, 2] = hit[2, 0] = hit[n - 1, 3] = True
    assert torch.isnan(o[:n][hit]).all() and torch.isnan(lse[:n][hit]).all()
    assert torch.equal(o[:n][~hit], clean[:n][~hit]) and torch.equal(lse[:n][~hit], lc[:n][~hit])
    pool.k.view(torch.uint8)[table[2, 0], 0, 3, 9] = 0x7f      # a key of the last request
    o, lse = sp.attn_cache_fwd(pool, q, start, ln, table, max(add))
    mine = slice(n - add[2], n)
    assert torch.isnan(o[mine]).all() and torch.isnan(lse[mine]).all()
    assert torch.equal(o[: n - add[2]], clean[: n - add[2]]) and torch.equal(lse[: n - add[2]], lc[: n - add[2]])


@pytest.mark.parametrize("add", [[1, 2, 1], [1, 70, 1], [20, 2, 300]])
def test_attn_bad_data(add):
    lengths, n, most = [100, 200, 300], sum(add), max(add)
    one, two, three = slice(0, add[0]), slice(add[0], add[0] + add[1]), slice(add[0] + add[1], n)
    s1, s2 = add[0], add[0] + add[1]
    pool, table, start, ln, q = check_attn(lengths, add, 2, 2, 64, 64, True)
    want = sp.attn_cache_fwd(pool, q, start, ln, table, most)

    # the work is dealt out by the lengths of the whole call, so that the others' rows may be summed in
    # another order: two results, each within 2^-8 |o| + (2^-11 + delta) max |v| of the same value
    near = lambda x, y: torch.allclose(x.float(), y.float(), atol=2.0 ** -6, rtol=2.0 ** -7)

    def call(start=start, ln=ln, table=table, max_add=most, **kw):
        o, lse = torch.full_like(want[0], 5.0), torch.full_like(want[1], 5.0)
        status = word()
        sp.attn_cache_fwd(pool, q, start, ln, table, max_add, o=o, lse=lse, status=status, **kw)
        return o, lse, int(status)

    for page in (pool.shape.blocks, -1, 2 ** 31 - 1, -2 ** 31):       # a bad page: its keys are left out
        bad = table.clone()
        bad[1, 1] = page
        o, lse, st = call(table=bad)
        assert st == sp.DATA
        seen = [torch.ones(2, -(-n // 64), dtype=torch.bool, device="cuda") for n in lengths]
        seen[1][:, 1] = False
        row_ptr, col = csr(seen)
        o2, lse2, st2 = call(row_ptr=row_ptr, col_idx=col)
        assert st2 == 0
        assert near(o[two], o2[two]) and near(o[one], want[0][one]) and near(o[three], want[0][three])
    for bad_len in (-1, 2 ** 31 - 1, table.shape[1] * 64 + 1):        # a bad length counts as 0
        o, lse, st = call(ln=i32([100, bad_len, 300]))
        assert st == sp.DATA and (o[two] == 0).all() and torch.isinf(lse[two]).all()
        assert near(o[three], want[0][three])
    for s in ([0, s1, s2, 2 ** 31 - 1], [0, s1, n, s2], [-1, s1, s2, n], [0, s1, s2, 1000], [-2 ** 31, s1, s2, n]):   # rows that are none: left out
        o, lse, st = call(start=i32(s))
        assert st == sp.DATA and torch.equal(o[n:], torch.full_like(o[n:], 5.0))
    o, lse, st = call(max_add=most - 1)                               # more rows than announced
    over = [p for p, a in zip((one, two, three), add) if a == most][0]
    assert st == sp.DATA and (o[over] == 5).all()
    assert all(near(o[p], want[0][p]) for p in (one, two, three) if p is not over)
    seen = [torch.ones(2, -(-n // 64), dtype=torch.bool, device="cuda") for n in lengths]
    row_ptr, col = csr(seen)
    for at, v in ((3, 4), (4, -1), (5, 2 ** 31 - 1)):                 # blocks without tokens: left out
        c = col.clone()
        c[at] = v
        o, lse, st = call(row_ptr=row_ptr, col_idx=c)
        assert st == sp.DATA and torch.isfinite(o.float()).all()
        assert near(o[three], want[0][three])
    for at, v in ((2, 0), (2, 2 ** 31 - 1), (6, 1000), (3, -4)):      # rows of lists that make no sense: empty
        r = row_ptr.clone()
        r[at] = v
        o, lse, st = call(row_ptr=r, col_idx=col)
        assert st == sp.DATA and torch.isfinite(o.float()).all() and near(o[one, :2], want[0][one, :2])


def test_attn_stream_capture_and_two_graphs():
    lengths, add = [1000, 300, 64], [1, 1, 1]
    pool, table, start, ln, q = check_attn(lengths, add, 2, 2, 128, 64, True, behind=0)
    want = sp.attn_cache_fwd(pool, q, start, ln, table, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sp.attn_cache_fwd(pool, q, start, ln, table, 1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # two graphs that share a workspace, replayed in turn, lengths and queries changed between
    ws = torch.empty(sp.attn_cache_workspace_size(pool.shape, 3, 4, 3, 1, table.shape[1]), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for scale in (0.0, 0.5):
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sp.attn_cache_fwd(pool, q, start, ln, table, 1, scale, o=o, lse=lse, ws=ws)
        graphs.append(graph)
        outs.append((o, lse))
    for lengths in ([1000, 300, 64], [1, 299, 0], [777, 65, 63]):
        ln.copy_(i32(lengths))
        for graph in graphs * 2:
            graph.replay()
        for scale, (o, lse) in zip((0.0, 0.5), outs):
            ref = sp.attn_cache_fwd(pool, q, start, ln, table, 1, scale)
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_attn_many_rows_stream_and_two_graphs():
    """As above, for requests of many rows and of few in one call, the two graphs on streams of their own."""
    lengths, add = [1000, 300, 64], [150, 1, 40]
    pool, table, start, ln, q = check_attn(lengths, add, 2, 2, 128, 64, True, behind=0)
    graphs, outs, sides = [], [], [torch.cuda.Stream() for _ in range(2)]
    for scale in (0.0, 0.5):
        o, lse = torch.empty(191, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(191, 4, device="cuda")
        ws = torch.empty(sp.attn_cache_workspace_size(pool.shape, 3, 4, 191, 150, table.shape[1]), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sp.attn_cache_fwd(pool, q, start, ln, table, 150, scale, o=o, lse=lse, ws=ws)
        graphs.append(graph)
        outs.append((o, lse, ws))
    for lengths in ([1000, 300, 64], [151, 299, 40], [777, 65, 63]):
        ln.copy_(i32(lengths))
        for side, graph in zip(sides, graphs):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph.replay()
                graph.replay()
        for side in sides:
            torch.cuda.current_stream().wait_stream(side)
        for scale, (o, lse, _) in zip((0.0, 0.5), outs):
            ref = sp.attn_cache_fwd(pool, q, start, ln, table, 150, scale)
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("add", [1, 100])
def test_far_offsets(add):
    """A pool of more than 2^32 bytes of codes: the same as a small one whose blocks hold the same."""
    n, heads, d, bt, g = 300, 30, 128, 128, gen(8)
    k, v = (torch.randn(n, heads, d, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(add, heads, d, generator=g, device="cuda").bfloat16()
    results, codes = [], []
    for blocks, page in ((9000, [8999, 3, 8998]), (3, [2, 0, 1])):
        pool, table = sp.block_pool(blocks, heads, d, bt), i32([page])
        slots = (table[0].long()[:, None] * bt + torch.arange(bt, device="cuda")).flatten()[:n].int()
        sp.cache_write(pool, k, v, slots)
        codes.append([t.view(torch.uint8)[page] for t in (pool.k, pool.v)] + [t[page] for t in (pool.k_scale, pool.v_scale)])
        results.append(sp.attn_cache_fwd(pool, q, i32([0, add]), i32([n]), table, add))
        del pool
    for a, b in zip(codes[0] + list(results[0]), codes[1] + list(results[1])):
        assert torch.equal(a, b)
    assert 9000 * heads * d * bt > 2 ** 32


def test_no_tokens():
    """A step in which nothing is new."""
    pool, status = fresh_pool(4, 2, 64, 64), word()
    before = [t.clone() for t in (pool.k.view(torch.uint8), pool.k_scale, pool.v.view(torch.uint8), pool.v_scale)]
    ln, start, slots, used = sp.cache_extend(pool.shape, i32([5, 0]), i32([0, 0]), i32([]), i32([[1], [2]]), 0, status=status)
    assert ln.tolist() == [5, 0] and start.tolist() == [0, 0, 0] and slots.numel() == 0 and int(used) == 0
    x = torch.empty(0, 2, 64, device="cuda")
    sp.cache_write(pool, x, x, slots, status=status)
    o, lse = sp.attn_cache_fwd(pool, x.bfloat16(), start, ln, i32([[1], [2]]), 1, status=status)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2) and int(status) == 0
    for a, b in zip(before, (pool.k.view(torch.uint8), pool.k_scale, pool.v.view(torch.uint8), pool.v_scale)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------- as they are used together

@pytest.mark.parametrize("heads,group,d,bt", [(2, 2, 64, 64), (3, 1, 128, 128)])
def test_generation(heads, group, d, bt):
    """Requests that start at different steps and grow by whole chunks and single tokens: norm
    and rotation of the new tokens, tables and slots, the write, attention; against
    attention in float64 over the values that the cache holds and, with the error of 8 bits
    (2^-4 of a value, 2^-10 of a block's largest, either way), over the values before."""
    B, H, width = 4, heads * group, 12
    pool = fresh_pool(B * width, heads, d, bt)
    free = torch.randperm(pool.shape.blocks, generator=gen(1), device="cuda").int()
    table = torch.full((B, width), -1, **I32)
    length, used, status = i32([0] * B), word(), word()
    g = gen(2)
    shape1 = sp.make_shape(1, H, 1, 1, 1, d, 1, 1, 1, "bf16")
    rope = sp.rope_table(shape1, (d, 0, 0), extent=(width * bt, 1, 1))
    w = [1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    past = [(torch.zeros(heads, 0, d, device="cuda"), torch.zeros(heads, 0, d, device="cuda")) for _ in range(B)]
    total = [0] * B
    for add in ([5, 0, 150, 1], [1, 70, 1, 1], [1, 1, 1, 1], [1, 1, 200, 0], [3, 64, 1, 1], [1, 1, 1, 1]):
        n = sum(add)
        x = torch.randn(1, n, H + 2 * heads, d, generator=g, device="cuda").bfloat16()
        pos = torch.zeros(1, n, 3, **I32)
        pos[0, :, 0] = torch.cat([torch.arange(t, t + a, device="cuda") for t, a in zip(total, add)])
        s = sp.make_shape(1, H, n, 1, 1, d, 1, 1, 1, "bf16")
        q, k = sp.norm_rope_fwd(s, rope, x[:, :, :H], x[:, :, H:H + heads], *w, rms=True, pos=pos, out_blocked=False,
                                status=status)
        v = x[0, :, H + heads:]
        _, start, slots, _ = sp.cache_extend(pool.shape, length, i32(add), free, table, n, used=used, len_out=length,
                                             used_out=used, status=status)
        sp.cache_write(pool, k[0], v, slots, status=status)
        o, lse = sp.attn_cache_fwd(pool, q[0], start, length, table, max(add), status=status)
        assert int(status) == 0
        total = [t + a for t, a in zip(total, add)]
        assert length.tolist() == total
        held, at = [], 0
        for b, a in enumerate(add):
            past[b] = tuple(torch.cat([old, new[at: at + a].float().transpose(0, 1)], 1) for old, new in zip(past[b], (k[0], v)))
            at += a
            page = table[b, : -(-total[b] // bt)].long()
            held.append(tuple((values(c)[page] * sc.double()[page][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :total[b]]
                              for c, sc in ((pool.k, pool.k_scale), (pool.v, pool.v_scale))))
            for was, now in zip(past[b], held[b]):
                if total[b]:
                    near = (now - was).abs() <= 2 * (2.0 ** -4 * was.double().abs() + 2.0 ** -10 * was.abs().amax((1, 2), keepdim=True))
                    assert near.all()
        O, L, to, tl = attn_ref(q[0], held, add, total, d ** -0.5, True, bt)
        assert ((o.double() - O).abs() <= to).all() and ((lse.double() - L).abs() <= tl).all()
    assert int(used) == sum(-(-t // bt) for t in total)
