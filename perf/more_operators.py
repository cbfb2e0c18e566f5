"""Cases that time the operators of generation with a block cache: the per-head norm of
queries and keys with the rotary positions in the same pass (and its backward), block
tables and slots from request lengths, the write of new keys and values into a cache
held in 8 bits, and attention over that cache. Each case runs in a plain form
(elementary torch operations in fp32) or, where `own` is true, through this package's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# ------------------------------------------------------------------- cases


def listed():
    return [
        # one step of serving: a token of each of 64 requests, queries sharing key heads; latency
        dict(name="qk_fwd_64_tokens", op="qk", bwd=False, B=1, H=32, Hk=8, grid="64x1x1", tile="", d=128, dtype="bf16",
             rms=True, half=True, positions=True, packed=True, means=False),
        # a 30k-token clip of 40 heads out of the fused projection, into tile order with the tile means
        dict(name="qk_fwd_30k", op="qk", bwd=False, B=1, H=40, Hk=40, grid="20x32x48", tile="2x8x8", d=128,
             dtype="bf16", rms=True, half=False, positions=False, packed=True, means=True),
        # the same clip in training: gradients in raster order, into the fused projection's gradient
        dict(name="qk_bwd_30k", op="qk", bwd=True, B=1, H=40, Hk=40, grid="20x32x48", tile="2x8x8", d=128,
             dtype="bf16", rms=True, half=False, positions=False, packed=True, means=False),
        # training on 8k-token clips in fp32, layer norm with biases, d = 64
        dict(name="qk_bwd_8k_f32", op="qk", bwd=True, B=1, H=12, Hk=12, grid="8x32x32", tile="4x4x4", d=64,
             dtype="f32", rms=False, half=False, positions=True, packed=False, means=False),
        # the tables of one serving step: a token more for each of 64 requests
        dict(name="extend_64_tokens", op="extend", B=64, most=4096, new=1, bt=64, mix=1),
        # a step that admits many requests of up to a few hundred tokens
        dict(name="extend_4k_requests", op="extend", B=4096, most=1024, new=127, bt=64, mix=2),
        # the write of one serving step: a token of each of 256 requests, most into half-filled blocks
        dict(name="write_256_tokens", op="write", B=256, most=2048, new=1, bt=64, Hk=8, d=128, dtype="bf16",
             packed=True, mix=3),
        # the write of a whole 30k-token clip of 40 heads
        dict(name="write_30k", op="write", B=1, most=0, new=30720, bt=128, Hk=40, d=128, dtype="bf16", packed=True,
             mix=4),
        # one token over one short request: the smallest call, latency
        dict(name="attn_one_1k", op="attn", B=1, most=1024, even=True, new=1, H=12, Hk=12, d=64, bt=64, causal=True,
             density=0.0, mix=5),
        # a token of each of 64 requests of very uneven length, four queries to a key head
        dict(name="attn_64_uneven", op="attn", B=64, most=32768, even=False, new=1, H=32, Hk=8, d=128, bt=64,
             causal=True, density=0.0, mix=6),
        # a few tokens over long caches, a tenth of the blocks of each head
        dict(name="attn_8_long_sparse", op="attn", B=8, most=131072, even=True, new=4, H=32, Hk=8, d=128, bt=128,
             causal=True, density=0.1, mix=7),
        # the next frame of a 30k-token clip: 1,536 queries of 40 heads that see the cache and one another
        dict(name="attn_frame_30k", op="attn", B=1, most=30720, even=True, new=1536, H=40, Hk=40, d=128, bt=128,
             causal=False, density=0.0, mix=8),
    ]


_TILES = [(4, 4, 4), (1, 8, 8), (2, 4, 8), (2, 8, 8), (8, 4, 4), (1, 8, 16)]


def _text(sizes):
    return "x".join(str(v) for v in sizes)


def _sizes(text):
    return [int(v) for v in text.split("x")]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_grid(rng, n_lo, n_hi):
    """A tile and a grid of whole tiles with about n_lo .. n_hi tokens, odd tile counts among them."""
    tile = rng.choice(_TILES)
    bt = tile[0] * tile[1] * tile[2]
    blocks = max(1, _log_int(rng, n_lo, n_hi) // bt)
    c = [1, 1, 1]
    while c[0] * c[1] * c[2] < blocks:
        a = rng.randrange(3)
        if (c[0] * c[1] * c[2]) // c[a] * (c[a] + 1) > blocks:
            break
        c[a] += 1
    return [c[i] * tile[i] for i in range(3)], tile


def _draw_heads(rng, most=40):
    """Query heads and key heads, one to eight of the first to one of the second."""
    group = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
    hk = max(1, _log_int(rng, 1, max(1, most // group)))
    return hk * group, hk


def draw(rng):
    """One more case of the listed ranges: single tokens to whole clips, 1 to 40 heads, 1 to 4,096 requests."""
    op = rng.choice(["qk", "qk", "extend", "write", "attn", "attn", "attn"])
    mix = rng.randrange(1 << 30)
    d = rng.choice([64, 128])
    if op == "qk":
        H, Hk = _draw_heads(rng)
        bwd = rng.random() < 0.5
        base = dict(op=op, bwd=bwd, H=H, Hk=Hk, d=d, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    rms=rng.random() < 0.5, half=rng.random() < 0.4, packed=rng.random() < 0.5)
        if rng.random() < 0.4:   # tokens of a batch of requests, no grid
            return dict(base, B=1, grid="%dx1x1" % _log_int(rng, 1, 8192), tile="", positions=True, means=False)
        most = min(65536, 30720 * 40 * 128 // (2 * max(H, Hk) * d) if base["dtype"] == "f32" else
                   30720 * 40 * 128 // (max(H, Hk) * d))
        grid, tile = _draw_grid(rng, 64, most)
        return dict(base, B=1 if grid[0] * grid[1] * grid[2] * 2 > most else rng.choice([1, 2]), grid=_text(grid),
                    tile=_text(tile), positions=rng.random() < 0.4, means=not bwd and rng.random() < 0.7)
    bt = rng.choice([64, 128])
    if op == "extend":
        B = _log_int(rng, 1, 4096)
        return dict(op=op, B=B, most=_log_int(rng, 1, 16384 if B < 256 else 1024),
                    new=_log_int(rng, 1, max(1, min(8192, 262144 // B))), bt=bt, mix=mix)
    H, Hk = _draw_heads(rng)
    if op == "write":
        B = _log_int(rng, 1, 256)
        new = _log_int(rng, 1, max(1, int(30720 * 40 * 128 / (Hk * d * B))))
        return dict(op=op, B=B, most=_log_int(rng, 1, 2048), new=min(new, 32768), bt=bt, Hk=Hk, d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]) if B * new * Hk * d < 50000000 else "bf16",
                    packed=rng.random() < 0.5, mix=mix)
    B = _log_int(rng, 1, 64)
    most = _log_int(rng, 1, min(131072, max(1, (1 << 31) // (B * Hk * d * 4))))
    # the pairs of the frame case at most
    new = max(1, min(_log_int(rng, 1, 2048), int(1536 * 30720 * 40 * 128 / (B * H * d * most)), most))
    if rng.random() < 0.5:
        new = min(new, rng.randint(1, 4))
    return dict(op=op, B=B, most=most, even=rng.random() < 0.3, new=new, H=H, Hk=Hk, d=d, bt=bt,
                causal=rng.random() < 0.6, density=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 3)]), mix=mix)


# ------------------------------------------------------------------- shapes

EPS = 1e-6
THETA = 10000.0


def _torch_dtype(case):
    return torch.float32 if case.get("dtype", "bf16") == "f32" else torch.bfloat16


def _ceil(a, b):
    return -(-a // b)


def _sections(d):
    """Columns of the time, height and width axes: the height and width axes get 2 * (d // 6) each."""
    side = 2 * (d // 6)
    return d - 2 * side, side, side


def _columns(case):
    """Without a grid (tokens of requests) every column turns with the one position."""
    return _sections(case["d"]) if case["tile"] else (case["d"], 0, 0)


def _grid(case):
    T, Y, X = _sizes(case["grid"])
    bt = math.prod(_sizes(case["tile"])) if case["tile"] else 0
    return T * Y * X, bt


def _block_order(case, device):
    """Raster token index of every token in tile order."""
    (T, Y, X), (a, b, c) = _sizes(case["grid"]), _sizes(case["tile"])
    n = torch.arange(T * Y * X, device=device).view(T // a, a, Y // b, b, X // c, c)
    return n.permute(0, 2, 4, 1, 3, 5).reshape(-1)


def _requests(case):
    """Per request the tokens held before the step and the new ones, of the case alone."""
    rng = random.Random(case["mix"])
    B, most, new = case["B"], case["most"], case["new"]
    if case["op"] == "attn":
        add = [new if B == 1 else rng.randint(1, new) for _ in range(B)]
        held = [most if case["even"] else _log_int(rng, 1, most) for _ in range(B)]
        return [max(0, h - a) for h, a in zip(held, add)], add
    held = [_log_int(rng, 1, most) if most else 0 for _ in range(B)]
    # mostly `new` at most; where many requests come, some bring nothing
    add = [new if new == 1 or B == 1 else rng.randint(0, new) for _ in range(B)]
    return held, [max(1, add[0])] + add[1:]


def _width(case):
    held, add = _requests(case)
    return max(1, max(_ceil(h + a, case["bt"]) for h, a in zip(held, add)))


def _rows_seen(case, b, held, add):
    """Keys that each new token of request b may see."""
    return [held[b] + i + 1 if case["causal"] else held[b] + add[b] for i in range(add[b])]


def _picks(case, blocks):
    """How many blocks of a row of that many a list takes."""
    return blocks if case["density"] == 0.0 else max(1, int(round(case["density"] * blocks)))


def work(case):
    e = 4 if case.get("dtype", "bf16") == "f32" else 2
    if case["op"] == "qk":
        n, bt = _grid(case)
        values = case["B"] * n * (case["H"] + case["Hk"]) * case["d"]
        params = 4 * case["d"] * (2 if case["rms"] else 4)
        pos = 12 * case["B"] * n if case["positions"] else 0
        means = 4 * values // bt if case["means"] else 0
        if case["bwd"]:
            return {"bytes": 3 * e * values + 2 * params + pos, "flops": 20 * values}
        return {"bytes": 2 * e * values + params + pos + means, "flops": 9 * values}
    held, add = _requests(case)
    if case["op"] == "extend":
        fresh = sum(_ceil(h + a, case["bt"]) - _ceil(h, case["bt"]) for h, a in zip(held, add))
        return {"bytes": 4 * (4 * case["B"] + 2 * fresh + sum(add)), "flops": 10 * case["B"] + 2 * sum(add)}
    if case["op"] == "write":
        values = 2 * sum(add) * case["Hk"] * case["d"]
        touched = sum(_ceil(h + a, case["bt"]) - h // case["bt"] for h, a in zip(held, add) if a)
        return {"bytes": (e + 1) * values + 4 * sum(add) + 16 * touched * case["Hk"], "flops": 3 * values}
    keys = pairs = 0
    for b in range(case["B"]):
        blocks = _ceil(held[b] + add[b], case["bt"])
        share = _picks(case, blocks) / max(1, blocks)
        keys += share * (held[b] + add[b])
        pairs += share * sum(_rows_seen(case, b, held, add))
    rows = sum(add) * case["H"]
    return {"bytes": int(2 * keys * case["Hk"] * case["d"] * (1 + 4 / (case["bt"] * case["d"]))
                         + rows * (4 * case["d"] + 4)),
            "flops": int(4 * case["d"] * case["H"] * pairs)}


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"qk": _prepare_qk, "extend": _prepare_extend, "write": _prepare_write, "attn": _prepare_attn}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_qk(case, g):
    n, bt = _grid(case)
    B, d, dt = case["B"], case["d"], _torch_dtype(case)
    heads = (case["H"], case["Hk"])
    rows = sum(heads) + heads[1] if case["packed"] else 0     # queries, keys and values of a token side by side
    st = dict(case=case, x=[], w=[], b=[], dy=[])
    if case["packed"]:
        # activations of a projection: unit scale, an offset per channel
        x = torch.empty(B, n, rows, d, device="cuda", dtype=dt)
        x[:, :, : sum(heads)] = (_randn(g, B, n, sum(heads), d) + 0.5 * _randn(g, sum(heads), d)).to(dt)
        st["x"] = [x[:, :, : heads[0]], x[:, :, heads[0]: sum(heads)]]
    else:
        st["x"] = [(_randn(g, B, n, h, d) + 0.5 * _randn(g, h, d)).to(dt) for h in heads]
    for h in heads:
        st["w"].append(1.0 + 0.2 * _randn(g, d))
        st["b"].append(None if case["rms"] else 0.1 * _randn(g, d))
        if case["bwd"]:
            st["dy"].append((0.1 * _randn(g, B, n, h, d)).to(dt))
    T, Y, X = _sizes(case["grid"])
    st["pos"] = None
    if not case["tile"]:
        # tokens of requests: each at its own place in a long sequence
        st["extent"] = (65536, 1, 1)
        st["pos"] = torch.zeros(B, n, 3, dtype=torch.int32, device="cuda")
        st["pos"][..., 0] = torch.randint(0, 65536, (B, n), generator=g, device="cuda")
    elif case["positions"]:
        # packed clips: the frame index starts over, the frame is shifted inside the table
        shift = torch.randint(0, 4, (B, 1, 3), generator=g, device="cuda")
        tok = torch.arange(n, device="cuda")
        grid = torch.stack([tok // (Y * X) % max(1, T // 2), tok // X % Y, tok % X], -1)
        st["pos"], st["extent"] = (grid[None] + shift).int().contiguous(), (T + 4, Y + 4, X + 4)
    else:
        st["extent"] = (T, Y, X)
    if own:
        import block_sparse_attention_token_gb300 as sp
        tile = _sizes(case["tile"]) if case["tile"] else (1, 1, 1)
        st["shape"] = s = sp.make_shape(B, case["H"], T, Y, X, d, *tile, case["dtype"])
        st["table"] = sp.rope_table(s, _columns(case), THETA, extent=st["extent"], half=case["half"])
        if case["bwd"]:
            # the gradient of the fused projection, or tensors of their own
            if case["packed"]:
                dx = torch.zeros(B, n, rows, d, device="cuda", dtype=dt)
                st["out"] = [dx[:, :, : heads[0]], dx[:, :, heads[0]: sum(heads)]]
            else:
                st["out"] = [torch.empty(B, n, h, d, device="cuda", dtype=dt) for h in heads]
            st["dw"] = [torch.empty(d, device="cuda") for _ in heads]
            st["db"] = [None if case["rms"] else torch.empty(d, device="cuda") for _ in heads]
            st["ws"] = torch.empty(sp.norm_rope_workspace_size(s, case["Hk"]), dtype=torch.uint8, device="cuda")
        else:
            st["out"] = [torch.empty((B, h, n, d) if case["tile"] else (B, n, h, d), device="cuda", dtype=dt)
                         for h in heads]
            st["means"] = [torch.empty(B, h, n // bt, d, device="cuda") if case["means"] else None for h in heads]
    else:
        st["angles"] = []
        for ext, cols in zip(st["extent"], _columns(case)):
            freq = THETA ** (-torch.arange(0, cols, 2, dtype=torch.float64, device="cuda") / max(cols, 1))
            ang = torch.arange(ext, dtype=torch.float64, device="cuda")[:, None] * freq
            st["angles"].append((ang.cos().float(), ang.sin().float()))
        st["order"] = _block_order(case, "cuda") if case["tile"] else None
    return st


def _prepare_extend(case, g):
    held, add = _requests(case)
    B, bt, width = case["B"], case["bt"], _width(case)
    held_blocks = [_ceil(h, bt) for h in held]
    fresh = sum(_ceil(h + a, bt) - n for h, a, n in zip(held, add, held_blocks))
    # a pool about a quarter larger than needed, its blocks handed out in any order; now and then too small
    blocks = sum(held_blocks) + fresh + max(1, fresh // 4)
    order = torch.randperm(blocks, generator=g, device="cuda").int()
    st = dict(case=case, blocks=blocks, n=sum(add))
    st["len"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    st["add"] = torch.tensor(add, dtype=torch.int32, device="cuda")
    st["table"] = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    own_blocks = torch.tensor(held_blocks, device="cuda")
    mine = torch.arange(width, device="cuda") < own_blocks[:, None]
    st["table"][mine] = order[: sum(held_blocks)]
    st["free"] = order[sum(held_blocks):].contiguous()
    if case["mix"] % 5 == 0 and fresh > 1:
        st["free"] = st["free"][: fresh // 2].contiguous()
    if own:
        import block_sparse_attention_token_gb300 as sp
        st["pool"] = sp.CacheShape(blocks, 1, 64, bt)
        i32 = dict(dtype=torch.int32, device="cuda")
        st["out"] = dict(len_out=torch.empty(B, **i32), start=torch.empty(B + 1, **i32),
                         slots=torch.empty(max(1, st["n"]), **i32)[: st["n"]], used_out=torch.empty(1, **i32))
        st["status"] = torch.zeros(1, **i32)
    return st


def _codes_at(codes, index):
    """codes[index] of an e4m3 tensor (indexing moves bytes)."""
    return codes.view(torch.uint8)[index].view(torch.float8_e4m3fn)


def _quantized(x, scale):
    """Codes of x (float) under a scale that broadcasts, rounded to nearest, ties to even."""
    return (x / scale).to(torch.float8_e4m3fn)


def _scale_of(most):
    """The smallest power of two under which a magnitude fits e4m3 (448 = 1.75 * 2^8), at least 2^-100."""
    m, e = torch.frexp(most)                       # most = m 2^e, 1/2 <= m < 1
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(most), torch.where(most > 0, e, -100).clamp(min=-100))


def _prepare_write(case, g):
    held, add = _requests(case)
    B, bt, Hk, d, dt = case["B"], case["bt"], case["Hk"], case["d"], _torch_dtype(case)
    n, width = sum(add), _width(case)
    blocks = sum(_ceil(h + a, bt) for h, a in zip(held, add)) + 3
    st = dict(case=case, n=n)
    order = torch.randperm(blocks, generator=g, device="cuda")
    slots, runs, at, row = [], [], 0, 0            # runs: (first row, rows, block, first token in it)
    for h, a in zip(held, add):
        for p in range(h // bt, _ceil(h + a, bt) if a else 0):
            lo, hi = max(h, p * bt), min(h + a, (p + 1) * bt)
            runs.append((row, hi - lo, at + p, lo - p * bt))
            slots.append((at + p, lo - p * bt, hi - lo))
            row += hi - lo
        at += _ceil(h + a, bt)
    host = torch.tensor([s for s in slots for _ in range(s[2])] or [(0, 0, 0)], device="cuda")[: n]
    first = torch.tensor([r[0] for r in runs for _ in range(r[1])] or [0], device="cuda")[: n]
    st["slots"] = (order[host[:, 0]] * bt + host[:, 1] + torch.arange(n, device="cuda") - first).int()
    st["runs"] = torch.tensor(runs or [(0, 0, 0, 0)], device="cuda")[: len(runs)]
    st["run_of"] = torch.repeat_interleave(torch.arange(len(runs), device="cuda"), st["runs"][:, 1], output_size=n)
    st["block_of"] = order[st["runs"][:, 2]]
    # keys with a few strong channels, as normed and turned keys have; values of unit scale, tokens of uneven size
    strong = 1.0 + 3.0 * (torch.rand(Hk, d, generator=g, device="cuda") < 0.05)
    parts = 3 if case["packed"] else 1
    x = torch.empty(max(1, n), parts, Hk, d, device="cuda", dtype=dt)[: n]
    y = torch.empty(max(1, n), parts, Hk, d, device="cuda", dtype=dt)[: n] if parts == 1 else x
    x[:, parts - 2 if parts > 1 else 0] = (_randn(g, n, Hk, d) * strong).to(dt)
    y[:, parts - 1] = (_randn(g, n, Hk, d) * torch.exp(0.5 * _randn(g, n, Hk, 1))).to(dt)
    st["k"], st["v"] = x[:, parts - 2 if parts > 1 else 0], y[:, parts - 1]
    # what the blocks held before, under scales of a few values like it
    st["pool"] = []
    for _ in range(2):
        st["pool"].append((2.0 ** 5 * _randn(g, blocks, Hk, bt, d)).clamp(-448, 448).to(torch.float8_e4m3fn))
        st["pool"].append(torch.exp2(torch.randint(-8, -5, (blocks, Hk), generator=g, device="cuda").float()))
    if own:
        import block_sparse_attention_token_gb300 as sp
        st["own_pool"] = sp.CachePool(sp.CacheShape(blocks, Hk, d, bt), *st["pool"])
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


def _prepare_attn(case, g):
    held, add = _requests(case)
    B, bt, H, Hk, d = case["B"], case["bt"], case["H"], case["Hk"], case["d"]
    total = [h + a for h, a in zip(held, add)]
    each = [_ceil(t, bt) for t in total]
    blocks, width = sum(each) + 2, max(each)
    st = dict(case=case, scale=1.0 / math.sqrt(d), total=total, add=add, each=each, max_add=max(add))
    order = torch.randperm(blocks, generator=g, device="cuda").int()
    st["table"] = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    st["table"][torch.arange(width, device="cuda") < torch.tensor(each, device="cuda")[:, None]] = order[: sum(each)]
    st["len"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    st["start"] = torch.tensor([0] + add, device="cuda").cumsum(0).int()
    # normed queries and keys with a shared direction: scores spread over several units. The blocks' tails, past a
    # request's last token, hold what an earlier request left there
    common = _randn(g, Hk, 1, d)
    st["pool"] = []
    for shared in (0.5 * common, 0.0):
        codes = torch.empty(blocks, Hk, bt, d, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(blocks, Hk, device="cuda")
        step = max(1, (1 << 27) // (Hk * bt * d))
        for i in range(0, blocks, step):
            x = 1.2 * _randn(g, min(step, blocks - i), Hk, bt, d) + shared
            s = _scale_of(x.abs().amax((2, 3)))
            codes[i: i + step], scales[i: i + step] = _quantized(x, s[..., None, None]), s
        st["pool"] += [codes, scales]
    n = sum(add)
    st["q"] = (1.2 * _randn(g, n, Hk, H // Hk, d) + 0.5 * common[:, None, 0]).view(n, H, d).bfloat16()
    st["row_ptr"] = st["col_idx"] = st["chosen"] = None
    if case["density"] > 0.0:
        # per request and key head a share of its blocks, ascending
        chosen = []
        for b in range(B):
            rank = torch.rand(Hk, each[b], generator=g, device="cuda").argsort(-1).argsort(-1)
            chosen.append(rank < _picks(case, each[b]))
        st["chosen"] = chosen
        counts = torch.cat([c.sum(1) for c in chosen])
        st["row_ptr"] = torch.zeros(B * Hk + 1, dtype=torch.int32, device="cuda")
        st["row_ptr"][1:] = counts.cumsum(0)
        st["col_idx"] = torch.cat([c.nonzero()[:, 1] for c in chosen]).int().contiguous()
    if own:
        import block_sparse_attention_token_gb300 as sp
        shape = sp.CacheShape(blocks, Hk, d, bt)
        st["own_pool"] = sp.CachePool(shape, *st["pool"])
        st["ws"] = torch.empty(sp.attn_cache_workspace_size(shape, B, H, n, st["max_add"], width), dtype=torch.uint8,
                               device="cuda")
        st["o"], st["lse"] = torch.empty_like(st["q"]), torch.empty(n, H, device="cuda")
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    name = case["op"] + ("_bwd" if case.get("bwd") else "")
    return (_OWN if own else _PLAIN)[name](state)


def _drop_none(outs):
    return tuple(t for t in outs if t is not None)


def _own_qk(st):
    import block_sparse_attention_token_gb300 as sp
    c = st["case"]
    q, k = sp.norm_rope_fwd(st["shape"], st["table"], *st["x"], *st["w"], *st["b"], eps=EPS, rms=c["rms"],
                            pos=st["pos"], q_out=st["out"][0], k_out=st["out"][1], out_blocked=bool(c["tile"]),
                            q_means=st["means"][0], k_means=st["means"][1])
    return _drop_none((q, k, *st["means"]))


def _own_qk_bwd(st):
    import block_sparse_attention_token_gb300 as sp
    c = st["case"]
    dq, dk, dw, db = sp.norm_rope_bwd(st["shape"], st["table"], *st["dy"], *st["x"], *st["w"], eps=EPS, rms=c["rms"],
                                      pos=st["pos"], dq=st["out"][0], dk=st["out"][1], dw=st["dw"], db=st["db"],
                                      ws=st["ws"])
    return _drop_none((dq, dk, *dw, *db))


def _own_extend(st):
    import block_sparse_attention_token_gb300 as sp
    out = st["out"]
    sp.cache_extend(st["pool"], st["len"], st["add"], st["free"], st["table"], st["n"], status=st["status"], **out)
    return st["table"], out["len_out"], out["start"], out["slots"], out["used_out"]


def _own_write(st):
    import block_sparse_attention_token_gb300 as sp
    sp.cache_write(st["own_pool"], st["k"], st["v"], st["slots"], status=st["status"])
    return tuple(st["pool"])


def _own_attn(st):
    import block_sparse_attention_token_gb300 as sp
    return sp.attn_cache_fwd(st["own_pool"], st["q"], st["start"], st["len"], st["table"], st["max_add"], st["scale"],
                             causal=st["case"]["causal"], row_ptr=st["row_ptr"], col_idx=st["col_idx"], o=st["o"],
                             lse=st["lse"], ws=st["ws"], status=st["status"])


def _cos_sin(st, x):
    B, n = x.shape[:2]
    T, Y, X = _sizes(st["case"]["grid"])
    if st["pos"] is None:
        tok = torch.arange(n, device=x.device)
        idx = [t.expand(B, n) for t in (tok // (Y * X), tok // X % Y, tok % X)]
    else:
        idx = [st["pos"][..., a].long() for a in range(3)]
    return (torch.cat([st["angles"][a][part][idx[a]] for a in range(3)], -1)[:, :, None] for part in range(2))


def _turned(case, x, cos, sin):
    d = x.shape[-1]
    a, b = (x[..., : d // 2], x[..., d // 2:]) if case["half"] else (x[..., 0::2], x[..., 1::2])
    rot = [a * cos - b * sin, a * sin + b * cos]
    return torch.cat(rot, -1) if case["half"] else torch.stack(rot, -1).flatten(-2)


def _normed(case, x):
    x32 = x.float()
    if not case["rms"]:
        x32 = x32 - x32.mean(-1, keepdim=True)
    rstd = ((x32 * x32).mean(-1, keepdim=True) + EPS).rsqrt()
    return x32 * rstd, rstd


def _plain_qk(st):
    case = st["case"]
    n, bt = _grid(case)
    outs, means = [], []
    for x, w, b in zip(st["x"], st["w"], st["b"]):
        y = _normed(case, x)[0] * w
        if b is not None:
            y = y + b
        y = _turned(case, y, *_cos_sin(st, x))
        if case["tile"]:
            y = y[:, st["order"]].transpose(1, 2).contiguous()
        outs.append(y.to(x.dtype))
        means.append(y.view(*y.shape[:2], n // bt, bt, case["d"]).mean(3) if case["means"] else None)
    return _drop_none((*outs, *means))


def _plain_qk_bwd(st):
    case, d = st["case"], st["case"]["d"]
    dxs, dws, dbs = [], [], []
    for x, w, dy in zip(st["x"], st["w"], st["dy"]):
        cos, sin = _cos_sin(st, x)
        g = _turned(case, dy.float(), cos, -sin)
        xh, rstd = _normed(case, x)
        gw = g * w
        dx = gw - xh * (gw * xh).mean(-1, keepdim=True)
        if not case["rms"]:
            dx = dx - gw.mean(-1, keepdim=True)
        dxs.append((dx * rstd).to(x.dtype))
        dws.append((g * xh).view(-1, d).sum(0))
        dbs.append(None if case["rms"] else g.view(-1, d).sum(0))
    return _drop_none((*dxs, *dws, *dbs))


def _plain_extend(st):
    bt, n, table = st["case"]["bt"], st["n"], st["table"]
    length, add, free = st["len"], st["add"], st["free"]
    before = (length + (bt - 1)) // bt
    need = (length + add + (bt - 1)) // bt - before
    upto = need.cumsum(0)
    admitted = (need == 0) | (upto <= free.numel())
    start = torch.zeros(add.numel() + 1, dtype=torch.int32, device="cuda")
    start[1:] = add.cumsum(0)
    col = torch.arange(table.shape[1], device="cuda")
    fresh = admitted[:, None] & (col >= before[:, None]) & (col < (before + need)[:, None])
    take = ((upto - need - before)[:, None] + col).clamp(0, max(0, free.numel() - 1))
    table = torch.where(fresh, free[take.long()], table)
    tok = torch.arange(n, device="cuda")
    req = torch.searchsorted(start[1:], tok, right=True)
    p = length[req] + tok - start[req]
    slots = table[req, (p // bt).clamp(max=table.shape[1] - 1)] * bt + p % bt
    slots = torch.where(admitted[req], slots, -1).int()
    used = torch.where(admitted, need, 0).sum().int().view(1)
    return table, torch.where(admitted, length + add, length).int(), start, slots, used


def _plain_write(st):
    case = st["case"]
    bt, runs, run_of, block = case["bt"], st["runs"], st["run_of"], st["block_of"]
    slots = st["slots"].long()
    outs = []
    for x, codes, scales in ((st["k"], *st["pool"][:2]), (st["v"], *st["pool"][2:])):
        codes, scales = codes.clone(), scales.clone()
        x32 = x.float()
        most = torch.zeros(runs.shape[0], case["Hk"], device="cuda")
        most.index_reduce_(0, run_of, x32.abs().amax(-1), "amax")
        need = _scale_of(most)
        old = scales[block]
        held = torch.arange(bt, device="cuda") < runs[:, 3:4]              # tokens that the blocks held before
        scale = torch.where(runs[:, 3:4] > 0, torch.maximum(old, need), need)
        step = max(1, (1 << 27) // (case["Hk"] * bt * case["d"]))
        for i in range(0, runs.shape[0], step):
            at, keep = block[i: i + step], held[i: i + step]
            was = _codes_at(codes, at).float()
            again = _quantized(was * old[i: i + step, :, None, None], scale[i: i + step, :, None, None])
            kept = torch.where(keep[:, None, :, None], again.float(), was).to(codes.dtype)
            codes.view(torch.uint8)[at] = kept.view(torch.uint8)
        scales[block] = scale
        new = _quantized(x32, scale[run_of][..., None])
        codes.view(torch.uint8)[slots // bt, :, slots % bt] = new.view(torch.uint8)
        outs += [codes, scales]
    return tuple(outs)


def _keys(st, b, part):
    """Keys or values of request b, [Hk, tokens, d] in fp32."""
    codes, scales = st["pool"][2 * part], st["pool"][2 * part + 1]
    at = st["table"][b, : st["each"][b]].long()
    x = _codes_at(codes, at).float() * scales[at][..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, : st["total"][b]]


def _plain_attn(st):
    case = st["case"]
    H, Hk, d, bt = case["H"], case["Hk"], case["d"], case["bt"]
    G = H // Hk
    o = torch.empty_like(st["q"])
    lse = torch.empty(o.shape[:2], device="cuda")
    at = 0
    for b, (total, n) in enumerate(zip(st["total"], st["add"])):
        q = st["q"][at: at + n].float().view(n, Hk, G, d).permute(1, 0, 2, 3).reshape(Hk, n * G, d)
        k, v = _keys(st, b, 0), _keys(st, b, 1)
        key = torch.arange(total, device="cuda")
        last = (total - n + torch.arange(n, device="cuda")) if case["causal"] else torch.full((n,), total, device="cuda")
        seen = (key <= last.repeat_interleave(G)[:, None])[None]
        step = max(1, int(1.5e9 / (8 * n * G * total)))
        for h in range(0, Hk, step):
            see = seen
            if st["chosen"] is not None:
                see = seen & st["chosen"][b][h: h + step].repeat_interleave(bt, 1)[:, None, :total]
            s = torch.bmm(q[h: h + step], k[h: h + step].transpose(1, 2)) * st["scale"]
            s = torch.where(see, s, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            p = torch.exp(s - m)
            l = p.sum(-1, keepdim=True)
            out = torch.bmm(p, v[h: h + step]) / torch.where(l > 0, l, 1.0)
            heads = slice(h * G, h * G + out.shape[0] * G)
            o[at: at + n, heads] = out.view(-1, n, G, d).permute(1, 0, 2, 3).reshape(n, -1, d).to(o.dtype)
            lse[at: at + n, heads] = (m + torch.log(l)).view(-1, n, G).permute(1, 0, 2).reshape(n, -1)
        at += n
    return o, lse


_PLAIN = {"qk": _plain_qk, "qk_bwd": _plain_qk_bwd, "extend": _plain_extend, "write": _plain_write, "attn": _plain_attn}
_OWN = {"qk": _own_qk, "qk_bwd": _own_qk_bwd, "extend": _own_extend, "write": _own_write, "attn": _own_attn}


# ------------------------------------------------------------------- 64-bit values


def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] > 4e12:
        return None   # scores in 64 bits would take longer than some seconds
    st = prepare(case, seed)
    return {"qk": _exact_qk, "extend": _exact_extend, "write": _exact_write, "attn": _exact_attn}[case["op"]](case, st)


def _exact_turn(case, st, B, n):
    """exp(i angle) of every token and pair."""
    T, Y, X = _sizes(case["grid"])
    if st["pos"] is None:
        pos = torch.cartesian_prod(torch.arange(T), torch.arange(Y), torch.arange(X)).cuda().double().expand(B, n, 3)
    else:
        pos = st["pos"].double()
    angles = []
    for axis, cols in enumerate(_columns(case)):
        i = torch.arange(cols // 2, dtype=torch.float64, device="cuda")
        angles.append(pos[..., axis, None] * torch.exp(-2.0 * i / max(cols, 1) * math.log(THETA)))
    turn = torch.cat(angles, -1)[:, :, None]
    return torch.polar(torch.ones_like(turn), turn)


def _exact_rotate(case, x, turn):
    B, n, H, d = x.shape
    pairs = x.view(B, n, H, 2, d // 2).transpose(-1, -2) if case["half"] else x.view(B, n, H, d // 2, 2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    return (z.transpose(-1, -2) if case["half"] else z).reshape(B, n, H, d)


def _exact_qk(case, st):
    n, bt = _grid(case)
    d = case["d"]
    turn = _exact_turn(case, st, case["B"], n)
    first, second, third = [], [], []
    for i, x in enumerate(st["x"]):
        x = x.double()
        mu = 0.0 if case["rms"] else x.sum(-1, keepdim=True) / d
        r = 1.0 / torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / d + EPS)
        hat = (x - mu) * r
        w = st["w"][i].double()
        if not case["bwd"]:
            y = hat * w
            if st["b"][i] is not None:
                y += st["b"][i].double()
            y = _exact_rotate(case, y, turn)
            if case["tile"]:
                (T, Y, X), (a, b, c) = _sizes(case["grid"]), _sizes(case["tile"])
                B, _, H, _ = y.shape
                y = y.view(B, T // a, a, Y // b, b, X // c, c, H, d).permute(0, 7, 1, 3, 5, 2, 4, 6, 8)
                y = y.reshape(B, H, n, d)
            first.append(y)
            if case["means"]:
                second.append(y.view(*y.shape[:2], -1, bt, d).mean(3))
            continue
        dy = _exact_rotate(case, st["dy"][i].double(), turn.conj())
        up = dy * w
        back = up - hat * ((up * hat).sum(-1, keepdim=True) / d)
        if not case["rms"]:
            back -= up.sum(-1, keepdim=True) / d
            third.append(dy.sum((0, 1, 2)))
        first.append(back * r)
        second.append(torch.einsum("bnhd,bnhd->d", dy, hat))
    return (*first, *second, *third)


def _exact_extend(case, st):
    """Request by request on the host."""
    table, free = st["table"].tolist(), st["free"].tolist()
    start, slots, length, used, waiting = [0], [], [], 0, False
    bt = case["bt"]
    for b, (h, a) in enumerate(zip(st["len"].tolist(), st["add"].tolist())):
        have, want = _ceil(h, bt), _ceil(h + a, bt)
        # whoever finds too few blocks waits, and so does everyone behind who needs any
        waiting = waiting or used + want - have > len(free)
        refused = waiting and want > have
        if not refused:
            for j in range(have, want):
                table[b][j] = free[used]
                used += 1
        slots += [-1 if refused else table[b][p // bt] * bt + p % bt for p in range(h, h + a)]
        length.append(h if refused else h + a)
        start.append(start[-1] + a)
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (table, length, start, slots, [used]))


def _exact_write(case, st):
    """Codes before rounding: a value over its block's scale."""
    bt, outs = case["bt"], []
    slots = st["slots"].tolist()
    for x, codes, scales in ((st["k"], *st["pool"][:2]), (st["v"], *st["pool"][2:])):
        codes, scales, x = codes.double(), scales.double(), x.double()
        for row, count, _, first in st["runs"].tolist():
            block = slots[row] // bt
            new = x[row: row + count].transpose(0, 1)                     # [Hk, count, d]
            most = new.abs().amax((1, 2))
            scale = torch.exp2(torch.floor(torch.log2(most / 448.0) - 0.5).clamp(min=-100))   # at most what is needed
            for _ in range(2):
                scale = torch.where(448.0 * scale < most, 2.0 * scale, scale)
            if first > 0:
                scale = torch.maximum(scale, scales[block])
                codes[block, :, :first] *= (scales[block] / scale)[:, None, None]
            codes[block, :, first: first + count] = new / scale[:, None, None]
            scales[block] = scale
        outs += [codes, scales]
    return tuple(outs)


def _exact_attn(case, st):
    """One request and key head at a time, dense scores."""
    H, Hk, d, bt = case["H"], case["Hk"], case["d"], case["bt"]
    G = H // Hk
    outs, lses, at = [], [], 0
    for b, (total, n) in enumerate(zip(st["total"], st["add"])):
        blocks = st["table"][b, : st["each"][b]].long()
        out = torch.zeros(n, H, d, dtype=torch.float64, device="cuda")
        lse = torch.zeros(n, H, dtype=torch.float64, device="cuda")
        hidden = torch.zeros(n, total, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = torch.ones(n, total, dtype=torch.bool, device="cuda").triu(total - n + 1)
        for hk in range(Hk):
            k, v = (_codes_at(st["pool"][2 * i], (blocks, hk)).double() * st["pool"][2 * i + 1][blocks, hk].double()[:, None, None]
                    for i in range(2))
            k, v = k.reshape(-1, d)[:total], v.reshape(-1, d)[:total]
            hide = hidden
            if st["chosen"] is not None:
                hide = hidden | ~st["chosen"][b][hk].repeat_interleave(bt)[:total]
            for h in range(hk * G, hk * G + G):
                score = (st["q"][at: at + n, h].double() @ k.T * st["scale"]).masked_fill_(hide, -math.inf)
                lse[:, h] = torch.logsumexp(score, 1)
                weight = torch.exp(score - lse[:, h, None]).masked_fill_(hide, 0.0)
                out[:, h] = weight @ v
        outs.append(out)
        lses.append(lse)
        at += n
    return torch.cat(outs), torch.cat(lses)
