"""Cases that time the operators around block-sparse attention of a video DiT layer:
the token norm (layer norm, RMS norm) and its backward, the three-axis rotary
positions with the tile reorder, and attention with a token mask and a score cap,
forward and backward. Each case runs in a plain form (elementary torch operations
in fp32) or, where `own` is true, through this package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

# ------------------------------------------------------------------- cases


def listed():
    return [
        # query/key norm per head on a 1k-token clip in fp32: the smallest call, latency
        dict(name="norm_fwd_head_1k_f32", op="norm", bwd=False, B=1, H=2, grid="4x16x16", tile="4x4x4", d=64,
             dtype="f32", rms=False, head=True, packed=False),
        # a 30k-token clip of 40 heads, RMS norm over the whole token, read out of the fused QKV projection
        dict(name="norm_fwd_token_30k_rms", op="norm", bwd=False, B=1, H=40, grid="20x32x48", tile="2x8x8", d=128,
             dtype="bf16", rms=True, head=False, packed=True),
        # the same clip in training: layer norm over the whole token, backward with both weight gradients
        dict(name="norm_bwd_token_30k", op="norm", bwd=True, B=1, H=40, grid="20x32x48", tile="2x8x8", d=128,
             dtype="bf16", rms=False, head=False, packed=False),
        # training at 64k tokens: per-head norm, one weight vector shared by 24 heads and all tokens
        dict(name="norm_bwd_head_64k", op="norm", bwd=True, B=1, H=24, grid="16x64x64", tile="2x8x8", d=128,
             dtype="bf16", rms=False, head=True, packed=False),
        # an 8k-token clip, d = 64: rotation, tile order and tile means in one pass
        dict(name="rope_fwd_8k_d64", op="rope", bwd=False, B=1, H=12, grid="8x32x32", tile="4x4x4", d=64,
             dtype="bf16", half=False, positions=False, means=True),
        # the 30k-token clip of 40 heads
        dict(name="rope_fwd_30k", op="rope", bwd=False, B=1, H=40, grid="20x32x48", tile="2x8x8", d=128,
             dtype="bf16", half=False, positions=False, means=True),
        # gradients of a 64k-token training step: raster in and out, per-token positions (packed clips), half pairing
        dict(name="rope_bwd_64k_positions", op="rope", bwd=True, B=1, H=24, grid="16x64x64", tile="2x8x8", d=128,
             dtype="bf16", half=True, positions=True, means=False),
        # attention on a 1k-token clip pair: the smallest call, latency
        dict(name="attn_fwd_1k_docs", op="attn", bwd=False, B=1, H=2, grid="4x16x16", tile="4x4x4", d=64,
             density=0.75, mask="docs", docs=2, prefix=0, cap=0.0),
        # packed clips of 8k tokens, d = 64 in 64-token blocks
        dict(name="attn_fwd_8k_docs", op="attn", bwd=False, B=1, H=12, grid="8x32x32", tile="4x4x4", d=64,
             density=0.8, mask="docs", docs=3, prefix=0, cap=0.0),
        # frame-by-frame generation on the 30k-token clip: causal in frames, two conditioning frames, capped scores
        dict(name="attn_fwd_30k_frames_cap", op="attn", bwd=False, B=1, H=40, grid="20x32x48", tile="2x8x8", d=128,
             density=0.5, mask="frames", docs=1, prefix=2, cap=30.0),
        # backward of the packed 8k clips
        dict(name="attn_bwd_8k_docs_cap", op="attn", bwd=True, B=1, H=12, grid="8x32x32", tile="4x4x4", d=64,
             density=0.8, mask="docs", docs=3, prefix=0, cap=20.0),
        # backward of a 64k-token training step over packed clips, a tenth of the blocks
        dict(name="attn_bwd_64k_docs", op="attn", bwd=True, B=1, H=24, grid="16x64x64", tile="2x8x8", d=128,
             density=0.1, mask="docs", docs=3, prefix=0, cap=0.0),
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


def draw(rng):
    """One more case of the listed ranges: 64 tokens to 65,536, 1 to 40 heads."""
    op = rng.choice(["norm", "rope", "attn"])
    d = rng.choice([64, 128])
    bwd = rng.random() < 0.5
    if op == "attn":
        grid, tile = _draw_grid(rng, 128, 24576)
        n = grid[0] * grid[1] * grid[2]
        heads = max(1, min(_log_int(rng, 1, 24), int(12 * 16384 ** 2 / n ** 2) + 1))
        mask = rng.choice(["docs", "frames", "none"])
        return dict(op=op, bwd=bwd, B=rng.choice([1, 1, 2]), H=heads, grid=_text(grid), tile=_text(tile), d=d,
                    density=round(rng.uniform(0.1, 0.9), 3), mask=mask, docs=rng.randint(1, 5),
                    prefix=rng.randint(0, 3), cap=rng.choice([0.0, 0.0, round(rng.uniform(5.0, 60.0), 2)]))
    grid, tile = _draw_grid(rng, 64, 65536)
    n = grid[0] * grid[1] * grid[2]
    heads = max(1, min(_log_int(rng, 1, 40), 30720 * 40 * 128 // (n * d)))
    base = dict(op=op, bwd=bwd, B=1 if n * heads > 400000 else rng.choice([1, 2]), H=heads, grid=_text(grid),
                tile=_text(tile), d=d,
                dtype=rng.choice(["bf16", "bf16", "f32"]) if n * heads * d < 50000000 else "bf16")
    if op == "norm":
        return dict(base, rms=rng.random() < 0.4, head=rng.random() < 0.5, packed=rng.random() < 0.4)
    return dict(base, half=rng.random() < 0.4, positions=rng.random() < 0.4, means=not bwd and rng.random() < 0.7)


# ------------------------------------------------------------------- shapes

EPS = 1e-6
THETA = 10000.0


def _dims(case):
    (T, Y, X), (a, b, c) = _sizes(case["grid"]), _sizes(case["tile"])
    bt = a * b * c
    return T * Y * X, bt, T * Y * X // bt


def _torch_dtype(case):
    return torch.float32 if case.get("dtype", "bf16") == "f32" else torch.bfloat16


def _shape(sp, case):
    return sp.make_shape(case["B"], case["H"], *_sizes(case["grid"]), case["d"], *_sizes(case["tile"]),
                         case.get("dtype", "bf16"))


def _sections(d):
    """Columns of the time, height and width axes: the height and width axes get 2 * (d // 6) each."""
    side = 2 * (d // 6)
    return d - 2 * side, side, side


def _block_order(case, device="cpu"):
    """Raster token index of every token in tile order."""
    (T, Y, X), (a, b, c) = _sizes(case["grid"]), _sizes(case["tile"])
    n = torch.arange(T * Y * X, device=device).view(T // a, a, Y // b, b, X // c, c)
    return n.permute(0, 2, 4, 1, 3, 5).reshape(-1)


def _token_mask(case, device="cpu"):
    """pos, lo, hi of every raster token: query n sees key m where lo[n] <= pos[m] < hi[n].

    docs: clips packed one after another, their borders inside frames, the last tokens
    padding that sees and is seen by nothing. frames: a token sees its own and earlier
    frames and the first `prefix` frames; none: every key."""
    T, Y, X = _sizes(case["grid"])
    n = T * Y * X
    tok = torch.arange(n, device=device)
    if case["mask"] == "docs":
        docs, pad = case["docs"], n // 50
        # borders at uneven places: clip i takes a share proportional to i + 2
        total = sum(i + 2 for i in range(docs))
        borders, acc = [], 0
        for i in range(docs):
            acc += i + 2
            borders.append((n - pad) * acc // total)
        ids = torch.bucketize(tok, torch.tensor(borders, device=device), right=True)
        live = ids < docs
        pos = torch.where(live, ids, -1)
        lo, hi = torch.where(live, ids, 0), torch.where(live, ids + 1, 0)
    elif case["mask"] == "frames":
        pos = tok // (Y * X)
        lo, hi = torch.zeros_like(pos), torch.clamp(pos + 1, min=min(case["prefix"], T))
    else:
        pos, lo, hi = torch.zeros_like(tok), torch.zeros_like(tok), torch.ones_like(tok)
    return pos.int(), lo.int(), hi.int()


def _visible_pairs(case):
    """[nb, nb]: how many token pairs of a block pair the mask lets through."""
    n, bt, nb = _dims(case)
    order = _block_order(case)
    pos, lo, hi = (t[order].long() for t in _token_mask(case))
    keys = pos.view(nb, bt).sort(1).values
    out = torch.zeros(nb, nb)
    for j in range(nb):
        count = torch.searchsorted(keys[j], hi) - torch.searchsorted(keys[j], lo)
        out[:, j] = count.clamp(min=0).view(nb, bt).sum(1).float()
    return out


def work(case):
    n, bt, nb = _dims(case)
    values = case["B"] * n * case["H"] * case["d"]
    e = 4 if case.get("dtype", "bf16") == "f32" else 2
    if case["op"] == "norm":
        cols = case["d"] if case["head"] else case["H"] * case["d"]
        stats = (values // cols) * (4 if case["rms"] else 8)
        params = 4 * cols * (1 if case["rms"] else 2)
        if case["bwd"]:
            return {"bytes": 3 * e * values + stats + 4 * cols + params, "flops": 14 * values}
        return {"bytes": 2 * e * values + stats + params, "flops": 8 * values}
    if case["op"] == "rope":
        means = 4 * values // bt if case["means"] else 0
        pos = 12 * case["B"] * n if case["positions"] else 0
        return {"bytes": 2 * e * values + means + pos, "flops": 3 * values + (values if case["means"] else 0)}
    pairs = _visible_pairs(case)
    seen = (pairs > 0).sum(1).clamp(min=1)
    per_row = pairs.sum(1) / seen                       # mean over the blocks a row can see at all
    picks = torch.minimum(seen.float(), torch.full_like(per_row, max(1.0, case["density"] * nb)))
    total = float((per_row * picks).sum()) * case["B"] * case["H"]
    rows = case["B"] * case["H"] * n
    index = 4 * case["B"] * case["H"] * nb * max(1.0, case["density"] * nb)
    if case["bwd"]:   # q, k, v, o, dO in; dQ, dK, dV out; LSE
        return {"bytes": 16 * values + 4 * rows + index, "flops": 10 * case["d"] * total}
    return {"bytes": 8 * values + 4 * rows + index, "flops": 4 * case["d"] * total}


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_norm(case, g):
    n, _, _ = _dims(case)
    B, H, d, dt = case["B"], case["H"], case["d"], _torch_dtype(case)
    cols = d if case["head"] else H * d
    parts = 3 if case["packed"] else 1
    # activations of a projection: unit scale, an offset per channel
    x = torch.empty(B, n, parts, H, d, device="cuda", dtype=dt)
    for p in range(parts):
        x[:, :, p] = (_randn(g, B, n, H, d) + 0.5 * _randn(g, H, d)).to(dt)
    st = dict(case=case, x=x[:, :, parts - 1], w=1.0 + 0.2 * _randn(g, cols),
              b=None if case["rms"] else 0.1 * _randn(g, cols))
    if case["bwd"]:
        st["dy"] = (0.1 * _randn(g, B, n, H, d)).to(dt)
        _, st["mean"], st["rstd"] = _norm_fwd_plain(case, st["x"], st["w"], st["b"])
    if own:
        import block_sparse_attention_token_gb300 as sp
        st["shape"] = s = _shape(sp, case)
        if case["bwd"]:
            st["ws"] = torch.empty(sp.norm_workspace_size(s, rms=case["rms"], per_head=case["head"]),
                                   dtype=torch.uint8, device="cuda")
            st["out"] = [torch.empty(B, n, H, d, dtype=dt, device="cuda"), torch.empty_like(st["w"]),
                         None if case["rms"] else torch.empty_like(st["w"])]
        else:
            stat = (B, n, H) if case["head"] else (B, n)
            st["out"] = [torch.empty(B, n, H, d, dtype=dt, device="cuda"),
                         None if case["rms"] else torch.empty(stat, device="cuda"), torch.empty(stat, device="cuda")]
    return st


def _prepare_rope(case, g):
    n, bt, nb = _dims(case)
    B, H, d, dt = case["B"], case["H"], case["d"], _torch_dtype(case)
    st = dict(case=case, x=_randn(g, B, n, H, d).to(dt), pos=None)
    T, Y, X = _sizes(case["grid"])
    if case["positions"]:
        # packed clips: the frame index starts over, the frame is shifted inside the table
        shift = torch.randint(0, 4, (B, 1, 3), generator=g, device="cuda")
        tok = torch.arange(n, device="cuda")
        grid = torch.stack([tok // (Y * X) % max(1, T // 2), tok // X % Y, tok % X], -1)
        st["pos"] = (grid[None] + shift).int().contiguous()
    st["extent"] = tuple(v + 4 for v in (T, Y, X)) if case["positions"] else (T, Y, X)
    st["order"] = _block_order(case, "cuda")
    if own:
        import block_sparse_attention_token_gb300 as sp
        st["shape"] = s = _shape(sp, case)
        st["table"] = sp.rope_table(s, _sections(d), THETA, extent=st["extent"], half=case["half"])
        blocked = not case["bwd"]
        st["out"] = torch.empty((B, H, n, d) if blocked else (B, n, H, d), dtype=dt, device="cuda")
        st["means"] = torch.empty(B, H, nb, d, device="cuda") if case["means"] else None
    else:
        st["angles"] = _rope_angles(case, st["extent"], "cuda")
    return st


def _rope_angles(case, extent, device):
    """(cos, sin) [extent, columns / 2] of each axis in fp32, from angles in 64 bits."""
    out = []
    for ext, cols in zip(extent, _sections(case["d"])):
        freq = THETA ** (-torch.arange(0, cols, 2, dtype=torch.float64, device=device) / cols)
        ang = torch.arange(ext, dtype=torch.float64, device=device)[:, None] * freq
        out.append((ang.cos().float(), ang.sin().float()))
    return out


def _prepare_attn(case, g):
    n, bt, nb = _dims(case)
    B, H, d = case["B"], case["H"], case["d"]
    scale = 1.0 / math.sqrt(d)
    # normed queries and keys with a shared direction: scores spread over several units, some above the cap
    common = _randn(g, B, H, 1, d)
    st = dict(case=case, scale=scale)
    st["q"] = (1.2 * _randn(g, B, H, n, d) + 0.5 * common).bfloat16()
    st["k"] = (1.2 * _randn(g, B, H, n, d) + 0.5 * common).bfloat16()
    st["v"] = _randn(g, B, H, n, d).bfloat16()
    st["mask"] = tuple(t.expand(B, n).contiguous() for t in _token_mask(case, "cuda"))
    # the selection: per row about density * nb blocks, those that the mask lets through first
    order = _block_order(case, "cuda")
    pos, lo, hi = (t[0][order].view(nb, bt) for t in st["mask"])
    live = lo < hi
    far = torch.iinfo(torch.int32).max
    lo_min = torch.where(live, lo, far).amin(1)
    hi_max = torch.where(live, hi, -far).amax(1)
    seen = (pos.amax(1)[None] >= lo_min[:, None]) & (pos.amin(1)[None] < hi_max[:, None])
    rank = torch.rand(B * H, nb, nb, generator=g, device="cuda") + 2.0 * seen
    length = case["density"] * nb * (0.5 + torch.rand(B * H, nb, 1, generator=g, device="cuda"))
    length = length.round().clamp(1, nb).long()
    place = rank.argsort(-1, descending=True).argsort(-1)
    chosen = place < length
    st["chosen"] = chosen
    flat = chosen.view(-1, nb)
    st["row_ptr"] = torch.zeros(B * H * nb + 1, dtype=torch.int32, device="cuda")
    st["row_ptr"][1:] = flat.sum(1).cumsum(0)
    st["col_idx"] = flat.nonzero()[:, 1].int().contiguous()
    st["order"] = order
    # the same rows as a padded table of the longest row's width (plain form)
    width = int(length.max())
    table = torch.where(chosen, torch.arange(nb, device="cuda"), nb).sort(-1).values[..., :width]
    st["table_ok"] = table < nb
    st["table"] = torch.where(st["table_ok"], table, 0)
    if case["bwd"]:
        st["do"] = _randn(g, B, H, n, d).bfloat16()
        st["o"], st["lse"] = _attn_fwd_plain(st)
    if own:
        import block_sparse_attention_token_gb300 as sp
        st["shape"] = s = _shape(sp, case)
        st["plan"] = None if case["mask"] == "none" else sp.mask_plan(s, *st["mask"])
        st["ws"] = torch.empty(sp.attn_masked_workspace_size(s, case["bwd"]), dtype=torch.uint8, device="cuda")
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["bwd"]:
            st["out"] = [torch.empty_like(st["q"]) for _ in range(3)]
        else:
            st["out"] = [torch.empty_like(st["q"]), torch.empty(B, H, n, device="cuda")]
    return st


# ------------------------------------------------------------------- one pass


def run(state):
    case = state["case"]
    name = case["op"] + ("_bwd" if case["bwd"] else "_fwd")
    return (_OWN if own else _PLAIN)[name](state)


def _drop_none(*outs):
    return tuple(t for t in outs if t is not None)


def _own_norm_fwd(st):
    import block_sparse_attention_token_gb300 as sp
    c, (y, mean, rstd) = st["case"], st["out"]
    return _drop_none(*sp.norm_fwd(st["shape"], st["x"], st["w"], st["b"], eps=EPS, rms=c["rms"], per_head=c["head"],
                                   out=y, mean=mean, rstd=rstd))


def _own_norm_bwd(st):
    import block_sparse_attention_token_gb300 as sp
    c, (dx, dw, db) = st["case"], st["out"]
    return _drop_none(*sp.norm_bwd(st["shape"], st["dy"], st["x"], st["w"], st["mean"], st["rstd"], rms=c["rms"],
                                   per_head=c["head"], dx=dx, dw=dw, db=db, ws=st["ws"]))


def _own_rope(st):
    import block_sparse_attention_token_gb300 as sp
    c = st["case"]
    out = sp.rope(st["shape"], st["table"], st["x"], out=st["out"], inverse=c["bwd"], out_blocked=not c["bwd"],
                  pos=st["pos"], means=st["means"])
    return (out, st["means"]) if c["means"] else (out,)


def _own_attn_fwd(st):
    import block_sparse_attention_token_gb300 as sp
    o, lse = st["out"]
    return sp.attn_masked_fwd(st["shape"], st["q"], st["k"], st["v"], st["row_ptr"], st["col_idx"], st["scale"],
                              cap=st["case"]["cap"], mask=st["plan"], o=o, lse=lse, ws=st["ws"], status=st["status"])


def _own_attn_bwd(st):
    import block_sparse_attention_token_gb300 as sp
    dq, dk, dv = st["out"]
    return sp.attn_masked_bwd(st["shape"], st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["row_ptr"],
                              st["col_idx"], st["scale"], cap=st["case"]["cap"], mask=st["plan"], dq=dq, dk=dk, dv=dv,
                              ws=st["ws"], status=st["status"])


def _norm_fwd_plain(case, x, w, b):
    x32 = x.float() if case["head"] else x.float().flatten(2)
    mean = None if case["rms"] else x32.mean(-1, keepdim=True)
    xc = x32 if case["rms"] else x32 - mean
    rstd = ((xc * xc).mean(-1, keepdim=True) + EPS).rsqrt()
    y = xc * rstd * w
    if b is not None:
        y = y + b
    return (y.view(x.shape).to(x.dtype), None if mean is None else mean.squeeze(-1), rstd.squeeze(-1))


def _plain_norm_fwd(st):
    return _drop_none(*_norm_fwd_plain(st["case"], st["x"], st["w"], st["b"]))


def _plain_norm_bwd(st):
    case, x = st["case"], st["x"]
    per_row = (lambda t: t.float()) if case["head"] else (lambda t: t.float().flatten(2))
    x32, dy = per_row(x), per_row(st["dy"])
    rstd = st["rstd"].unsqueeze(-1)
    xh = x32 * rstd if case["rms"] else (x32 - st["mean"].unsqueeze(-1)) * rstd
    g = dy * st["w"]
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if not case["rms"]:
        dx = dx - g.mean(-1, keepdim=True)
    dx = (dx * rstd).view(x.shape).to(x.dtype)
    cols = dy.shape[-1]
    dw = (dy * xh).view(-1, cols).sum(0)
    return (dx, dw) if case["rms"] else (dx, dw, dy.view(-1, cols).sum(0))


def _plain_rope(st):
    case, x = st["case"], st["x"]
    B, n, H, d = x.shape
    T, Y, X = _sizes(case["grid"])
    if st["pos"] is None:
        tok = torch.arange(n, device=x.device)
        idx = [t.expand(B, n) for t in (tok // (Y * X), tok // X % Y, tok % X)]
    else:
        idx = [st["pos"][..., a].long() for a in range(3)]
    cos = torch.cat([st["angles"][a][0][idx[a]] for a in range(3)], -1)[:, :, None]
    sin = torch.cat([st["angles"][a][1][idx[a]] for a in range(3)], -1)[:, :, None]
    if case["bwd"]:
        sin = -sin
    x32 = x.float()
    first, second = (x32[..., : d // 2], x32[..., d // 2:]) if case["half"] else (x32[..., 0::2], x32[..., 1::2])
    rot = [first * cos - second * sin, first * sin + second * cos]
    y = torch.cat(rot, -1) if case["half"] else torch.stack(rot, -1).flatten(-2)
    if case["bwd"]:
        return (y.to(x.dtype),)
    y = y[:, st["order"]].transpose(1, 2).contiguous()
    if not case["means"]:
        return (y.to(x.dtype),)
    bt = _dims(case)[1]
    return y.to(x.dtype), y.view(B, H, n // bt, bt, d).mean(3)   # the means before rounding


def _chunks(st, bytes_per_score):
    """Ranges of query blocks whose scores fit in about 1.5 GB."""
    n, bt, nb = _dims(st["case"])
    step = max(1, int(1.5e9 / (bytes_per_score * bt * bt * st["table"].shape[-1])))
    return [(i, min(nb, i + step)) for i in range(0, nb, step)]


def _plain_scores(st, bh, i0, i1, q, k):
    """Scaled and capped scores of query blocks i0 .. i1 over their padded rows, the pairs that count, and tanh."""
    case = st["case"]
    n, bt, nb = _dims(case)
    idx, ok = st["table"][bh, i0:i1], st["table_ok"][bh, i0:i1]
    kg = k[idx].flatten(1, 2)
    s = torch.bmm(q, kg.transpose(1, 2)) * st["scale"]
    t = None
    if case["cap"] > 0:
        t = torch.tanh(s / case["cap"])
        s = t * case["cap"]
    pos, lo, hi = (m[bh // case["H"]][st["order"]].view(nb, bt) for m in st["mask"])
    pk = pos[idx].flatten(1, 2)[:, None]
    see = (pk >= lo[i0:i1, :, None]) & (pk < hi[i0:i1, :, None]) & ok.repeat_interleave(bt, 1)[:, None]
    return s, see, t, idx, kg


def _attn_fwd_plain(st):
    case = st["case"]
    n, bt, nb = _dims(case)
    B, H, d = case["B"], case["H"], case["d"]
    o = torch.empty(B, H, n, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, H, n, device="cuda")
    for bh in range(B * H):
        q, k, v = (st[x].view(B * H, nb, bt, d)[bh].float() for x in "qkv")
        for i0, i1 in _chunks(st, 4):
            s, see, _, idx, _ = _plain_scores(st, bh, i0, i1, q[i0:i1], k)
            s = torch.where(see, s, -math.inf)
            m = s.amax(-1, keepdim=True)
            m = torch.where(m == -math.inf, 0.0, m)
            p = torch.exp(s - m)
            total = p.sum(-1, keepdim=True)
            out = torch.bmm(p, v[idx].flatten(1, 2)) / torch.where(total > 0, total, 1.0)
            o.view(B * H, nb, bt, d)[bh, i0:i1] = out.to(o.dtype)
            lse.view(B * H, nb, bt)[bh, i0:i1] = (m + torch.log(total)).squeeze(-1)
    return o, lse


def _attn_bwd_plain(st):
    case = st["case"]
    n, bt, nb = _dims(case)
    B, H, d = case["B"], case["H"], case["d"]
    grads = [torch.empty(B, H, n, d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    for bh in range(B * H):
        q, k, v, o, do = (st[x].view(B * H, nb, bt, d)[bh].float() for x in ("q", "k", "v", "o", "do"))
        lse = st["lse"].view(B * H, nb, bt, 1)[bh]
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        for i0, i1 in _chunks(st, 4):
            s, see, t, idx, kg = _plain_scores(st, bh, i0, i1, q[i0:i1], k)
            p = torch.where(see, torch.exp(s - lse[i0:i1]), 0.0)
            dp = torch.bmm(do[i0:i1], v[idx].flatten(1, 2).transpose(1, 2))
            ds = p * (dp - (do[i0:i1] * o[i0:i1]).sum(-1, keepdim=True))
            if t is not None:
                ds = ds * (1 - t * t)
            ds = ds * st["scale"]
            dq[i0:i1] = torch.bmm(ds, kg)
            dk.index_add_(0, idx.flatten(), torch.bmm(ds.transpose(1, 2), q[i0:i1]).view(-1, bt, d))
            dv.index_add_(0, idx.flatten(), torch.bmm(p.transpose(1, 2), do[i0:i1]).view(-1, bt, d))
        for out, acc in zip(grads, (dq, dk, dv)):
            out.view(B * H, nb, bt, d)[bh] = acc.to(out.dtype)
    return tuple(grads)


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "rope_fwd": _plain_rope, "rope_bwd": _plain_rope,
          "attn_fwd": _attn_fwd_plain, "attn_bwd": _attn_bwd_plain}
_OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "rope_fwd": _own_rope, "rope_bwd": _own_rope,
        "attn_fwd": _own_attn_fwd, "attn_bwd": _own_attn_bwd}


# ------------------------------------------------------------------- 64-bit values


def exact(case, seed):
    n, bt, nb = _dims(case)
    if case["op"] == "attn":
        dense = (10 if case["bwd"] else 4) * case["B"] * case["H"] * case["d"] * float(n) * n
        if dense > 6e12:   # dense scores in 64 bits would take longer than some seconds
            return None
    st = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](case, st)


def _exact_norm(case, st):
    x = st["x"].double()
    cols = case["d"] if case["head"] else case["H"] * case["d"]
    rows = x.reshape(-1, cols)
    w = st["w"].double()
    if not case["bwd"]:
        mu = torch.zeros(rows.shape[0], dtype=torch.float64, device=x.device) if case["rms"] else rows.sum(1) / cols
        var = ((rows - mu[:, None]) ** 2).sum(1) / cols
        r = 1.0 / torch.sqrt(var + EPS)
        y = (rows - mu[:, None]) * r[:, None] * w
        if st["b"] is not None:
            y += st["b"].double()
        stat = x.shape[:3] if case["head"] else x.shape[:2]
        return _drop_none(y.view(x.shape), None if case["rms"] else mu.view(stat), r.view(stat))
    dy = st["dy"].double().reshape(-1, cols)
    r = st["rstd"].double().reshape(-1, 1)
    hat = rows * r if case["rms"] else (rows - st["mean"].double().reshape(-1, 1)) * r
    up = dy * w
    back = up - hat * ((up * hat).sum(1, keepdim=True) / cols)
    if not case["rms"]:
        back -= up.sum(1, keepdim=True) / cols
    grads = [(back * r).view(x.shape), torch.einsum("rc,rc->c", dy, hat)]
    if not case["rms"]:
        grads.append(dy.sum(0))
    return tuple(grads)


def _exact_rope(case, st):
    """Each pair as a complex number times exp(i angle)."""
    x = st["x"].double()
    B, n, H, d = x.shape
    T, Y, X = _sizes(case["grid"])
    if st["pos"] is None:
        lattice = torch.cartesian_prod(torch.arange(T), torch.arange(Y), torch.arange(X)).cuda()
        pos = lattice.double().expand(B, n, 3)
    else:
        pos = st["pos"].double()
    angles = []
    for axis, cols in enumerate(_sections(d)):
        i = torch.arange(cols // 2, dtype=torch.float64, device=x.device)
        angles.append(pos[..., axis, None] * torch.exp(-2.0 * i / cols * math.log(THETA)))
    turn = torch.cat(angles, -1)[:, :, None]
    turn = torch.polar(torch.ones_like(turn), -turn if case["bwd"] else turn)
    pairs = x.view(B, n, H, 2, d // 2).transpose(-1, -2) if case["half"] else x.view(B, n, H, d // 2, 2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = (z.transpose(-1, -2) if case["half"] else z).reshape(B, n, H, d)
    if case["bwd"]:
        return (y,)
    a, b, c = _sizes(case["tile"])
    y = y.view(B, T // a, a, Y // b, b, X // c, c, H, d).permute(0, 7, 1, 3, 5, 2, 4, 6, 8).reshape(B, H, n, d)
    if not case["means"]:
        return (y,)
    return y, y.view(B, H, -1, a * b * c, d).mean(3)


def _exact_attn(case, st):
    """Dense scores of one head at a time, the selection and the mask as a matrix of pairs."""
    n, bt, nb = _dims(case)
    B, H, d = case["B"], case["H"], case["d"]
    results = [[] for _ in range(3 if case["bwd"] else 2)]
    for b in range(B):
        pos, lo, hi = (m[b][st["order"]] for m in st["mask"])
        sees = (lo[:, None] <= pos[None]) & (pos[None] < hi[:, None])
        for h in range(H):
            pick = st["chosen"][b * H + h].repeat_interleave(bt, 0).repeat_interleave(bt, 1) & sees
            q, k, v = (st[x][b, h].double() for x in "qkv")
            score = (q @ k.T).mul_(st["scale"])
            slope = None
            if case["cap"] > 0:
                score = torch.tanh(score / case["cap"])
                slope = 1.0 - score ** 2
                score *= case["cap"]
            score.masked_fill_(~pick, -math.inf)
            if not case["bwd"]:
                lse = torch.logsumexp(score, 1)
                prob = torch.exp(score - lse[:, None]).masked_fill_(~pick, 0.0)
                results[0].append(prob @ v)
                results[1].append(lse)
                continue
            prob = torch.exp(score - st["lse"][b, h].double()[:, None]).masked_fill_(~pick, 0.0)
            do, o = st["do"][b, h].double(), st["o"][b, h].double()
            ds = prob * (do @ v.T - (do * o).sum(1, keepdim=True))
            if slope is not None:
                ds *= slope
            ds *= st["scale"]
            for out, value in zip(results, (ds @ k, ds.T @ q, prob.T @ do)):
                out.append(value)
    return tuple(torch.stack(r).view(B, H, *r[0].shape) for r in results)
