"""The per-head norm and the rotary positions in one pass against plain float64 forms.

Tolerances. One rounding to the stored type is off by at most half a step (eps/2
relative: bf16 2^-8, fp32 2^-24). fp32 arithmetic before it: a row's sums have at most
128 terms, taken by lanes and then a tree, at most 24 roundings deep; products, root,
quotient and rotation add a few more. `DEEP` = 64 2^-24 covers them, applied to the
magnitudes that enter. Sums over rows (dw, db) are taken in parts of at most 64 x 8 rows per
thread and warp, then over the parts: at most 600 roundings deep in the shapes here, of
which a term meets a random few; `LONG` = 640 2^-24 of the sum of magnitudes bounds all."""
import numpy as np
import pytest
import torch

import block_sparse_attention_token_gb300 as sp

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

U32 = 2.0 ** -24
DEEP, LONG = 64 * U32, 640 * U32
EPS = 1e-6

# B, H, Hk, grid, tile (None: tokens without tiles), d
SHAPES = [
    (1, 1, 1, (4, 4, 4), (4, 4, 4), 64),
    (2, 6, 2, (2, 24, 8), (2, 8, 8), 64),
    (1, 8, 1, (3, 8, 40), (1, 8, 8), 128),
    (2, 5, 5, (2, 8, 24), (2, 8, 8), 128),
    (1, 40, 40, (8, 8, 16), (1, 8, 16), 128),
    (1, 1, 1, (1, 1, 1), None, 128),
    (1, 32, 8, (77, 1, 1), None, 128),
    (3, 3, 1, (1, 5, 13), None, 64),
    (1, 2, 2, (1301, 1, 1), None, 64),
]
CASES = [("bf16", True, False, True), ("bf16", False, True, False), ("f32", True, True, False), ("f32", False, False, True)]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def shape_of(dims, dtype):
    B, H, Hk, grid, tile, d = dims
    return sp.make_shape(B, H, *grid, d, *(tile or (1, 1, 1)), dtype)


def cols_of(d):
    side = 2 * (d // 6)
    return d - 2 * side, side, side


def inputs(dims, s, g, packed):
    """q and k, slices of one projection or tensors of their own."""
    B, H, Hk, _, _, d = dims
    make = lambda h: (torch.randn(B, s.N, h, d, generator=g, device="cuda") + 0.7).to(s.torch_dtype)
    if packed:
        x = make(H + 2 * Hk)
        return x[:, :, :H], x[:, :, H:H + Hk]
    return make(H), make(Hk)


def angles(s, pos, cols, theta=1e4):
    B, N = s.B, s.N
    if pos is None:
        grid = torch.cartesian_prod(*(torch.arange(v) for v in (s.T, s.Y, s.X))).reshape(-1, 3).cuda()
        pos = grid.expand(B, N, 3)
    out = []
    for a in range(3):
        i = torch.arange(cols[a] // 2, dtype=torch.float64, device="cuda")
        out.append(pos[..., a, None].double() * theta ** (-2 * i / max(cols[a], 1)))
    ang = torch.cat(out, -1)
    rest = s.d // 2 - ang.shape[-1]
    return torch.cat([ang, torch.zeros(*ang.shape[:-1], rest, dtype=torch.float64, device="cuda")], -1)[:, :, None]


def rotate(x, ang, half):
    d = x.shape[-1]
    a, b = (x[..., :d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    c, s = ang.cos(), ang.sin()
    r = (a * c - b * s, a * s + b * c)
    return torch.cat(r, -1) if half else torch.stack(r, -1).flatten(-2)


def magnitude(m, half):
    """Of each turned value: those of its pair, added."""
    d = m.shape[-1]
    a, b = (m[..., :d // 2], m[..., d // 2:]) if half else (m[..., 0::2], m[..., 1::2])
    t = a + b
    return torch.cat([t, t], -1) if half else torch.stack([t, t], -1).flatten(-2)


def order(s):
    n = torch.arange(s.N, device="cuda").view(s.T // s.ta, s.ta, s.Y // s.tb, s.tb, s.X // s.tc, s.tc)
    return n.permute(0, 2, 4, 1, 3, 5).reshape(-1)


def ref_norm(x, w, b, rms, eps=EPS):
    x = x.double()
    mu = torch.zeros_like(x[..., :1]) if rms else x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mu) * rstd
    y = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return y, xh, rstd


def close(got, ref, tol, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off"


def setup(dims, dtype, rms, half, packed, seed):
    s = shape_of(dims, dtype)
    g = gen(seed)
    q, k = inputs(dims, s, g, packed)
    cols = cols_of(s.d) if dims[4] else (s.d, 0, 0)
    if not half and dims[4]:
        cols = (cols[0] - 6, cols[1], cols[2])    # some pairs do not turn
    pos, ext = None, (s.T, s.Y, s.X)
    if packed:
        ext = tuple(v + 9 for v in ext)
        pos = torch.stack([torch.randint(0, v, (s.B, s.N), generator=g, device="cuda") for v in ext], -1).int()
    table = sp.rope_table(s, cols, extent=ext, half=half)
    w = [1 + 0.3 * torch.randn(s.d, generator=g, device="cuda") for _ in range(2)]
    b = [None if rms else 0.5 * torch.randn(s.d, generator=g, device="cuda") for _ in range(2)]
    return s, g, q, k, table, pos, angles(s, pos, cols), w, b


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("dtype,rms,half,packed", CASES)
def test_forward(dims, dtype, rms, half, packed):
    s, g, q, k, table, pos, ang, w, b = setup(dims, dtype, rms, half, packed, 1)
    tiles = dims[4] is not None
    means = [torch.full((s.B, x.shape[2], s.nb, s.d), 9.0, device="cuda") if tiles else None for x in (q, k)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = sp.norm_rope_fwd(s, table, q, k, *w, *b, eps=EPS, rms=rms, pos=pos, out_blocked=tiles, q_means=means[0],
                            k_means=means[1], status=status)
    assert int(status) == 0
    alone, none = sp.norm_rope_fwd(s, table, q, None, w[0], None, b[0], None, eps=EPS, rms=rms, pos=pos, out_blocked=False)
    assert none is None
    for x, got, m, wi, bi in zip((q, k), outs, means, w, b):
        y, xh, rstd = ref_norm(x, wi, bi, rms)
        mag = (x.double().abs() * rstd + 1) * (1 + xh.abs()) * wi.double().abs() + (0 if bi is None else bi.double().abs())
        y, mag = rotate(y, ang, half), magnitude(mag, half)
        tol = sp_half(s) * y.abs() + DEEP * mag
        if x is q:
            close(alone, y, tol, "q alone, raster")
        if tiles:
            y, tol, mag = (t[:, order(s)].transpose(1, 2) for t in (y, tol, mag))
            cut = lambda t: t.reshape(s.B, -1, s.nb, s.Bt, s.d).mean(3)
            close(m, cut(y), 2 * DEEP * cut(mag), "means")
        close(got, y, tol, "y")


def sp_half(s):
    return torch.finfo(s.torch_dtype).eps / 2


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("dtype,rms,half,packed", CASES)
def test_backward(dims, dtype, rms, half, packed):
    s, g, q, k, table, pos, ang, w, b = setup(dims, dtype, rms, half, packed, 2)
    blocked = dims[4] is not None and dtype == "f32"
    raster = [(0.1 * torch.randn(s.B, s.N, x.shape[2], s.d, generator=g, device="cuda")).to(s.torch_dtype) for x in (q, k)]
    dy = [t[:, order(s)].transpose(1, 2).contiguous() for t in raster] if blocked else raster
    H, Hk = q.shape[2], k.shape[2]
    wide = torch.full((s.B, s.N, H + 2 * Hk, s.d), 7.0, device="cuda", dtype=s.torch_dtype)
    db = [torch.empty(s.d, device="cuda") for _ in range(2)]
    dq, dk, dw, db = sp.norm_rope_bwd(s, table, *dy, q, k, *w, eps=EPS, rms=rms, pos=pos, in_blocked=blocked,
                                      dq=wide[:, :, :H], dk=wide[:, :, H:H + Hk], db=db)
    assert (wide[:, :, H + Hk:] == 7.0).all()   # the rest of the wider tensor is left as it was
    for x, up, wi, got, gw_, gb_ in zip((q, k), raster, w, (dq, dk), dw, db):
        _, xh, rstd = ref_norm(x, wi, None, rms)
        gr = rotate(up.double(), -ang, half)
        gmag = magnitude(up.double().abs(), half)
        xmag = x.double().abs() * rstd + 1
        gw, gwm = gr * wi.double(), gmag * wi.double().abs()
        mean = lambda t: t.mean(-1, keepdim=True)
        ref = gw - xh * mean(gw * xh)
        mag = gwm + xmag * (1 + xh.abs()) * mean(gwm * xmag) * 2
        if not rms:
            ref, mag = ref - mean(gw), mag + mean(gwm)
        close(got, ref * rstd, sp_half(s) * (ref * rstd).abs() + DEEP * mag * (1 + xh.abs()) * rstd, "dx")
        tot = lambda t: t.sum((0, 1, 2))
        close(gw_, tot(gr * xh), (LONG + DEEP) * tot(gmag * xmag * (1 + xh.abs())), "dw")
        close(gb_, tot(gr), (LONG + DEEP) * tot(gmag), "db")
    again = sp.norm_rope_bwd(s, table, *dy, q, k, *w, eps=EPS, rms=rms, pos=pos, in_blocked=blocked)
    assert torch.equal(again[0], dq) and torch.equal(again[1], dk)
    assert torch.equal(again[2][0], dw[0]) and torch.equal(again[2][1], dw[1])


@pytest.mark.parametrize("rms,half", [(True, False), (False, True)])
def test_backward_against_differences(rms, half):
    """<dx, v> against the central difference of sum(dy y) along v in float64: its own error
    is h^2 / 6 times a third derivative of order 1 per value, its rounding 2^-53 / h."""
    dims = (1, 3, 2, (2, 8, 8), (2, 8, 8), 64)
    s, g, q, k, table, pos, ang, w, b = setup(dims, "f32", rms, half, False, 3)
    dy = [torch.randn(s.B, s.N, x.shape[2], s.d, generator=g, device="cuda") for x in (q, k)]
    dq, dk, dw, db = sp.norm_rope_bwd(s, table, *dy, q, k, *w, eps=EPS, rms=rms)
    h = 1e-4
    for x, up, wi, dx, gw in zip((q, k), dy, w, (dq, dk), dw):
        f = lambda x, wt: (rotate(ref_norm(x, wt, None, rms)[0], ang, half) * up.double()).sum()
        v = torch.randn(x.shape, generator=g, device="cuda").double()
        diff = (f(x.double() + h * v, wi.double()) - f(x.double() - h * v, wi.double())) / (2 * h)
        scale = (dx.double().abs() * v.abs()).sum()
        assert abs(float((dx.double() * v).sum() - diff)) <= 1e-6 * float(scale)
        u = torch.randn(s.d, generator=g, device="cuda").double()
        diff = (f(x.double(), wi.double() + h * u) - f(x.double(), wi.double() - h * u)) / (2 * h)
        scale = x[..., 0].numel() * float(u.abs().sum())
        assert abs(float((gw.double() * u).sum() - diff)) <= 1e-6 * scale


def test_positions_outside_the_table():
    s = sp.make_shape(1, 2, 70, 1, 1, 64, 1, 1, 1, "bf16")
    g = gen(5)
    x = torch.randn(1, 70, 2, 64, generator=g, device="cuda").bfloat16()
    table = sp.rope_table(s, (64, 0, 0), extent=(100, 1, 1))
    pos = torch.randint(0, 100, (1, 70, 3), generator=g, device="cuda").int()
    good = sp.norm_rope_fwd(s, table, x, rms=True, pos=pos, out_blocked=False)[0]
    bad = pos.clone()
    bad[0, 3, 0], bad[0, 69, 0] = 100, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sp.norm_rope_fwd(s, table, x, rms=True, pos=bad, out_blocked=False, status=status)[0]
    assert int(status) == sp.DATA
    bad[0, 3, 0] = bad[0, 69, 0] = 0        # not turned
    assert torch.equal(got, sp.norm_rope_fwd(s, table, x, rms=True, pos=bad, out_blocked=False)[0])
    keep = [i for i in range(70) if i not in (3, 69)]
    assert torch.equal(got[:, keep], good[:, keep])
    pos[..., 1:] = -5                       # axes without columns are not looked at
    status.zero_()
    assert torch.equal(sp.norm_rope_fwd(s, table, x, rms=True, pos=pos, out_blocked=False, status=status)[0], good)
    assert int(status) == 0


def test_given_stream_and_capture():
    dims = (1, 8, 2, (4, 8, 8), (1, 8, 8), 128)
    s, g, q, k, table, pos, ang, w, b = setup(dims, "bf16", True, True, True, 6)
    want = sp.norm_rope_fwd(s, table, q, k, *w, rms=True, pos=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sp.norm_rope_fwd(s, table, q, k, *w, rms=True, pos=pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.norm_rope_fwd(s, table, q, k, *w, rms=True, pos=pos, q_out=out[0], k_out=out[1])
    q.copy_(q.flip(1))
    graph.replay()
    assert torch.equal(out[1], want[1])
    assert torch.equal(out[0], sp.norm_rope_fwd(s, table, q, k, *w, rms=True, pos=pos)[0])
