"""Token norm and three-axis rotary positions against plain float64 forms.

Tolerances. One rounding to the stored type is off by at most half a step:
eps/2 relative (bf16 2^-8, fp32 2^-24). fp32 arithmetic before it: a sum of n
terms in any order is off by at most n 2^-24 times the sum of their magnitudes,
and a row's statistics are sums of C terms taken by threads and then a tree, at
most 64 roundings deep in every shape here; the handful of products around
them add a few 2^-24. `DEEP` = 96 2^-24 covers both, applied to the magnitudes
that enter (not to the result, which may cancel)."""
import numpy as np
import pytest
import torch

import block_sparse_attention_token_gb300 as sp

pytestmark = [pytest.mark.gpu, pytest.mark.timeout(300)]

U32 = 2.0 ** -24
DEEP = 96 * U32
EPS = 1e-6

# B, H, T, Y, X, d, ta, tb, tc: one token tile, odd tile counts, several batches, rows of every kernel variant
# (8, 16, 32, 64, 128 vectors, CTA rows of two and four vectors a thread)
SHAPES = [
    (1, 1, 4, 4, 4, 64, 4, 4, 4),
    (2, 3, 2, 24, 8, 64, 2, 8, 8),
    (1, 2, 3, 8, 40, 128, 1, 8, 8),
    (1, 5, 2, 8, 24, 128, 2, 8, 8),
    (2, 7, 4, 8, 12, 128, 4, 4, 4),
    (1, 40, 2, 8, 8, 128, 2, 8, 8),
    (1, 127, 1, 8, 16, 128, 1, 8, 16),
]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def raster(shape, g, parts=1, mean=0.7, scale=1.0):
    """A raster tensor, the last of `parts` slices of a fused projection."""
    x = torch.randn(shape.B, shape.N, parts, shape.H, shape.d, generator=g, device="cuda") * scale + mean
    return x.to(shape.torch_dtype)[:, :, parts - 1]


def norm_ref(x, w, b, rms, per_head, eps=EPS):
    rows = x.double() if per_head else x.double().flatten(2)
    mu = torch.zeros_like(rows[..., :1]) if rms else rows.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((rows - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh = (rows - mu) * rstd
    y = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return y.view(x.shape), mu.squeeze(-1), rstd.squeeze(-1), xh, rows


def close(got, ref, tol, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of tol"


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rms,per_head,parts", [(False, False, 1), (True, False, 3), (False, True, 3), (True, True, 1)])
def test_norm_forward(dims, dtype, rms, per_head, parts):
    s = sp.make_shape(*dims, dtype)
    g = gen(1)
    x = raster(s, g, parts)
    cols = s.d if per_head else s.H * s.d
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    b = None if rms else 0.5 * torch.randn(cols, generator=g, device="cuda")
    y, mean, rstd = sp.norm_fwd(s, x, w, b, EPS, rms, per_head)
    yr, mu, rs, xh, rows = norm_ref(x, w, b, rms, per_head)
    big = rows.abs().amax(-1)
    if rms:
        assert mean is None
    else:
        close(mean, mu, DEEP * big, "mean")
    close(rstd, rs, DEEP * (1 + (big * rs) ** 2) * rs, "rstd")   # the error of the mean enters through x - mean
    mag = (rows.abs() * rs[..., None] + 1) * (1 + xh.abs()) * w.double().abs() + (0 if b is None else b.double().abs())
    close(y, yr, half_step(s.torch_dtype) * yr.abs() + DEEP * mag.view(yr.shape), "y")


@pytest.mark.parametrize("dims", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rms,per_head,parts", [(False, False, 3), (True, False, 1), (False, True, 1), (True, True, 3)])
def test_norm_backward(dims, dtype, rms, per_head, parts):
    s = sp.make_shape(*dims, dtype)
    g = gen(2)
    x, dy = raster(s, g, parts), raster(s, g, 1, 0.1)
    dy = dy.contiguous()
    cols = s.d if per_head else s.H * s.d
    w = 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")
    _, mean, rstd = sp.norm_fwd(s, x, w, None, EPS, rms, per_head)
    wide = torch.full((s.B, s.N, 2, s.H, s.d), 7.0, device="cuda", dtype=s.torch_dtype)
    db = torch.empty(cols, device="cuda")
    dx, dw, db = sp.norm_bwd(s, dy, x, w, mean, rstd, rms, per_head, dx=wide[:, :, 1], db=db)
    assert (wide[:, :, 0] == 7.0).all()   # the other slice is left as it was
    # the formula at the statistics the kernel is given
    rows, up = (x.double(), dy.double()) if per_head else (x.double().flatten(2), dy.double().flatten(2))
    rs = rstd.double()[..., None]
    xh = rows * rs if rms else (rows - mean.double()[..., None]) * rs
    gw = up * w.double()
    ref = gw - xh * (gw * xh).mean(-1, keepdim=True)
    mag = gw.abs() + xh.abs() * (gw * xh).abs().mean(-1, keepdim=True)
    if not rms:
        ref = ref - gw.mean(-1, keepdim=True)
        mag = mag + gw.abs().mean(-1, keepdim=True)
    mag = mag + (gw * rows.abs() * rs).abs().mean(-1, keepdim=True) * (1 + xh.abs())   # x - mean cancels in fp32
    ref, mag = (ref * rs).view(x.shape), (mag * rs).view(x.shape)
    close(dx, ref, half_step(s.torch_dtype) * ref.abs() + DEEP * mag, "dx")
    n = up.numel() // cols
    terms = (up.abs() * (rows.abs() * rs + xh.abs())).reshape(-1, cols).sum(0)
    close(dw, (up * xh).reshape(-1, cols).sum(0), (n + 16) * U32 * terms, "dw")
    close(db, up.reshape(-1, cols).sum(0), n * U32 * up.abs().reshape(-1, cols).sum(0), "db")


def test_norm_backward_is_the_derivative():
    """Central differences of sum(dy * y) in float64 of the forward's formula."""
    s = sp.make_shape(1, 2, 4, 4, 4, 64, 4, 4, 4, "f32")
    g = gen(3)
    x, dy = raster(s, g), raster(s, g).contiguous()
    w, b = (torch.randn(128, generator=g, device="cuda") for _ in range(2))
    _, mean, rstd = sp.norm_fwd(s, x, w, b, 1e-3)
    dx, dw, db = sp.norm_bwd(s, dy, x, w, mean, rstd)
    leaves = [t.double().requires_grad_() for t in (x, w, b)]
    rows = leaves[0].flatten(2)
    mu = rows.mean(-1, keepdim=True)
    y = (rows - mu) / torch.sqrt(((rows - mu) ** 2).mean(-1, keepdim=True) + 1e-3) * leaves[1] + leaves[2]

    def loss(x_, w_, b_):
        r = x_.flatten(2)
        m = r.mean(-1, keepdim=True)
        z = (r - m) / torch.sqrt(((r - m) ** 2).mean(-1, keepdim=True) + 1e-3) * w_ + b_
        return float((z.view(dy.shape) * dy.double()).sum())

    (y.view(dy.shape) * dy.double()).sum().backward()
    for name, got, leaf in zip(("dx", "dw", "db"), (dx, dw, db), leaves):
        tol = 1e-4 * leaf.grad.abs().max()    # 64-term sums of fp32 terms of magnitude up to 10: 64 * 10 * 2^-24
        close(got, leaf.grad, torch.full_like(leaf.grad, float(tol)), name)
    base = [t.detach().double() for t in (x, w, b)]
    for which, got in ((0, dx), (1, dw), (2, db)):
        for at in (0, 37, 111):
            step = 1e-4
            moved = []
            for sign in (1, -1):
                args = [t.clone() for t in base]
                args[which].view(-1)[at] += sign * step
                moved.append(loss(*args))
            diff = (moved[0] - moved[1]) / (2 * step)
            # differences: step^2 of the third derivative (order 1) and 2^-52 * |loss| / step
            assert abs(diff - float(got.view(-1)[at])) <= 1e-4 * max(1.0, abs(diff)), (which, at)


def test_norm_special_rows():
    """A constant row has variance 0 (y = b); a row of large mean keeps its digits;
    NaN and infinity stay in their row."""
    s = sp.make_shape(1, 2, 4, 4, 4, 64, 4, 4, 4, "f32")
    g = gen(4)
    x = raster(s, g)
    x[0, 0] = 3.0
    x[0, 1] = 4096.0 + torch.randn(2, 64, generator=g, device="cuda")
    x[0, 2, 1, 5] = float("nan")
    x[0, 3, 0, 7] = float("inf")
    w, b = torch.ones(128, device="cuda"), torch.full((128,), 0.25, device="cuda")
    y, mean, rstd = sp.norm_fwd(s, x, w, b, EPS)
    assert (y[0, 0] == 0.25).all()
    yr = norm_ref(x, w, b, False, False)[0]
    # x has 2^-24 * 4096 of resolution and mean as much error: both relative to a deviation of order 1
    close(y[0, 1], yr[0, 1], torch.full_like(yr[0, 1], 4096 * DEEP), "large mean")
    assert not torch.isfinite(y[0, 2:4]).any(-1).all()
    assert torch.isfinite(y[0, 4:]).all()
    y2, _, _ = sp.norm_fwd(s, x, None, None, EPS, per_head=True)
    assert torch.isnan(y2[0, 2, 1]).all() and torch.isfinite(y2[0, 2, 0]).all()


@pytest.mark.parametrize("per_head", [False, True])
def test_norm_backward_with_some_gradients(per_head):
    """dw and db are written only where asked for (through the C call: the binding always asks for dw)."""
    import ctypes
    s = sp.make_shape(1, 20, 4, 16, 16, 64, 4, 4, 4, "bf16")
    g = gen(10)
    x, dy = raster(s, g), raster(s, g).contiguous()
    w = torch.rand(64 if per_head else 1280, generator=g, device="cuda")
    _, mean, rstd = sp.norm_fwd(s, x, w, per_head=per_head)
    want = sp.norm_bwd(s, dy, x, w, mean, rstd, per_head=per_head)
    ws = torch.empty(sp.norm_workspace_size(s, per_head=per_head), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for ask_w, ask_b in ((False, False), (True, False), (False, True)):
        dx = torch.empty_like(dy)
        dw, db = torch.full_like(w, 7.0), torch.full_like(w, 7.0)
        code = sp.lib().sparsp_norm_bwd(
            ctypes.byref(s), sp.NORM_HEAD if per_head else 0, dy.data_ptr(), x.data_ptr(), 0, w.data_ptr(),
            mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), 0, dw.data_ptr() if ask_w else None,
            db.data_ptr() if ask_b else None, ws.data_ptr() if ask_w or ask_b else None, ws.numel(), stream)
        assert code == sp.OK and torch.equal(dx, want[0])
        assert torch.equal(dw, want[1]) if ask_w else (dw == 7.0).all()
        assert torch.equal(db, want[2]) if ask_b else (db == 7.0).all()


def test_norm_no_weight_and_repeatable():
    s = sp.make_shape(2, 12, 4, 16, 16, 128, 2, 8, 8, "bf16")
    g = gen(5)
    x, dy = raster(s, g), raster(s, g).contiguous()
    y, mean, rstd = sp.norm_fwd(s, x)
    ones = torch.ones(s.H * s.d, device="cuda")
    assert torch.equal(y, sp.norm_fwd(s, x, ones, torch.zeros_like(ones))[0])
    first = sp.norm_bwd(s, dy, x, None, mean, rstd)
    for _ in range(3):
        for a, b in zip(first, sp.norm_bwd(s, dy, x, ones, mean, rstd)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------- rotary positions

COLS = {64: [(24, 20, 20), (16, 16, 16), (0, 32, 32), (64, 0, 0)],
        128: [(44, 42, 42), (32, 32, 32), (2, 0, 126), (0, 0, 0)]}


def angles(shape, cols, theta, offset, scale, pos):
    """[B, N, sum(cols)/2] float64 angles."""
    out = []
    for ax in range(3):
        i = torch.arange(cols[ax] // 2, dtype=torch.float64, device="cuda")
        freq = theta ** (-2 * i / max(cols[ax], 1))
        out.append((offset[ax] + scale[ax] * pos[..., ax, None].double()) * freq)
    return torch.cat(out, -1)


def grid_pos(shape):
    n = torch.arange(shape.N, device="cuda")
    p = torch.stack([n // (shape.Y * shape.X), n // shape.X % shape.Y, n % shape.X], -1)
    return p.expand(shape.B, shape.N, 3)


def turn(x, phi, half):
    """float64 rotation of raster x by phi [B, N, pairs]."""
    x = x.double()
    d, m = x.shape[-1], phi.shape[-1]
    full = torch.zeros(*phi.shape[:2], d // 2, dtype=torch.float64, device="cuda")
    full[..., :m] = phi
    c, s = full.cos()[:, :, None], full.sin()[:, :, None]
    a, b = (x[..., : d // 2], x[..., d // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * s, a * s + b * c
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def to_blocked(shape, x):
    s = shape
    v = x.reshape(s.B, s.T // s.ta, s.ta, s.Y // s.tb, s.tb, s.X // s.tc, s.tc, s.H, s.d)
    return v.permute(0, 7, 1, 3, 5, 2, 4, 6, 8).reshape(s.B, s.H, s.N, s.d)


def rope_tol(dtype, ref, x):
    """cos and sin are rounded once (2^-24), each product and the sum once, the result to its type; the pair's
    magnitudes are at most |x| of the row's largest pair."""
    return half_step(dtype) * ref.abs() + 4 * U32 * 2 * x.double().abs().amax()


@pytest.mark.parametrize("dims", SHAPES[:6])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(5))
def test_rope_forward(dims, dtype, case):
    s = sp.make_shape(*dims, dtype)
    g = gen(6)
    half = case == 4
    cols = (s.d - 32, 16, 16) if half else COLS[s.d][case]
    off, scale, theta = (0.5, 0.0, 100000.0), (1.0, 0.5, 1.0), 10000.0   # far positions keep their angles
    tab = sp.rope_table(s, cols, theta, off, scale, half=half)
    x = raster(s, g, 1 + case % 3)
    means = torch.empty(s.B, s.H, s.nb, s.d, device="cuda")
    y = sp.rope(s, tab, x, means=means)
    ref = turn(x, angles(s, cols, theta, off, scale, grid_pos(s)), half)
    blocked = to_blocked(s, ref)
    close(y, blocked, rope_tol(s.torch_dtype, blocked, x), "blocked")
    m = blocked.view(s.B, s.H, s.nb, s.Bt, s.d)
    close(means, m.mean(3), (DEEP + 8 * U32) * 2 * x.double().abs().amax(), "means")
    flat = sp.rope(s, tab, x, out_blocked=False)
    assert torch.equal(to_blocked(s, flat), y)


@pytest.mark.parametrize("dims", SHAPES[:5])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_inverse_positions_and_layouts(dims, half, dtype):
    s = sp.make_shape(*dims, dtype)
    g = gen(7)
    cols = (s.d - 48, 24, 24)
    tab = sp.rope_table(s, cols, 500.0, extent=(9, 50, 60), half=half)
    pos = torch.stack([torch.randint(0, e, (s.B, s.N), generator=g, device="cuda") for e in (9, 50, 60)], -1).int()
    x = raster(s, g)
    phi = angles(s, cols, 500.0, (0,) * 3, (1,) * 3, pos)
    ref = turn(x, -phi, half)
    tol = rope_tol(s.torch_dtype, ref, x)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    back = sp.rope(s, tab, x, inverse=True, out_blocked=False, pos=pos, status=st)
    close(back, ref, tol, "raster")
    wide = torch.full((s.B, s.N, 2, s.H, s.d), 3.0, device="cuda", dtype=s.torch_dtype)
    xb = to_blocked(s, x).contiguous()
    sp.rope(s, tab, xb, out=wide[:, :, 0], inverse=True, in_blocked=True, out_blocked=False, pos=pos, status=st)
    assert torch.equal(wide[:, :, 0], back) and (wide[:, :, 1] == 3.0).all()
    bb = sp.rope(s, tab, xb, inverse=True, in_blocked=True, pos=pos, status=st)
    assert torch.equal(bb, to_blocked(s, back))
    # the inverse is the transpose: <turn x, z> = <x, turn^T z>
    if dtype == "f32":
        z = raster(s, g)
        left = (sp.rope(s, tab, x, out_blocked=False, pos=pos).double() * z.double()).sum()
        right = (x.double() * sp.rope(s, tab, z, inverse=True, out_blocked=False, pos=pos).double()).sum()
        bound = 8 * U32 * 2 * (x.double().abs().amax() * z.double().abs().sum() + z.double().abs().amax()
                               * x.double().abs().sum())
        assert abs(float(left - right)) <= float(bound)
    assert int(st) == 0


def test_rope_position_out_of_range():
    s = sp.make_shape(1, 2, 4, 4, 4, 64, 4, 4, 4, "f32")
    tab = sp.rope_table(s, (24, 20, 20))
    pos = grid_pos(s).int().contiguous()
    pos[0, 5] = torch.tensor([4, -1, 2], dtype=torch.int32)
    x = raster(s, gen(8))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sp.rope(s, tab, x, out_blocked=False, pos=pos, status=st)
    assert int(st) == sp.DATA
    want = sp.rope(s, tab, x, out_blocked=False)
    keep = [n for n in range(s.N) if n != 5]
    assert torch.equal(y[0, keep], want[0, keep])
    assert torch.equal(y[0, 5, :, :44], x[0, 5, :, :44])          # frame and row pairs are not turned


def test_norm_rope_on_another_stream_and_captured():
    s = sp.make_shape(1, 4, 4, 16, 16, 64, 4, 4, 4, "bf16")
    g = gen(9)
    x, dy = raster(s, g), raster(s, g).contiguous()
    w = torch.rand(s.d, generator=g, device="cuda") + 0.5
    tab = sp.rope_table(s, (24, 20, 20))
    ws = torch.empty(sp.norm_workspace_size(s, per_head=True), dtype=torch.uint8, device="cuda")

    def step():
        y, mean, rstd = sp.norm_fwd(s, x, w, per_head=True)
        z = sp.rope(s, tab, y)
        up = sp.rope(s, tab, dy, inverse=True, out_blocked=False)
        return (z, *sp.norm_bwd(s, up, x, w, mean, rstd, per_head=True, ws=ws))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    x.mul_(1.5)
    want = [t.clone() for t in step()]
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
