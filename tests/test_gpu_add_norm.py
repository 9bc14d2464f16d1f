"""GPU parity of the residual addition with RMS norm, and of the rotary positions, with the
float64 oracles.

u = 2^-24 is fp32's half step, U the output type's. A row's sum of squares is 38 additions deep
at most (16 elements a lane, 6 steps across a wave, 16 waves) with one rounding a product: 40 u
of it, half of that for rstd and 4 u for its root. Forward, from the stored h: y is off by 27 u
|y| and U |y|; its 8-bit form by half a step of e4m3, 2^-4 of the value or 2^-10 of the block's
power, besides; a block's power is the one of some y within 27 u. Backward, from given rstd:
n = h rstd is off by u |n|, a = dy (offset + w) by 2 u |a|, mean(a n) by 45 u mean |a n|, so d by
rstd times (4 u |a| + 50 u |n| mean |a n|), 3 u (|dh| + |d|) and U |d|. The weight's gradient: as
the norms' own (a lane's rows, a block's teams, the blocks' sums).
Rotary: the fraction of a turn is rounded to fp32 (2^-25 of a half turn: pi 2^-25), the sine
and cosine are off by 2 u more and the two products and their sum by 3 u: 8 u (|p| + |q|), U |y|.
"""
import numpy as np
import pytest

from oracle import blocks8_oracle as Q
from oracle import norm_oracle as N
from oracle import rotary_oracle as R
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B

from test_gpu_blocks8 import decode, dtype_of, log, torch_dev  # noqa: F401
from test_gpu_norm import TYPES, U32, draw, host, round_tol, row_depth, within

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-6))


def check_forward(torch, name, rname, x, r, w, offset, **more):  # noqa: F811
    rows, cols = x.numel() // x.shape[-1], x.shape[-1]
    kept = None if r is None else host(r)
    h, y, y8, rstd = muon.add_rms_norm_forward(x, r, w, eps=1e-6, weight_offset=offset, codes=True, **more)
    torch.cuda.synchronize()
    if r is None:
        assert h is None
        hs = host(x)
    else:
        assert h.dtype == r.dtype and h.shape == x.shape
        want = host(x) + kept
        within(host(h), want, U32 * np.abs(want) + round_tol(rname, want) * (1 + 2 * U32), "h")
        hs = host(h)
    ry, _, rrstd, _, _ = N.norm_forward(hs, None if w is None else host(w).reshape(-1), None, "rms", EPS, offset)
    ry, rrstd = ry[0], rrstd[0]
    within(host(rstd), rrstd, 24 * U32 * rrstd, "rstd")
    worst = within(host(y).reshape(ry.shape), ry, 27 * U32 * np.abs(ry) + round_tol(name, ry), "y")
    assert y.dtype == x.dtype and y.shape == x.shape and y8.shape == (rows, cols) and not y8.tiles
    vals, e = decode(y8)
    s = 2.0 ** Q.spread(e, ry.shape).astype(float)
    within(vals, ry, 28 * U32 * np.abs(ry) + np.maximum(2.0 ** -4 * np.abs(ry) * 1.001, 2.0 ** -10 * s * 1.001), "codes")
    low, high = Q.powers(ry * (1 - 28 * U32)), Q.powers(ry * (1 + 28 * U32))
    assert ((e == low) | (e == high)).all(), "powers"
    return h, rstd, worst


def check_backward(torch, name, rname, dy, dh, h, w, rstd, offset, **more):  # noqa: F811
    rows, cols = h.numel() // h.shape[-1], h.shape[-1]
    g, hh, dd = host(dy).reshape(rows, cols), host(h).reshape(rows, cols), 0.0 if dh is None else host(dh).reshape(rows, cols)
    dx, dr, dw = muon.add_rms_norm_backward(dy, dh, h, w, rstd, weight_offset=offset, **more)
    torch.cuda.synchronize()
    rdx, rdw, _, n, a = N.norm_backward(g, hh, None if w is None else host(w).reshape(-1), None, host(rstd), "rms", offset)
    rd, n, a, r = rdx[0] + dd, n[0], a[0], host(rstd).reshape(-1, 1)
    mean = np.abs(a * n).mean(1, keepdims=True)
    tol = r * (4 * U32 * np.abs(a) + 50 * U32 * np.abs(n) * mean) + 3 * U32 * (np.abs(dd) + np.abs(rd))
    worst = within(host(dr).reshape(rd.shape), rd, tol + round_tol(rname, rd), "dr")
    within(host(dx).reshape(rd.shape), rd, tol + round_tol(name, rd), "dx")
    assert dr.dtype == h.dtype and dx.dtype == dy.dtype and dx.shape == dy.shape
    if w is None:
        assert dw is None
    else:
        mag = (np.abs(g) * np.abs(n)).sum(0)
        wname = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[w.dtype]
        within(host(dw).reshape(-1), rdw[0], (row_depth(name, cols, rows, 1) + 4) * U32 * mag + round_tol(wname, rdw[0]), "dw")
        assert dw.shape == w.shape and dw.dtype == w.dtype
    return worst


COLS = [1, 2, 3, 5, 7, 8, 9, 31, 64, 65, 100, 127, 128, 129, 250, 256, 300, 512, 513, 1000, 1153, 2048, 2050, 4097, 5120, 9000, 16384]


@pytest.mark.parametrize("name,rname,wname", [("f32", "f32", "f32"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"),
                                              ("f16", "f32", "f32"), ("f16", "f16", "f16")])
def test_add_norm(torch_dev, name, rname, wname):  # noqa: F811
    """Every width's split over lanes and waves, with and without residual, dh and weight."""
    torch, dev = torch_dev
    dt, rdt, wdt = dtype_of(torch, name), dtype_of(torch, rname), dtype_of(torch, wname)
    for i, cols in enumerate(COLS):
        rows = (1, 3, 70)[i % 3]
        offset = float(i % 2)
        x = draw(torch, dev, 600 + i, 0, (rows, cols), dt, 0.5)
        r = draw(torch, dev, 600 + i, 1, (rows, cols), rdt, 1.5, 0.3)
        w = draw(torch, dev, 600 + i, 2, (cols,), wdt, 0.3, 1.0 - offset) if i % 4 else None
        h, rstd, wf = check_forward(torch, name, rname, x, r, w, offset)
        dy = draw(torch, dev, 600 + i, 3, (rows, cols), dt)
        dh = draw(torch, dev, 600 + i, 4, (rows, cols), rdt) if i % 5 else None
        wb = check_backward(torch, name, rname, dy, dh, h, w, rstd, offset)
        _, rstd, _ = check_forward(torch, name, name, x, None, w, offset)
        check_backward(torch, name, name, dy, None, x, w, rstd, offset)
        log(f"{name} residual {rname} w {wname} {rows} x {cols}: {wf:.2f}, {wb:.2f} of the bound")


@pytest.mark.parametrize("rows,cols,name", [(4999, 1153, "f32"), (8192, 512, "bf16"), (70000, 96, "bf16"), (2050, 5120, "bf16"), (900, 12000, "f16")])
def test_many_rows(torch_dev, rows, cols, name):  # noqa: F811
    torch, dev = torch_dev
    dt = dtype_of(torch, name)
    x, r, dy, dh = (draw(torch, dev, 640, i, (rows, cols), dt, 1.0 + i) for i in range(4))
    w = draw(torch, dev, 640, 5, (cols,), torch.float32, 0.3, 1.0)
    h, rstd, _ = check_forward(torch, name, name, x, r, w, 0.0)
    check_backward(torch, name, name, dy, dh, h, w, rstd, 0.0)
    again = muon.add_rms_norm_backward(dy, dh, h, w, rstd)
    assert all(torch.equal(a, b) for a, b in zip(again, muon.add_rms_norm_backward(dy, dh, h, w, rstd)))


@pytest.mark.parametrize("cols", [7, 129, 1153, 2050, 6001])
@pytest.mark.parametrize("name,rname", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_in_place_and_strides(torch_dev, cols, name, rname):  # noqa: F811
    """h over the residual, d over dh, rows inside larger ones whose rest stays."""
    torch, dev = torch_dev
    rows, dt, rdt = 300, dtype_of(torch, name), dtype_of(torch, rname)
    big = draw(torch, dev, 650, 0, (rows, 2, cols + 3), dt)
    stream = draw(torch, dev, 650, 1, (rows, cols + 5), rdt, 1.5)
    x, r = big[:, 1, 1:-2], stream[:, 2:-3]
    w = draw(torch, dev, 650, 2, (cols,), torch.float32, 0.3, 1.0)
    want = muon.add_rms_norm_forward(x, r, w, codes=True)
    kept = stream.clone()
    h, rstd, _ = check_forward(torch, name, rname, x, r, w, 0.0, residual_out=r)
    assert h is r and torch.equal(r, want[0]) and torch.equal(rstd, want[3])
    kept[:, 2:-3] = r
    assert torch.equal(stream, kept)
    dy, dh = draw(torch, dev, 650, 3, (rows, cols), dt), draw(torch, dev, 650, 4, (rows, cols + 1), rdt)[:, 1:]
    ref = muon.add_rms_norm_backward(dy, dh, h, w, rstd)
    check_backward(torch, name, rname, dy, dh, h, w, rstd, 0.0, out=dh)
    assert torch.equal(dh, ref[1])
    over = h.clone()
    got = muon.add_rms_norm_backward(dy, None, over, w, rstd, out=over)
    assert torch.equal(got[1], muon.add_rms_norm_backward(dy, None, h, w, rstd)[1])
    if name == rname:
        same = dy.clone()
        got = muon.add_rms_norm_backward(same, None, h, w, rstd, out=same)
        assert got[0] is same and torch.equal(same, muon.add_rms_norm_backward(dy, None, h, w, rstd)[0])


def test_special_rows(torch_dev):  # noqa: F811
    """Rows of zeros, with infinities and NaN, the largest and smallest values: what they touch
    is their row alone, and the 8-bit form follows the norm's output."""
    torch, dev = torch_dev
    x = draw(torch, dev, 660, 0, (12, 700), torch.float32)
    r = torch.zeros_like(x)
    x[0] = 0.0
    x[1, 3], x[2, 699] = float("nan"), float("inf")
    x[3] *= 1e18
    x[4] *= 1e-30
    x[5, 5], r[5, 5] = float("inf"), float("-inf")
    h, y, y8, rstd = muon.add_rms_norm_forward(x, r, codes=True)
    clean = muon.add_rms_norm_forward(x[6:], r[6:], codes=True)
    torch.cuda.synchronize()
    assert torch.equal(y[6:], clean[1]) and torch.equal(y8.codes[6:].view(torch.uint8), clean[2].codes.view(torch.uint8))
    assert not y[0].any() and not y8.dequantise()[0].any()
    assert float(rstd[2]) == 0.0 and bool(y[2, 699].isnan()) and not y[2, :699].any()
    assert bool(y[1].isnan().all()) and bool(y[5].isnan().all()) and bool(h[5, 5].isnan())
    assert bool(y[3:5].isfinite().all())
    back = y8.dequantise()
    assert torch.equal(back.isnan(), y.isnan())


@pytest.mark.parametrize("name,rname", [("bf16", "f32"), ("f32", "f32")])
def test_add_norm_autograd(torch_dev, name, rname):  # noqa: F811
    """Two steps of a residual stream against torch's own gradients in float64."""
    torch, dev = torch_dev
    dt, rdt = dtype_of(torch, name), dtype_of(torch, rname)
    x1, x2 = (draw(torch, dev, 670, i, (5, 40, 200), dt).requires_grad_() for i in (0, 1))
    r = draw(torch, dev, 670, 2, (5, 40, 200), rdt, 1.5).requires_grad_()
    w = draw(torch, dev, 670, 3, (200,), torch.float32, 0.3, 1.0).requires_grad_()
    g1, g2 = (draw(torch, dev, 670, i, (5, 40, 200), dt) for i in (4, 5))
    y1, h1 = muon.add_rms_norm(x1, r, w)
    y2, h2 = muon.add_rms_norm(x2, h1, w)
    ((y1.float() * g1).sum() + (y2.float() * g2).sum() + h2.float().square().sum()).backward()
    leaves = [t.detach().double().requires_grad_() for t in (x1, x2, r, w)]

    def norm(h, w):
        return h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w

    a = leaves[0] + leaves[2]
    b = leaves[1] + a
    ((norm(a, leaves[3]) * g1).sum() + (norm(b, leaves[3]) * g2).sum() + b.square().sum()).backward()
    # fp32 throughout but for the types' roundings on the way: y and its gradient, dx
    step = TYPES[name][0]
    for got, ref, tol in ((x1.grad, leaves[0].grad, step), (x2.grad, leaves[1].grad, step), (r.grad, leaves[2].grad, 2.0 ** -20), (w.grad, leaves[3].grad, 2.0 ** -18)):
        assert got.dtype in (torch.float32, dt)
        assert float((got.double() - ref).norm() / ref.norm()) < 2 * tol + 2.0 ** -18
    # outputs that are not used
    for use in (0, 1):
        t = x1.detach().requires_grad_()
        out = muon.add_rms_norm(t, r.detach(), w.detach())[use]
        out.float().sum().backward()
        assert bool(t.grad.isfinite().all())
        if use:
            assert bool((t.grad == 1).all())
    y, h = muon.add_rms_norm(x1, None, w)
    assert h is None
    x1.grad = None
    y.float().sum().backward()
    assert bool(x1.grad.isfinite().all())


# ---------------------------------------------------------------- rotary ----

def check_rotary(torch, name, x, pos, sections, layout, inverse=False, axes=None, ladder=None, **more):  # noqa: F811
    axes = axes or muon.RotaryAxes(sections, layout=layout, device=x.device)
    freq, axis = ladder or R.ladder(sections)
    hx = host(x)
    got = muon.rotary_apply(x, pos, axes, inverse=inverse, **more)
    torch.cuda.synchronize()
    want = R.rotate(hx, host(pos), freq, axis, layout, inverse)
    n = len(freq)
    mag = np.zeros(hx.shape)
    p, q = (slice(0, n), slice(n, 2 * n)) if layout == "halves" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    mag[..., p] = mag[..., q] = np.abs(hx[..., p]) + np.abs(hx[..., q])
    # the angle itself in float64: a position of 2^40 leaves 2^-12 of a radian
    far = np.abs(host(pos)).max(initial=0.0) * 2.0 ** -51
    within(host(got), want, (8 * U32 + far) * mag + round_tol(name, want) * (mag > 0), "y")
    assert got.shape == x.shape and got.dtype == x.dtype
    return got


@pytest.mark.parametrize("layout", ["halves", "adjacent"])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_rotary(torch_dev, name, layout):  # noqa: F811
    """Head sizes and sections that vectors divide and do not, one token to many, every type of
    position, forward and back."""
    torch, dev = torch_dev
    dt = dtype_of(torch, name)
    cases = [((16, 24, 24), 128, 1, 32), ((64,), 128, 5, 3), ((7, 13, 13), 90, 130, 5), ((1,), 2, 3, 1), ((1,), 3, 4, 2), ((2, 0, 3), 11, 6, 7),
             ((16, 56, 56), 256, 20, 3), ((128, 128), 513, 9, 2), ((20, 20), 80, 700, 1), ((4,), 8, 3000, 16), ((8, 12, 12), 72, 65, 24), ((512,), 1024, 4, 3)]
    for i, (sections, dim, tokens, heads) in enumerate(cases):
        x = draw(torch, dev, 700 + i, 0, (tokens, heads, dim), dt, 1.5)
        pos = torch.from_numpy(np.random.default_rng(i).integers(-50, 20000, (tokens, len(sections)))).to(dev)
        for j, kind in enumerate((torch.int32, torch.int64, torch.float32)):
            p = pos.to(kind) if j < 2 else pos.to(kind) * 0.375
            check_rotary(torch, name, x, p, sections, layout, inverse=bool((i + j) % 2))
        log(f"{name} {layout} {sections} of {dim}, {tokens} tokens x {heads}")


def test_rotary_far_positions(torch_dev):  # noqa: F811
    """Positions past 2^24, past 2^31, below zero and at zero; infinite ones give NaN."""
    torch, dev = torch_dev
    pos = torch.tensor([[0], [-1], [2 ** 24 + 1], [2 ** 31 + 7], [-2 ** 33 - 3], [2 ** 40 + 1]], device=dev)
    x = draw(torch, dev, 720, 0, (6, 3, 64), torch.float32)
    got = check_rotary(torch, "f32", x, pos, (32,), "halves")
    assert torch.equal(got[0], x[0])
    bad = torch.tensor([[float("inf")], [float("nan")], [1.0]], device=dev)
    y = muon.rotary_apply(x[:3], bad, muon.RotaryAxes((30,), device=dev))
    assert bool(y[:2, :, :60].isnan().all()) and bool(y[2].isfinite().all()) and torch.equal(y[..., 60:], x[:3, :, 60:])


@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("dim,sections", [(128, (16, 24, 24)), (90, (7, 13, 13))])
def test_rotary_views_and_in_place(torch_dev, name, dim, sections):  # noqa: F811
    """Query and key heads of a fused projection in place, heads before tokens, a batch with the
    same positions, infinities in elements that are not turned."""
    torch, dev = torch_dev
    dt, axes = dtype_of(torch, name), muon.RotaryAxes(sections, device=dev)
    batch, tokens, heads = 3, 70, 4
    qkv = draw(torch, dev, 730, 0, (batch, tokens, 3 * heads, dim), dt)
    pos = torch.from_numpy(np.random.default_rng(3).integers(0, 500, (tokens, 3)).astype(np.int32)).to(dev)
    want = check_rotary(torch, name, qkv[:, :, :2 * heads], pos.expand(batch, tokens, 3), sections, "halves")
    for p in (pos, pos[None], pos.expand(batch, tokens, 3), pos.expand(batch, tokens, 3).contiguous()):
        assert torch.equal(muon.rotary_apply(qkv[:, :, :2 * heads], p, axes), want)
    kept = qkv.clone()
    out = muon.rotary_apply(qkv[:, :, :2 * heads], pos, axes, out=qkv[:, :, :2 * heads])
    assert torch.equal(out, want) and torch.equal(qkv[:, :, 2 * heads:], kept[:, :, 2 * heads:])
    turned = kept[:, :, :2 * heads].permute(0, 2, 1, 3).contiguous()  # [batch, heads, tokens, dim]
    got = muon.rotary_apply(turned.transpose(1, 2), pos, axes, out=turned.transpose(1, 2))
    assert torch.equal(got, want) and torch.equal(turned.transpose(1, 2), want)
    one = muon.rotary_apply(kept[0, 0, :2 * heads], pos[0], axes)
    assert torch.equal(one, want[0, 0])
    if dim > 2 * axes.pairs:
        kept[..., -1] = float("inf")
        assert bool((muon.rotary_apply(kept, pos, axes)[..., -1] == float("inf")).all())
        assert torch.equal(muon.rotary_apply(kept, pos, axes)[:, :, :2 * heads, :-1], want[..., :-1])
    empty = muon.rotary_apply(kept[:, :0], pos[:0], axes)
    assert empty.shape == (batch, 0, 3 * heads, dim)


@pytest.mark.parametrize("layout", ["halves", "adjacent"])
@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_rotary_in_place_of_odd_heads(torch_dev, name, layout):  # noqa: F811
    """Heads that vectors do not divide, of fewer elements than a vector and of more vectors than
    a wave has lanes."""
    torch, dev = torch_dev
    for i, (pairs, dim) in enumerate(((3, 7), (1, 2), (9, 19), (61, 125), (300, 601), (509, 1019))):
        x = draw(torch, dev, 735 + i, 0, (40, 5, dim), dtype_of(torch, name))
        pos = torch.arange(40, device=dev)[:, None]
        want = check_rotary(torch, name, x, pos, (pairs,), layout)
        assert torch.equal(check_rotary(torch, name, x, pos, (pairs,), layout, out=x), want)
        log(f"{name} {layout} {pairs} pairs of {dim}")


def test_rotary_own_frequencies(torch_dev):  # noqa: F811
    """Axes dealt out pair by pair."""
    torch, dev = torch_dev
    freq, axis = R.ladder((12,))[0], np.arange(12) % 3
    axes = muon.RotaryAxes((4, 4, 4), frequencies=freq, axis_of_pair=axis, layout="adjacent", device=dev)
    x = draw(torch, dev, 740, 0, (50, 2, 24), torch.float32)
    pos = torch.from_numpy(np.random.default_rng(5).integers(0, 300, (50, 3))).to(dev)
    check_rotary(torch, "f32", x, pos, None, "adjacent", axes=axes, ladder=(freq, axis))


def test_rotary_far_apart_rows(torch_dev):  # noqa: F811
    """Heads past 2^32 elements from the start."""
    torch, dev = torch_dev
    x = torch.empty((600, 1 << 23), dtype=torch.bfloat16, device=dev)[:, :128].view(600, 2, 64)
    x.copy_(draw(torch, dev, 745, 0, (600, 2, 64), torch.bfloat16))
    pos = torch.arange(600, device=dev)[:, None]
    check_rotary(torch, "bf16", x, pos, (32,), "halves")
    check_rotary(torch, "bf16", x, pos, (32,), "halves", out=x)


def test_rotary_autograd(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    axes = muon.RotaryAxes((3, 5, 5), device=dev)
    pos = torch.from_numpy(np.random.default_rng(6).integers(0, 90, (33, 3))).to(dev)
    x = draw(torch, dev, 750, 0, (2, 33, 4, 30), torch.float32).requires_grad_()
    g = draw(torch, dev, 750, 1, (2, 33, 4, 30), torch.float32)
    y = muon.rotary(x, pos, axes)
    y.backward(g)
    assert torch.equal(x.grad, muon.rotary_apply(g, pos, axes, inverse=True))
    # the map is linear: a difference of any size is the gradient's
    move = draw(torch, dev, 750, 2, x.shape, torch.float32)
    diff = float(((muon.rotary_apply(x.detach() + move, pos, axes).double() - y.detach().double()) * g.double()).sum())
    slope = float((x.grad.double() * move.double()).sum())
    # 26 (x + move and its rotation, y: 13 roundings of |x| + |move| each) u a product
    size = float(((x.detach().abs() + move.abs()).double() * g.double().abs().sum(-1, keepdim=True)).sum())
    assert abs(diff - slope) <= 26 * U32 * size
    x.grad = None
    muon.rotary(x, pos, axes).transpose(1, 2).sum(-1).square().sum().backward()
    assert bool(x.grad.isfinite().all())


def test_streams_and_graph(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    x, r = draw(torch, dev, 760, 0, (300, 640), torch.bfloat16), draw(torch, dev, 760, 1, (300, 640), torch.bfloat16)
    w = draw(torch, dev, 760, 2, (640,), torch.float32, 0.3, 1.0)
    axes, pos = muon.RotaryAxes((8, 12, 12), device=dev), torch.arange(900, device=dev).view(300, 3)

    def step():
        h, y, y8, rstd = muon.add_rms_norm_forward(x, r, w, codes=True)
        q = muon.rotary_apply(y.view(300, 10, 64), pos, axes)
        dx, _, dw = muon.add_rms_norm_backward(q.view(300, 640), h, h, w, rstd)
        return h, y, y8.codes.view(torch.uint8), q, dx, dw

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [step() for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for t in got for a, b in zip(t, want))
    h = muon.add_rms_norm_forward(x, r, w, stream=streams[0])[0]
    q = muon.rotary_apply(h.view(300, 10, 64), pos, axes, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(h, want[0]) and q.shape == (300, 10, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(draw(torch, dev, 770 + i, 0, (300, 640), torch.bfloat16))
        pos += 3
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))


def test_python_refusals_on_the_gpu(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    x, w = torch.zeros(4, 16, device=dev), torch.ones(16, device=dev)
    bf, rstd = x.bfloat16(), torch.ones(4, device=dev)
    axes, pos = muon.RotaryAxes((2, 2), device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev)
    heads = torch.zeros(4, 2, 8, device=dev)
    cases = [(lambda: muon.add_rms_norm_forward(x, bf), "dtype"), (lambda: muon.add_rms_norm_forward(x, x[:3]), "shape"),
             (lambda: muon.add_rms_norm_forward(x, x.cpu()), "live on"), (lambda: muon.add_rms_norm_forward(x, x, w[:8]), "elements"),
             (lambda: muon.add_rms_norm_forward(x, x, w.bfloat16()), "dtype"), (lambda: muon.add_rms_norm_forward(x, x, w.view(1, 16).expand(4, 16)), "rows"),
             (lambda: muon.add_rms_norm_forward(x, residual_out=x), "without a residual"), (lambda: muon.add_rms_norm_forward(x.t(), x.t()), "adjacent"),
             (lambda: muon.add_rms_norm_forward(x, x, residual_out=bf), "dtype"),
             (lambda: muon.add_rms_norm_backward(x, bf, x, w, rstd), "dtype"), (lambda: muon.add_rms_norm_backward(x, None, bf, w, rstd), "dtype"),
             (lambda: muon.add_rms_norm_backward(x, None, x, w, rstd[:3]), "entry per row"),
             (lambda: muon.add_rms_norm_backward(x, None, x, w, rstd, out=bf), "dtype"),
             (lambda: muon.add_rms_norm_backward(x, None, x, w, rstd, workspace=torch.zeros(4, device=dev)), "uint8"),
             (lambda: muon.rotary_apply(heads, pos[:3], axes), "does not fit"), (lambda: muon.rotary_apply(heads, pos[:, :1], axes), "2 axes"),
             (lambda: muon.rotary_apply(heads[..., :6], pos, axes), "turn 8 elements"), (lambda: muon.rotary_apply(heads[0, 0], pos, axes), "last two"),
             (lambda: muon.rotary_apply(heads.double(), pos, axes), "float32"), (lambda: muon.rotary_apply(heads, pos.double(), axes), "positions must be"),
             (lambda: muon.rotary_apply(heads, pos.cpu(), axes), "live on"), (lambda: muon.rotary_apply(heads, pos, axes, out=heads[:3]), "out must"),
             (lambda: muon.rotary_apply(heads.transpose(1, 2), pos, muon.RotaryAxes((1, 0), device=dev)), "adjacent")]
    for call, text in cases:
        with pytest.raises(ValueError, match=text):
            call()
    for call in (lambda: muon.add_rms_norm_forward(x, x, residual_out=torch.zeros(64, device=dev).as_strided((4, 16), (8, 1))),
                 lambda: muon.rotary_apply(heads, pos, axes, out=torch.zeros(8, device=dev).as_strided((4, 2, 8), (0, 0, 1)))):
        with pytest.raises(B.MuonError):  # rows that overlap
            call()
