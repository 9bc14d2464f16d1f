"""GPU parity of the normalisation layers and their gradients with the float64 oracle.

Every tolerance is a bound by arithmetic, element by element. u = 2^-24 is fp32's half
step, U the output type's (2^-24, bf16 2^-8, fp16 2^-11, with 2^-25 for fp16 subnormals).
A row sum adds at most 16 elements in a lane, then 6 steps across a wave and 16 waves:
its error is at most DEPTH u times the sum of magnitudes with DEPTH = 38 and one more for
each product's own rounding, 40 in all.
  forward: the mean is off by at most 40 u mean|x|; rstd by half of the variance's
  relative error and its own 3 operations, 24 u; so h = (x - mean) rstd is off by
  40 u rstd mean|x| + 27 u |h|, y by |scale| times that, 3 u (|h scale| + |b|) more, and U |y|.
  backward (from given statistics): h is off by 2 u |h|, a by 2 u |a| (weight + offset and
  the product); mean(a) by 42 u mean|a|, mean(a h) by 45 u mean|a h|; dx by rstd times
  (3 u |a| + 43 u mean|a| + |h| 48 u mean|a h|), 4 u of rstd (|a| + |mean a| + |h mean(a h)|)
  more, and U |dx|.
  weight gradients: a lane adds at most ROWS rows (the rows of a block divided by the rows
  it holds at once), then the block's teams, then the blocks' sums: (depth + 3) u times the
  sum of magnitudes, with the depth that the split gives; and U of the result.
"""
import sys

import numpy as np
import pytest

from oracle import norm_oracle as N
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B
from matrix_orthogonalising_optimizer_02_amd import workloads as WL

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
TYPES = {"f32": (2.0 ** -24, 0.0), "bf16": (2.0 ** -8, 0.0), "f16": (2.0 ** -11, 2.0 ** -25)}


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a visible GPU"
    B.load_library()
    return torch, torch.device("cuda:0")


def dtype_of(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def host(t):
    return t.detach().double().cpu().numpy()


def draw(torch, dev, key, i, shape, dt, scale=1.0, shift=0.0):
    return (torch.from_numpy(WL.host_normal(key, WL.ROLE_G, i, shape, 1.0)) * scale + shift).to(dev).to(dt)


def within(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    worst = np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)) if got.size else 0.0
    assert not bad.any(), (what, int(bad.sum()), float(worst))
    return float(worst)


def round_tol(name, ref):
    step, least = TYPES[name]
    return step * 1.001 * np.abs(ref) + least


def row_depth(name, cols, rows, groups):
    """How many additions deep a weight gradient's sum is (see the module's text)."""
    vec = 4 if name == "f32" else 8
    vectors = -(-cols // vec)
    teams = 256 // max(8, 1 << max(0, vectors - 1).bit_length()) if vectors <= 64 else 1
    per_group = rows // groups
    chunks = max(1, 256 // groups)  # the backward split never has fewer blocks, but for few rows
    block_rows = max(per_group / chunks, 64 * teams)
    return block_rows / teams + teams + 1024 / 16 + 16


def check_forward(torch, name, wname, kind, x, w, b, offset, groups, eps=1e-6, **more):
    y, mean, rstd = muon.norm_forward(x, w, b, kind=kind, eps=eps, weight_offset=offset, **more)
    torch.cuda.synchronize()
    ry, rmean, rrstd, h, scale = N.norm_forward(host(x), None if w is None else host(w), None if b is None else host(b),
                                                kind, float(np.float32(eps)), offset, groups)
    mag = np.abs(host(x).reshape(h.shape)).mean(2, keepdims=True) if kind == "layer" else np.zeros(h.shape[:2] + (1,))
    bias = 0.0 if b is None else np.abs(host(b)).reshape(groups, 1, -1)
    tol = np.abs(scale) * (40 * U32 * rrstd[..., None] * mag + 27 * U32 * np.abs(h)) \
        + 3 * U32 * (np.abs(h * scale) + bias) + round_tol(name, ry)
    worst = within(host(y).reshape(ry.shape), ry, tol, "y")
    within(host(rstd).reshape(rrstd.shape), rrstd, 24 * U32 * rrstd + 1600 * U32 ** 2 * rrstd ** 3 * mag[..., 0] ** 2, "rstd")
    if kind == "layer":
        within(host(mean).reshape(rmean.shape), rmean, 41 * U32 * mag[..., 0], "mean")
    else:
        assert mean is None
    assert y.dtype == x.dtype and y.shape == x.shape
    return mean, rstd, worst


def check_backward(torch, name, wname, kind, dy, x, w, mean, rstd, offset, groups, bias=True, **more):
    dx, dw, db = muon.norm_backward(dy, x, w, mean, rstd, kind=kind, weight_offset=offset, bias_grad=bias, **more)
    torch.cuda.synchronize()
    rdx, rdw, rdb, h, a = N.norm_backward(host(dy), host(x), None if w is None else host(w),
                                          None if mean is None else host(mean), host(rstd), kind, offset, groups)
    r = host(rstd).reshape(groups, -1, 1)
    ma = np.abs(a).mean(2, keepdims=True) if kind == "layer" else 0.0
    mah = np.abs(a * h).mean(2, keepdims=True)
    ca = np.abs(a.mean(2, keepdims=True)) if kind == "layer" else 0.0
    tol = r * (3 * U32 * np.abs(a) + 43 * U32 * ma + np.abs(h) * 48 * U32 * mah) \
        + 4 * U32 * r * (np.abs(a) + ca + np.abs(h * (a * h).mean(2, keepdims=True))) + round_tol(name, rdx)
    worst = within(host(dx).reshape(rdx.shape), rdx, tol, "dx")
    depth = row_depth(name, x.shape[-1], x.numel() // x.shape[-1], groups) + 3
    g = host(dy).reshape(h.shape)
    if w is not None and dw is not None:
        within(host(dw).reshape(rdw.shape), rdw, depth * U32 * np.abs(g * h).sum(1) + round_tol(wname, rdw), "dw")
        assert dw.shape == w.shape and dw.dtype == w.dtype
    if bias:
        within(host(db).reshape(rdb.shape), rdb, depth * U32 * np.abs(g).sum(1) + round_tol(wname, rdb), "db")
    else:
        assert db is None
    return worst


# rows, cols, groups: one element, one row, every lane count with and without a ragged
# end, sizes that no vector divides, rows of a whole block, the widest row
SHAPES = [(1, 1, 1), (3, 1, 1), (1, 8, 1), (5, 7, 5), (33, 64, 1), (40, 65, 4), (17, 127, 1), (64, 128, 2), (130, 129, 1),
          (31, 255, 1), (64, 256, 8), (9, 511, 3), (48, 512, 1), (50, 513, 2), (6, 1153, 1), (25, 2048, 5), (12, 4097, 1),
          (10, 5120, 2), (3, 8193, 1), (4, 16383, 2), (2, 16384, 1)]


@pytest.mark.parametrize("rows,cols,groups", SHAPES)
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_forward_and_backward_vs_oracle(torch_dev, name, rows, cols, groups):
    torch, dev = torch_dev
    dt = dtype_of(torch, name)
    for kind, wname, offset, bias in (("layer", "f32", 0.0, True), ("layer", name, 1.0, True), ("rms", "f32", 0.0, False)):
        wdt = dtype_of(torch, wname)
        key = 500 + cols % 97
        x = draw(torch, dev, key, 0, (rows, cols), dt, 2.0, 0.5)
        w = draw(torch, dev, key, 1, (groups, cols), wdt, 0.3, 1.0 - offset)
        b = draw(torch, dev, key, 2, (groups, cols), wdt, 0.2) if bias else None
        dy = draw(torch, dev, key, 3, (rows, cols), dt)
        mean, rstd, wf = check_forward(torch, name, wname, kind, x, w, b, offset, groups)
        wb = check_backward(torch, name, wname, kind, dy, x, w, mean, rstd, offset, groups, bias)
        log(f"{name} {kind} w {wname} {rows} x {cols}, {groups} groups: {wf:.2f}, {wb:.2f} of the bound")


@pytest.mark.parametrize("rows,cols,groups", [(4999, 1153, 1), (8192, 512, 8), (70000, 128, 1), (3000, 64, 2), (2050, 5120, 1),
                                              (700, 12000, 7)])
def test_many_rows_weight_gradient(torch_dev, rows, cols, groups):
    """Weight gradients over many blocks, fp32 and bf16."""
    torch, dev = torch_dev
    for name in ("f32", "bf16"):
        dt = dtype_of(torch, name)
        x = draw(torch, dev, 520, 0, (rows, cols), dt, 1.5, 0.2)
        w = draw(torch, dev, 520, 1, (groups, cols), torch.float32, 0.3, 1.0)
        b = draw(torch, dev, 520, 2, (groups, cols), torch.float32, 0.2)
        dy = draw(torch, dev, 520, 3, (rows, cols), dt)
        mean, rstd, _ = check_forward(torch, name, "f32", "layer", x, w, b, 0.0, groups)
        check_backward(torch, name, "f32", "layer", dy, x, w, mean, rstd, 0.0, groups)
        log(f"{name} {rows} x {cols}, {groups} groups")


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("heads,cols", [(1, 128), (3, 72), (16, 128), (5, 33)])
def test_strided_query_view(torch_dev, name, heads, cols):
    """Rows of a query view of a fused projection, written back in place and to a gradient's view."""
    torch, dev = torch_dev
    tokens = 37
    dt = dtype_of(torch, name)
    qkv = draw(torch, dev, 530, heads, (tokens, 3, heads, cols), dt, 1.5, 0.1)
    w = draw(torch, dev, 530, 50, (cols,), torch.float32, 0.3, 1.0)
    q = qkv[:, 1]
    mean, rstd, _ = check_forward(torch, name, "f32", "rms", q, w, None, 0.0, 1)
    dqkv = torch.full_like(qkv, 7.0)
    dy = draw(torch, dev, 530, 60, (tokens, heads, cols), dt)
    check_backward(torch, name, "f32", "rms", dy, q, w, mean, rstd, 0.0, 1, False, out=dqkv[:, 1])
    assert bool((dqkv[:, 0] == 7.0).all()) and bool((dqkv[:, 2] == 7.0).all())
    want, _, _ = muon.norm_forward(q, w, kind="rms")
    kept = qkv.clone()
    muon.norm_forward(q, w, kind="rms", out=q)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(qkv[:, 0], kept[:, 0]) and torch.equal(qkv[:, 2], kept[:, 2])


def test_modulation_slices_and_three_dims(torch_dev):
    """adaLN as a block has it: x [samples, tokens, H], scale and shift strided slices of
    the modulation [samples, 6H]."""
    torch, dev = torch_dev
    s, t, h = 3, 29, 320
    mod = draw(torch, dev, 540, 0, (s, 6 * h), torch.bfloat16, 0.3)
    x = draw(torch, dev, 540, 1, (s, t, h), torch.bfloat16, 2.0)
    dy = draw(torch, dev, 540, 2, (s, t, h), torch.bfloat16)
    shift, scale = mod[:, None, :h], mod[:, None, h:2 * h]
    mean, rstd, _ = check_forward(torch, "bf16", "bf16", "layer", x, scale, shift, 1.0, s)
    check_backward(torch, "bf16", "bf16", "layer", dy, x, scale, mean, rstd, 1.0, s)
    # an expanded gradient (stride 0 over the rows) needs no copy
    check_backward(torch, "bf16", "bf16", "layer", dy[:1, :1].expand(s, t, h), x, scale, mean, rstd, 1.0, s)
    # tokens before samples: two strides of rows
    xt = x.transpose(0, 1)
    y, _, _ = muon.norm_forward(xt)
    want, _, _ = muon.norm_forward(xt.contiguous())
    assert torch.equal(y, want)


def test_without_weight_and_bias_alone(torch_dev):
    torch, dev = torch_dev
    x = draw(torch, dev, 550, 0, (19, 384), torch.float32, 1.0, 0.3)
    dy = draw(torch, dev, 550, 1, (19, 384), torch.float32)
    b = draw(torch, dev, 550, 2, (384,), torch.float32)
    mean, rstd, _ = check_forward(torch, "f32", "f32", "layer", x, None, None, 0.0, 1)
    check_forward(torch, "f32", "f32", "layer", x, None, b, 1.0, 1)
    check_backward(torch, "f32", "f32", "layer", dy, x, None, mean, rstd, 1.0, 1)
    dx, dw, db = muon.norm_backward(dy, x, None, mean, rstd, bias_grad=False)
    assert dw is None and db is None
    y, m, r = muon.norm_forward(x, stats=False)
    assert m is None and r is None and torch.equal(y, muon.norm_forward(x)[0])


def test_in_place_and_unaligned_rows(torch_dev):
    torch, dev = torch_dev
    for name in ("f32", "bf16", "f16"):
        dt = dtype_of(torch, name)
        base = draw(torch, dev, 560, 0, (11 * 640 + 3,), dt, 1.5)
        x = base[3:].view(11, 640)  # no row starts at 16 bytes
        w = draw(torch, dev, 560, 1, (640 + 1,), torch.float32)[1:]
        dy = draw(torch, dev, 560, 2, (11 * 640 + 1,), dt)[1:].view(11, 640)
        mean, rstd, _ = check_forward(torch, name, "f32", "layer", x, w, w, 0.0, 1)
        check_backward(torch, name, "f32", "layer", dy, x, w, mean, rstd, 0.0, 1)
        want, wdw, wdb = muon.norm_backward(dy, x, w, mean, rstd)
        for target in ("dy", "x"):
            a, g = x.clone(), dy.clone()
            dx, dw, db = muon.norm_backward(g, a, w, mean, rstd, out=g if target == "dy" else a)
            assert torch.equal(dx, want) and torch.equal(dw, wdw) and torch.equal(db, wdb), (name, target)
        assert float(base[:3].float().abs().sum()) > 0  # untouched, as drawn
        assert torch.equal(base[:3], draw(torch, dev, 560, 0, (11 * 640 + 3,), dt, 1.5)[:3])


def test_constant_rows_large_offsets_and_non_finite(torch_dev):
    """A constant row gives h = 0 up to the mean's rounding; a row far from zero keeps its
    digits; a NaN or an infinity stays within its row (forward, dx)."""
    torch, dev = torch_dev
    x = draw(torch, dev, 570, 0, (8, 1000), torch.float32)
    x[1] = 3.3
    x[2] += 1e4
    x[3] = 0.0
    w = draw(torch, dev, 570, 1, (1000,), torch.float32)
    mean, rstd, _ = check_forward(torch, "f32", "f32", "layer", x, w, None, 0.0, 1)
    check_backward(torch, "f32", "f32", "layer", draw(torch, dev, 570, 2, (8, 1000), torch.float32), x, w, mean, rstd, 0.0, 1)
    y0 = muon.norm_forward(x, w)[0]
    x[4, 17] = float("nan")
    x[5, 3] = float("inf")
    y, mean, rstd = muon.norm_forward(x, w)
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(y[keep], y0[keep])
    assert bool(torch.isnan(y[4]).all()) and bool(torch.isnan(y[5]).any())
    dx, dw, _ = muon.norm_backward(torch.ones_like(x), x, w, mean, rstd)
    assert bool(torch.isfinite(dx[keep]).all()) and bool(torch.isnan(dx[4]).all())
    assert bool(torch.isnan(dw).all())


def test_no_rows(torch_dev):
    torch, dev = torch_dev
    x = torch.empty(0, 96, device=dev)
    w = torch.ones(96, device=dev)
    y, mean, rstd = muon.norm_forward(x, w, w)
    assert y.shape == (0, 96) and mean.numel() == 0
    dx, dw, db = muon.norm_backward(x, x, w, mean, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 96) and float(dw.abs().sum()) == 0.0 and float(db.abs().sum()) == 0.0
    e = torch.empty(4, 0, device=dev)
    assert muon.norm_forward(e)[0].shape == (4, 0)


def test_repeats_bitwise_and_on_a_side_stream(torch_dev):
    torch, dev = torch_dev
    x = draw(torch, dev, 580, 0, (6000, 768), torch.bfloat16)
    dy = draw(torch, dev, 580, 1, (6000, 768), torch.bfloat16)
    w = draw(torch, dev, 580, 2, (768,), torch.float32)
    y, mean, rstd = muon.norm_forward(x, w, w)
    ref = (y, mean, rstd) + muon.norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (side, None):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(torch.cuda.current_stream() if given is not None else side):
            f = muon.norm_forward(x, w, w, stream=given)
            b = muon.norm_backward(dy, x, w, f[1], f[2], stream=given)
            junk = torch.full((4 << 20,), float("nan"), device=dev)
            del junk
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(f + b, ref))


def test_captured_forward_and_backward_replay_bitwise(torch_dev):
    torch, dev = torch_dev
    x = draw(torch, dev, 590, 0, (4096, 640), torch.bfloat16)
    dy = draw(torch, dev, 590, 1, (4096, 640), torch.bfloat16)
    w = draw(torch, dev, 590, 2, (4, 640), torch.bfloat16)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y, mean, rstd = muon.norm_forward(x, w, w, weight_offset=1.0)
        outs = (y, mean, rstd) + muon.norm_backward(dy, x, w, mean, rstd, weight_offset=1.0)
    for r in range(3):
        x.copy_(draw(torch, dev, 591 + r, 0, (4096, 640), torch.bfloat16))
        fy, fm, fr = muon.norm_forward(x, w, w, weight_offset=1.0)
        want = (fy, fm, fr) + muon.norm_backward(dy, x, w, fm, fr, weight_offset=1.0)
        for o in outs:
            o.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), r
        assert float(torch.randn(1 << 18, device=dev).sum()) != 0.0


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_autograd_against_differences(torch_dev, kind):
    """The gradients of sum(y c) against central differences of the float64 oracle."""
    torch, dev = torch_dev
    rows, cols, groups = 6, 40, 2
    x = draw(torch, dev, 600, 0, (rows, cols), torch.float32).requires_grad_()
    w = draw(torch, dev, 600, 1, (groups, cols), torch.float32).requires_grad_()
    b = draw(torch, dev, 600, 2, (groups, cols), torch.float32).requires_grad_() if kind == "layer" else None
    c = draw(torch, dev, 600, 3, (rows, cols), torch.float32)
    y = muon.layer_norm(x, w, b, 1e-5, 1.0) if kind == "layer" else muon.rms_norm(x, w, 1e-5, 1.0)
    (y * c).sum().backward()
    vals = [host(x), host(w)] + ([host(b)] if b is not None else [])

    def loss(v):
        ry = N.norm_forward(v[0], v[1], v[2] if len(v) > 2 else None, kind, float(np.float32(1e-5)), 1.0, groups)[0]
        return float((ry.reshape(rows, cols) * host(c)).sum())

    rng = WL.rng(600, 0, 9)
    for i, leaf in enumerate([x, w] + ([b] if b is not None else [])):
        for _ in range(12):
            at = tuple(int(rng.integers(n)) for n in vals[i].shape)
            step = 1e-5
            up, down = [v.copy() for v in vals], [v.copy() for v in vals]
            up[i][at] += step
            down[i][at] -= step
            diff = (loss(up) - loss(down)) / (2 * step)
            # the difference's own error is of order step^2 and 1e-16 / step; the fp32 pass's
            # is at most some 100 u of the magnitudes summed (about 40 of order 1 each)
            assert abs(float(leaf.grad[at]) - diff) < 100 * U32 * 200 + 1e-7, (i, at)


def test_autograd_expanded_gradient_and_frozen_inputs(torch_dev):
    torch, dev = torch_dev
    x = draw(torch, dev, 610, 0, (4, 5, 96), torch.float32).requires_grad_()
    w = draw(torch, dev, 610, 1, (96,), torch.float32)
    muon.layer_norm(x, w).sum().backward()  # dy is one expanded element
    _, mean, rstd = muon.norm_forward(x.detach(), w)
    want, _, _ = muon.norm_backward(torch.ones(4, 5, 96, device=dev), x.detach(), w, mean, rstd)
    assert torch.equal(x.grad, want) and w.grad is None
    b = torch.zeros(96, device=dev, requires_grad=True)
    muon.layer_norm(x.detach(), None, b).sum().backward()
    assert torch.equal(b.grad, torch.full((96,), 20.0, device=dev))


def test_in_place_gradient_that_overflows(torch_dev):
    """fp16 gradients that overflow to infinity, written over dy and over x: the weight's
    gradient is the one of separate buffers, for row counts that leave teams without a row."""
    torch, dev = torch_dev
    for rows, cols in ((5, 64), (37, 128), (70, 320), (131, 1024), (300, 640)):
        x = draw(torch, dev, 620, 0, (rows, cols), torch.float16, 1e-3)
        dy = draw(torch, dev, 620, 1, (rows, cols), torch.float16, 300.0)
        w = draw(torch, dev, 620, 2, (cols,), torch.float32)
        _, mean, rstd = muon.norm_forward(x, w, eps=1e-8)
        want = muon.norm_backward(dy, x, w, mean, rstd)
        assert bool(torch.isinf(want[0]).any()) and bool(torch.isfinite(want[1]).all())
        for target in ("dy", "x"):
            a, g = x.clone(), dy.clone()
            got = muon.norm_backward(g, a, w, mean, rstd, out=g if target == "dy" else a)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (rows, cols, target)


def test_offsets_past_32_bits(torch_dev):
    """A tensor of more than 2^32 elements: its last rows as those of a small one."""
    torch, dev = torch_dev
    cols, rows = 4096, (1 << 20) + 7
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev).normal_(0.0, 1.0, generator=torch.Generator(dev).manual_seed(3))
    w = draw(torch, dev, 630, 1, (cols,), torch.float32, 0.3, 1.0)
    y, mean, rstd = muon.norm_forward(x, w)
    for part in (slice(rows - 9, rows), slice((1 << 20) - 3, (1 << 20) + 2), slice(0, 5)):
        p, m, r = muon.norm_forward(x[part].clone(), w)
        assert torch.equal(p, y[part]) and torch.equal(m, mean[part]) and torch.equal(r, rstd[part])
    dx, _, _ = muon.norm_backward(y, x, w, mean, rstd, out=y)
    for part in (slice(rows - 9, rows), slice(0, 5)):
        xs = x[part].clone()
        p, m, r = muon.norm_forward(xs, w)
        want, _, _ = muon.norm_backward(p, xs, w, m, r)
        assert torch.equal(want, dx[part])


def test_two_streams_at_once(torch_dev):
    """Two calls at the same time on two streams, each with its own workspace."""
    torch, dev = torch_dev
    xs = [draw(torch, dev, 640 + i, 0, (8192, 1024), torch.bfloat16) for i in range(2)]
    w = draw(torch, dev, 640, 1, (1024,), torch.float32)
    refs = []
    for x in xs:
        y, m, r = muon.norm_forward(x, w, w)
        refs.append((y, m, r) + muon.norm_backward(x, x, w, m, r))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = []
        for x, s in zip(xs, streams):
            y, m, r = muon.norm_forward(x, w, w, stream=s)
            outs.append((y, m, r) + muon.norm_backward(x, x, w, m, r, stream=s))
        torch.cuda.synchronize()
        for got, want in zip(outs, refs):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
