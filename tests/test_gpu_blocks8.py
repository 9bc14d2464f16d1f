"""GPU parity of the 8-bit matrices and their products with the float64 oracle.

Quantising is exact arithmetic and one rounding: codes and powers have to be the oracle's.
Products, with u = 2^-24 (fp32's half step), S = sum over k of |a b| and U the result's half
step (2^-24, bf16 2^-8, fp16 2^-11 with 2^-25 for subnormals): K products are added in fp32
one after the other at worst, and the parts of k after that, so that a sum is off by at most
(K + 64) u S, and the result by U of it. The 8-bit instructions drop, in each group of eight
products, bits below 2^-13 of the largest: each of the eight loses at most that, and the
largest is at most the group's sum of magnitudes: 8 2^-13 = 2^-10 of S.
"""
import sys

import numpy as np
import pytest

from oracle import blocks8_oracle as Q
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


def draw(torch, dev, i, shape, dt, scale=1.0):
    """Rows and columns of unlike sizes."""
    x = WL.host_normal(810, 0, i, shape, scale)
    x = x * np.exp(WL.host_normal(810, 1, i, shape[-1:], 1.0)) * np.exp(WL.host_normal(810, 2, i, shape[:-1] + (1,), 1.0))
    return torch.from_numpy(x.astype(np.float32)).to(dev).to(dt)


VALUES = Q.e4m3_values()


def decode(q):
    """(values, exponents) of a Blocks8, by the bytes alone; its padding has to be zero."""
    codes = q.codes.view(__import__("torch").uint8).cpu().numpy()
    e = q.scales.cpu().numpy().astype(int)
    blocks = -(-q.cols // 128)
    assert not codes[:, q.cols:blocks * 128].any(), "padding"
    e = e[:, :blocks] - 127
    return VALUES[codes[:, :q.cols]] * 2.0 ** Q.spread(e, (q.rows, q.cols), q.tiles).astype(float), e


def check_codes(torch, x, tiles, what, **more):
    host = x.double().cpu().numpy()
    q, qt = muon.quantise8(x, tiles=tiles, direct=True, transposed=True, **more)
    torch.cuda.synchronize()
    for got, ref in ((q, host), (qt, host.T)):
        assert got.shape == ref.shape
        vals, e = decode(got)
        want, we = Q.quantise(ref, tiles)
        assert np.array_equal(e, we), (what, "powers")
        assert np.array_equal(vals, want, equal_nan=True), (what, "codes")
        near = np.where(Q.spread(e, ref.shape, tiles) > -127, want, 0.0 * want)
        for dt in (torch.float32, torch.bfloat16):
            back = got.dequantise(dt).double().cpu().numpy()
            fine = np.abs(near) >= 2.0 ** -126
            assert np.array_equal(back[fine], near[fine]) and np.array_equal(np.isnan(back), np.isnan(near)), (what, dt)
            assert (np.abs(back[~fine & np.isfinite(near)]) < 2.0 ** -125).all()
    return q, qt


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tiles", [False, True])
def test_codes_and_powers(torch_dev, name, tiles):
    torch, dev = torch_dev
    for i, (r, c) in enumerate(((1, 1), (1, 128), (128, 1), (3, 7), (5, 129), (127, 128), (129, 127), (128, 128), (130, 260),
                                (257, 384), (300, 515), (64, 1000), (1000, 64), (513, 513))):
        check_codes(torch, draw(torch, dev, i, (r, c), dtype_of(torch, name)), tiles, (name, tiles, r, c))
        log(f"{name} tiles {tiles} {r} x {c}")


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tiles", [False, True])
def test_special_values(torch_dev, name, tiles):
    """Zeros, one value, values at a power's border, infinities and NaN in every block's reach,
    the smallest and the largest magnitudes, subnormals."""
    torch, dev = torch_dev
    dt = dtype_of(torch, name)
    info = torch.finfo(dt)
    x = draw(torch, dev, 40, (260, 390), torch.float32)
    x[0] = 0.0
    x[1, :128] = 0.0
    x[2, 130] = float("inf")
    x[3, 140], x[3, 141] = float("-inf"), float("nan")
    x[4, :128] = float("nan")
    x[5, :128] = float("inf")
    x[6, 128:256] = 448.0 * 2.0 ** -6
    x[7, 128:256] = 448.0 * 2.0 ** -6 * (1 + 2.0 ** -8)
    x[8, :] = info.max / 4  # the largest fp32 itself rounds to 2^128
    x[9, :] = info.tiny
    x[10, :] = info.smallest_normal / 4
    x[11, :] = -info.max / 4
    x[12, 256:] = 2.0 ** -24
    x[200:, 300:] = 0.0
    check_codes(torch, x.to(dt), tiles, (name, tiles))


@pytest.mark.parametrize("tiles", [False, True])
def test_strides_and_what_lies_beside(torch_dev, tiles):
    """Rows apart, unaligned, expanded; results inside larger buffers, which stay as they are."""
    torch, dev = torch_dev
    big = draw(torch, dev, 50, (140, 701), torch.bfloat16)
    for x in (big[:, :300], big[:, 1:400], big[3::2, 5:300], big[:1].expand(70, 701)):
        check_codes(torch, x, tiles, x.stride())
    lead = draw(torch, dev, 51, (3, 43, 200), torch.float16)
    q, _ = check_codes(torch, lead.view(129, 200), tiles, "flat")
    again, _ = muon.quantise8(lead, tiles=tiles)
    assert torch.equal(q.codes.view(torch.uint8), again.codes.view(torch.uint8)) and torch.equal(q.scales, again.scales)
    rows, cols = 129, 200
    srows = 2 if tiles else rows
    codes, scales = torch.full((rows + 2, 400), 7, dtype=torch.uint8, device=dev), torch.full((srows + 2, 12), 7, dtype=torch.uint8, device=dev)
    out = muon.Blocks8(codes[1:-1, 16:272].view(torch.float8_e4m3fn), scales[1:-1, 4:8], cols, tiles)
    muon.quantise8(lead, tiles=tiles, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out.codes.view(torch.uint8), q.codes.view(torch.uint8)) and torch.equal(out.scales[:, :2], q.scales[:, :2])
    codes[1:-1, 16:272], scales[1:-1, 4:8] = 7, 7
    assert bool((codes == 7).all()) and bool((scales == 7).all())
    y = torch.full((rows + 2, 250), 7.0, dtype=torch.float32, device=dev)
    q.dequantise(out=y[1:-1, 10:210])
    torch.cuda.synchronize()
    assert torch.equal(y[1:-1, 10:210], q.dequantise())
    y[1:-1, 10:210] = 7.0
    assert bool((y == 7.0).all())


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tiles", [False, True])
def test_reading_back_to_any_place(torch_dev, name, tiles):
    """Into rows that fill whole lines and rows that do not, from every offset, beside what stays."""
    torch, dev = torch_dev
    for i, (rows, cols) in enumerate(((1, 1), (3, 7), (5, 130), (200, 256), (131, 1001), (40, 4096))):
        q, _ = muon.quantise8(draw(torch, dev, 60 + i, (rows, cols), torch.float32), tiles=tiles)
        want = q.dequantise(torch.float32).to(dtype_of(torch, name))  # float32 holds the values exactly
        assert torch.equal(q.dequantise(dtype_of(torch, name)), want)
        for lead, beside in ((0, 0), (0, 64), (1, 0), (3, 6), (8, 24)):
            full = torch.full((rows + 2, lead + cols + beside), 7.0, dtype=dtype_of(torch, name), device=dev)
            q.dequantise(out=full[1:-1, lead:lead + cols])
            torch.cuda.synchronize()
            assert torch.equal(full[1:-1, lead:lead + cols], want), (rows, cols, lead, beside)
            full[1:-1, lead:lead + cols] = 7.0
            assert bool((full == 7.0).all()), (rows, cols, lead, beside)


def test_nothing_to_quantise(torch_dev):
    torch, dev = torch_dev
    for shape in ((0, 5), (5, 0), (0, 0)):
        q, qt = muon.quantise8(torch.zeros(shape, device=dev), transposed=True)
        assert q.shape == shape and qt.shape == shape[::-1]
        assert q.dequantise().shape == shape
    a, _ = muon.quantise8(torch.zeros(3, 0, device=dev))
    b, _ = muon.quantise8(torch.zeros(200, 0, device=dev))
    for x, y in ((a, b), (b, a), (b, b)):
        assert not muon.matmul8(x, y, dtype=torch.float32, out=torch.full((x.rows, y.rows), 3.0, device=dev)).any()
        kept = muon.matmul8(x, y, out=torch.full((x.rows, y.rows), 3.0, device=dev), accumulate=True)
        assert bool((kept == 3.0).all())
    none, _ = muon.quantise8(torch.zeros(0, 8, device=dev))
    some, _ = muon.quantise8(torch.ones(4, 8, device=dev))
    assert muon.matmul8(none, some).shape == (0, 4) and muon.matmul8(some, none).shape == (4, 0)


# ---------------------------------------------------------------- products ----

def operand(torch, dev, i, rows, k, tiles=False, scale=0.05):
    q, _ = muon.quantise8(draw(torch, dev, i, (rows, k), torch.float32, scale), tiles=tiles)
    return q


def exact(q):
    """The values in float64, on the GPU, by the bytes alone."""
    import torch
    table = torch.from_numpy(VALUES).to(q.device)
    s = torch.pow(2.0, q.scales.double() - 127.0).repeat_interleave(128, 1)
    if q.tiles:
        s = s.repeat_interleave(128, 0)
    return table[q.codes.view(torch.uint8).long()][:, :q.cols] * s[:q.rows, :q.cols]


def bound(name, products, k, ref, mag):
    step, least = TYPES[name]
    rel = (k + 64) * U32 + (2.0 ** -10 if products == 8 else 0.0)
    return rel * mag + (step * (1.0 + rel)) * (ref.abs() + rel * mag) + least


def check_product(torch, a, b, name, products, what, old=None, **more):
    va, vb = exact(a), exact(b)
    ref, mag = va @ vb.t().contiguous(), va.abs() @ vb.abs().t().contiguous()
    if old is not None:
        ref, mag = ref + old.double(), mag + old.double().abs()
    got = muon.matmul8(a, b, dtype=dtype_of(torch, name), products=products, **more)
    torch.cuda.synchronize()
    tol = bound(name, products, a.cols, ref, mag)
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((off / tol).max()))
    return got


SIZES = [(1, 1, 1), (1, 16, 128), (1, 17, 129), (2, 300, 127), (15, 100, 640), (16, 129, 513), (17, 33, 1000), (33, 513, 130),
         (48, 64, 2011), (64, 1000, 384), (64, 16, 5000), (65, 65, 65), (65, 1, 700), (127, 129, 128), (128, 128, 256),
         (129, 257, 385), (200, 70, 4224), (300, 1153, 900), (1003, 300, 2011)]


@pytest.mark.parametrize("name,products", [("bf16", 8), ("f16", 8), ("f32", 8), ("f32", 16), ("bf16", 16)])
def test_products(torch_dev, name, products):
    torch, dev = torch_dev
    for i, (m, n, k) in enumerate(SIZES):
        for tiles in (False, True):
            a, b = operand(torch, dev, 100 + i, m, k), operand(torch, dev, 200 + i, n, k, tiles, 0.02)
            check_product(torch, a, b, name, products, (name, products, m, n, k, tiles))
            if tiles:  # and as the first operand
                check_product(torch, b, a, name, products, (name, products, n, m, k, "tiles first"))
        log(f"{name} products {products} [{m}, {k}] x [{n}, {k}]")


@pytest.mark.parametrize("products", [8, 16])
@pytest.mark.parametrize("m,n", [(130, 140), (4095, 4001)])
def test_every_length_of_the_loop(torch_dev, products, m, n):
    """1 to 11 steps of 128 along k, whole and ragged, on both tile sizes."""
    torch, dev = torch_dev
    for steps in range(1, 12):
        k = steps * 128 - (5 if steps % 2 else 0)
        a, b = operand(torch, dev, 300 + steps, m, k), operand(torch, dev, 320 + steps, n, k, steps % 3 == 0)
        check_product(torch, a, b, "f32", products, (products, m, n, k))
        log(f"products {products} [{m}, {k}] x [{n}, {k}]")


@pytest.mark.parametrize("m,n,k,name", [(128, 128, 1 << 16, "f32"), (500, 600, 20000, "bf16"), (7, 9000, 16384 + 300, "bf16"),
                                        (33, 3000, 40000, "f32"), (60, 70, 70000, "f16"), (256, 256, 33000, "f32")])
def test_parts_of_k(torch_dev, m, n, k, name):
    torch, dev = torch_dev
    assert muon.matmul8_workspace_bytes(m, n, k, dtype_of(torch, name)) > 0
    a, b = operand(torch, dev, 400, m, k), operand(torch, dev, 401, n, k)
    one = check_product(torch, a, b, name, None if name == "f32" else 8, (m, n, k))
    assert torch.equal(one, muon.matmul8(a, b, dtype=dtype_of(torch, name)))


@pytest.mark.parametrize("m,n,k", [(5, 200, 300), (64, 9000, 2500), (130, 140, 700), (140, 130, 33000), (4095, 4001, 260)])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_accumulate_into_a_view(torch_dev, m, n, k, name):
    """c += a b^T inside a larger buffer whose rest stays, in every form of the product."""
    torch, dev = torch_dev
    a, b = operand(torch, dev, 410, m, k), operand(torch, dev, 411, n, k, True)
    buf = draw(torch, dev, 412, (m + 2, n + 7), dtype_of(torch, name), 0.1)
    kept = buf.clone()
    out = buf[1:-1, 3:-4]
    check_product(torch, a, b, name, 16 if name == "f32" else 8, (m, n, k, name), old=out.clone(), out=out, accumulate=True)
    buf[1:-1, 3:-4], kept[1:-1, 3:-4] = 0, 0
    assert torch.equal(buf, kept)


@pytest.mark.parametrize("m,n,k", [(3, 100, 600), (20, 9000, 2500), (200, 260, 900), (4095, 4001, 260)])
def test_nan_stays_in_its_row(torch_dev, m, n, k):
    """NaN codes, and powers of 255, reach the rows and columns they belong to alone; so do the
    rows that a tile has beyond the matrix's end."""
    torch, dev = torch_dev
    a, b = operand(torch, dev, 420, m, k), operand(torch, dev, 421, n, k)
    clean = muon.matmul8(a, b, dtype=torch.float32, products=8)
    a.codes.view(torch.uint8)[m - 1, k - 1] = 0x7F
    b.codes.view(torch.uint8)[5, 0] = 0xFF
    b.scales[n - 1, (k - 1) // 128] = 255
    for products in (8, 16):
        got = muon.matmul8(a, b, dtype=torch.float32, products=products)
        torch.cuda.synchronize()
        if products == 16:  # a power of 255 is a matter of the 8-bit instructions
            got[:, n - 1] = float("nan")
        want = torch.zeros(m, n, dtype=torch.bool, device=dev)
        want[m - 1], want[:, 5], want[:, n - 1] = True, True, True
        assert torch.equal(got.isnan(), want)
        if products == 8:
            assert torch.equal(got[~want], clean[~want])


def test_eight_bit_products_on_normal_values(torch_dev):
    """The documented size of what the 8-bit instructions drop: 2^-16 of the result, root mean
    square, on normally distributed values (asserted to twice that), and less than fp32's own
    2^-20 when widened."""
    torch, dev = torch_dev
    a, b = (muon.quantise8(torch.from_numpy(WL.host_normal(830, 0, i, (512, 4096), 1.0)).to(dev))[0] for i in (0, 1))
    ref = exact(a) @ exact(b).t().contiguous()
    off = {p: float((muon.matmul8(a, b, dtype=torch.float32, products=p).double() - ref).norm() / ref.norm()) for p in (8, 16)}
    log(f"relative: {off}")
    assert off[8] < 2.0 ** -15 and off[16] < 2.0 ** -20


def test_slices_and_large_strides(torch_dev):
    """Operands that are rows of larger ones, rows megabytes apart, offsets past 2^32."""
    torch, dev = torch_dev
    whole = operand(torch, dev, 430, 400, 700)
    part = muon.Blocks8(whole.codes[30:333], whole.scales[30:333], 700)
    b = operand(torch, dev, 431, 150, 700)
    full = muon.matmul8(whole, b)
    assert torch.equal(muon.matmul8(part, b), full[30:333]) and torch.equal(muon.matmul8(b, part), muon.matmul8(b, whole)[:, 30:333])
    # codes 4 MiB apart: 1100 rows are past 2^32 bytes; a result whose rows are 2^22 elements apart
    ld = 1 << 22
    far = torch.empty((1100, ld), dtype=torch.float8_e4m3fn, device=dev)[:, :768]
    a = operand(torch, dev, 432, 1100, 700)
    far.copy_(a.codes)
    out = torch.empty((1100, 1 << 22), dtype=torch.bfloat16, device=dev)[:, :150]
    got = muon.matmul8(muon.Blocks8(far, a.scales, 700), b, out=out)
    assert torch.equal(got, muon.matmul8(a, b))
    few = muon.Blocks8(far[:9], a.scales[:9], 700)
    assert torch.equal(muon.matmul8(few, muon.Blocks8(far, a.scales, 700)),
                       muon.matmul8(muon.Blocks8(a.codes[:9], a.scales[:9], 700), a))
    del out, got
    x = torch.empty((1100, 1 << 22), dtype=torch.bfloat16, device=dev)[:, :300]
    x.copy_(draw(torch, dev, 433, (1100, 300), torch.bfloat16))
    check_codes(torch, x, False, "far rows")


def test_streams_and_graph(torch_dev):
    """On a stream of the caller's, two products at once, and captured and replayed with new
    values, each replay against the eager result."""
    torch, dev = torch_dev
    x, w = draw(torch, dev, 440, (200, 700), torch.bfloat16), draw(torch, dev, 441, (300, 700), torch.float32, 0.02)
    long = draw(torch, dev, 442, (130, 20000), torch.bfloat16)

    def step():
        a, at = muon.quantise8(x, transposed=True)
        b, bt = muon.quantise8(w, tiles=True, transposed=True)
        q, _ = muon.quantise8(long)
        y = muon.matmul8(a, b)
        dy, dyt = muon.quantise8(y, transposed=True)
        few = muon.Blocks8(a.codes[:5], a.scales[:5], 700)
        return y, muon.matmul8(dy, bt), muon.matmul8(dyt, at, dtype=torch.float32), muon.matmul8(q, q), muon.matmul8(few, b)

    want = step()
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [step() for _ in range(3)]
    with torch.cuda.stream(other):
        second = [step() for _ in range(3)]
    torch.cuda.synchronize()
    for got in first + second:
        assert all(torch.equal(g, t) for g, t in zip(got, want))
    a, _ = muon.quantise8(x, stream=side)
    b, _ = muon.quantise8(w, tiles=True, stream=side)
    y = muon.matmul8(a, b, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(draw(torch, dev, 450 + i, (200, 700), torch.bfloat16))
        w.copy_(draw(torch, dev, 460 + i, (300, 700), torch.float32, 0.02))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for g, t in zip(got, step()):
            assert torch.equal(g, t)


def test_python_refusals_on_the_gpu(torch_dev):
    torch, dev = torch_dev
    a, b = operand(torch, dev, 470, 20, 300), operand(torch, dev, 471, 30, 301)
    cases = [(lambda: muon.matmul8(a, b), "same number of columns"), (lambda: muon.matmul8(a, a, products=4), "products"),
             (lambda: muon.matmul8(a, a, accumulate=True), "needs out"), (lambda: muon.matmul8(a, a, dtype=torch.float64), "dtype"),
             (lambda: muon.matmul8(a, a, out=torch.zeros(20, 21, device=dev)), "shape"),
             (lambda: muon.matmul8(a, a, out=torch.zeros(20, 40, device=dev)[:, ::2]), "adjacent"),
             (lambda: muon.matmul8(a, a, out=torch.zeros(20, 20, device=dev), dtype=torch.bfloat16), "dtype"),
             (lambda: muon.quantise8(torch.zeros(4, 4, dtype=torch.float64, device=dev)), "float32"),
             (lambda: muon.quantise8(torch.zeros(4, 8, device=dev).t()), "adjacent"),
             (lambda: muon.quantise8(torch.zeros(4, 6, 8, device=dev)[:, :3]), "one stride"),
             (lambda: muon.quantise8(torch.zeros(4, 8, device=dev), direct=False), "neither"),
             (lambda: muon.quantise8(torch.zeros(4, 8, device=dev), out=a), "must be a Blocks8 of"),
             (lambda: muon.Blocks8(a.codes, a.scales, 385), "columns"), (lambda: muon.Blocks8(a.codes, a.scales[:, :2], 300), "scales must have"),
             (lambda: muon.Blocks8(a.codes, a.scales, 300, tiles=True), "scales must have"),
             (lambda: muon.Blocks8(a.codes.view(torch.uint8), a.scales, 300), "2-D"),
             (lambda: muon.Blocks8(a.codes, a.scales.cpu(), 300), "GPU"), (lambda: a.dequantise(torch.float64), "dtype"),
             (lambda: muon.linear8(torch.zeros(3, 7, device=dev), torch.zeros(5, 7, device=dev),
                                   muon.Weight8(torch.zeros(5, 8, device=dev))), "weight8 must have")]
    for call, text in cases:
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(B.MuonError):  # codes off their 16 bytes
        muon.matmul8(muon.Blocks8(torch.zeros(4, 200, dtype=torch.uint8, device=dev)[:, 8:136].view(torch.float8_e4m3fn),
                                  torch.zeros(4, 4, dtype=torch.uint8, device=dev), 128), operand(torch, dev, 472, 5, 128))
    with pytest.raises(B.MuonError):  # the result on an operand
        muon.matmul8(a, a, out=a.codes.view(torch.bfloat16)[:, :20])


# ---------------------------------------------------------------- the layer ----

@pytest.mark.parametrize("name,wname,lead", [("bf16", "f32", (150,)), ("f16", "f32", (3, 50)), ("f32", "f32", (1,)), ("bf16", "bf16", (2, 3, 70))])
def test_linear8_and_its_gradients(torch_dev, name, wname, lead):
    """The layer's three products against those of the values that its quantised operands stand
    for, with a weight's form of its own and a kept one."""
    torch, dev = torch_dev
    dt, wdt = dtype_of(torch, name), dtype_of(torch, wname)
    x = draw(torch, dev, 500, lead + (300,), dt).requires_grad_()
    w = draw(torch, dev, 501, (200, 300), wdt, 0.02).requires_grad_()
    g = draw(torch, dev, 502, lead + (200,), dt)
    flat, gflat = x.detach().reshape(-1, 300), g.reshape(-1, 200)
    x8, xt8 = muon.quantise8(flat, transposed=True)
    w8, wt8 = muon.quantise8(w.detach(), tiles=True, transposed=True)
    g8, gt8 = muon.quantise8(gflat, transposed=True)
    for kept in (None, muon.Weight8(w.detach())):
        x.grad = w.grad = None
        y = muon.linear8(x, w, kept)
        assert y.shape == lead + (200,) and y.dtype == dt
        y.backward(g)
        products = 16 if name == "f32" else 8
        for got, (a, b), kind, p in ((y.detach().reshape(-1, 200), (x8, w8), name, products), (x.grad.reshape(-1, 300), (g8, wt8), name, products),
                                     (w.grad, (gt8, xt8), wname, 16 if wname == "f32" else 8)):
            va, vb = exact(a), exact(b)
            ref, mag = va @ vb.t().contiguous(), va.abs() @ vb.abs().t().contiguous()
            assert bool(((got.double() - ref).abs() <= bound(kind, p, a.cols, ref, mag)).all())
    # an expanded gradient, one input's gradient alone, and a form that has moved on
    kept = muon.Weight8(w.detach())
    y = muon.linear8(x.detach(), w, kept)
    w.grad = None
    y.backward(torch.ones((), dtype=dt, device=dev).expand(y.shape))
    assert w.grad is not None and bool(w.grad.isfinite().all())
    y = muon.linear8(x, w, kept)
    kept.update(w.detach())
    with pytest.raises(RuntimeError, match="updated after"):
        y.backward(g)


def test_linear8_gradient_is_the_difference(torch_dev):
    """Moves of the input and the weight that 8 bits hold exactly move the output by the
    gradient: small whole numbers, where nothing is rounded."""
    torch, dev = torch_dev
    gen = np.random.default_rng(7)
    x = torch.from_numpy(gen.integers(-3, 4, (40, 256)).astype(np.float32)).to(dev).requires_grad_()
    w = torch.from_numpy(gen.integers(-3, 4, (70, 256)).astype(np.float32)).to(dev).requires_grad_()
    g = torch.from_numpy(gen.integers(-2, 3, (40, 70)).astype(np.float32)).to(dev)
    (muon.linear8(x, w) * g).sum().backward()
    dx, dw = (torch.from_numpy(gen.integers(-1, 2, t.shape).astype(np.float32)).to(dev) for t in (x, w))

    def loss(a, b):
        return float((muon.linear8(a, b).double() * g).sum())

    with torch.no_grad():
        for step in (1.0, -1.0):
            assert loss(x + step * dx, w) - loss(x, w) == step * float((x.grad.double() * dx).sum())
            assert loss(x, w + step * dw) - loss(x, w) == step * float((w.grad.double() * dw).sum())
