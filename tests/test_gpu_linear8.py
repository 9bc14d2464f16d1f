"""linear8 on the GPU: what stays allocated, the same gradients through offloading and
checkpointing, sums that cancel; and the ends of the powers' range."""
import numpy as np
import pytest

from oracle import blocks8_oracle as Q
import matrix_orthogonalising_optimizer_02_amd as muon
from test_gpu_blocks8 import VALUES, draw, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


def layer(torch, dev, rows=300, cols=520, out=260):
    x = draw(torch, dev, 510, (rows, cols), torch.bfloat16).requires_grad_()
    w = draw(torch, dev, 511, (out, cols), torch.float32, 0.02).requires_grad_()
    return x, w, draw(torch, dev, 512, (rows, out), torch.bfloat16)


def test_memory_after_the_backward_pass(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    x, w, g = layer(torch, dev, 1024, 1024, 1024)
    muon.linear8(x, w).backward(g)  # x.grad and w.grad have their memory
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = muon.linear8(x, w)
    assert torch.cuda.memory_allocated() - before >= y.numel() * 2 + x.numel() + w.numel()
    y.backward(g)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before == y.numel() * 2
    with pytest.raises(RuntimeError, match="second time"):
        y.backward(g)


def test_offloaded_and_checkpointed(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    x, w, g = layer(torch, dev)
    kept = muon.Weight8(w)

    def gradients(call):
        x.grad = w.grad = None
        y = call()
        y.backward(g)
        torch.cuda.synchronize()
        return y.detach(), x.grad, w.grad

    def offloaded(w8):
        with torch.autograd.graph.save_on_cpu():
            return muon.linear8(x, w, w8)

    for w8 in (None, kept):
        want = gradients(lambda: muon.linear8(x, w, w8))
        for call in (lambda: offloaded(w8),
                     lambda: torch.utils.checkpoint.checkpoint(lambda a, b: muon.linear8(a, b, w8), x, w, use_reentrant=False)):
            assert all(torch.equal(a, b) for a, b in zip(want, gradients(call)))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("kept", [False, True])
def test_sums_that_cancel(torch_dev, dtype, kept):  # noqa: F811
    """products=16: small products beside large ones that cancel each other. Every product and
    partial sum is a multiple of 2^-16 below 2^17 in magnitude that eleven significant bits or a
    few more hold, so that sums as of fp32 additions are exact; the 8-bit instructions drop what
    lies 2^-13 below the largest of eight products."""
    torch, dev = torch_dev
    v = torch.ones(16, device=dev)
    v[0] = v[8] = 256.0
    s = v.clone()
    s[8] = -256.0
    w = (v[:, None] * v[None, :] / 256.0).requires_grad_()
    x = s[None, :].repeat(3, 1).to(getattr(torch, dtype)).requires_grad_()
    y = muon.linear8(x, w, muon.Weight8(w) if kept else None, products=16)
    y.backward(x.detach())
    want = (v * 14.0 / 256.0)[None, :].repeat(3, 1)  # v . s = 14
    assert torch.equal(y.detach().float(), want) and torch.equal(x.grad.float(), want)


def every_code(torch, dev, byte, rows):
    """A Blocks8 [rows, 256] of all codes by turns under one power, and its values in float64."""
    codes = (torch.arange(256, device=dev, dtype=torch.uint8)[None, :] + torch.arange(rows, device=dev, dtype=torch.uint8)[:, None])
    q = muon.Blocks8(codes.view(torch.float8_e4m3fn), torch.full((rows, 4), byte, dtype=torch.uint8, device=dev), 256)
    return q, torch.from_numpy(VALUES).to(dev)[codes.long()] * (2.0 ** (byte - 127) if byte < 255 else float("nan"))


@pytest.mark.parametrize("byte", [0, 1, 2, 3, 8, 127, 247, 254, 255])
def test_one_meaning_of_a_power(torch_dev, byte):  # noqa: F811
    """code 2^(byte - 127), from the smallest byte to the largest, 255 a NaN: read back, and
    multiplied by the identity at 1 in both widths. fp32 holds all of it that is below its
    largest; bf16, and the products through it, round what has bits below 2^-133."""
    torch, dev = torch_dev
    q, want = every_code(torch, dev, byte, 40)
    assert torch.equal(q.dequantise().cpu().nan_to_num(7.0), want.cpu().float().nan_to_num(7.0))
    assert torch.equal(q.dequantise(torch.bfloat16).cpu().nan_to_num(7.0), want.cpu().float().to(torch.bfloat16).nan_to_num(7.0))
    clean = want.isfinite() & (want.abs() < 2.0 ** 119)  # times 2^(130 - 127), within bf16
    codes = q.codes.view(torch.uint8).clone()
    codes[~clean] = 0
    if byte == 255:
        codes[:] = 0x38
    unit = torch.zeros(256, 256, dtype=torch.uint8, device=dev)
    unit.fill_diagonal_(0x38)  # 1
    for m in (40, 140):  # few rows, and tiles
        a = muon.Blocks8(codes.repeat(4, 1)[:m].view(torch.float8_e4m3fn), q.scales.repeat(4, 1)[:m], 256)
        b = muon.Blocks8(unit.view(torch.float8_e4m3fn), torch.full((256, 4), 130, dtype=torch.uint8, device=dev), 256)
        exact = torch.where(clean, want, 0.0 * want.nan_to_num()).repeat(4, 1)[:m] * 8.0
        for products in (8, 16):
            got = muon.matmul8(a, b, dtype=torch.float32, products=products)
            torch.cuda.synchronize()
            if byte == 255:
                assert bool(got.isnan().all()), (m, products)
            else:
                # eight times half a step of bf16's subnormals
                assert bool(((got.double() - exact).abs() <= (8.0 * 2.0 ** -134 if products == 16 and byte < 3 else 0.0)).all()), (m, products)


def test_blocks_of_subnormals(torch_dev):  # noqa: F811
    """Blocks below 2^-118 are read back as they were rounded."""
    torch, dev = torch_dev
    x = draw(torch, dev, 513, (20, 300), torch.float32).clamp(-50, 50) * 2.0 ** -126
    for tiles in (False, True):
        q, qt = muon.quantise8(x, tiles=tiles, transposed=True)
        for got, ref in ((q, x.double().cpu().numpy()), (qt, x.double().cpu().numpy().T)):
            want, e = Q.quantise(ref, tiles)
            assert (e == -127).any() and np.array_equal(got.dequantise().double().cpu().numpy(), want)


def test_no_rows_and_one_row(torch_dev):  # noqa: F811
    """Empty batches through the autograd forms, and inputs that are a single row."""
    torch, dev = torch_dev
    w = draw(torch, dev, 514, (30, 40), torch.float32, 0.02).requires_grad_()
    n = torch.ones(40, device=dev, requires_grad=True)
    axes = muon.RotaryAxes((2, 3), device=dev)
    for lead in ((0,), (2, 0)):
        x = torch.zeros(lead + (40,), device=dev, dtype=torch.bfloat16, requires_grad=True)
        y, h = muon.add_rms_norm(x, torch.zeros_like(x), n)
        z = muon.linear8(y, w)
        q = muon.rotary(z.view(lead + (3, 10)), torch.zeros(lead + (2,), device=dev, dtype=torch.int32), axes)
        (q.float().sum() + h.float().sum()).backward()
        torch.cuda.synchronize()
        assert x.grad.shape == x.shape and z.shape == lead + (30,)
        assert not w.grad.any() and not n.grad.any() and w.grad.shape == w.shape
        w.grad = n.grad = None
    x, w8 = draw(torch, dev, 515, (1, 40), torch.bfloat16), muon.Weight8(w)
    flat = x[0].clone().requires_grad_()
    y = muon.linear8(flat, w, w8)
    y.backward(torch.ones_like(y))
    want = x.clone().requires_grad_()
    z = muon.linear8(want, w, w8)
    z.backward(torch.ones_like(z))
    assert y.shape == (30,) and torch.equal(y, z[0]) and torch.equal(flat.grad, want.grad[0])
