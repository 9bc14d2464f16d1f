"""The block's 8-bit path as a model uses it: two pre-norm layers (residual norm, fused
projection in 8 bits, query and key norms, rotary positions, an output projection) forward and
backward, stepped by the hybrid optimizer which keeps the weights' 8-bit forms, and the same
forward pass for a single token.

Tolerances, relative Frobenius, against the same network with torch's float64 autograd over the
values that the 8-bit operands stand for (quantising has the identity's gradient): a chain of fp32
steps is off by 2^-20 or so, which puts a share of 2^-16 of the values on the other side of a
code's border (codes are 2^-4 apart at least), and each of those moves by 2^-3 at most: 2^-8 2^-3
= 2^-11 behind a quantising, asserted to 2^-8. The backward pass starts from that difference:
a share of 2^-7 of the gradients' codes, 2^-3.5 2^-3 = 2^-6.5, asserted to 2^-4.
"""
import numpy as np
import pytest

import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B
from matrix_orthogonalising_optimizer_02_amd import hybrid as H

from test_gpu_blocks8 import exact, log, torch_dev  # noqa: F401
from test_gpu_norm import draw

pytestmark = pytest.mark.gpu

TOKENS, HIDDEN, HEADS = 150, 384, 3
DIM = HIDDEN // HEADS
SECTIONS = (16, 24, 24)
EPS = float(np.float32(1e-6))
SHAPES = {"blocks.0.qkv.weight": (3 * HIDDEN, HIDDEN), "blocks.0.proj.weight": (HIDDEN, HIDDEN), "blocks.0.norm.weight": (HIDDEN,),
          "blocks.0.q_norm.weight": (DIM,), "final.norm.weight": (HIDDEN,)}


def parameters(torch, dev):
    p = {}
    for i, (n, s) in enumerate(SHAPES.items()):
        p[n] = draw(torch, dev, 900, i, s, torch.float32, 0.05, 0.0 if len(s) == 2 else 1.0)
    return p


def network(torch, p, x, r, pos, axes, w8):
    """A layer by the library's operators, all for torch.autograd."""
    y, h = muon.add_rms_norm(x, r, p["blocks.0.norm.weight"])
    qkv = muon.linear8(y, p["blocks.0.qkv.weight"], w8.get("blocks.0.qkv.weight")).view(TOKENS, 3 * HEADS, DIM)
    qk = muon.rms_norm(qkv[:, :2 * HEADS], p["blocks.0.q_norm.weight"])
    qk = muon.rotary(qk, pos, axes)
    mix = qk[:, :HEADS] * qk[:, HEADS:] + qkv[:, 2 * HEADS:]  # in attention's place
    out = muon.linear8(mix.reshape(TOKENS, HIDDEN), p["blocks.0.proj.weight"], w8.get("blocks.0.proj.weight"))
    y, h = muon.add_rms_norm(out, h, p["final.norm.weight"])
    return y, h


def plain(torch, p, x, r, pos, freq):
    """The same in float64, with the operands of each product replaced by what they stand for in
    8 bits and the gradients of that replacement taken as the identity's, themselves quantised."""
    def norm(h, w):
        return h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w

    class Product(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a, w):
            qa, qat = muon.quantise8(a.float(), transposed=True)
            qw, qwt = muon.quantise8(w.float(), tiles=True, transposed=True)
            ctx.kept = qat, qwt
            return exact(qa) @ exact(qw).t().contiguous()

        @staticmethod
        def backward(ctx, g):
            qat, qwt = ctx.kept
            qg, qgt = muon.quantise8(g.float().contiguous(), transposed=True)
            return exact(qg) @ exact(qwt).t().contiguous(), exact(qgt) @ exact(qat).t().contiguous()

    h = x + r
    qkv = Product.apply(norm(h, p["blocks.0.norm.weight"]), p["blocks.0.qkv.weight"]).view(TOKENS, 3 * HEADS, DIM)
    qk = norm(qkv[:, :2 * HEADS], p["blocks.0.q_norm.weight"])
    angle = (pos.double()[:, np.repeat(np.arange(3), SECTIONS)] * freq)[:, None]
    a, b = qk[..., :DIM // 2], qk[..., DIM // 2:]
    qk = torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)
    mix = qk[:, :HEADS] * qk[:, HEADS:] + qkv[:, 2 * HEADS:]
    out = Product.apply(mix.reshape(TOKENS, HIDDEN), p["blocks.0.proj.weight"])
    h = out + h
    return norm(h, p["final.norm.weight"]), h


def far(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def test_a_layer_forward_backward_and_its_step(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    p = {n: t.requires_grad_() for n, t in parameters(torch, dev).items()}
    opt = H.HybridOptimizer({n: t.detach() for n, t in p.items()}, adamw_state_bits=8, max_grad_norm=1.0,
                            weights8=["blocks.0.qkv.weight", "blocks.0.proj.weight"])
    axes = muon.RotaryAxes(SECTIONS, device=dev)
    freq = torch.tensor(axes.frequencies, dtype=torch.float64, device=dev)
    pos = torch.from_numpy(np.random.default_rng(1).integers(0, 64, (TOKENS, 3)).astype(np.int32)).to(dev)
    for step in range(3):
        x, r, g = (draw(torch, dev, 910 + step, i, (TOKENS, HIDDEN), torch.float32, 1.0) for i in range(3))
        x.requires_grad_()
        y, h = network(torch, p, x, r, pos, axes, opt.weights8)
        ((y * g).sum() + (h * g).sum()).backward()
        ref = {n: t.detach().double().requires_grad_() for n, t in p.items()}
        xd = x.detach().double().requires_grad_()
        yd, hd = plain(torch, ref, xd, r.double(), pos, freq)
        ((yd * g).sum() + (hd * g).sum()).backward()
        errs = {"y": far(y, yd), "h": far(h, hd), "x": far(x.grad, xd.grad), **{n: far(t.grad, ref[n].grad) for n, t in p.items()}}
        log(f"step {step}: " + ", ".join(f"{n} {e:.1e}" for n, e in errs.items()))
        assert max(errs["y"], errs["h"]) < 2.0 ** -8
        assert errs["final.norm.weight"] < 2.0 ** -8 and errs["blocks.0.proj.weight"] < 2.0 ** -4
        assert max(errs.values()) < 2.0 ** -4
        opt.step({n: t.grad for n, t in p.items()})
        for n, w in opt.weights8.items():
            q, qt = muon.quantise8(p[n].detach(), tiles=True, transposed=True)
            for a, b in ((w.direct, q), (w.transposed, qt)):
                assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)
        for t in p.values():
            t.grad = None


def test_a_token_alone_is_the_batch_s(torch_dev):  # noqa: F811
    """The forward pass for one token, by the calls that write in place and the norm's own 8-bit
    output, against the same token inside a batch: the same codes, and sums in another order."""
    torch, dev = torch_dev
    p = parameters(torch, dev)
    w8 = {n: muon.Weight8(t) for n, t in p.items() if t.dim() == 2}
    axes = muon.RotaryAxes(SECTIONS, device=dev)
    x, r = (draw(torch, dev, 930, i, (TOKENS, HIDDEN), torch.bfloat16, 1.0) for i in range(2))
    pos = torch.from_numpy(np.random.default_rng(2).integers(0, 64, (TOKENS, 3))).to(dev)

    def forward(x, r, pos):
        h, _, y8, _ = muon.add_rms_norm_forward(x, r, p["blocks.0.norm.weight"], y=False, codes=True, stats=False)
        qkv = muon.matmul8(y8, w8["blocks.0.qkv.weight"].direct).view(len(x), 3 * HEADS, DIM)
        qk = qkv[:, :2 * HEADS]
        muon.norm_forward(qk, p["blocks.0.q_norm.weight"], kind="rms", out=qk, stats=False)
        muon.rotary_apply(qk, pos, axes, out=qk)
        return h, y8, qkv

    hb, yb, qb = forward(x, r.clone(), pos)
    for t in (0, 77, TOKENS - 1):
        h, y8, qkv = forward(x[t:t + 1], r[t:t + 1].clone(), pos[t:t + 1])
        assert torch.equal(h, hb[t:t + 1]) and torch.equal(y8.scales, yb.scales[t:t + 1])
        assert torch.equal(y8.codes.view(torch.uint8), yb.codes[t:t + 1].view(torch.uint8))
        # sums of 384 in another order, and one rounding of 2^-8 apart at each of three steps
        assert far(qkv, qb[t:t + 1]) < 3 * 2.0 ** -8


def test_hybrid_optimizer_names_its_weights(torch_dev):  # noqa: F811
    torch, dev = torch_dev
    p = parameters(torch, dev)
    for bad in (["blocks.0.norm.weight"], ["missing"]):
        with pytest.raises(ValueError, match="no 2-D parameter"):
            H.HybridOptimizer(p, weights8=bad)
    opt = H.HybridOptimizer(p, weights8=["blocks.0.proj.weight"])
    kept = opt.weights8["blocks.0.proj.weight"]
    before, version = kept.direct.codes.view(torch.uint8).clone(), kept.version
    p["blocks.0.proj.weight"].mul_(-1.0)
    opt.update_weights8()
    assert kept.version == version + 1
    assert torch.equal(kept.direct.codes.view(torch.uint8) ^ 0x80, before)
    assert B.MUON_OK == 0 and H.HybridOptimizer(p).weights8 == {}
