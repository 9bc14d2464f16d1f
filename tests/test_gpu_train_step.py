"""The training-step operators together, as a transformer's step uses them: adaLN and the
query norm forward, their gradients, the gradient norm with its clip factor, and the
hybrid optimizer's step (Muon on the block matrix, AdamW with 8- or 32-bit states on the
norm weight and the biases), against the float64 oracles step by step.

Tolerances: the network's gradients are those of torch's float64 autograd on the same
fp32 parameters; the GPU's pass is fp32 (torch's own fp32 products between the norms), of
some 200 roundings deep at most along any path, relative Frobenius 2e-5. The optimizer's
parts: Muon's momentum 1e-6 against the oracle and its weights bit for bit against
muon_step on gradients that torch clipped (the modulation's gradient has rank 3 here, one
a sample, and the bf16 Newton-Schulz has nothing to be compared with in the other 189
directions: rounding noise of 2^-9 there grows by 3.4445^5 = 485); AdamW's update 4e-5 lr
besides W's own rounding, its moments as their own tests have them.
"""
import sys

import numpy as np
import pytest

from oracle import adamw8_oracle as O8
from oracle import adamw_oracle as A
from oracle import muon_oracle as O
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B
from matrix_orthogonalising_optimizer_02_amd import hybrid as H
from matrix_orthogonalising_optimizer_02_amd import workloads as WL

pytestmark = pytest.mark.gpu

SAMPLES, TOKENS, HIDDEN, HEADS = 3, 40, 192, 3
DIM = HIDDEN // HEADS
SHAPES = {"blocks.0.mod.weight": (2 * HIDDEN, HIDDEN), "blocks.0.mod.bias": (2 * HIDDEN,),
          "blocks.0.q.weight": (HIDDEN, HIDDEN), "blocks.0.q.bias": (HIDDEN,), "blocks.0.q_norm.weight": (DIM,),
          "final.norm.weight": (HIDDEN,), "final.norm.bias": (HIDDEN,)}


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a visible GPU"
    B.load_library()
    return torch, torch.device("cuda:0")


def network(torch, p, x, cond, norms):
    """A block's adaLN, query projection and query norm, and a final affine norm."""
    mod = cond @ p["blocks.0.mod.weight"].t() + p["blocks.0.mod.bias"]
    shift, scale = mod[:, :HIDDEN], mod[:, HIDDEN:]
    h = norms["adaln"](x, scale, shift)
    q = (h @ p["blocks.0.q.weight"].t() + p["blocks.0.q.bias"]).view(SAMPLES, TOKENS, HEADS, DIM)
    q = norms["rms"](q, p["blocks.0.q_norm.weight"])
    y = x + q.reshape(SAMPLES, TOKENS, HIDDEN)
    return norms["affine"](y, p["final.norm.weight"], p["final.norm.bias"])


def own_norms():
    return {"adaln": lambda x, s, b: muon.layer_norm(x, s, b, 1e-6, 1.0), "rms": lambda x, w: muon.rms_norm(x, w, 1e-6),
            "affine": lambda x, w, b: muon.layer_norm(x, w, b, 1e-6)}


def plain_norms(torch):
    eps = float(np.float32(1e-6))

    def layer(x):
        d = x - x.mean(-1, keepdim=True)
        return d / (d.square().mean(-1, keepdim=True) + eps).sqrt()

    return {"adaln": lambda x, s, b: layer(x) * (1.0 + s[:, None]) + b[:, None],
            "rms": lambda x, w: x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w,
            "affine": lambda x, w, b: layer(x) * w + b}


def host(t):
    return t.detach().double().cpu().numpy()


def rel(a, b):
    return float(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300))


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_of_a_small_block(torch_dev, bits):
    torch, dev = torch_dev
    params = {n: torch.from_numpy(WL.host_normal(900, 0, i, s, 0.05)).to(dev) for i, (n, s) in enumerate(SHAPES.items())}
    for n in ("blocks.0.q_norm.weight", "final.norm.weight"):
        params[n] += 1.0
    mhp = O.OracleHParams()
    ahp = A.AdamWHParams(**{f: float(np.float32(getattr(A.AdamWHParams(), f))) for f in
                            ("lr", "beta1", "beta2", "eps", "weight_decay")})
    opt = H.HybridOptimizer(params, adamw_state_bits=bits, max_grad_norm=0.5, seed=17)
    assert set(opt.muon_names) == {"blocks.0.mod.weight", "blocks.0.q.weight"}
    for step in range(4):
        x = torch.from_numpy(WL.host_normal(901, 0, step, (SAMPLES, TOKENS, HIDDEN), 1.0)).to(dev)
        cond = torch.from_numpy(WL.host_normal(902, 0, step, (SAMPLES, HIDDEN), 1.0)).to(dev)
        target = torch.from_numpy(WL.host_normal(903, 0, step, (SAMPLES, TOKENS, HIDDEN), 1.0)).to(dev)
        leaves = {n: p.detach().requires_grad_() for n, p in params.items()}
        loss = (network(torch, leaves, x, cond, own_norms()) - target).square().sum() / 100.0
        grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
        ref = {n: p.detach().double().cpu().requires_grad_() for n, p in params.items()}
        rloss = (network(torch, ref, x.double().cpu(), cond.double().cpu(), plain_norms(torch)) - target.double().cpu())
        rgrads = dict(zip(ref, torch.autograd.grad(rloss.square().sum() / 100.0, list(ref.values()))))
        worst = max(rel(host(grads[n]), host(rgrads[n])) for n in grads)
        assert worst < 2e-5, worst
        # the step from the GPU's own gradients and states
        before = {n: host(p) for n, p in params.items()}
        mom = {n: host(t) for n, t in opt.momenta.items()}
        ad = {n: [host(t) for t in opt._adamw.moments(i)] for i, n in enumerate(opt.adamw_names)}
        g_h = {n: host(g) for n, g in grads.items()}
        _, total, factor = O8.grad_norm(list(g_h.values()), 0.5)
        clip = torch.tensor([factor], device=dev)
        alone = {n: (params[n].clone(), opt.momenta[n].clone(), grads[n] * clip) for n in opt.muon_names}
        B.muon_step(*[[t[k] for t in alone.values()] for k in range(3)], step)
        opt.step({n: g.contiguous() for n, g in grads.items()})
        torch.cuda.synchronize()
        got = host(opt.grad_norm)
        assert abs(got[0] / total - 1) < 1e-6 and abs(got[1] / factor - 1) < 1e-6 and factor < 1.0
        for n in opt.muon_names:
            w_ref, m_ref = O.muon_step(before[n], mom[n], g_h[n] * factor, step, mhp)
            assert rel(host(opt.momenta[n]), m_ref) < 1e-6
            # W: what muon_step gives for the clipped gradients, to the bit
            assert torch.equal(params[n], alone[n][0]) and torch.equal(opt.momenta[n], alone[n][1]), (n, step)
        for i, n in enumerate(opt.adamw_names):
            w_ref, m_ref, v_ref = A.adamw_step(before[n], g_h[n] * factor, ad[n][0], ad[n][1], step, ahp)
            err = np.abs(host(params[n]) - w_ref)
            assert (err <= 1e-5 * ahp.lr * 4 + 2.0 ** -22 * np.abs(before[n])).all(), (n, step)
            if bits == 32:
                assert rel(host(opt._adamw.moments(i)[0]), m_ref) < 1e-6
                assert rel(host(opt._adamw.moments(i)[1]), v_ref) < 1e-6
            else:  # one code's step at most: 1/8 of the value, or 2^-9 of the scale
                m1, v1 = (host(t) for t in opt._adamw.moments(i))
                top = np.abs(m_ref).max() / 448 * 2.0 ** -9 * 1.01
                assert (np.abs(m1 - m_ref) <= np.abs(m_ref) / 8 * 1.01 + top).all(), (n, step)
                utop = np.sqrt(v_ref).max() / 448 * 2.0 ** -9 * 1.01
                assert (np.abs(np.sqrt(v1) - np.sqrt(v_ref)) <= np.sqrt(v_ref) / 8 * 1.01 + utop).all(), (n, step)
        log(f"step {step}: gradients {worst:.1e}, norm {total:.3f}")


def test_default_hybrid_optimizer_is_unchanged_and_kinds_do_not_mix(torch_dev):
    torch, dev = torch_dev
    params = {n: torch.from_numpy(WL.host_normal(910, 0, i, s, 0.05)).to(dev) for i, (n, s) in enumerate(SHAPES.items())}
    plain = H.HybridOptimizer({n: p.clone() for n, p in params.items()})
    multi = H.HybridOptimizer({n: p.clone() for n, p in params.items()}, adamw_state_bits=32)
    for step in range(3):
        grads = {n: torch.from_numpy(WL.host_normal(911, 2, i, s, 1e-3, step)).to(dev) for i, (n, s) in enumerate(SHAPES.items())}
        plain.step(grads)
        multi.step(grads)
    torch.cuda.synchronize()
    for n in SHAPES:
        if n in plain.muon_names:
            assert torch.equal(plain.params[n], multi.params[n])
        else:
            assert float((plain.params[n] - multi.params[n]).abs().max()) <= 2.0 ** -22
    with pytest.raises(ValueError):
        plain.load_state_dict(multi.state_dict())
    with pytest.raises(ValueError):
        multi.load_state_dict(plain.state_dict())
    with pytest.raises(ValueError):
        H.HybridOptimizer(params, max_grad_norm=1.0)
    with pytest.raises(ValueError):
        H.HybridOptimizer(params, adamw_state_bits=16)


@pytest.mark.parametrize("bits", [8, 32])
def test_hybrid_save_and_resume_bitwise(torch_dev, bits):
    torch, dev = torch_dev

    def fresh():
        return H.HybridOptimizer({n: torch.from_numpy(WL.host_normal(920, 0, i, s, 0.05)).to(dev)
                                  for i, (n, s) in enumerate(SHAPES.items())}, adamw_state_bits=bits, max_grad_norm=0.01, seed=3)

    def grads(step):
        return {n: torch.from_numpy(WL.host_normal(921, 2, i, s, 1e-3, step)).to(dev) for i, (n, s) in enumerate(SHAPES.items())}

    straight = fresh()
    for s in range(6):
        straight.step(grads(s))
    first = fresh()
    for s in range(3):
        first.step(grads(s))
    second = fresh()
    second.load_state_dict(first.state_dict())
    for n, p in second.params.items():
        p.copy_(first.params[n])
    for s in range(3, 6):
        second.step(grads(s))
    torch.cuda.synchronize()
    assert all(torch.equal(straight.params[n], second.params[n]) for n in SHAPES)


def test_whole_step_captured_and_replayed(torch_dev):
    """Norm forward and backward, clipping and the hybrid step in one graph: three replays,
    each against the same calls made eagerly. A first step within a capture is refused."""
    torch, dev = torch_dev
    x = torch.from_numpy(WL.host_normal(930, 0, 0, (512, HIDDEN), 1.0)).to(dev)
    dy = torch.from_numpy(WL.host_normal(930, 1, 0, (512, HIDDEN), 1.0)).to(dev)
    dw0 = torch.from_numpy(WL.host_normal(930, 2, 0, (HIDDEN, HIDDEN), 1e-2)).to(dev)

    def fresh():
        p = {"blocks.0.q.weight": torch.from_numpy(WL.host_normal(931, 0, 0, (HIDDEN, HIDDEN), 0.05)).to(dev),
             "n.weight": torch.ones(HIDDEN, device=dev), "n.bias": torch.zeros(HIDDEN, device=dev)}
        g = {n: torch.zeros_like(t) for n, t in p.items()}
        return p, g, H.HybridOptimizer(p, muon.default_hparams(period_k=1), adamw_state_bits=8, max_grad_norm=0.5)

    def one(p, g, opt):
        y, mean, rstd = muon.norm_forward(x, p["n.weight"], p["n.bias"])
        dx, dw, db = muon.norm_backward(dy, x, p["n.weight"], mean, rstd)
        g["n.weight"].copy_(dw)
        g["n.bias"].copy_(db)
        g["blocks.0.q.weight"].copy_(dw0)
        opt.step_count = 5  # a captured step keeps the step that it was captured at
        opt.step(g)
        return y, dx

    side = torch.cuda.Stream()
    p, g, opt = fresh()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with pytest.raises(B.MuonError, match="captured"):
        with torch.cuda.graph(graph, stream=side):
            one(p, g, opt)
    torch.cuda.synchronize()
    states = []
    for _ in range(2):
        p, g, opt = fresh()
        one(p, g, opt)  # the tables are written
        states.append((p, g, opt))
    torch.cuda.synchronize()
    (p1, g1, o1), (p2, g2, o2) = states
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        outs = one(p2, g2, o2)
    for r in range(3):
        want = one(p1, g1, o1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), r
        assert all(torch.equal(p1[n], p2[n]) and torch.equal(g1[n], g2[n]) for n in p1), r
        assert torch.equal(o1.grad_norm, o2.grad_norm)
        assert float(torch.randn(1 << 18, device=dev).sum()) != 0.0
