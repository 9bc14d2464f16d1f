"""GPU parity of AdamW over many tensors (32-bit and 8-bit states), of the gradient norm
with its clip factor, and of scaling in place, with the float64 oracles.

u = 2^-24. Tolerances by arithmetic:
  m: b1 m and (1 - b1) g' with g' = s g, four roundings: 4 u (|b1 m| + |(1 - b1) g'|), and
  u of the stored scale where the state has 8 bits; v likewise with 6, both addends > 0.
  update d = lr/(1 - b1^t) m / (u/sqrt(1 - b2^t) + eps): the error of m, and relative to d
  half of v's (3 u), root 2 u, the fused denominator u, reciprocal and product 3 u,
  the factor from the host 2 u (its two halves rounded): 12 u with 1 to spare.
  W: the factor (1 - lr wd) and its product with W, and the last rounding: 3 u |W|.
  8-bit codes: m / scale is off by the error of m and 3 u (the scale's product, the
  reciprocal's two roundings): the code has to be the neighbour that the rounding bits
  choose, or the other one where the fraction is that close to the bits' edge (2^-16 of
  a gap and the error); scales 4 u and the error of the largest magnitude.
  norms: fp64 sums rounded once, u (1 + 2^-20).
"""
import sys

import numpy as np
import pytest

from oracle import adamw8_oracle as O8
from oracle import adamw_oracle as A
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B
from matrix_orthogonalising_optimizer_02_amd import workloads as WL

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def as_hp(**over):
    base = dict(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
    base.update(over)
    return A.AdamWHParams(**{k: float(np.float32(v)) for k, v in base.items()}), muon.adamw_default_hparams(**base)


def log(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch_dev():
    import torch
    assert torch.cuda.is_available(), "the gpu tests need a visible GPU"
    B.load_library()
    return torch, torch.device("cuda:0")


def types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def host(t):
    return t.detach().double().cpu().numpy().ravel()


def codes(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


def tensors(torch, dev, key, role, shapes, std, dt=None, step=0):
    out = [torch.from_numpy(WL.host_normal(key, role, i, s, std, step)).to(dev) for i, s in enumerate(shapes)]
    return out if dt is None else [t.to(dt) for t in out]


def check_codes(got, scale, x, err, bits, floor, what):
    """Codes against the values before rounding (float64) and what they may be off."""
    ref_scale = O8.block_scales(x)
    top = np.pad(err, (0, -err.size % O8.BLOCK)).reshape(-1, O8.BLOCK).max(1) / O8.E4M3_MAX
    assert (np.abs(scale - ref_scale) <= 4 * U * ref_scale + top).all(), what
    lo, hi, frac = O8.candidates(x, ref_scale)
    s = np.repeat(ref_scale, O8.BLOCK)[:x.size]
    gap = np.maximum(O8.VALUES[hi] - O8.VALUES[lo], 2.0 ** -9)
    mag = np.abs(x)
    slack = np.divide(err + (3 * U + 4 * U) * mag + np.repeat(top, O8.BLOCK)[:x.size] * mag / np.maximum(s, 1e-300) , s * gap,
                      out=np.zeros_like(mag), where=s > 0)
    up = frac + bits / 65536.0 >= 1.0
    close = np.abs(frac + bits / 65536.0 - 1.0) <= slack + 2.0 ** -16
    # right at a code, the neighbour below is as near
    at_code = frac <= slack
    mags = got & 127
    least = np.where((floor > 0) & (mag > 0), floor, 0)
    want = np.maximum(np.where(up, hi, lo), least)
    other = np.maximum(np.where(up, lo, hi), least)
    below = np.maximum(np.maximum(lo - 1, 0), least)
    ok = (mags == want) | (close & (mags == other)) | (at_code & ((mags == below) | (mags == lo)))
    assert ok.all(), (what, int((~ok).sum()), mags[~ok][:5], want[~ok][:5])
    assert (mags[x == 0] == 0).all(), what
    signed = mags > 0
    assert ((got[signed] >> 7) == (x[signed] < 0)).all(), what
    return float(np.count_nonzero(mags != want)) / max(1, mags.size)


def run_steps(torch, dev, shapes, bits, gname, copy, steps, key, start=0, seed=7, scale=None, lr_scales=None, wd_scales=None,
              g_std=1e-3, w_std=0.02, hp=None):
    """Teacher-forced steps on the GPU against the oracle."""
    ohp, hp = hp or as_hp()
    dt = types(torch)[gname]
    w = tensors(torch, dev, key, WL.ROLE_W, shapes, w_std)
    cp = [torch.zeros(s, dtype=types(torch)[copy], device=dev) for s in shapes] if copy else None
    opt = muon.AdamWMulti(w, tensors(torch, dev, key, WL.ROLE_G, shapes, g_std, dt), hp, state_bits=bits, copies=cp, seed=seed,
                          lr_scales=lr_scales, wd_scales=wd_scales)
    factor = None if scale is None else torch.tensor([scale], device=dev)
    gs = 1.0 if scale is None else float(np.float32(scale))
    differ = 0.0
    for step in range(start, start + steps):
        g = tensors(torch, dev, key, WL.ROLE_G, shapes, g_std, dt, step)
        before = [(host(w[i]), codes(opt.exp_avg[i]).copy() if bits == 8 else host(opt.exp_avg[i]),
                   codes(opt.exp_avg_sq[i]).copy() if bits == 8 else host(opt.exp_avg_sq[i])) for i in range(len(shapes))]
        scales = [(host(opt.exp_avg_scale[i]), host(opt.exp_avg_sq_scale[i])) for i in range(len(shapes))] if bits == 8 else None
        opt.step(step, grad_scale=factor, grads=g)
        torch.cuda.synchronize()
        for i, s in enumerate(shapes):
            w0, m0, v0 = before[i]
            gv = host(g[i]) * gs
            lrs = 1.0 if lr_scales is None else float(np.float32(lr_scales[i]))
            wds = 1.0 if wd_scales is None else float(np.float32(wd_scales[i]))
            ohi = A.AdamWHParams(ohp.lr * lrs, ohp.beta1, ohp.beta2, ohp.eps, ohp.weight_decay * wds)
            if bits == 8:
                n = w0.size
                md = O8.decode(m0) * np.repeat(scales[i][0], O8.BLOCK)[:n]
                vd = (O8.decode(v0) * np.repeat(scales[i][1], O8.BLOCK)[:n]) ** 2
            else:
                md, vd = m0, v0
            rw, rm, rv = A.adamw_step(w0, gv, md, vd, step, ohi)
            em = 5 * U * (np.abs(ohi.beta1 * md) + np.abs((1 - ohi.beta1) * gv)) + 2.0 ** -148
            ev = 8 * U * rv + 2.0 ** -148
            ru = np.sqrt(rv)
            t = step + 1
            den = ru / np.sqrt(1 - ohi.beta2 ** t) + ohi.eps
            k = abs(ohi.lr) / (1 - ohi.beta1 ** t)
            tol = k * (em + 13 * U * np.abs(rm)) / den + 3 * U * np.abs(w0)
            got = host(w[i])
            assert (np.abs(got - rw) <= tol).all(), (s, step, float(np.max(np.abs(got - rw) / tol)))
            if copy:
                assert torch.equal(cp[i], w[i].to(cp[i].dtype)), (s, step)
            if bits == 32:
                assert (np.abs(host(opt.exp_avg[i]) - rm) <= em).all(), (s, step)
                assert (np.abs(host(opt.exp_avg_sq[i]) - rv) <= ev).all(), (s, step)
            else:
                bm, bv = O8.rounding_bits(seed, step, i, np.arange(w0.size))
                eu = 0.5 * np.divide(ev, ru, out=np.full_like(ru, 2.0 ** -74), where=ru > 1e-18) + 2 * U * ru
                differ = max(differ, check_codes(codes(opt.exp_avg[i]), host(opt.exp_avg_scale[i]), rm, em, bm, 0, (s, step, "m")))
                differ = max(differ, check_codes(codes(opt.exp_avg_sq[i]), host(opt.exp_avg_sq_scale[i]), ru, eu, bv, 1,
                                                 (s, step, "u")))
    return opt, differ


RAGGED = [(1,), (3,), (255,), (256,), (257,), (4095,), (4096,), (4097,), (10001,), (7, 33), (128, 256), (3, 5, 7)]


@pytest.mark.parametrize("gname", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_ragged_sizes_vs_oracle(torch_dev, bits, gname):
    torch, dev = torch_dev
    _, differ = run_steps(torch, dev, RAGGED, bits, gname, "bf16" if gname != "f16" else "f16", 3, 700)
    log(f"{bits} bits, {gname} gradients: {differ:.2e} of the codes at the edge of their bits")


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_empty_ones_and_scales(torch_dev, bits):
    torch, dev = torch_dev
    shapes = [(0,), (5,), (0,)] + [(37 * (i % 7) + 5,) for i in range(150)] + [(70000,), (0,)]
    n = len(shapes)
    run_steps(torch, dev, shapes, bits, "f32", None, 2, 701, scale=0.37, lr_scales=[1.0 + (i % 3) for i in range(n)],
              wd_scales=[float(i % 2) for i in range(n)])


@pytest.mark.parametrize("bits", [32, 8])
def test_late_step_other_hyperparameters_and_seeds(torch_dev, bits):
    torch, dev = torch_dev
    hp = as_hp(lr=3e-3, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.0)
    run_steps(torch, dev, [(5000,), (64, 64)], bits, "bf16", None, 2, 702, start=(1 << 32) + 5, seed=(5 << 40) + 3, hp=hp)
    run_steps(torch, dev, [(700,)], bits, "f32", None, 2, 703, hp=as_hp(beta1=0.0, beta2=0.0), g_std=30.0)


def test_32_bit_states_agree_with_adamw_step(torch_dev):
    """The same formula as the library's adamw_step, within both calls' rounding."""
    torch, dev = torch_dev
    shapes = [(5000,), (33, 77)]
    w = tensors(torch, dev, 704, WL.ROLE_W, shapes, 0.0)
    w2 = [x.clone() for x in w]
    m, v = [torch.zeros_like(x) for x in w], [torch.zeros_like(x) for x in w]
    opt = muon.AdamWMulti(w2, w2[:0] + [torch.zeros_like(x) for x in w])
    for step in range(4):
        g = tensors(torch, dev, 704, WL.ROLE_G, shapes, 1e-3, None, step)
        B.adamw_step(w, g, m, v, step)
        opt.step(step, grads=g)
    torch.cuda.synchronize()
    for a, b in zip(w, w2):
        # four steps, each off by at most 13 u of its update on either side (and u of W)
        assert float((a - b).abs().max()) <= 4 * 30 * U * 4e-4


def test_8_bit_rounding_is_unbiased_and_never_drops_a_root(torch_dev):
    """v decays by 0.1% a step without a gradient: rounded to nearest it would stay for
    good. Stochastically, 200 steps bring its mean to 0.999^200 within 5 standard errors:
    a code's step is 1/8 at most of its value, so one rounding's variance is below
    (1/16)^2 (largest for a fraction of one half), and 200 of them on 2^16 elements give a
    mean off by at most sqrt(200) / 16 / 256 = 0.0035 (of u, relative)."""
    torch, dev = torch_dev
    n = 1 << 16
    w = [torch.zeros(n, device=dev)]
    g = [torch.from_numpy(WL.host_normal(705, 0, 0, (n,), 1.0)).to(dev).abs() + 0.5]
    g[0][::256] = 60.0  # a block's largest, so that the others lie between the codes
    opt = muon.AdamWMulti(w, g, state_bits=8, seed=11)
    opt.step(0)
    v0 = opt.moments(0)[1]
    zero = [torch.zeros(n, device=dev)]
    for step in range(1, 201):
        opt.step(step, grads=zero)
    v1 = opt.moments(0)[1]
    keep = torch.arange(n, device=dev) % 256 != 0
    ratio = float((v1.sqrt()[keep] / v0.sqrt()[keep]).mean())
    want = 0.999 ** 100
    log(f"mean root after 200 decays: {ratio:.4f} of the first, {want:.4f} expected")
    assert abs(ratio / want - 1.0) < 5 * 0.0035
    assert bool((v1 > 0).all())
    # a root far below its block's largest keeps the least code
    g2 = [torch.full((512,), 1e-9, device=dev)]
    g2[0][0], g2[0][300] = 1.0, 0.0
    opt = muon.AdamWMulti([torch.zeros(512, device=dev)], g2, state_bits=8)
    opt.step(0)
    c = opt.exp_avg_sq[0].view(torch.uint8)
    assert int(c[0]) == 126 and bool((c[1:256] == 1).all())
    assert int(c[300]) == 0


def test_non_finite_gradients_stay_in_their_block(torch_dev):
    torch, dev = torch_dev
    for bits in (8, 32):
        shapes = [(1000,), (300,)]
        w = tensors(torch, dev, 706, WL.ROLE_W, shapes, 0.02)
        g = tensors(torch, dev, 706, WL.ROLE_G, shapes, 1e-3)
        w2, g2 = [x.clone() for x in w], [x.clone() for x in g]
        g2[0][300] = float("nan")
        g2[0][700] = float("inf")
        a, b = muon.AdamWMulti(w, g, state_bits=bits, seed=3), muon.AdamWMulti(w2, g2, state_bits=bits, seed=3)
        a.step(0)
        b.step(0)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(w2[0])
        assert bad.nonzero().flatten().tolist() == [300, 700] and torch.equal(w[0][~bad], w2[0][~bad])
        a.step(1)
        b.step(1, grads=g)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(w2[0])
        want = torch.zeros(1000, dtype=torch.bool, device=dev)
        if bits == 8:  # the blocks of 256 that had them
            want[256:768] = True
        else:
            want[300] = want[700] = True
        assert bool((bad == want).all())
        assert torch.equal(w[0][~bad], w2[0][~bad]) and torch.equal(w[1], w2[1])


def test_save_and_resume_bitwise_and_seed_matters(torch_dev):
    torch, dev = torch_dev
    shapes = [(3000,), (17, 65)]
    grads = [tensors(torch, dev, 707, WL.ROLE_G, shapes, 1e-3, None, s) for s in range(6)]

    def fresh(seed=5):
        w = tensors(torch, dev, 707, WL.ROLE_W, shapes, 0.02)
        return w, muon.AdamWMulti(w, grads[0], state_bits=8, seed=seed)

    w, opt = fresh()
    for s in range(6):
        opt.step(s, grads=grads[s])
    w1, opt1 = fresh()
    for s in range(3):
        opt1.step(s, grads=grads[s])
    saved, ws = opt1.state_dict(), [x.clone() for x in w1]
    w2, opt2 = fresh(seed=99)
    opt2.load_state_dict(saved)
    for a, b in zip(w2, ws):
        a.copy_(b)
    for s in range(3, 6):
        opt2.step(s, grads=grads[s])
    torch.cuda.synchronize()
    for a, b in zip(w, w2):
        assert torch.equal(a, b)
    for a, b in zip(opt.exp_avg_sq, opt2.exp_avg_sq):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    _, opt3 = fresh(seed=6)
    for s in range(6):
        opt3.step(s, grads=grads[s])
    assert any(not torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(opt.exp_avg, opt3.exp_avg))


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_clip_and_step_replay_bitwise(torch_dev, bits):
    torch, dev = torch_dev
    shapes = [(5000,), (64, 130), (9,)]
    g = tensors(torch, dev, 708, WL.ROLE_G, shapes, 1.0)

    def fresh():
        w = tensors(torch, dev, 708, WL.ROLE_W, shapes, 0.02)
        return w, muon.AdamWMulti(w, g, state_bits=bits, seed=1), muon.GradNorm(g)

    w1, opt1, norm1 = fresh()
    w2, opt2, norm2 = fresh()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        norm2.measure(0.5)
        opt2.step(3, grad_scale=norm2.factor)
    assert all(torch.equal(a, b) for a, b in zip(w1, w2))
    for r in range(3):
        for i, t in enumerate(g):
            t.copy_(tensors(torch, dev, 709 + r, WL.ROLE_G, shapes, 1.0)[i])
        norm1.measure(0.5)
        opt1.step(3, grad_scale=norm1.factor)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm1.total, norm2.total) and torch.equal(norm1.norms, norm2.norms)
        for a, b in zip(w1 + opt1.exp_avg + opt1.exp_avg_sq, w2 + opt2.exp_avg + opt2.exp_avg_sq):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), r
        assert float(torch.randn(1 << 18, device=dev).sum()) != 0.0


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_step_with_a_counter_on_the_device(torch_dev, bits):
    """A captured step whose counter and learning rate are on the device: each replay is the
    next step, with other rounding bits, as a host loop of steps (the bias corrections, made
    in double on either side, may differ in fp32's last place: u of the update, 4 u with
    the update's own roundings)."""
    torch, dev = torch_dev
    shapes = [(5000,), (64, 130), (9,)]
    g = tensors(torch, dev, 750, WL.ROLE_G, shapes, 1e-3)

    def fresh():
        w = tensors(torch, dev, 750, WL.ROLE_W, shapes, 0.02)
        return w, muon.AdamWMulti(w, g, state_bits=bits, seed=1 << 33)

    w1, eager = fresh()
    w2, counted = fresh()
    counter, lr = torch.tensor([3], device=dev), torch.tensor([1e-4], device=dev)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        counted.step(counter, lr=lr)
    assert int(counter) == 3
    for r in range(4):
        for i, t in enumerate(g):
            t.copy_(tensors(torch, dev, 751 + r, WL.ROLE_G, shapes, 1e-3)[i])
        rate = float(np.float32(1e-4 * (r + 1)))
        lr.fill_(rate)
        eager.hp.lr = rate
        eager.step(3 + r)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert int(counter) == 4 + r
        for a, b in zip(eager.exp_avg + eager.exp_avg_sq, counted.exp_avg + counted.exp_avg_sq):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), r
        for a, b in zip(w1, w2):
            # updates of at most 4 lr a step so far, 4 u of each, and W's own rounding
            assert float((a - b).abs().max()) <= (r + 1) * (4 * U * 4 * rate * 4 + 2 * U * 0.2), r
        assert float(torch.randn(1 << 18, device=dev).sum()) != 0.0
    with pytest.raises(ValueError):
        counted.step(torch.tensor([3.0], device=dev))
    with pytest.raises(ValueError):
        counted.step(3, lr=lr)


def test_side_stream_step(torch_dev):
    torch, dev = torch_dev
    shapes = [(50000,), (77,)]
    g = tensors(torch, dev, 715, WL.ROLE_G, shapes, 1e-3)
    w1, w2 = tensors(torch, dev, 715, WL.ROLE_W, shapes, 0.02), tensors(torch, dev, 715, WL.ROLE_W, shapes, 0.02)
    a = muon.AdamWMulti(w1, g, state_bits=8)
    a.step(0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = muon.AdamWMulti(w2, g, state_bits=8, stream=side)
    norm = muon.GradNorm(g, stream=side)
    side.wait_stream(torch.cuda.current_stream())
    norm.measure(1e9, stream=side)
    b.step(0, grad_scale=norm.factor, stream=side)
    torch.full((1 << 20,), float("nan"), device=dev)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(w1, w2))


@pytest.mark.parametrize("gname", ["f32", "bf16", "f16"])
def test_grad_norm_vs_oracle(torch_dev, gname):
    torch, dev = torch_dev
    shapes = [(1,), (0,), (7, 33), (8192,), (16384,), (16385,), (300, 1000), (5,), (0,)] + [(11 + i,) for i in range(120)]
    dt = types(torch)[gname]
    g = tensors(torch, dev, 720, WL.ROLE_G, shapes, 0.7, dt)
    norm = muon.GradNorm(g)
    for max_norm in (0.25, 1e4):
        total, norms = norm.measure(max_norm)
        torch.cuda.synchronize()
        rn, rt, rf = O8.grad_norm([host(t) for t in g], float(np.float32(max_norm)))
        assert (np.abs(host(norms) - rn) <= U * (1 + 2.0 ** -20) * rn).all()
        got = host(total)
        assert abs(got[0] - rt) <= U * 1.001 * rt and abs(got[1] - rf) <= U * 1.001 * rf
        assert (got[1] == 1.0) == (max_norm > 1.0)
    # in place: each element times the factor, rounded once
    norm.measure(0.25)
    f = float(host(norm.total)[1])
    kept = [t.clone() for t in g]
    norm.scale_()
    torch.cuda.synchronize()
    for a, b in zip(g, kept):
        assert torch.equal(a, (b.float() * f).to(dt))
    kept = [t.clone() for t in g]
    norm.scale_(torch.ones(1, device=dev))
    norm.measure(1e9)
    norm.scale_()
    assert all(torch.equal(a, b) for a, b in zip(g, kept))


def test_grad_norm_range_unaligned_and_non_finite(torch_dev):
    torch, dev = torch_dev
    base = torch.zeros(70003, device=dev)
    g = [base[1:40002], base[40002:70003]]  # neither starts at 16 bytes
    g[0].fill_(3e25)
    g[1].fill_(2e-30)
    norm = muon.GradNorm(g)
    total, norms = norm.measure(1.0)
    want = float(np.float32(3e25)) * np.sqrt(40001.0), float(np.float32(2e-30)) * np.sqrt(30001.0)
    assert abs(float(norms[0]) / want[0] - 1) < 2 * U and abs(float(norms[1]) / want[1] - 1) < 2 * U
    norm.scale_(torch.tensor([0.5], device=dev))
    assert float(base[0]) == 0.0 and bool((g[0] == torch.tensor(3e25).to(dev) * 0.5).all())
    g[1][12345] = float("inf")
    assert float(norm.measure(1.0)[0][0]) == float("inf") and float(norm.total[1]) == 0.0
    g[0][39999] = float("nan")
    total, norms = norm.measure(1.0)
    assert bool(torch.isnan(total).all()) and bool(torch.isnan(norms[0])) and float(norms[1]) == float("inf")


def test_large_tensor_norm_and_step_repeat_bitwise(torch_dev):
    """More than 8192 runs of 16384 elements (longer runs), twice the same bits; against
    torch's float64 sum."""
    torch, dev = torch_dev
    gen = torch.Generator(device=dev)
    gen.manual_seed(5)
    n = 8192 * 16384 + 12345
    g = [torch.randn(n, generator=gen, device=dev, dtype=torch.bfloat16), torch.ones(3, device=dev)]
    norm = muon.GradNorm(g)
    a = [t.clone() for t in norm.measure(1.0)]
    b = norm.measure(1.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    sq = sum(float(p.double().square().sum()) for p in g[0].split(1 << 24))
    assert abs(float(a[1][0]) / np.sqrt(sq) - 1) < 1.01 * U


def test_new_gradients_at_other_addresses(torch_dev):
    torch, dev = torch_dev
    shapes = [(1000,), (77,)]
    w = tensors(torch, dev, 730, WL.ROLE_W, shapes, 0.02)
    g1, g2 = tensors(torch, dev, 730, WL.ROLE_G, shapes, 1.0), tensors(torch, dev, 731, WL.ROLE_G, shapes, 1.0)
    norm = muon.GradNorm(g1)
    first = norm.measure(1.0)[1].clone()
    norm.set_grads(g2)
    second = norm.measure(1.0)[1].clone()
    assert not torch.equal(first, second)
    norm.set_grads([t.bfloat16() for t in g1])
    third = norm.measure(1.0)[1]
    assert float((third / first - 1).abs().max()) < 2.0 ** -8
    opt = muon.AdamWMulti(w, g1)
    with pytest.raises(ValueError):
        opt.step(0, grads=g2[:1])
    with pytest.raises(ValueError):
        opt.step(0, grads=[g2[1], g2[0]])
    with pytest.raises(ValueError):
        opt.step(0, grad_scale=torch.ones(2, device=dev))


def test_offsets_past_32_bits(torch_dev):
    """One tensor of more than 2^32 elements with 8-bit states: its last blocks against the
    oracle (the rounding bits have the index's high word in them), and its norm."""
    torch, dev = torch_dev
    ohp, hp = as_hp()
    n = (1 << 32) + 4096 + 700
    gen = torch.Generator(dev).manual_seed(9)
    w = torch.zeros(n, device=dev)
    g = torch.empty(n, dtype=torch.bfloat16, device=dev).normal_(0.0, 1e-3, generator=gen)
    opt = muon.AdamWMulti([w], [g], hp, state_bits=8, seed=21)
    norm = muon.GradNorm([g])
    norm.measure(1e9)
    opt.step(0, grad_scale=norm.factor)
    torch.cuda.synchronize()
    sq = sum(float(p.double().square().sum()) for p in g.split(1 << 28))
    assert abs(float(norm.total[0]) / np.sqrt(sq) - 1) < 1.01 * U
    for first, count in ((n - 700 - 2048, 2748), ((1 << 32) - 512, 1024), (0, 512), (1 << 31, 256)):
        gv = host(g[first:first + count])
        rw, rm, rv = A.adamw_step(np.zeros(count), gv, np.zeros(count), np.zeros(count), 0, ohp)
        got = host(w[first:first + count])
        assert (np.abs(got - rw) <= 14 * U * np.abs(rw) + 2.0 ** -148).all()
        bm, bv = O8.rounding_bits(21, 0, 0, np.arange(first, first + count))
        blocks = slice(first // 256, -(-(first + count) // 256))
        em, eu = 5 * U * np.abs(rm) + 2.0 ** -148, 6 * U * np.sqrt(rv)
        check_codes(codes(opt.exp_avg[0][first:first + count]), host(opt.exp_avg_scale[0][blocks]), rm, em, bm, 0, first)
        check_codes(codes(opt.exp_avg_sq[0][first:first + count]), host(opt.exp_avg_sq_scale[0][blocks]), np.sqrt(rv), eu, bv, 1,
                    first)


def test_both_widths_in_one_plan(torch_dev):
    """The C call takes states of both widths in one list: the same as two lists, apart from
    the position that the rounding bits know."""
    import ctypes
    torch, dev = torch_dev
    shapes = [(5000,), (300,), (9000,)]
    w1, g = tensors(torch, dev, 740, WL.ROLE_W, shapes, 0.02), tensors(torch, dev, 740, WL.ROLE_G, shapes, 1e-3)
    w2 = [x.clone() for x in w1]
    small, wide = muon.AdamWMulti(w1, g, state_bits=8, seed=4), muon.AdamWMulti(w2, g, state_bits=32, seed=4)
    mixed_w = [x.clone() for x in w1]
    a, b = muon.AdamWMulti(mixed_w, g, state_bits=8, seed=4), muon.AdamWMulti(mixed_w, g, state_bits=32, seed=4)
    arr = (B.AdamWTensor * 3)(a._arr[0], b._arr[1], a._arr[2])
    need, plan = ctypes.c_size_t(), B.TensorPlan()
    lib = B.load_library()
    assert lib.adamw_multi_plan_bytes(arr, 3, need) == 0
    table = torch.empty(need.value, dtype=torch.uint8, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.adamw_multi_plan(arr, 3, table.data_ptr(), table.numel(), plan, stream) == 0
    for step in range(2):
        small.step(step)
        wide.step(step)
        assert lib.adamw_multi_step(plan, small.hp, step, 4, None, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(mixed_w[0], w1[0]) and torch.equal(mixed_w[1], w2[1]) and torch.equal(mixed_w[2], w1[2])
    assert torch.equal(a.exp_avg[2].view(torch.uint8), small.exp_avg[2].view(torch.uint8))


def test_overflowing_second_moment(torch_dev):
    """|g| above 1.8e19: v is infinite, the update 0 (fp32's own answer); 32-bit states keep
    it to the element."""
    torch, dev = torch_dev
    for bits in (8, 32):
        g = [torch.full((600,), 1e-3, device=dev)]
        g[0][10] = 3e25
        w = [torch.ones(600, device=dev)]
        opt = muon.AdamWMulti(w, g, muon.adamw_default_hparams(weight_decay=0.0), state_bits=bits)
        opt.step(0)
        torch.cuda.synchronize()
        assert float(w[0][10]) == 1.0 and bool(torch.isfinite(w[0]).all())
        g[0][10] = 0.0
        opt.step(1)
        bad = ~torch.isfinite(w[0])
        assert int(bad.sum()) == (256 if bits == 8 else 0)


@pytest.mark.parametrize("eps", [1e-30, 1e-18, 2.0 ** -126])
@pytest.mark.parametrize("bits", [32, 8])
def test_small_second_moments_and_small_eps(torch_dev, bits, eps):
    """Gradients of 1e-20 to 1e-17: v is a subnormal fp32 number, and eps no cover for its root.

    v is off by at most 2^-149 besides 8 u of itself (g'^2, its product, the decoded root's
    square and b2 times it each round to a multiple of 2^-149 there, to half a step, the
    first and the third times a factor below 1), so its root lies between those of v - e and
    v + e; the update is off by 16 u besides that and m's own error (the module's text)."""
    torch, dev = torch_dev
    ohp, hp = as_hp(lr=1e-3, eps=eps, weight_decay=0.0)
    sizes, n = [1e-17, 1e-18, 1e-19, 3e-20, 1e-20], 700
    rng = np.random.default_rng(5)
    w = [torch.zeros(n, device=dev) for _ in sizes]
    opt = muon.AdamWMulti(w, [torch.zeros(n, device=dev) for _ in sizes], hp, state_bits=bits, seed=9)
    for step in range(3):
        g = [torch.from_numpy((s * rng.uniform(0.9, 1.1, n) * rng.choice([-1.0, 1.0], n)).astype(np.float32)).to(dev)
             for s in sizes]
        if bits == 8:
            scales = [(host(opt.exp_avg_scale[i]), host(opt.exp_avg_sq_scale[i])) for i in range(len(sizes))]
            md = [O8.decode(codes(opt.exp_avg[i])) * np.repeat(s[0], O8.BLOCK)[:n] for i, s in enumerate(scales)]
            vd = [(O8.decode(codes(opt.exp_avg_sq[i])) * np.repeat(s[1], O8.BLOCK)[:n]) ** 2 for i, s in enumerate(scales)]
        else:
            md, vd = [host(t) for t in opt.exp_avg], [host(t) for t in opt.exp_avg_sq]
        before = [host(t) for t in w]
        opt.step(step, grads=g)
        torch.cuda.synchronize()
        for i, size in enumerate(sizes):
            gv, t = host(g[i]), step + 1
            _, rm, rv = A.adamw_step(before[i], gv, md[i], vd[i], step, ohp)
            ev = 1.5 * 2.0 ** -149 + 8 * U * rv
            em = 5 * U * (np.abs(ohp.beta1 * md[i]) + np.abs((1 - ohp.beta1) * gv)) + 2.0 ** -148
            lo, hi = np.sqrt(np.maximum(rv - ev, 0.0)), np.sqrt(rv + ev)
            k, bc = ohp.lr / (1 - ohp.beta1 ** t), np.sqrt(1 - ohp.beta2 ** t)
            least = k * np.maximum(np.abs(rm) - em, 0.0) / (hi / bc + ohp.eps) * (1 - 16 * U)
            most = k * (np.abs(rm) + em) / (lo / bc + ohp.eps) * (1 + 16 * U)
            got = (before[i] - host(w[i])) * np.sign(rm)
            tol = U * (np.abs(before[i]) + np.abs(host(w[i])))
            ok = (got >= least - tol) & (got <= most + tol)
            assert ok.all(), (size, step, float((got / most).max()), float((got / np.maximum(least, 1e-300)).min()))
            if bits == 32:
                assert (np.abs(host(opt.exp_avg_sq[i]) - rv) <= ev).all(), (size, step)
            else:  # the stored root: a code's step (1/8, or 2^-9 of the scale) either way
                top = np.repeat(host(opt.exp_avg_sq_scale[i]), O8.BLOCK)[:n]
                u1 = O8.decode(codes(opt.exp_avg_sq[i])) * top
                assert (u1 >= lo * 0.87 - top * 2.0 ** -9).all() and (u1 <= hi * 1.13 + top * 2.0 ** -9).all(), (size, step)
        log(f"{bits} bits, eps {eps:.1e}, step {step}: largest update {max(float(np.abs(host(t)).max()) for t in w):.2e}")


def test_gradients_changed_in_place_are_seen(torch_dev):
    """The same tensor objects with another size or layout are checked again, and other
    objects at the same addresses need no new table."""
    torch, dev = torch_dev
    g = [torch.zeros(1000, device=dev), torch.zeros(8, 4, device=dev)]
    w = [torch.zeros(1000, device=dev), torch.zeros(8, 4, device=dev)]
    opt, norm = muon.AdamWMulti(w, g), muon.GradNorm(g)
    opt.step(0, grads=g)
    B.timing_read()
    B.timing_enable()
    opt.step(1, grads=[t.view(t.shape) for t in g])
    norm.set_grads([t.view(t.shape) for t in g])
    plans = B.timing_read()["tensor_plan"][1]
    B.timing_enable(False)
    assert plans == 0
    opt.set_grads(g)
    g[0].resize_(500)
    for call in (lambda: opt.step(2, grads=g), lambda: norm.set_grads(g)):
        with pytest.raises(ValueError, match="1000 elements"):
            call()
    g[0].resize_(1000)
    g[1].t_()
    for call in (lambda: opt.step(2, grads=g), lambda: norm.set_grads(g)):
        with pytest.raises(ValueError, match="contiguous"):
            call()
    g[1].t_()
    opt.step(2, grads=g)
    with pytest.raises(TypeError):
        opt.step(3, grads=[None, g[1]])


@pytest.mark.parametrize("bits", [8, 32])
def test_refused_gradients_leave_those_given_before(torch_dev, bits):
    """A list that set_grads or a step refuses (off 16 bytes, on a weight, within a capture)
    changes nothing: the earlier gradients are kept, and steps and replays go on with them."""
    torch, dev = torch_dev
    shapes = [(1000,), (64, 9)]
    flat = torch.zeros(1001, device=dev)
    g = tensors(torch, dev, 760, WL.ROLE_G, shapes, 1e-3)
    want = [t.clone() for t in g]

    def fresh(grads):
        w = tensors(torch, dev, 760, WL.ROLE_W, shapes, 0.02)
        return w, muon.AdamWMulti(w, grads, state_bits=bits), muon.GradNorm(grads)

    w1, straight, norm1 = fresh(want)
    w2, opt, norm2 = fresh(g)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        norm2.measure(1.0)
        opt.step(0, norm2.factor)
    bad = [flat[1:], w2[0]]
    other = [t.clone() for t in g]
    del g
    for step in range(3):
        for first in bad:
            with pytest.raises(B.MuonError):
                opt.step(step, grads=[first, opt.grads[1]])
        with pytest.raises(B.MuonError):
            norm2.set_grads([other[0], other[0].view(-1)[:576].view(64, 9)])
        with pytest.raises(ValueError):
            norm2.set_grads(other[:1])
        if step == 1:
            second = torch.cuda.CUDAGraph()
            with pytest.raises(B.MuonError, match="captured"):
                with torch.cuda.graph(second, stream=side):
                    opt.step(step, grads=other)
            torch.cuda.synchronize()
        straight.step(step, norm1.measure(1.0)[0][1:])
        opt.step(step, norm2.measure(1.0)[0][1:])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w1 + [norm1.total, norm1.norms], w2 + [norm2.total, norm2.norms])), step
    norm1.measure(1.0)
    straight.step(0, norm1.factor)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(w1, w2))
    opt.step(4, grads=other)
    straight.step(4)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(w1, w2))


def test_tensors_that_got_other_memory_are_refused(torch_dev):
    """p.data = ... after the construction: a step would write where the tensor was."""
    torch, dev = torch_dev
    shapes = [(1000,), (64, 9)]
    for bits in (8, 32):
        w, g = tensors(torch, dev, 770, WL.ROLE_W, shapes, 0.02), tensors(torch, dev, 770, WL.ROLE_G, shapes, 1e-3)
        copies = [t.bfloat16() for t in w]
        opt, norm = muon.AdamWMulti(w, g, state_bits=bits, copies=copies), muon.GradNorm(g)
        opt.step(0)
        norm.measure(1.0)
        saved = opt.state_dict()
        for moved, calls in ((w[1], [lambda: opt.step(1), lambda: opt.step(1, grads=g), lambda: opt.check_step(1)]),
                             (copies[0], [lambda: opt.step(1)]),
                             (g[0], [lambda: norm.scale_()]),
                             (opt.exp_avg[0], [opt.state_dict, lambda: opt.moments(0), lambda: opt.load_state_dict(saved)])):
            old, kept = moved.data, [t.clone() for t in w + copies + opt.exp_avg]
            new = old.clone()
            moved.data = new
            for call in calls:
                with pytest.raises(ValueError, match="other memory"):
                    call()
            torch.cuda.synchronize()
            moved.data = old
            assert all(torch.equal(a, b) for a, b in zip([t.view(torch.uint8) for t in w + copies + opt.exp_avg],
                                                         [t.view(torch.uint8) for t in kept]))
        # a gradient's memory is the one that it had, and kept, until it is given again
        first = norm.measure(1.0)[1].clone()
        g[0].data = g[0].data * 3.0
        junk = torch.full((1000,), float("nan"), device=dev)
        assert torch.equal(norm.measure(1.0)[1], first)
        norm.set_grads(g)
        assert abs(float(norm.measure(1.0)[1][0] / first[0]) - 3.0) < 1e-5
        opt.step(1, grads=g)
        del junk


def test_scalars_within_the_tensors_are_refused(torch_dev):
    """A factor inside the gradients that it scales, or inside the weights, would be read by
    some blocks before and by others after it is written; beside them is fine."""
    torch, dev = torch_dev
    flat = torch.ones(4096, device=dev)
    g = [flat[:1000], flat[1024:2048]]
    norm = muon.GradNorm(g)
    norm.measure(1.0)
    for i in (0, 999, 1024, 2047):
        with pytest.raises(ValueError, match="within the tensors"):
            norm.scale_(flat[i:i + 1])
    torch.cuda.synchronize()
    assert bool((flat == 1.0).all())
    flat[1000] = 0.5
    norm.scale_(flat[1000:1001])
    assert bool((g[0] == 0.5).all()) and bool((g[1] == 0.5).all()) and float(flat[1001]) == 1.0 and float(flat[2048]) == 1.0
    for bits in (8, 32):
        w = [torch.ones(1000, device=dev), torch.ones(1, device=dev)]
        gw = [torch.ones(1000, device=dev), torch.ones(1, device=dev)]
        opt = muon.AdamWMulti(w, gw, state_bits=bits)
        ok, count = torch.ones(1, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
        wrong = [dict(grad_scale=w[1]), dict(grad_scale=w[0][7:8])]
        wrong += [dict(grad_scale=opt.exp_avg_scale[0][2:3])] if bits == 8 else [dict(grad_scale=opt.exp_avg[0][3:4])]
        for more in wrong:
            with pytest.raises(ValueError, match="within the tensors"):
                opt.step(0, **more)
        for step, lr in ((gw[0].view(torch.int64)[3:4], None), (w[0].view(torch.int64)[0:1], None), (count, w[0][1:2])):
            with pytest.raises(ValueError, match="within"):
                opt.step(step, lr=lr)
        torch.cuda.synchronize()
        assert bool((w[0] == 1.0).all()) and bool((gw[0] == 1.0).all()) and int(count) == 0
        opt.step(0, grad_scale=gw[1])  # a gradient is only read
        opt.step(count, grad_scale=ok, lr=ok)
        assert int(count) == 1
