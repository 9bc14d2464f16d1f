"""Workloads of the training-step operators: normalisation layers with their gradients,
AdamW over many tensors with 32-bit or 8-bit states, and the gradient norm with its clip
factor. Each case can be run in a plain form (elementary torch operations in fp32) or
through the library, and against the definition in float64.

A case is a dict of plain values; `op` is one of

  norm_fwd   y = (x - mean) rstd (offset + w[g]) + b[g] over rows of `cols` elements
  norm_bwd   its input, weight and bias gradients
  adamw      one AdamW step over `count` tensors of `low` .. `high` elements
  grad_norm  l2 norm of every gradient, their total and the clip factor

Rows of a norm are split evenly into `groups`, each with its own weight and bias row
(adaLN: one group a sample). `heads` > 0: the rows are tokens x heads of a query view
inside a fused query-key-value projection, and are read strided.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
QBLOCK = 256          # elements of 8-bit state that share a scale
E4M3_MAX = 448.0
MAX_NORM = 1.0
CLIP_EPS = 1e-6
# the hyperparameters as the device holds them (fp32 values)
LR, BETA1, BETA2, ADAM_EPS, DECAY = (float(np.float32(v)) for v in (1e-4, 0.9, 0.999, 1e-8, 0.1))
FIRST_STEP = 100      # 0-based step of a state's first pass: the middle of a run's warm-up


def _norm(name, op, kind, rows, cols, groups, dtype, wdtype, offset, bias, heads=0):
    return {"name": name, "op": op, "kind": kind, "rows": rows, "cols": cols, "groups": groups, "dtype": dtype,
            "wdtype": wdtype, "offset": offset, "bias": bias, "heads": heads}


def _adamw(name, bits, count, low, high, gdtype, copy):
    return {"name": name, "op": "adamw", "bits": bits, "count": count, "low": low, "high": high, "gdtype": gdtype,
            "copy": copy}


def _gnorm(name, count, low, high, gdtype):
    return {"name": name, "op": "grad_norm", "count": count, "low": low, "high": high, "gdtype": gdtype}


def listed():
    return [
        # the pooled-text or timestep vector of one sample at H = 2048: all latency
        _norm("ln fwd one row", "norm_fwd", "layer", 1, 2048, 1, "bf16", "f32", 0.0, True),
        # adaLN before the attention of a 15B-scale block: eight images of 1024 tokens, H = 5120,
        # the scale and shift of each image from its modulation projection
        _norm("adaln fwd", "norm_fwd", "layer", 8192, 5120, 8, "bf16", "bf16", 1.0, True),
        # an affine layer norm in fp32 at sizes that no vector width divides
        _norm("ln bwd odd", "norm_bwd", "layer", 4999, 1153, 1, "f32", "f32", 0.0, True),
        # the backward pass of the adaLN above: the modulation's gradients are per image
        _norm("adaln bwd", "norm_bwd", "layer", 8192, 5120, 8, "bf16", "bf16", 1.0, True),
        # query norm of a 1.3B-scale block (16 heads of 128) over 8192 tokens, read from the
        # fused projection; its one weight row gathers a gradient over 131072 rows
        _norm("q norm bwd", "norm_bwd", "rms", 131072, 128, 1, "bf16", "f32", 0.0, False, 16),
        # a whole step's worth of tokens, 64 images, in one backward call
        _norm("adaln bwd large", "norm_bwd", "layer", 65536, 5120, 64, "bf16", "bf16", 1.0, True),
        # the norms and biases of one small block: all latency
        _adamw("adamw8 small", 8, 48, 128, 6144, "f32", False),
        # everything that Muon leaves to AdamW in a 16-block model: 238 tensors, bf16 gradients,
        # a bf16 copy of the weights for the next forward pass; first with 8-bit states, then 32
        _adamw("adamw8 model", 8, 238, 128, 8000000, "bf16", True),
        _adamw("adamw32 model", 32, 238, 128, 8000000, "bf16", True),
        # one large table (an embedder or an output projection) with fp32 gradients
        _adamw("adamw8 large", 8, 1, 268435456, 268435456, "f32", False),
        # the gradient norm of the same small block, and of a 15B-scale block's ten matrices
        _gnorm("grad norm small", 48, 128, 6144, "f32"),
        _gnorm("grad norm block", 10, 26214400, 157286400, "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "adamw", "grad_norm"])
    if op.startswith("norm"):
        kind = rng.choice(["layer", "rms"])
        dtype = rng.choice(["f32", "bf16", "f16"])
        c = {"op": op, "kind": kind, "dtype": dtype, "wdtype": rng.choice(["f32", dtype]),
             "offset": rng.choice([0.0, 1.0]), "bias": kind == "layer" and rng.random() < 0.8}
        if rng.random() < 0.25:
            heads = rng.choice([1, 3, 8, 16, 40])
            tokens = _log_int(rng, 1, 30000)
            c.update(rows=tokens * heads, cols=rng.choice([64, 72, 96, 128, 256]), groups=1, heads=heads)
        else:
            cols = _log_int(rng, 8, 16384)
            groups = rng.choice([1, 1, 2, 5, 8, 32])
            per = max(1, min(_log_int(rng, 1, 65536), 150000000 // (cols * groups)))
            c.update(rows=groups * per, cols=cols, groups=groups, heads=0)
        return c
    count = _log_int(rng, 1, 500)
    high = _log_int(rng, 256, max(300, min(100000000, 150000000 // count)))
    low = max(1, min(high, _log_int(rng, 1, high)))
    c = {"op": op, "count": count, "low": low, "high": high, "gdtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "adamw":
        c.update(bits=rng.choice([8, 8, 32]), copy=rng.random() < 0.5)
    return c


def _sizes(case):
    """Element counts between low and high, spread evenly over the logarithm."""
    lo, ratio = case["low"], case["high"] / case["low"]
    n = case["count"]
    return [max(1, int(lo * ratio ** ((i * 0.6180339887498949 + 0.5) % 1.0))) if ratio > 1 else lo for i in range(n)]


def _starts(sizes):
    """Each tensor's first element in one flat buffer, every start a multiple of QBLOCK."""
    at, starts = 0, []
    for n in sizes:
        starts.append(at)
        at += -(-n // QBLOCK) * QBLOCK
    return starts, at


def _heavy(n, scale, gen):
    """scale * Student-t(3): gradients have heavy tails."""
    z = torch.randn(n, generator=gen, device=DEV)
    chi = torch.zeros_like(z)
    for _ in range(3):
        chi += torch.randn(n, generator=gen, device=DEV).square_()
    return z.mul_(chi.div_(3.0).rsqrt_()).mul_(scale)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 2 + 1)
    return _prepare_norm(case, gen) if case["op"].startswith("norm") else _prepare_tensors(case, gen, int(seed))


def _prepare_norm(case, gen):
    rows, cols, groups, heads = case["rows"], case["cols"], case["groups"], case["heads"]
    dt, wdt = DT[case["dtype"]], DT[case["wdtype"]]

    def activations(scale, shift):
        if heads:  # the query part of [tokens, 3, heads, cols]
            full = torch.randn(rows // heads, 3, heads, cols, generator=gen, device=DEV)
            return (full * scale + shift).to(dt)[:, 0]
        x = torch.randn(rows, cols, generator=gen, device=DEV)
        return (x * scale + shift).to(dt)

    # channels of unlike sizes and offsets, as a residual stream has them
    chan = torch.randn(cols, generator=gen, device=DEV)
    st = {"case": case, "x": activations(torch.exp(0.5 * chan), 0.5 * torch.randn(cols, generator=gen, device=DEV))}
    centre = 0.0 if case["offset"] else 1.0
    st["w"] = (centre + 0.2 * torch.randn(groups, cols, generator=gen, device=DEV)).to(wdt)
    st["b"] = (0.2 * torch.randn(groups, cols, generator=gen, device=DEV)).to(wdt) if case["bias"] else None
    if case["op"] == "norm_bwd":
        st["dy"] = activations(1.0, 0.0) if not heads else \
            torch.randn(rows // heads, heads, cols, generator=gen, device=DEV).to(dt)
        mean, rstd = [], []
        for part in st["x"].reshape(rows, cols).split(8192):
            p = part.double()
            mu = p.mean(1) if case["kind"] == "layer" else torch.zeros_like(p[:, 0])
            mean.append(mu.float())
            rstd.append(((p - mu[:, None]).square().mean(1) + EPS).rsqrt().float())
        st["mean"], st["rstd"] = torch.cat(mean), torch.cat(rstd)
        if case["kind"] == "rms":
            st["mean"] = None
    return st


def _prepare_tensors(case, gen, seed):
    sizes = _sizes(case)
    starts, total = _starts(sizes)
    keep = torch.zeros(total, dtype=torch.bool, device=DEV)
    for a, n in zip(starts, sizes):
        keep[a:a + n] = True
    # every eleventh block of 256 is a table's row that no sample of the batch touched
    touched = (torch.arange(total // QBLOCK, device=DEV) % 11 != 5).repeat_interleave(QBLOCK) & keep
    g = torch.where(touched, _heavy(total, 1e-3, gen), 0.0).to(DT[case["gdtype"]])

    def views(flat):
        return [flat[a:a + n] for a, n in zip(starts, sizes)]

    st = {"case": case, "g": g, "starts": starts, "sizes": sizes}
    if case["op"] == "grad_norm":
        ids = torch.arange(len(sizes), device=DEV)
        ids = ids.repeat_interleave(torch.tensor([-(-n // QBLOCK) for n in sizes], device=DEV))
        # the blocks of a tensor are added up in 1024 sums, and then those
        st["sum_of_block"] = ids * 1024 + torch.arange(total // QBLOCK, device=DEV) % 1024
        if own:
            import matrix_orthogonalising_optimizer_02_amd as muon
            st["norm"] = muon.GradNorm(views(g))
        return st
    st["w"] = torch.where(keep, 0.02 * torch.randn(total, generator=gen, device=DEV), 0.0)
    st["m"] = torch.where(touched, 3e-4 * torch.randn(total, generator=gen, device=DEV), 0.0)
    st["v"] = torch.where(touched, (1e-3 * (0.5 + torch.rand(total, generator=gen, device=DEV))).square(), 0.0)
    st["copy"] = torch.zeros(total, dtype=torch.bfloat16, device=DEV) if case["copy"] else None
    st["scale"] = torch.tensor([0.75], device=DEV)
    st["step"], st["seed"] = FIRST_STEP, seed
    if case["bits"] == 8:
        for name, scale, x in (("m", "ms", st["m"]), ("v", "vs", st["v"].sqrt())):
            x = x.view(-1, QBLOCK)
            s = x.abs().amax(1) / E4M3_MAX
            st[name] = (x / torch.where(s > 0, s, 1.0)[:, None]).to(torch.float8_e4m3fn).reshape(-1)
            st[scale] = s
        first = torch.tensor([a // QBLOCK for a in starts], device=DEV)
        st["block_tensor"] = torch.bucketize(torch.arange(total // QBLOCK, device=DEV), first, right=True) - 1
        st["block_start"] = (torch.arange(total // QBLOCK, device=DEV) - first[st["block_tensor"]]) * QBLOCK
    if own:
        import matrix_orthogonalising_optimizer_02_amd as muon
        states = {"exp_avg": views(st["m"]), "exp_avg_sq": views(st["v"])}
        if case["bits"] == 8:
            for name, key in (("exp_avg_scale", "ms"), ("exp_avg_sq_scale", "vs")):
                states[name] = [st[key][a // QBLOCK:a // QBLOCK + -(-n // QBLOCK)] for a, n in zip(starts, sizes)]
        hp = muon.adamw_default_hparams(lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY)
        st["opt"] = muon.AdamWMulti(views(st["w"]), views(g), hp, state_bits=case["bits"], states=states, seed=seed,
                                    copies=views(st["copy"]) if case["copy"] else None)
    return st


def run(st):
    op = st["case"]["op"]
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "adamw": _adamw_step, "grad_norm": _grad_norm}[op](st)


def _norm_fwd(st):
    c = st["case"]
    if own:
        import matrix_orthogonalising_optimizer_02_amd as muon
        y, mean, rstd = muon.norm_forward(st["x"], st["w"], st["b"], kind=c["kind"], eps=EPS,
                                          weight_offset=c["offset"])
        return {"y": y, "mean": mean, "rstd": rstd}
    x = st["x"].float().reshape(c["groups"], -1, c["cols"])
    mean = x.mean(2, keepdim=True) if c["kind"] == "layer" else None
    d = x if mean is None else x - mean
    rstd = (d.square().mean(2, keepdim=True) + EPS).rsqrt()
    y = d * rstd * (c["offset"] + st["w"].float()[:, None])
    if st["b"] is not None:
        y = y + st["b"].float()[:, None]
    return {"y": y.to(DT[c["dtype"]]).reshape(st["x"].shape), "mean": None if mean is None else mean.reshape(-1),
            "rstd": rstd.reshape(-1)}


def _norm_bwd(st):
    c = st["case"]
    if own:
        import matrix_orthogonalising_optimizer_02_amd as muon
        dx, dw, db = muon.norm_backward(st["dy"], st["x"], st["w"], st["mean"], st["rstd"], kind=c["kind"],
                                        weight_offset=c["offset"], bias_grad=c["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    shape = (c["groups"], -1, c["cols"])
    dy, h = st["dy"].float().reshape(shape), st["x"].float().reshape(shape)
    r = st["rstd"].view(c["groups"], -1, 1)
    if st["mean"] is not None:
        h = h - st["mean"].view(c["groups"], -1, 1)
    h = h * r
    a = dy * (c["offset"] + st["w"].float()[:, None])
    dx = a - h * (a * h).mean(2, keepdim=True)
    if st["mean"] is not None:
        dx = dx - a.mean(2, keepdim=True)
    wdt = DT[c["wdtype"]]
    return {"dx": (r * dx).to(DT[c["dtype"]]).reshape(st["x"].shape), "dw": (dy * h).sum(1).to(wdt),
            "db": dy.sum(1).to(wdt) if c["bias"] else None}


def _mix(x):
    """A 32-bit multiply-xorshift hash of int64 values below 2^32."""
    x = (x ^ (x >> 16)) * 0x6A09E667 & 0xFFFFFFFF
    x = (x ^ (x >> 15)) * 0xBB67AE85 & 0xFFFFFFFF
    return x ^ (x >> 16)


def _round_bits(seed, step, tensor, index):
    """32 bits for element `index` of tensor `tensor` (int64 arrays): the low 16 round the
    first moment, the high 16 the second."""
    key = _mix(_mix(_mix(seed & 0xFFFFFFFF) + (seed >> 32) & 0xFFFFFFFF) + step & 0xFFFFFFFF)
    key = _mix(key + tensor * 0x510E527F & 0xFFFFFFFF)
    lo, hi = index & 0xFFFFFFFF, index >> 32
    return _mix(lo * 0x9E3779B9 + hi * 0x510E527F + key & 0xFFFFFFFF)


def _stochastic_e4m3(a, bits16):
    """e4m3 codes of 0 <= a <= 448 (fp32), rounded up where the 16 bits say so."""
    raw = a.view(torch.int32).long()
    normal = ((raw + (bits16 << 4)) >> 20) - (120 << 3)
    small = ((a * 2.0 ** 25).long() + bits16) >> 16
    return torch.where(a >= 2.0 ** -6, normal, small)


def _quantise(x, bits16, floor_code):
    """(codes, scales) of x [blocks, QBLOCK]; a magnitude above 0 gets at least floor_code."""
    amax = x.abs().amax(1, keepdim=True)
    some = amax >= 1e-30
    a = (x.abs() * torch.where(some, E4M3_MAX / amax, 0.0)).clamp(max=E4M3_MAX)
    code = torch.maximum(_stochastic_e4m3(a, bits16), (a > 0).long() * floor_code) | ((x < 0).long() << 7)
    return code.to(torch.uint8).view(torch.float8_e4m3fn).reshape(-1), torch.where(some, amax / E4M3_MAX, 0.0).view(-1)


def _adamw_step(st):
    c = st["case"]
    step = st["step"]
    st["step"] += 1
    out = {k: st[k] for k in ("w", "copy", "m", "v", "ms", "vs") if st.get(k) is not None}
    if own:
        st["opt"].step(step, grad_scale=st["scale"])
        return out
    g = st["g"].float() * st["scale"]
    if c["bits"] == 8:
        m = st["m"].float().view(-1, QBLOCK) * st["ms"][:, None]
        v = (st["v"].float().view(-1, QBLOCK) * st["vs"][:, None]).square()
        g = g.view(-1, QBLOCK)
    else:
        m, v = st["m"], st["v"]
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g.square()
    u = v.sqrt()
    t = step + 1
    upd = (LR / (1.0 - BETA1 ** t)) * m / (u / math.sqrt(1.0 - BETA2 ** t) + ADAM_EPS)
    st["w"].copy_((1.0 - LR * DECAY) * st["w"] - upd.reshape(-1))
    if c["copy"]:
        st["copy"].copy_(st["w"])
    if c["bits"] == 8:
        index = st["block_start"][:, None] + torch.arange(QBLOCK, device=DEV)
        bits = _round_bits(st["seed"], step, st["block_tensor"][:, None], index)
        code, s = _quantise(m, bits & 0xFFFF, 0)
        st["m"].copy_(code)
        st["ms"].copy_(s)
        code, s = _quantise(u, bits >> 16, 1)
        st["v"].copy_(code)
        st["vs"].copy_(s)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return out


def _grad_norm(st):
    if own:
        total, norms = st["norm"].measure(MAX_NORM)
        return {"total": total, "norms": norms}
    sums = st["g"].float().view(-1, QBLOCK).square().sum(1)
    sq = torch.zeros(len(st["sizes"]) * 1024, device=DEV, dtype=torch.float64)
    sq = sq.index_add_(0, st["sum_of_block"], sums.double()).view(-1, 1024).sum(1)
    norm = sq.sum().sqrt()
    clip = (MAX_NORM / (norm + CLIP_EPS)).clamp(max=1.0)
    return {"total": torch.stack([norm, clip]).float(), "norms": sq.sqrt().float()}


def work(case):
    if case["op"].startswith("norm"):
        n, e = case["rows"] * case["cols"], SIZE[case["dtype"]]
        per_group = case["groups"] * case["cols"] * SIZE[case["wdtype"]]
        stats = case["rows"] * 4 * (2 if case["kind"] == "layer" else 1)
        rows_of = 2 if case["bias"] else 1
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * n * e + stats + rows_of * per_group, "flops": 8 * n}
        return {"bytes": 3 * n * e + stats + (1 + rows_of) * per_group, "flops": 14 * n}
    n, e = sum(_sizes(case)), SIZE[case["gdtype"]]
    if case["op"] == "grad_norm":
        return {"bytes": n * e + 4 * case["count"], "flops": 2 * n}
    per = 8 + e + (2 if case["copy"] else 0) + (16 if case["bits"] == 32 else 4 + 16 / QBLOCK)
    return {"bytes": n * per, "flops": (15 if case["bits"] == 32 else 40) * n}


def exact(case, seed):
    """The operators by their definitions in float64, tensor by tensor."""
    st = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(case, st)
    if case["op"] == "grad_norm":
        norms = torch.stack([st["g"][a:a + n].double().norm() for a, n in zip(st["starts"], st["sizes"])])
        total = norms.norm()
        return {"total": torch.stack([total, (MAX_NORM / (total + CLIP_EPS)).clamp(max=1.0)]), "norms": norms}
    return _exact_adamw(case, st)


def _exact_norm(case, st):
    groups, cols = case["groups"], case["cols"]
    per = case["rows"] // groups
    xs = st["x"].reshape(groups, per, cols)
    layer = case["kind"] == "layer"
    if case["op"] == "norm_fwd":
        out = {"y": torch.empty(groups, per, cols, dtype=torch.float64, device=DEV)}
        mean, var = torch.zeros(groups, per, dtype=torch.float64, device=DEV), []
        for k in range(groups):
            x = xs[k].double()
            if layer:
                mean[k] = x.sum(1) / cols
                x = x - mean[k][:, None]
            var.append((x * x).sum(1) / cols)
            y = x / (var[-1] + EPS).sqrt()[:, None] * (st["w"][k].double() + case["offset"])
            out["y"][k] = y if st["b"] is None else y + st["b"][k].double()
        out["y"] = out["y"].reshape(st["x"].shape)
        out["mean"] = mean.reshape(-1) if layer else None
        out["rstd"] = 1.0 / (torch.cat(var) + EPS).sqrt()
        return out
    dys = st["dy"].reshape(groups, per, cols)
    dx = torch.empty(groups, per, cols, dtype=torch.float64, device=DEV)
    dw, db = [], []
    for k in range(groups):
        rows = slice(k * per, (k + 1) * per)
        r = st["rstd"][rows].double()[:, None]
        h = (xs[k].double() - (st["mean"][rows].double()[:, None] if layer else 0.0)) * r
        dy = dys[k].double()
        a = dy * (st["w"][k].double() + case["offset"])
        inner = a - h * ((a * h).sum(1, keepdim=True) / cols)
        dx[k] = r * (inner - a.sum(1, keepdim=True) / cols if layer else inner)
        dw.append((dy * h).sum(0))
        db.append(dy.sum(0))
    return {"dx": dx.reshape(st["x"].shape), "dw": torch.stack(dw), "db": torch.stack(db) if case["bias"] else None}


def _exact_adamw(case, st):
    step, t = st["step"], st["step"] + 1
    w = st["w"].double()
    out = {"w": w, "m": torch.zeros_like(w), "v": torch.zeros_like(w)}
    if case["copy"]:
        out["copy"] = torch.zeros_like(w)
    if case["bits"] == 8:
        out["ms"], out["vs"] = st["ms"].double(), st["vs"].double()
    for i, (a, n) in enumerate(zip(st["starts"], st["sizes"])):
        at, pad = slice(a, a + n), -n % QBLOCK
        g = st["g"][at].double() * st["scale"].double()
        m, v = st["m"][at].double(), st["v"][at].double()
        if case["bits"] == 8:
            blocks = slice(a // QBLOCK, (a + n + pad) // QBLOCK)
            m = m * st["ms"][blocks].double().repeat_interleave(QBLOCK)[:n]
            v = (v * st["vs"][blocks].double().repeat_interleave(QBLOCK)[:n]) ** 2
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + g * g * (1.0 - BETA2)
        mhat, vhat = m / (1.0 - BETA1 ** t), v / (1.0 - BETA2 ** t)
        w[at] -= LR * (mhat / (vhat.sqrt() + ADAM_EPS) + DECAY * w[at])
        if case["copy"]:
            out["copy"][at] = w[at]
        if case["bits"] == 32:
            out["m"][at], out["v"][at] = m, v
            continue
        bits = _round_bits(st["seed"], step, torch.tensor([i], device=DEV), torch.arange(n, device=DEV))
        for name, scale, x, b in (("m", "ms", m, bits & 0xFFFF), ("v", "vs", v.sqrt(), bits >> 16)):
            s = torch.nn.functional.pad(x.abs(), (0, pad)).view(-1, QBLOCK).amax(1) / E4M3_MAX
            out[scale][blocks] = s
            mag = x.abs() / torch.where(s > 0, s, 1.0).repeat_interleave(QBLOCK)[:n]
            # the spacing of e4m3 around mag: 2^(e - 3), e the exponent, at least -6
            ulp = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3.0)
            down = torch.floor(mag / ulp)
            up = down + (mag / ulp - down + b.double() / 65536.0 >= 1.0)
            val = up * ulp
            if name == "v":
                val = torch.where(mag > 0, val.clamp(min=2.0 ** -9), val)
            out[name][at] = torch.where(x < 0, -val, val)
    return out
