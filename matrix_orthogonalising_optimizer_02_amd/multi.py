"""AdamW and gradient clipping over many tensors, one launch a step whatever their count.

`AdamWMulti` is the AdamW side of the hybrid optimizer for large parameter lists: fp32
weights, gradients in any type, states in 32 bits or in 8, an optional 16-bit copy of the
weights, and a gradient factor that stays on the device. `GradNorm` measures the
gradients' norms and the clip factor that feeds it.
"""
from __future__ import annotations

import bisect
import ctypes
import operator
from typing import Optional

from . import binding as B

STATE_BLOCK = 256  # elements of an 8-bit state that share a scale


def _check_list(tensors, name, device=None, dtypes=None, numels=None):
    torch = B._torch()
    if device is not None and device.type == "cuda" and dtypes is not None and B.plainly_right(tensors, set(dtypes), device) \
            and (numels is None or list(map(torch.Tensor.numel, tensors)) == numels):
        return
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name}[{i}] must be a torch.Tensor")
        if dtypes is not None and t.dtype not in dtypes:
            raise ValueError(f"{name}[{i}] must have dtype {' or '.join(str(d) for d in dtypes)}")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        if numels is not None and t.numel() != numels[i]:
            raise ValueError(f"{name}[{i}] must have {numels[i]} elements")
        if t.device.type != "cuda":
            raise ValueError(f"{name}[{i}] must live on a GPU")
        if device is not None and t.device != device:
            raise ValueError(f"{name}[{i}] must live on {device}")


def _device_of(tensors, name):
    """The first tensor's device; the current one of an empty list."""
    torch = B._torch()
    if not tensors:
        return torch.device("cuda", torch.cuda.current_device())
    if not isinstance(tensors[0], torch.Tensor):
        raise TypeError(f"{name}[0] must be a torch.Tensor")
    return tensors[0].device


def _per_tensor(values, n, name):
    if values is None:
        return [1.0] * n
    values = [float(v) for v in values]
    if len(values) != n:
        raise ValueError(f"one {name} per parameter")
    return values


_dtype = operator.attrgetter("dtype")


def _unchanged(grads, ptrs, numels, dtypes, plan):
    """Whether gradients are placed as those of the last table, and that was written."""
    if plan.kind == 0 or ptrs is None:
        return False
    t = B._torch().Tensor
    try:
        return list(map(t.data_ptr, grads)) == ptrs and list(map(t.numel, grads)) == numels \
            and list(map(_dtype, grads)) == dtypes and all(map(t.is_contiguous, grads))
    except (TypeError, AttributeError):  # not tensors: the checks say which
        return False


def _moved(tensors, ptrs):
    """Index of the first tensor that is no longer at its address, or None."""
    now = list(map(B._torch().Tensor.data_ptr, tensors))
    return None if now == ptrs else next(i for i, (a, b) in enumerate(zip(now, ptrs)) if a != b)


class _Watch:
    """Tensors (by list, in `parts`) whose addresses stand in a table, and those addresses."""

    def __init__(self, parts):
        self.parts = parts
        self.tensors = [t for tensors in parts.values() for t in tensors]
        self.data_ptr = B._torch().Tensor.data_ptr
        self.ptrs = list(map(self.data_ptr, self.tensors))

    def check(self):
        if list(map(self.data_ptr, self.tensors)) == self.ptrs:
            return
        i = _moved(self.tensors, self.ptrs)
        for name, tensors in self.parts.items():
            if i < len(tensors):
                raise ValueError(f"{name}[{i}] has other memory than when it was given")
            i -= len(tensors)


class _Spans:
    """The bytes at ptrs, as disjoint address ranges in order."""

    def __init__(self, ptrs, sizes):
        self.starts, self.ends = [], []
        last = 0
        for lo, size in sorted(zip(ptrs, sizes)):
            hi = lo + size
            if lo > last:
                if size:
                    self.starts.append(lo)
                    self.ends.append(hi)
                    last = hi
            elif hi > last:
                self.ends[-1] = last = hi

    def touch(self, ptr, nbytes):
        i = bisect.bisect_left(self.starts, ptr + nbytes) - 1
        return i >= 0 and self.ends[i] > ptr


def _need_grads(grads):
    if grads is None:
        raise ValueError("there are no gradients: give them first")


def _copy(arr):
    return type(arr).from_buffer_copy(arr)


def _next_plan(rc, new, old):
    """The plan to go on with after a plan call: the new one, or the old one where the call was
    refused before it wrote anything (a launch that failed leaves a plan that steps refuse)."""
    return old if rc and not new.device else new


def _scalar_ptr(t, name, device, written):
    """Device pointer of a one-element float32 tensor outside the spans that the call writes."""
    torch = B._torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() != 1:
        raise ValueError(f"{name} must be a float32 tensor of one element")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}")
    ptr = t.data_ptr()
    if written.touch(ptr, 4):
        raise ValueError(f"{name} lies within the tensors that the call writes")
    return ptr


class AdamWMulti:
    """AdamW over a list of fp32 parameters of any shapes, in one launch a step.

    The gradient tensors given here, or to set_grads() or step() later (float32, bfloat16
    or float16), are kept and read at every step until others are given or
    release_grads() lets go of them. Their addresses stand in a
    table on the device that is written when they change, which cannot be captured into a
    graph: give the gradients before a capture. Replayed steps read the table too, so new
    gradients are new for them as well. The parameters', copies' and states' addresses are
    those of the construction: a step refuses parameters and copies that have got other
    memory since (`p.data = ...`, a module moved or converted). Of a gradient the memory
    that it had when it was given is kept and read.
    state_bits: 32, or 8 for moments in e4m3 with one scale for every 256 elements (a
    quarter of the memory), rounded stochastically from `seed`, the step and the position.
    copies: optional 16-bit tensors that receive the updated weights.
    lr_scales, wd_scales: optional factors per parameter on lr and on weight decay.
    states: optional dict of existing states as state_dict() names them, used in place:
    lists `exp_avg` and `exp_avg_sq` (32 bits: float32; 8 bits: float8_e4m3fn, where
    exp_avg_sq holds square roots) and for 8 bits `exp_avg_scale`, `exp_avg_sq_scale`
    (float32, ceil(numel / 256) entries). Otherwise the states start at zero.
    """

    def __init__(self, params, grads=None, hp: Optional[B.AdamWHParams] = None, state_bits: int = 32, copies=None,
                 lr_scales=None, wd_scales=None, seed: int = 0, states=None, stream=None):
        torch = B._torch()
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be in [0, 2^64)")
        self.params, self.hp, self.state_bits, self.seed = list(params), hp or B.adamw_default_hparams(), state_bits, seed
        n = self.n = len(self.params)
        self.device = _device_of(self.params, "params")
        _check_list(self.params, "params", self.device, (torch.float32,))
        self._numels = [p.numel() for p in self.params]
        self.copies = None if copies is None else list(copies)
        if self.copies is not None:
            if len(self.copies) != n:
                raise ValueError("one copy per parameter")
            _check_list(self.copies, "copies", self.device, (torch.bfloat16, torch.float16), self._numels)
        lr_scales, wd_scales = _per_tensor(lr_scales, n, "lr_scale"), _per_tensor(wd_scales, n, "wd_scale")
        with B.device_and_stream(self.device, stream):
            self._make_states(states)
        codes = B.dtype_codes()
        self._arr = (B.AdamWTensor * max(n, 1))()
        small = state_bits == 8
        for i, p in enumerate(self.params):
            c = self.copies[i] if self.copies is not None else None
            self._arr[i] = B.AdamWTensor(
                self._numels[i], p.data_ptr() or None, c.data_ptr() or None if c is not None else None, None,
                self.exp_avg[i].data_ptr() or None, self.exp_avg_sq[i].data_ptr() or None,
                self.exp_avg_scale[i].data_ptr() or None if small else None,
                self.exp_avg_sq_scale[i].data_ptr() or None if small else None, 0,
                codes[c.dtype] if c is not None else 0, state_bits, lr_scales[i], wd_scales[i])
        # The kernel writes to all of these. The first are looked at in every step; the states, whose
        # memory is kept, where they are read or replaced by name.
        self._fixed = _Watch({"params": self.params, **({"copies": self.copies} if self.copies is not None else {})})
        self._states = _Watch({name: getattr(self, name) for name in self._state_names})
        sizes = [4 * k for k in self._numels] + [2 * k for k in self._numels if self.copies is not None]
        sizes += [k if small else 4 * k for k in self._numels] * 2
        sizes += [4 * -(-k // STATE_BLOCK) for k in self._numels if small] * 2
        self._written = _Spans(self._fixed.ptrs + self._states.ptrs, sizes)
        lists = self._states.parts.values()  # own states: a list has one memory
        self._states.memory = [t.untyped_storage() for ts in lists for t in (ts if states is not None else ts[:1])]
        self._plan = B.TensorPlan()
        self._empty = B.TensorPlan()
        B._check(B.load_library().adamw_multi_plan(None, 0, None, 0, self._empty, None), "adamw_multi_plan")
        self._table = None
        self.grads = self._ptrs = self._dtypes = self._read = None
        if grads is not None:
            self.set_grads(grads, stream)

    def _make_states(self, states):
        torch = B._torch()
        small = self.state_bits == 8
        dtype = torch.float8_e4m3fn if small else torch.float32
        scales = [-(-k // STATE_BLOCK) for k in self._numels]
        names = {"exp_avg": self._numels, "exp_avg_sq": self._numels}
        if small:
            names.update(exp_avg_scale=scales, exp_avg_sq_scale=scales)
        for name, sizes in names.items():
            kind = torch.float32 if name.endswith("scale") else dtype
            if states is not None:
                tensors = list(states[name])
                if len(tensors) != self.n:
                    raise ValueError(f"one {name} per parameter")
                _check_list(tensors, name, self.device, (kind,), sizes)
            else:
                # one zeroed buffer, every tensor at a multiple of 256 bytes
                size = torch.empty(0, dtype=kind).element_size()
                starts, at = [], 0
                for k in sizes:
                    starts.append(at)
                    at += -(-k * size // 256) * 256
                flat = torch.zeros(at, dtype=torch.uint8, device=self.device)
                tensors = [flat[a:a + k * size].view(kind) for a, k in zip(starts, sizes)]
            setattr(self, name, tensors)
        self._state_names = tuple(names)

    def set_grads(self, grads, stream=None):
        """New gradient tensors. Their addresses are written to the table on `stream` where
        one differs from before; steps that follow on the stream read them. Tensors that are
        refused leave those given before."""
        torch = B._torch()
        grads = list(grads)
        if _unchanged(grads, self._ptrs, self._numels, self._dtypes, self._plan):
            if self.grads is None or not all(map(operator.is_, grads, self.grads)):
                self._take(grads)
            return
        if len(grads) != self.n:
            raise ValueError("one gradient per parameter")
        _check_list(grads, "grads", self.device, (torch.float32, torch.bfloat16, torch.float16), self._numels)
        self._fixed.check()
        codes = B.dtype_codes()
        arr, ptrs, dtypes = _copy(self._arr), [g.data_ptr() for g in grads], [g.dtype for g in grads]
        for d, ptr, dtype in zip(arr, ptrs, dtypes):
            d.g, d.g_dtype = ptr or None, codes[dtype]
        lib = B.load_library()
        with B.device_and_stream(self.device, stream):
            if self._table is None:
                need = ctypes.c_size_t(0)
                B._check(lib.adamw_multi_plan_bytes(arr, self.n, need), "adamw_multi_plan_bytes")
                self._table = torch.empty(max(need.value, 1), dtype=torch.uint8, device=self.device)
            plan = B.TensorPlan()
            rc = lib.adamw_multi_plan(arr, self.n, self._table.data_ptr(), self._table.numel(), plan,
                                      B.raw_stream(stream, self.device))
        self._plan = _next_plan(rc, plan, self._plan)
        B._check(rc, "adamw_multi_plan")
        self._arr, self._ptrs, self._dtypes, self._read = arr, ptrs, dtypes, None
        self._take(grads)

    def _take(self, grads):
        self.grads, self._memory = grads, [g.untyped_storage() for g in grads]

    def release_grads(self):
        """Lets go of the gradient tensors: the next step needs some given first. Tensors at
        the same addresses then need no new table."""
        self.grads = self._memory = self._read = None

    def step(self, step, grad_scale=None, stream=None, grads=None, lr=None):
        """One step. step: the 0-based step number, or, for steps in a captured graph, a
        one-element int64 device tensor that holds it and is increased by the call, so each
        AdamWMulti has its own (a number would stay as it was at the capture, and with it
        the bias corrections and the rounding bits). grad_scale: optional one-element float32
        device tensor. lr: with a counter, an optional one-element float32 device tensor in
        place of hp.lr. None of the three may lie within what the step writes."""
        if grads is not None:
            self.set_grads(grads, stream)

    def _make_states(self, states):
        torch = B._torch()
        small = self.state_bits == 8
        dtype = torch.float8_e4m3fn if small else torch.float32
        scales = [-(-k // STATE_BLOCK) for k in self._numels]
        names = {"exp_avg": self._numels, "exp_avg_sq": self._numels}
        if small:
            names.update(exp_avg_scale=scales, exp_avg_sq_scale=scales)
        for name, sizes in names.items():
            kind = torch.float32 if name.endswith("scale") else dtype
            if states is not None:
                tensors = list(states[name])
                if len(tensors) != self.n:
                    raise ValueError(f"one {name} per parameter")
                _check_list(tensors, name, self.device, (kind,), sizes)
            else:
                # one zeroed buffer, every tensor at a multiple of 256 bytes
                size = torch.empty(0, dtype=kind).element_size()
                starts, at = [], 0
                for k in sizes:
                    starts.append(at)
                    at += -(-k * size // 256) * 256
                flat = torch.zeros(at, dtype=torch.uint8, device=self.device)
                tensors = [flat[a:a + k * size].view(kind) for a, k in zip(starts, sizes)]
            setattr(self, name, tensors)
        self._state_names = tuple(names)

    def set_grads(self, grads, stream=None):
        """New gradient tensors. Their addresses are written to the table on `stream` where
        one differs from before; steps that follow on the stream read them. Tensors that are
        refused leave those given before."""
        torch = B._torch()
        grads = list(grads)
        if _unchanged(grads, self._ptrs, self._numels, self._dtypes, self._plan):
            if self.grads is None or not all(map(operator.is_, grads, self.grads)):
                self._take(grads)
            return
        if len(grads) != self.n:
            raise ValueError("one gradient per parameter")
        _check_list(grads, "grads", self.device, (torch.float32, torch.bfloat16, torch.float16), self._numels)
        self._fixed.check()
        codes = B.dtype_codes()
        arr, ptrs, dtypes = _copy(self._arr), [g.data_ptr() for g in grads], [g.dtype for g in grads]
        for d, ptr, dtype in zip(arr, ptrs, dtypes):
            d.g, d.g_dtype = ptr or None, codes[dtype]
        lib = B.load_library()
        with B.device_and_stream(self.device, stream):
            if self._table is None:
                need = ctypes.c_size_t(0)
                B._check(lib.adamw_multi_plan_bytes(arr, self.n, need), "adamw_multi_plan_bytes")
                self._table = torch.empty(max(need.value, 1), dtype=torch.uint8, device=self.device)
            plan = B.TensorPlan()
            rc = lib.adamw_multi_plan(arr, self.n, self._table.data_ptr(), self._table.numel(), plan,
                                      B.raw_stream(stream, self.device))
        self._plan = _next_plan(rc, plan, self._plan)
        B._check(rc, "adamw_multi_plan")
        self._arr, self._ptrs, self._dtypes, self._read = arr, ptrs, dtypes, None
        self._take(grads)

    def _take(self, grads):
        self.grads, self._memory = grads, [g.untyped_storage() for g in grads]

    def release_grads(self):
        """Lets go of the gradient tensors: the next step needs some given first. Tensors at
        the same addresses then need no new table."""
        self.grads = self._memory = self._read = None

    def step(self, step, grad_scale=None, stream=None, grads=None, lr=None):
        """One step. step: the 0-based step number, or, for steps in a captured graph, a
        one-element int64 device tensor that holds it and is increased by the call, so each
        AdamWMulti has its own (a number would stay as it was at the capture, and with it
        the bias corrections and the rounding bits). grad_scale: optional one-element float32 device tensor. lr: with a
        counter, an optional one-element float32 device tensor in place of hp.lr."""
        if grads is not None:
            self.set_grads(grads, stream)
        _need_grads(self.grads)
        self._fixed.check()
        lib = B.load_library()
        scale = None if grad_scale is None else _scalar_ptr(grad_scale, "grad_scale", self.device, self._written)
        counter, rate = self._scalars(step, lr)
        with B.device_and_stream(self.device, stream):
            handle = B.raw_stream(stream, self.device)
            if counter is not None:
                rc = lib.adamw_multi_step_device(self._plan, self.hp, counter, rate, self.seed, scale, handle)
            else:
                rc = lib.adamw_multi_step(self._plan, self.hp, int(step), self.seed, scale, handle)
        B._check(rc, "adamw_multi_step")

    def check_step(self, step=0, lr=None):
        """Raises where step() would refuse the parameters, hp, the step's number or counter, or
        lr; enqueues nothing."""
        self._fixed.check()
        counter, _ = self._scalars(step, lr)
        rc = B.load_library().adamw_multi_step(self._empty, self.hp, 0 if counter else int(step), self.seed, None, None)
        B._check(rc, "adamw_multi_step")

    def _scalars(self, step, lr):
        """(address of the step's counter, of its learning rate), None where they are the host's."""
        torch = B._torch()
        if not isinstance(step, torch.Tensor):
            if lr is not None:
                raise ValueError("lr as a tensor goes with a step counter; otherwise set hp.lr")
            return None, None
        if step.dtype != torch.int64 or step.numel() != 1 or step.device != self.device:
            raise ValueError(f"a step counter must be an int64 tensor of one element on {self.device}")
        ptr = step.data_ptr()
        if self._read is None and self.grads is not None:
            self._read = _Spans(self._ptrs, [n * g.element_size() for n, g in zip(self._numels, self.grads)])
        if self._written.touch(ptr, 8) or (self._read is not None and self._read.touch(ptr, 8)):
            raise ValueError("the step counter lies within other tensors of the step")
        return ptr, None if lr is None else _scalar_ptr(lr, "lr", self.device, self._written)

    def moments(self, i: int):
        """The fp32 values of parameter i's first and second moment, in its shape."""
        self._states.check()
        p = self.params[i]
        if self.state_bits == 32:
            return self.exp_avg[i].view(p.shape).clone(), self.exp_avg_sq[i].view(p.shape).clone()
        out = []
        for codes, scale in ((self.exp_avg[i], self.exp_avg_scale[i]), (self.exp_avg_sq[i], self.exp_avg_sq_scale[i])):
            out.append((codes.float() * scale.repeat_interleave(STATE_BLOCK)[:p.numel()]).view(p.shape))
        return out[0], out[1].square()

    def state_dict(self):
        self._states.check()
        return {"state_bits": self.state_bits, "seed": self.seed,
                **{name: [t.clone() for t in getattr(self, name)] for name in self._state_names}}

    def load_state_dict(self, state):
        self._states.check()
        if state["state_bits"] != self.state_bits:
            raise ValueError(f"the saved states have {state['state_bits']} bits, these {self.state_bits}")
        seed = int(state["seed"])
        for name in self._state_names:
            if len(state[name]) != self.n:
                raise ValueError(f"one {name} per parameter")
            for dst, src in zip(getattr(self, name), state[name]):
                if dst.shape != src.shape or dst.dtype != src.dtype:
                    raise ValueError(f"{name} does not fit the parameters")
        self.seed = seed
        for name in self._state_names:
            for dst, src in zip(getattr(self, name), state[name]):
                dst.copy_(src)


class GradNorm:
    """l2 norms of a list of gradients, their total and the clip factor, on the device.

    The gradients' addresses are kept in a table, as AdamWMulti's (not within a capture);
    scale_() refuses gradients that have got other memory than when they were given.
    `total` (float32 [2]: the norm, the factor) and `norms` (float32 [count]) belong to the
    object and are overwritten by every measure(); calls on one object must not overlap.
    """

    def __init__(self, grads, stream=None):
        torch = B._torch()
        grads = list(grads)
        self.n = len(grads)
        self.device = _device_of(grads, "grads")
        self._arr = (B.GradTensor * max(self.n, 1))()
        self._plan = B.TensorPlan()
        self._table = self._numels = self.grads = self._ptrs = self._dtypes = None
        self.set_grads(grads, stream)
        with B.device_and_stream(self.device, stream):
            self.total = torch.empty(2, dtype=torch.float32, device=self.device)
            self.norms = torch.empty(self.n, dtype=torch.float32, device=self.device)
        self.norm, self.factor = self.total[0:1], self.total[1:2]

    def set_grads(self, grads, stream=None):
        """New gradient tensors of the same sizes; written to the table where an address differs."""
        torch = B._torch()
        grads = list(grads)
        if _unchanged(grads, self._ptrs, self._numels, self._dtypes, self._plan):
            if self.grads is None or not all(map(operator.is_, grads, self.grads)):
                self._take(grads)
            return
        if len(grads) != self.n:
            raise ValueError(f"{self.n} gradients are expected")
        _check_list(grads, "grads", self.device, (torch.float32, torch.bfloat16, torch.float16), self._numels)
        codes = B.dtype_codes()
        arr, ptrs, dtypes = _copy(self._arr), [g.data_ptr() for g in grads], [g.dtype for g in grads]
        numels = [g.numel() for g in grads]
        for d, ptr, numel, dtype in zip(arr, ptrs, numels, dtypes):
            d.g, d.numel, d.dtype = ptr or None, numel, codes[dtype]
        lib = B.load_library()
        with B.device_and_stream(self.device, stream):
            if self._table is None:
                need = ctypes.c_size_t(0)
                B._check(lib.grad_norm_plan_bytes(arr, self.n, need), "grad_norm_plan_bytes")
                self._table = torch.empty(max(need.value, 1), dtype=torch.uint8, device=self.device)
            plan = B.TensorPlan()
            rc = lib.grad_norm_plan(arr, self.n, self._table.data_ptr(), self._table.numel(), plan,
                                    B.raw_stream(stream, self.device))
        self._plan = _next_plan(rc, plan, self._plan)
        B._check(rc, "grad_norm_plan")
        self._arr, self._numels, self._ptrs, self._dtypes, self._written = arr, numels, ptrs, dtypes, None
        self._take(grads)

    def _take(self, grads):
        self.grads, self._memory = grads, [g.untyped_storage() for g in grads]

    def release_grads(self):
        """Lets go of the gradient tensors: the next call needs some given first. Tensors at
        the same addresses then need no new table."""
        self.grads = self._memory = None

    def measure(self, max_norm: float, stream=None):
        """(total, norms): total[0] the norm over all gradients, total[1] the factor
        min(1, max_norm / (norm + 1e-6)), norms[i] the norm of gradient i."""
        _need_grads(self.grads)
        with B.device_and_stream(self.device, stream):
            rc = B.load_library().grad_norm(self._plan, max_norm, self.total.data_ptr(), self.norms.data_ptr() or None,
                                            B.raw_stream(stream, self.device))
        B._check(rc, "grad_norm")
        return self.total, self.norms

    def scale_(self, factor=None, stream=None):
        """The gradients times `factor` in place (one-element float32 device tensor; by
        default the last measure()'s clip factor; not an element of the gradients). Nothing is
        read or written where it is 1."""
        _need_grads(self.grads)
        i = _moved(self.grads, self._ptrs)
        if i is not None:
            raise ValueError(f"grads[{i}] has other memory than when it was given")
        if self._written is None:
            self._written = _Spans(self._ptrs, [n * g.element_size() for n, g in zip(self._numels, self.grads)])
        ptr = _scalar_ptr(self.factor if factor is None else factor, "factor", self.device, self._written)
        with B.device_and_stream(self.device, stream):
            rc = B.load_library().grad_scale(self._plan, ptr, B.raw_stream(stream, self.device))
        B._check(rc, "grad_scale")
