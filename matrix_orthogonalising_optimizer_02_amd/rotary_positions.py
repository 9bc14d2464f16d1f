"""Rotary positions over several axes, over torch tensors.

For the query and key heads after their RMS norms: `RotaryAxes` says which pairs of a head's
elements go by which axis (time, height and width of an image or video token, or one axis
for text) and how fast they turn, `rotary_apply` turns them by their tokens' positions, and
`rotary` is the same for torch.autograd.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import binding as B

LAYOUTS = {"halves": 0, "adjacent": 1}

_pack_desc = struct.Struct("@4q6i").pack       # the C struct rotary_desc
_pack_rows = struct.Struct("@P3q").pack        # rotary_rows
_pack_positions = struct.Struct("@P2q").pack   # rotary_positions
_call = None
_position_types = None


def _entry_point():
    global _call
    if _call is None:
        _call = B.load_library()["rotary_apply"]
        _call.argtypes = [ctypes.c_void_p] * 7
    return _call


def _position_type(t):
    global _position_types
    if _position_types is None:
        torch = B._torch()
        _position_types = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
    return _position_types.get(t.dtype)


class RotaryAxes:
    """How the pairs of a head's elements turn; made once and kept.

    sections: pairs of each axis, in order; their sum is at most half of a head's elements,
    and elements past twice that are left as they are. base: one number, or one for each
    axis: pair i of an axis with n pairs turns by base^(-i / n) radians per unit of position.
    layout: "halves" pairs element i with i + pairs, "adjacent" 2 i with 2 i + 1.
    frequencies, axis_of_pair: radians per unit and axis of each pair in place of that rule,
    for models that deal the axes out otherwise (axis_of_pair without regard to sections'
    order; its axes still number len(sections)).
    """

    def __init__(self, sections, base=10000.0, layout: str = "halves", device="cuda", frequencies=None, axis_of_pair=None):
        torch = B._torch()
        self.sections = tuple(int(s) for s in sections)
        if not self.sections or min(self.sections) < 0 or sum(self.sections) < 1:
            raise ValueError("sections must name the pairs of each axis, one pair at least in all")
        if layout not in LAYOUTS:
            raise ValueError("layout must be 'halves' or 'adjacent'")
        self.layout, self.axes, self.pairs = layout, len(self.sections), sum(self.sections)
        if frequencies is None:
            bases = [float(base)] * self.axes if not hasattr(base, "__len__") else [float(b) for b in base]
            if len(bases) != self.axes or not all(b > 0 and math.isfinite(b) for b in bases):
                raise ValueError("base must be a finite number above 0, or one for each axis")
            frequencies = [b ** (-i / n) for b, n in zip(bases, self.sections) for i in range(n)]
        self.frequencies = tuple(float(f) for f in frequencies)
        if axis_of_pair is None:
            axis_of_pair = [a for a, n in enumerate(self.sections) for _ in range(n)]
        self.axis_of_pair = tuple(int(a) for a in axis_of_pair)
        if len(self.frequencies) != self.pairs or not all(math.isfinite(f) for f in self.frequencies):
            raise ValueError(f"frequencies must be {self.pairs} finite numbers")
        if len(self.axis_of_pair) != self.pairs or not all(0 <= a < self.axes for a in self.axis_of_pair):
            raise ValueError(f"axis_of_pair must name one of {self.axes} axes for each of {self.pairs} pairs")
        self._freq = torch.tensor([f / (2.0 * math.pi) for f in self.frequencies], dtype=torch.float64, device=device)
        self._axis = torch.tensor(self.axis_of_pair, dtype=torch.int32, device=device)
        self.device = self._freq.device


def _levels(lead, strides):
    """Leading dimensions as at most two (size, strides) levels, outer first: neighbours that
    are one run in every tensor become one."""
    levels = []
    for i, size in enumerate(lead):
        if size == 1:
            continue
        here = [s[i] for s in strides]
        if levels and all(o == size * h for o, h in zip(levels[-1][1], here)):
            levels[-1] = (levels[-1][0] * size, here)
        else:
            levels.append((size, here))
    if len(levels) > 2:
        raise ValueError("x, out and positions have tokens at more than two strides; make them contiguous")
    return [(1, [0] * len(strides))] * (2 - len(levels)) + levels


def rotary_apply(x, positions, axes: RotaryAxes, *, inverse: bool = False, out=None, stream=None):
    """x [..., tokens, heads, dim] with each head's pairs turned by its token's position
    (inverse: turned back, the gradient of the former).

    positions: int32, int64 or float32 [..., tokens, axes]; leading dimensions of size 1, or
    left out, are the same for all of x's. x may be strided (the query and key heads of a
    fused projection, or [batch, heads, tokens, dim] transposed), its last dimension adjacent.
    float32, bfloat16 or float16; angles in fp64, the rest in fp32, rounded once. out: receives
    the result, and may be x.
    """
    torch = B._torch()
    if not isinstance(x, torch.Tensor) or not isinstance(positions, torch.Tensor):
        raise TypeError("x and positions must be torch.Tensors")
    if not isinstance(axes, RotaryAxes):
        raise TypeError("axes must be a RotaryAxes")
    if not x.is_cuda:
        raise ValueError("x must live on a GPU")
    code, kind = B.dtype_codes().get(x.dtype), _position_type(positions)
    if code is None:
        raise ValueError("x must be float32, bfloat16 or float16")
    if kind is None:
        raise ValueError("positions must be int32, int64 or float32")
    device = x.device
    if positions.device != device or axes.device != device:
        raise ValueError(f"positions and axes must live on {device}")
    if x.dim() < 2:
        raise ValueError("x must have heads and their elements as its last two dimensions")
    lead, (heads, dim) = x.shape[:-2], x.shape[-2:]
    if positions.dim() < 1 or positions.shape[-1] != axes.axes:
        raise ValueError(f"positions must have {axes.axes} axes in its last dimension")
    if 2 * axes.pairs > dim:
        raise ValueError(f"axes turn {2 * axes.pairs} elements of a head, which has {dim}")
    if out is not None and (not isinstance(out, torch.Tensor) or out.shape != x.shape or out.dtype != x.dtype
                            or out.device != device):
        raise ValueError(f"out must have shape {tuple(x.shape)} and dtype {x.dtype} and live on {device}")
    for t, name in ((x, "x"), (out, "out")):
        if t is not None and dim > 1 and t.stride(-1) != 1 and t.numel():
            raise ValueError(f"{name} must have adjacent elements in its last dimension")
    if axes.axes > 1 and positions.stride(-1) != 1 and positions.numel():
        raise ValueError("positions must have adjacent elements in its last dimension")
    try:
        spread = positions.expand(*lead, axes.axes)
    except RuntimeError:
        raise ValueError(f"positions of shape {tuple(positions.shape)} does not fit tokens {tuple(lead)}") from None
    with B.device_and_stream(device, stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=device) if out is None else out
        if x.numel() == 0:
            return y
        (batch, sb), (tokens, st) = _levels(lead, (x.stride(), y.stride(), spread.stride()))
        rc = _entry_point()(_pack_desc(batch, tokens, heads, dim, axes.pairs, axes.axes, code, LAYOUTS[axes.layout], kind,
                                       bool(inverse)),
                            _pack_rows(x.data_ptr(), sb[0], st[0], x.stride(-2)),
                            _pack_positions(positions.data_ptr(), sb[2], st[2]), axes._freq.data_ptr(), axes._axis.data_ptr(),
                            _pack_rows(y.data_ptr(), sb[1], st[1], y.stride(-2)), B.raw_stream(stream, device))
    if rc:
        B._check(rc, "rotary_apply")
    return y


_function = None


def _autograd_function():
    """The autograd function, made at its first use: torch is imported lazily."""
    global _function
    if _function is not None:
        return _function
    torch = B._torch()

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, positions, axes):
            y = rotary_apply(x, positions, axes)  # checks its arguments
            ctx.save_for_backward(positions)
            ctx.axes = axes
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            positions, = ctx.saved_tensors
            try:
                return rotary_apply(dy, positions, ctx.axes, inverse=True), None, None
            except ValueError:  # an expanded or transposed gradient
                return rotary_apply(dy.contiguous(), positions, ctx.axes, inverse=True), None, None

    _function = Rotary
    return Rotary


def rotary(x, positions, axes: RotaryAxes):
    """rotary_apply for torch.autograd; positions have no gradient. To capture a backward pass into
    a HIP graph, call rotary_apply itself, inverse for the gradient: while an eager graph of the
    same leaves lives, torch ends a process that captures autograd's backward pass."""
    if getattr(positions, "requires_grad", False):
        raise ValueError("positions have no gradient")
    return _autograd_function().apply(x, positions, axes)
