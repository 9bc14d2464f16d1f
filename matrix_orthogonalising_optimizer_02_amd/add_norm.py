"""The residual's addition with the RMS norm that follows it, over torch tensors.

The step between two layers of a pre-norm block: `add_rms_norm_forward` adds a layer's
output to the residual stream and normalises the sum in one pass, with the norm's output in
x's type, in 8 bits for `matmul8`, or both; `add_rms_norm_backward` is its gradient, and
`add_rms_norm` the two for torch.autograd.
"""
from __future__ import annotations

import ctypes
import struct

from . import binding as B
from .blocks8 import _new, _rows_of
from .norms import _check_like, _like

_pack_desc = struct.Struct("@2q3i2fi").pack  # the C struct add_norm_desc
_pack_rows = struct.Struct("@P2q").pack
_pack_param = struct.Struct("@Pq").pack
_calls = None


def _entry_points():
    """add_rms_norm_forward, add_rms_norm_backward and the workspace query with plain pointer
    arguments."""
    global _calls
    if _calls is None:
        lib = B.load_library()
        vp = ctypes.c_void_p
        forward, backward = lib["add_rms_norm_forward"], lib["add_rms_norm_backward"]
        size = lib["add_rms_norm_backward_workspace_bytes"]
        forward.argtypes = [vp] * 9
        backward.argtypes = [vp] * 10 + [ctypes.c_size_t, vp]
        size.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
        _calls = forward, backward, size
    return _calls


def _strided(t, name):
    """(rows, cols, packed norm_rows) of a tensor as a matrix of its last dimension."""
    rows, cols, stride = _rows_of(t, name)
    return rows, cols, _pack_rows(t.data_ptr(), stride, 0)


def _check_beside(t, name, x, dtypes):
    """t has x's shape and device and one of dtypes."""
    torch = B._torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != x.shape:
        raise ValueError(f"{name} must have shape {tuple(x.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(str(d) for d in dict.fromkeys(dtypes))}")
    if t.device != x.device:
        raise ValueError(f"{name} must live on {x.device}")


def _weight(weight, x, cols):
    """(packed norm_param, dtype) of a weight of one row."""
    torch = B._torch()
    if weight is None:
        return None, torch.float32
    if not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor")
    if weight.dtype not in (torch.float32, x.dtype):
        raise ValueError(f"weight must have dtype torch.float32 or {x.dtype}")
    if weight.numel() != cols or weight.dim() < 1 or weight.shape[-1] != cols:
        raise ValueError(f"weight must have {cols} elements in its last dimension and no other rows")
    if weight.device != x.device:
        raise ValueError(f"weight must live on {x.device}")
    if cols > 1 and weight.stride(-1) != 1:
        raise ValueError("weight must have adjacent elements")
    return _pack_param(weight.data_ptr(), cols), weight.dtype


def add_rms_norm_forward(x, residual=None, weight=None, *, eps: float = 1e-6, weight_offset: float = 0.0, y: bool = True,
                         codes: bool = False, stats: bool = True, residual_out=None, stream=None):
    """(h, y, y8, rstd) of h = x + residual and y = h / sqrt(mean(h^2) + eps) (weight_offset +
    weight) over the last dimension.

    h is rounded to the residual's dtype, float32 or x's, and y is the norm of what h then
    holds; without a residual h is x (None is returned). y: the norm's output in x's dtype;
    codes: as a Blocks8 [rows, cols] for matmul8; both come from the same fp32 values, and
    each is None where not wanted. weight: float32 or x's dtype, [cols]. rstd: float32 [rows]
    for add_rms_norm_backward, None with stats=False. residual_out receives h, and may be
    residual (or x).
    """
    rows, cols, px = _strided(x, "x")
    torch = B._torch()
    device = x.device
    rdtype = x.dtype
    if residual is not None:
        _check_beside(residual, "residual", x, (torch.float32, x.dtype))
        rdtype = residual.dtype
        if residual_out is not None:
            _check_beside(residual_out, "residual_out", x, (rdtype,))
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    w, wdtype = _weight(weight, x, cols)
    kinds = B.dtype_codes()
    with B.device_and_stream(device, stream):
        h = pr = ph = out = py = y8 = p8 = rstd = None
        if residual is not None:
            pr = _strided(residual, "residual")[2]
            h = _like(residual) if residual_out is None else residual_out
            ph = _strided(h, "residual_out")[2]
        if y:
            out = _like(x)
            py = _pack_rows(out.data_ptr(), cols, 0)
        if codes:
            y8 = _new(x, rows, cols, False)
            p8 = y8._packed()
        if stats:
            rstd = x.new_empty(rows, dtype=torch.float32)
        rc = _entry_points()[0](_pack_desc(rows, cols, kinds[x.dtype], kinds[rdtype], kinds[wdtype], eps, weight_offset, 0), px,
                                pr, w, ph, py, p8, rstd.data_ptr() if stats else None, B.raw_stream(stream, device))
    if rc:
        B._check(rc, "add_rms_norm_forward")
    return h, out, y8, rstd


def add_rms_norm_backward_workspace_bytes(rows: int, cols: int, dtype=None) -> int:
    """Bytes of add_rms_norm_backward's workspace for [rows, cols] of dtype (default bfloat16)."""
    kind = B.dtype_codes()[dtype or B._torch().bfloat16]
    return _workspace_bytes(_pack_desc(rows, cols, kind, kind, 0, 1.0, 0.0, 0))


def _workspace_bytes(desc):
    out = ctypes.c_size_t(0)
    B._check(_entry_points()[2](desc, out), "add_rms_norm_backward_workspace_bytes")
    return out.value


def add_rms_norm_backward(dy, dh, h, weight, rstd, *, weight_offset: float = 0.0, weight_grad: bool = True, out=None,
                          workspace=None, stream=None):
    """(dx, dresidual, dweight) from the gradient dy of the norm's output and dh of h itself
    (None: 0), with the forward pass's h (x, without a residual) and rstd.

    The gradient of x and that of the residual are the same numbers: dresidual in h's dtype
    (dh's too), dx in dy's; one tensor where the two are the same. An output in 8 bits has the
    gradient of the one that was rounded. dweight has weight's shape and dtype, None when not
    asked for. out: receives dresidual, and may be dh, h, or dy of its dtype. workspace:
    optional uint8 buffer of add_rms_norm_backward_workspace_bytes().
    """
    rows, cols, pdy = _strided(dy, "dy")
    torch = B._torch()
    device = dy.device
    _check_beside(h, "h", dy, (torch.float32, dy.dtype))
    ph = _strided(h, "h")[2]
    pdh = None
    if dh is not None:
        _check_beside(dh, "dh", dy, (h.dtype,))
        pdh = _strided(dh, "dh")[2]
    w, wdtype = _weight(weight, dy, cols)
    if not isinstance(rstd, torch.Tensor) or rstd.dtype != torch.float32 or rstd.numel() != rows or not rstd.is_contiguous() \
            or rstd.device != device:
        raise ValueError(f"rstd must be a contiguous float32 tensor on {device} with one entry per row")
    if out is not None:
        _check_like(out, "out", h)
    kinds = B.dtype_codes()
    with B.device_and_stream(device, stream):
        dr = _like(h) if out is None else out
        pdr = _strided(dr, "out")[2]
        dx, pdx = dr, None
        if h.dtype != dy.dtype:
            dx = _like(dy)
            pdx = _pack_rows(dx.data_ptr(), cols, 0)
        desc = _pack_desc(rows, cols, kinds[dy.dtype], kinds[h.dtype], kinds[wdtype], 1.0, weight_offset, 0)
        dweight = pdw = None
        if weight_grad and weight is not None:
            dweight = weight.new_empty(weight.shape)
            pdw = _pack_param(dweight.data_ptr(), cols)
        ws, wsb = None, 0
        if workspace is not None:
            if workspace.device != device or not workspace.is_contiguous() or workspace.dtype != torch.uint8:
                raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
            ws, wsb = workspace.data_ptr(), workspace.numel()
        elif pdw is not None:
            wsb = _workspace_bytes(desc)
            if wsb:
                workspace = dy.new_empty(wsb, dtype=torch.uint8)
                ws = workspace.data_ptr()
        rc = _entry_points()[1](desc, pdy, pdh, ph, w, rstd.data_ptr(), pdr, pdx, pdw, ws, wsb, B.raw_stream(stream, device))
    if rc:
        B._check(rc, "add_rms_norm_backward")
    return dx, dr, dweight


_function = None


def _autograd_function():
    """The autograd function, made at its first use: torch is imported lazily."""
    global _function
    if _function is not None:
        return _function
    torch = B._torch()

    class AddRmsNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight, eps, weight_offset):
            h, y, _, rstd = add_rms_norm_forward(x, residual, weight, eps=eps, weight_offset=weight_offset)
            ctx.save_for_backward(x if h is None else h, weight, rstd)
            ctx.weight_offset, ctx.x_dtype = weight_offset, x.dtype
            ctx.set_materialize_grads(False)
            return (y, h) if h is not None else (y, None)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy, dh):
            h, weight, rstd = ctx.saved_tensors
            needs = ctx.needs_input_grad
            if dy is None:  # the norm's output was not used
                if dh is None:
                    return None, None, None, None, None
                return (dh.to(ctx.x_dtype) if needs[0] else None, dh if needs[1] else None, None, None, None)
            dy, dh = _rows_or_copy(dy), None if dh is None else _rows_or_copy(dh)
            dx, dr, dw = add_rms_norm_backward(dy, dh, h, weight, rstd, weight_offset=ctx.weight_offset, weight_grad=needs[2])
            return dx if needs[0] else None, dr if needs[1] else None, dw, None, None

    _function = AddRmsNorm
    return AddRmsNorm


def _rows_or_copy(t):
    """t, or its copy where its rows are at no one stride (an expanded or transposed gradient)."""
    try:
        _rows_of(t, "gradient")
    except ValueError:
        return t.contiguous()
    return t


def add_rms_norm(x, residual=None, weight=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """(y, h) of add_rms_norm_forward for torch.autograd: the norm's output, and the residual
    stream for the next addition (None without a residual). To capture a backward pass into a HIP
    graph, call add_rms_norm_forward and add_rms_norm_backward themselves: while an eager graph of
    the same leaves lives, torch ends a process that captures autograd's backward pass."""
    return _autograd_function().apply(x, residual, weight, eps, weight_offset)
