"""Normalisation layers with their gradients, over torch tensors.

The layers beside the block matrices of a transformer: the affine layer norm and the
query and key RMS norms, whose weights the hybrid optimizer keeps on AdamW, and the
modulated norm (adaLN) that takes a scale and a shift per sample from a [6H, H]
projection. `norm_forward` and `norm_backward` are the library's two calls; `layer_norm`
and `rms_norm` are the same for torch.autograd.
"""
from __future__ import annotations

import ctypes
import struct

from . import binding as B

NORM_LAYER, NORM_RMS = 0, 1
MAX_COLS = 16384
_KINDS = {"layer": NORM_LAYER, "rms": NORM_RMS}

# The C structs norm_desc, norm_rows and norm_param as bytes: a small call's time is the
# host's, and packing takes a fifth of building a ctypes.Structure.
_pack_desc = struct.Struct("@4q3i2f4x").pack
_pack_rows = struct.Struct("@P2q").pack
_pack_param = struct.Struct("@Pq").pack
_calls = None


def _entry_points():
    """norm_forward, norm_backward and the workspace query with plain pointer arguments."""
    global _calls
    if _calls is None:
        lib = B.load_library()
        vp = ctypes.c_void_p
        forward, backward, size = lib["norm_forward"], lib["norm_backward"], lib["norm_backward_workspace_bytes"]
        forward.argtypes = [vp] * 8
        backward.argtypes = [vp] * 10 + [ctypes.c_size_t, vp]
        size.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t)]
        _calls = forward, backward, size
    return _calls


def _row_levels(t, name):
    """The leading dimensions of t as at most two (size, stride) levels, innermost first."""
    shape = t.shape
    cols = shape[-1]
    if t.is_contiguous():
        n = t.numel() // cols if cols else 0
        return [(n, cols)] if n > 1 else []
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent elements in its last dimension")
    levels = []
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if levels and stride == levels[-1][0] * levels[-1][1]:
            levels[-1] = (levels[-1][0] * size, levels[-1][1])
        else:
            levels.append((size, stride))
    if len(levels) > 2:
        raise ValueError(f"{name} has rows at more than two strides; make it contiguous")
    return levels


def _layout(tensors):
    """(inner, packed norm_rows) for [(tensor, name)] of one shape."""
    for t, _ in tensors:
        if not t.is_contiguous():
            break
    else:
        cols = tensors[0][0].shape[-1]
        return 1, [_pack_rows(t.data_ptr(), cols, 0) for t, _ in tensors]
    levels = [_row_levels(t, name) for t, name in tensors]
    inner = 1
    for lv, (_, name) in zip(levels, tensors):
        if len(lv) == 2:
            if inner not in (1, lv[0][0]):
                raise ValueError(f"{name} splits its rows unlike another tensor of the call; make it contiguous")
            inner = lv[0][0]
    rows = []
    for lv, (t, _) in zip(levels, tensors):
        if len(lv) == 2:
            s0, s1 = lv[1][1], lv[0][1]
        else:
            s1 = lv[0][1] if lv else 0
            s0 = s1 * inner
        rows.append(_pack_rows(t.data_ptr(), s0, s1))
    return inner, rows


def _check_x(x):
    torch = B._torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError("x must live on a GPU")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    if x.dtype not in B.dtype_codes():
        raise ValueError("x must be float32, bfloat16 or float16")


def _check_like(t, name, x):
    """t has x's shape, type and device."""
    if not isinstance(t, B._torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != x.dtype:
        raise ValueError(f"{name} must have dtype {x.dtype}")
    if t.shape != x.shape:
        raise ValueError(f"{name} must have shape {tuple(x.shape)}")
    if t.device != x.device:
        raise ValueError(f"{name} must live on {x.device}")


def _param(t, name, cols, groups, x, dtypes):
    """(groups, packed norm_param) of a weight or bias whose last dimension is the row's."""
    if not isinstance(t, B._torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must have dtype {' or '.join(str(d) for d in dict.fromkeys(dtypes))}")
    if t.device != x.device:
        raise ValueError(f"{name} must live on {x.device}")
    if t.dim() < 1 or t.shape[-1] != cols:
        raise ValueError(f"{name} must have {cols} elements in its last dimension")
    n = t.numel() // cols if cols else 1
    if groups is not None and n != groups:
        raise ValueError(f"{name} must have {groups} rows, as the weight")
    if n > 1 and x.dim() > 2:
        _check_leading(t, n, name, x)
    stride = cols
    if not t.is_contiguous():
        levels = _row_levels(t, name)
        if len(levels) > 1:
            raise ValueError(f"{name} has rows at more than one stride; make it contiguous")
        stride = levels[0][1] if levels else cols
    return n, _pack_param(t.data_ptr(), stride)


def _check_leading(t, n, name, x):
    """t's n rows belong to x's leading dimensions, one or several of them in order."""
    lead = list(t.shape[:-1])
    while lead[-1] == 1:
        lead.pop()
    products = [1]
    for size in x.shape[:-1]:
        products.append(products[-1] * size)
    if n not in products or (len(lead) > 1 and lead != list(x.shape[:len(lead)])):
        raise ValueError(f"{name} of shape {tuple(t.shape)} has no row for each of the leading dimensions of x, {tuple(x.shape)}")


def _desc(x, rows, cols, weight, bias, kind, eps, weight_offset, inner):
    """(packed norm_desc, weight's, bias's packed norm_param) of a call on x."""
    if kind not in _KINDS:
        raise ValueError("kind must be 'layer' or 'rms'")
    codes = B.dtype_codes()
    float32 = B._torch().float32
    groups, w, b, wdtype = None, None, None, float32
    if weight is not None:
        groups, w = _param(weight, "weight", cols, None, x, (float32, x.dtype))
        wdtype = weight.dtype
    if bias is not None:
        groups, b = _param(bias, "bias", cols, groups, x, (float32, x.dtype) if weight is None else (wdtype,))
        wdtype = bias.dtype
    return _pack_desc(rows, cols, 1 if groups is None else groups, inner, _KINDS[kind], codes[x.dtype], codes[wdtype],
                      eps, weight_offset), w, b


def _like(x):
    """A new tensor of x's shape and type, rows adjacent."""
    return B._torch().empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def norm_forward(x, weight=None, bias=None, *, kind: str = "layer", eps: float = 1e-6,
                 weight_offset: float = 0.0, out=None, stats: bool = True, stream=None):
    """(y, mean, rstd) of y = (x - mean) rstd (weight_offset + weight) + bias over x's last dimension.

    kind "rms" takes no mean away (mean is None). weight and bias: float32 or x's dtype,
    [cols] for all rows, or one row for each of `groups` equal runs of x's rows (adaLN's
    scale and shift of each sample, e.g. [samples, cols], with weight_offset 1); where x has
    more than two dimensions, a run is what one or several leading ones number. x's rows
    may be strided (a slice of a fused projection). mean and rstd: float32 [rows], for
    norm_backward; neither is computed into memory with stats=False (both None then). out:
    receives y, and may be x.
    """
    _check_x(x)
    device = x.device
    if stream is not None or B._torch().cuda.current_device() != device.index:
        with B.device_and_stream(device, stream):
            return _forward(x, weight, bias, kind, eps, weight_offset, out, stats, B.raw_stream(stream, device))
    return _forward(x, weight, bias, kind, eps, weight_offset, out, stats, B.raw_stream(None, device))


def _forward(x, weight, bias, kind, eps, weight_offset, out, stats, stream):
    float32 = B._torch().float32
    if out is None:
        y = _like(x)
    else:
        _check_like(out, "out", x)
        y = out
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    inner, (rx, ry) = _layout(((x, "x"), (y, "out")))
    d, w, b = _desc(x, rows, cols, weight, bias, kind, eps, weight_offset, inner)
    mean = rstd = pm = pr = None
    if stats:
        rstd = x.new_empty(rows, dtype=float32)
        pr = rstd.data_ptr()
        if kind == "layer":
            mean = x.new_empty(rows, dtype=float32)
            pm = mean.data_ptr()
    rc = _entry_points()[0](d, rx, w, b, ry, pm, pr, stream)
    if rc:
        B._check(rc, "norm_forward")
    return y, mean, rstd


def _workspace_bytes(desc):
    out = ctypes.c_size_t(0)
    B._check(_entry_points()[2](desc, out), "norm_backward_workspace_bytes")
    return out.value


def norm_backward_workspace_bytes(rows: int, cols: int, groups: int = 1, kind: str = "layer", dtype=None,
                                  weight_dtype=None) -> int:
    """Bytes of norm_backward's workspace for [rows, cols] of dtype (default bfloat16) in
    `groups` groups, weights of weight_dtype (default float32)."""
    torch, codes = B._torch(), B.dtype_codes()
    if kind not in _KINDS:
        raise ValueError("kind must be 'layer' or 'rms'")
    return _workspace_bytes(_pack_desc(rows, cols, groups, 1, _KINDS[kind], codes[dtype or torch.bfloat16],
                                       codes[weight_dtype or torch.float32], 1.0, 0.0))


def norm_backward(dy, x, weight, mean, rstd, *, kind: str = "layer", weight_offset: float = 0.0,
                  weight_grad: bool = True, bias_grad: bool = True, out=None, workspace=None, stream=None,
                  grad_shape=None, grad_dtype=None):
    """(dx, dweight, dbias) from dy and the forward pass's x, mean and rstd.

    dweight and dbias have weight's shape and dtype; each is None when not asked for (and
    dweight without a weight). A norm with a bias and no weight names its bias's shape and
    dtype as grad_shape and grad_dtype. out: receives dx, and may be dy or x. workspace:
    optional uint8 device buffer of norm_backward_workspace_bytes().
    """
    _check_x(x)
    _check_like(dy, "dy", x)
    device = x.device
    args = (dy, x, weight, mean, rstd, kind, weight_offset, weight_grad, bias_grad, out, workspace)
    if stream is not None or B._torch().cuda.current_device() != device.index:
        with B.device_and_stream(device, stream):
            return _backward(*args, B.raw_stream(stream, device), grad_shape, grad_dtype)
    return _backward(*args, B.raw_stream(None, device), grad_shape, grad_dtype)


def _backward(dy, x, weight, mean, rstd, kind, weight_offset, weight_grad, bias_grad, out, workspace, stream, grad_shape,
              grad_dtype):
    torch = B._torch()
    device = x.device
    if out is None:
        dx = _like(x)
    else:
        _check_like(out, "out", x)
        dx = out
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    inner, (rdy, rx, rdx) = _layout(((dy, "dy"), (x, "x"), (dx, "out")))
    dbias = None
    if bias_grad:
        if weight is not None:
            dbias = _like(weight)
        else:
            dbias = x.new_empty(x.shape[-1:] if grad_shape is None else tuple(grad_shape),
                                dtype=grad_dtype or torch.float32)
    d, w, db = _desc(x, rows, cols, weight, dbias, kind, 1.0, weight_offset, inner)
    dweight = dw = None
    if weight_grad and weight is not None:
        dweight = _like(weight)
        dw = _pack_param(dweight.data_ptr(), cols)
    stats = []
    for t, nm in ((mean, "mean"), (rstd, "rstd")):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.numel() != rows
                              or not t.is_contiguous() or t.device != device):
            raise ValueError(f"{nm} must be a contiguous float32 tensor on {device} with one entry per row")
        stats.append(t.data_ptr() if t is not None else None)
    ws, wsb = None, 0
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous() or workspace.dtype != torch.uint8:
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
        ws, wsb = workspace.data_ptr(), workspace.numel()
    elif dw is not None or db is not None:
        wsb = _workspace_bytes(d)
        if wsb:
            workspace = x.new_empty(wsb, dtype=torch.uint8)
            ws = workspace.data_ptr()
    rc = _entry_points()[1](d, rdy, rx, w, stats[0], stats[1], rdx, dw, db, ws, wsb, stream)
    if rc:
        B._check(rc, "norm_backward")
    return dx, dweight, dbias


_function = None


def _autograd_function():
    """The autograd function, made at its first use: torch is imported lazily."""
    global _function
    if _function is not None:
        return _function
    torch = B._torch()

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, kind, eps, weight_offset):
            y, mean, rstd = norm_forward(x, weight, bias, kind=kind, eps=eps, weight_offset=weight_offset)
            ctx.save_for_backward(x, weight, mean, rstd)
            ctx.kind, ctx.weight_offset = kind, weight_offset
            ctx.bias = None if bias is None else (bias.shape, bias.dtype)
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, weight, mean, rstd = ctx.saved_tensors
            bias_grad = ctx.bias is not None and ctx.needs_input_grad[2]
            shape, dtype = ctx.bias or (None, None)
            try:
                _layout(((dy, "dy"), (x, "x")))
            except ValueError:  # an expanded or transposed gradient
                dy = dy.contiguous()
            dx, dw, db = norm_backward(dy, x, weight, mean, rstd, kind=ctx.kind, weight_offset=ctx.weight_offset,
                                       weight_grad=ctx.needs_input_grad[1], bias_grad=bias_grad,
                                       grad_shape=shape, grad_dtype=dtype)
            return dx if ctx.needs_input_grad[0] else None, dw, None if db is None else db.view(shape), None, None, None

    _function = Norm
    return Norm


def layer_norm(x, weight=None, bias=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """norm_forward's y for torch.autograd: affine with weight and bias of [cols], adaLN
    with one row a sample and weight_offset 1, plain without either. To capture a backward
    pass into a HIP graph, call norm_forward and norm_backward themselves: while an eager
    graph of the same leaves lives, a capture of autograd's backward pass waits for that
    graph's stream, which a capture does not allow, and torch ends the process."""
    return _autograd_function().apply(x, weight, bias, "layer", eps, weight_offset)


def rms_norm(x, weight=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """x / sqrt(mean(x^2) + eps) (weight_offset + weight) for torch.autograd."""
    return _autograd_function().apply(x, weight, None, "rms", eps, weight_offset)
