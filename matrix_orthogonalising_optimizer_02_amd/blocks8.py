"""Matrices in 8 bits with a power of two for every 128 elements, and their products.

The 8-bit path of the linear layers whose weights Muon steps: `quantise8` turns
activations, gradients and fp32 weights into e4m3 codes, `matmul8` multiplies them on the
scaled matrix instructions, and `linear8` is the layer with both gradients for
torch.autograd. The norm before a projection can write its output in this form itself
(`add_rms_norm_forward`).
"""
from __future__ import annotations

import ctypes
import struct

from . import binding as B

BLOCK = 128
_pack = struct.Struct("@2q2P2q2i").pack  # the C struct blocks8
_calls = None


def _entry_points():
    """quantise8, dequantise8, matmul8 and the workspace query with plain pointer arguments."""
    global _calls
    if _calls is None:
        lib = B.load_library()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        quantise, dequantise, product = lib["quantise8"], lib["dequantise8"], lib["matmul8"]
        size = lib["matmul8_workspace_bytes"]
        quantise.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp]
        dequantise.argtypes = [vp, vp, i64, i32, vp]
        product.argtypes = [vp, vp, vp, i64, i32, i32, i32, vp, ctypes.c_size_t, vp]
        size.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(ctypes.c_size_t)]
        _calls = quantise, dequantise, product, size
    return _calls


def _up(n, to):
    return -(-n // to) * to


class Blocks8:
    """A matrix [rows, cols] as codes and powers of two.

    codes: float8_e4m3fn [rows, at least cols rounded up to 128], zeros from cols to there.
    scales: uint8 [rows, at least cols / 128 rounded up, to a multiple of 4], the power of
    each 1 x 128 elements as its exponent + 127; with `tiles` a row for each 128 rows, the
    power of 128 x 128 elements. A value is code * 2^(scale - 127), NaN for a scale of 255. Rows
    may lie further apart than they are long.
    """

    __slots__ = ("codes", "scales", "rows", "cols", "tiles")

    def __init__(self, codes, scales, cols: int, tiles: bool = False):
        torch = B._torch()
        for t, name, dtype in ((codes, "codes", torch.float8_e4m3fn), (scales, "scales", torch.uint8)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype != dtype or t.dim() != 2:
                raise ValueError(f"{name} must be a 2-D {dtype} tensor")
            if not t.is_cuda:
                raise ValueError(f"{name} must live on a GPU")
            if t.shape[1] > 1 and t.stride(1) != 1:
                raise ValueError(f"{name} must have adjacent elements in its last dimension")
        if scales.device != codes.device:
            raise ValueError(f"scales must live on {codes.device}")
        self.codes, self.scales = codes, scales
        self.rows, self.cols, self.tiles = int(codes.shape[0]), int(cols), bool(tiles)
        blocks, high = -(-self.cols // BLOCK), -(-self.rows // BLOCK) if tiles else self.rows
        if self.cols < 0 or codes.shape[1] < blocks * BLOCK:
            raise ValueError(f"codes must have {blocks * BLOCK} columns for a matrix of {cols}")
        if scales.shape[0] != high or scales.shape[1] < _up(blocks, 4):
            raise ValueError(f"scales must have shape [{high}, {_up(blocks, 4)}] for a matrix [{self.rows}, {cols}]")

    @property
    def shape(self):
        return self.rows, self.cols

    @property
    def device(self):
        return self.codes.device

    def _packed(self):
        c, s = self.codes, self.scales
        # the stride of a single row is of no account
        ld = c.stride(0) if self.rows > 1 else _up(self.cols, BLOCK)
        scale_ld = s.stride(0) if s.shape[0] > 1 else _up(-(-self.cols // BLOCK), 4)
        return _pack(self.rows, self.cols, c.data_ptr(), s.data_ptr(), ld, scale_ld, self.tiles, 0)

    def dequantise(self, dtype=None, out=None, stream=None):
        """The values [rows, cols] in dtype (default float32; exact there, and in bfloat16 but
        for what has bits below 2^-133)."""
        torch = B._torch()
        device = self.device
        with B.device_and_stream(device, stream):
            if out is None:
                out = torch.empty((self.rows, self.cols), dtype=dtype or torch.float32, device=device)
            else:
                _check_out(out, (self.rows, self.cols), dtype, device)
            if out.dtype not in B.dtype_codes():
                raise ValueError("dtype must be float32, bfloat16 or float16")
            rc = _entry_points()[1](self._packed(), out.data_ptr(), out.stride(0), B.dtype_codes()[out.dtype],
                                    B.raw_stream(stream, device))
        if rc:
            B._check(rc, "dequantise8")
        return out


def _check_out(out, shape, dtype, device):
    torch = B._torch()
    if not isinstance(out, torch.Tensor):
        raise TypeError("out must be a torch.Tensor")
    if tuple(out.shape) != tuple(shape) or out.device != device:
        raise ValueError(f"out must have shape {tuple(shape)} and live on {device}")
    if dtype is not None and out.dtype != dtype:
        raise ValueError(f"out must have dtype {dtype}")
    if out.shape[-1] > 1 and out.stride(-1) != 1:
        raise ValueError("out must have adjacent elements in its last dimension")


def _new(like, rows, cols, tiles):
    """Memory for a matrix [rows, cols] in 8 bits, beside the tensor `like`."""
    torch = B._torch()
    blocks = -(-cols // BLOCK)
    return _made(like.new_empty((rows, blocks * BLOCK), dtype=torch.float8_e4m3fn),
                 like.new_empty((-(-rows // BLOCK) if tiles else rows, _up(blocks, 4)), dtype=torch.uint8), rows, cols, tiles)


def _made(codes, scales, rows, cols, tiles):
    """The Blocks8 of memory that is known to fit it."""
    q = Blocks8.__new__(Blocks8)
    q.codes, q.scales, q.rows, q.cols, q.tiles = codes, scales, rows, cols, tiles
    return q


def _rows_of(x, name):
    """(rows, cols, stride) of a tensor as a matrix of its last dimension."""
    torch = B._torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must live on a GPU")
    if x.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    if x.dtype not in B.dtype_codes():
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    cols = x.shape[-1]
    rows = 1
    for size in x.shape[:-1]:
        rows *= size
    if x.is_contiguous() or rows == 0 or cols == 0:
        return rows, cols, cols
    if cols > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name} must have adjacent elements in its last dimension")
    stride = span = None
    for size, step in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride, span = step, size * step
        elif step != span:
            raise ValueError(f"{name} has rows at more than one stride; make it contiguous")
        else:
            span *= size
    return rows, cols, cols if stride is None else stride


def _given(q, name, rows, cols, tiles, device):
    if not isinstance(q, Blocks8):
        raise TypeError(f"{name} must be a Blocks8")
    if (q.rows, q.cols, q.tiles) != (rows, cols, tiles) or q.device != device:
        raise ValueError(f"{name} must be a Blocks8 of [{rows}, {cols}] with tiles={tiles} on {device}")


def quantise8(x, *, tiles: bool = False, direct: bool = True, transposed: bool = False, out=None, out_transposed=None,
              stream=None):
    """(q, qt): x [..., cols] as Blocks8 [rows, cols] and its transpose [cols, rows], each None
    where not asked for, from one read of x.

    Each block of 128 elements along a result's rows (tiles: of 128 x 128) gets the least power
    of two that brings its largest finite magnitude to 448 or less; codes are rounded to
    nearest. Infinities and NaN become NaN, each for itself. x: float32, bfloat16 or float16,
    its rows at one stride. out, out_transposed: Blocks8 that are written in place of new ones.
    """
    rows, cols, stride = _rows_of(x, "x")
    device = x.device
    tiles = bool(tiles)
    if out is not None:
        _given(out, "out", rows, cols, tiles, device)
    if out_transposed is not None:
        _given(out_transposed, "out_transposed", cols, rows, tiles, device)
    if not (direct or transposed or out is not None or out_transposed is not None):
        raise ValueError("neither direct nor transposed is asked for")
    with B.device_and_stream(device, stream):
        q, qt = out, out_transposed
        if q is None and direct:
            q = _new(x, rows, cols, tiles)
        if qt is None and transposed:
            qt = _new(x, cols, rows, tiles)
        rc = _entry_points()[0](x.data_ptr(), rows, cols, stride, B.dtype_codes()[x.dtype], q and q._packed(),
                                qt and qt._packed(), B.raw_stream(stream, device))
    if rc:
        B._check(rc, "quantise8")
    return q, qt


def _check_products(products):
    if products not in (None, 8, 16):
        raise ValueError("products must be None, 8 or 16")


def matmul8_workspace_bytes(m: int, n: int, k: int, dtype=None, products=None) -> int:
    """Bytes of matmul8's workspace for [m, k] times [n, k] into dtype (default bfloat16)."""
    size = ctypes.c_size_t(0)
    dtype = B.dtype_codes()[dtype or B._torch().bfloat16]
    B._check(_entry_points()[3](m, n, k, dtype, products or 0, size), "matmul8_workspace_bytes")
    return size.value


def matmul8_plan(m: int, n: int, k: int, dtype=None, products=None):
    """How matmul8 cuts [m, k] times [n, k] into dtype (default bfloat16), host only: a dict of
    `tile` (a block's side of the result, 0 up to 64 rows), `parts` of k, and up to 64 rows the
    `groups` of 16 rows of a, whether b goes through LDS (`stream`), else the `waves` of a block
    and how many `share` the same rows of b."""
    out = (ctypes.c_int32 * 6)()
    B._check(B.load_library().matmul8_plan(m, n, k, B.dtype_codes()[dtype or B._torch().bfloat16], products or 0, out), "matmul8_plan")
    return dict(zip(("tile", "parts", "groups", "stream", "waves", "share"), out))


def matmul8(a: Blocks8, b: Blocks8, *, dtype=None, out=None, accumulate: bool = False, products=None, workspace=None,
            stream=None):
    """out[i, j] = sum_k a[i, k] b[j, k] (plus the old out with accumulate), fp32 sums rounded
    once to dtype (float32, bfloat16 or float16; default out's, or bfloat16).

    With quantise8's results of a layer's x, weight and dy: y = (x, weight), dx = (dy, weight
    transposed), dweight = (dy transposed, x transposed). products 8: by the 8-bit matrix
    instructions, which drop bits below 2^-13 of the largest in every eight products. The result
    is off by 2^-16 of it on normally distributed values, but by up to 2^-10 of the products'
    magnitudes: more than a 16-bit result's own rounding where sums cancel. 16: widened to
    bfloat16, exactly, with sums as of fp32 additions, at half the rate. None: 16 for a float32
    result, 8 for others. workspace: optional uint8 buffer of matmul8_workspace_bytes().
    """
    torch = B._torch()
    for q, name in ((a, "a"), (b, "b")):
        if not isinstance(q, Blocks8):
            raise TypeError(f"{name} must be a Blocks8")
    device = a.device
    if b.device != device:
        raise ValueError(f"b must live on {device}")
    if a.cols != b.cols:
        raise ValueError(f"a and b must have the same number of columns, {a.cols} and {b.cols}")
    _check_products(products)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if out is not None:
        _check_out(out, (a.rows, b.rows), dtype, device)
    dtype = out.dtype if out is not None else dtype or torch.bfloat16
    code = B.dtype_codes().get(dtype)
    if code is None:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    with B.device_and_stream(device, stream):
        if out is None:
            out = a.codes.new_empty((a.rows, b.rows), dtype=dtype)
        ws, wsb = None, 0
        if workspace is not None:
            if workspace.device != device or not workspace.is_contiguous() or workspace.dtype != torch.uint8:
                raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
            ws, wsb = workspace.data_ptr(), workspace.numel()
        else:
            wsb = matmul8_workspace_bytes(a.rows, b.rows, a.cols, dtype, products)
            if wsb:
                workspace = a.codes.new_empty(wsb, dtype=torch.uint8)
                ws = workspace.data_ptr()
        ldc = out.stride(0) if out.shape[0] > 1 else out.shape[1]
        rc = _entry_points()[2](a._packed(), b._packed(), out.data_ptr(), ldc, code, products or 0, bool(accumulate), ws, wsb,
                                B.raw_stream(stream, device))
    if rc:
        B._check(rc, "matmul8")
    return out


class Weight8:
    """A layer's weight [out, in] in 8 bits, as both products that read it want it: `direct`
    for y = x w^T and `transposed` for dx = dy w, a power of two for every 128 x 128 elements.
    Kept between steps; `update` follows the weight after one (HybridOptimizer does it for the
    weights that it is told of).

    `version` counts the updates that the host made: linear8's backward pass refuses a form that
    was updated after its forward pass. An update in a captured graph counts once, at the capture:
    its replays write new codes and are not seen there, so a step is replayed after the backward
    passes of the forward passes before it."""

    def __init__(self, weight, stream=None):
        if not isinstance(weight, B._torch().Tensor) or weight.dim() != 2:
            raise ValueError("weight must be a 2-D torch.Tensor")
        self.direct, self.transposed = quantise8(weight.detach(), tiles=True, transposed=True, stream=stream)
        self.version = 0

    @property
    def shape(self):
        return self.direct.shape

    def update(self, weight, stream=None):
        """Takes the weight's present values, into the same memory."""
        if tuple(weight.shape) != self.shape:
            raise ValueError(f"weight must have shape {self.shape}")
        quantise8(weight.detach(), tiles=True, out=self.direct, out_transposed=self.transposed, stream=stream)
        self.version += 1


_function = None


def _autograd_function():
    """The autograd function, made at its first use: torch is imported lazily."""
    global _function
    if _function is not None:
        return _function
    torch = B._torch()

    class Linear8(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, weight8, products, weight_products, grads):
            # needs_input_grad tells of the leaves alone; grads: whether autograd records this call
            need_x, need_w = (grads and need for need in ctx.needs_input_grad[:2])
            ctx.shape, ctx.dtype, ctx.weight_dtype, ctx.products = x.shape, x.dtype, weight.dtype, (products, weight_products)
            # the caller's Weight8 is the caller's to keep; what is made here is autograd's, which
            # frees it after the backward pass and shows it to saved_tensors_hooks
            ctx.weight8, ctx.version = weight8, weight8 and weight8.version
            if weight8 is None:
                w8, w8t = quantise8(weight, tiles=True, transposed=need_x)
            else:
                w8, w8t = weight8.direct, None
            x8, x8t = quantise8(x, transposed=need_w)
            ctx.rows = x8.rows
            ctx.save_for_backward(x8t and x8t.codes, x8t and x8t.scales, w8t and w8t.codes, w8t and w8t.scales)
            return matmul8(x8, w8, dtype=x.dtype, products=products).view(*x.shape[:-1], w8.rows)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x_codes, x_scales, w_codes, w_scales = ctx.saved_tensors
            if ctx.weight8 is not None and ctx.weight8.version != ctx.version:
                raise RuntimeError("the weight's 8-bit form was updated after the forward pass")
            want_x, want_w = ctx.needs_input_grad[:2]
            cols = ctx.shape[-1]
            try:
                _rows_of(dy, "dy")
            except ValueError:  # an expanded or transposed gradient
                dy = dy.contiguous()
            dy8, dy8t = quantise8(dy, direct=want_x, transposed=want_w) if want_x or want_w else (None, None)
            dx = dw = None
            if want_x:
                w8t = _made(w_codes, w_scales, cols, dy8.cols, True) if ctx.weight8 is None else ctx.weight8.transposed
                dx = matmul8(dy8, w8t, dtype=ctx.dtype, products=ctx.products[0]).view(ctx.shape)
            if want_w:
                x8t = _made(x_codes, x_scales, cols, ctx.rows, False)
                dw = matmul8(dy8t, x8t, dtype=ctx.weight_dtype, products=ctx.products[1])
            return dx, dw, None, None, None, None

    _function = Linear8
    return Linear8


def linear8(x, weight, weight8: Weight8 = None, *, products=None, weight_grad_products=None):
    """x weight^T for torch.autograd with all three products in 8 bits: the output, x's gradient
    (both in x's dtype) and the weight's (in the weight's dtype, fp32 as Muon takes it).

    x [..., in], weight [out, in], each float32, bfloat16 or float16. x and the gradient are
    quantised by 128 elements along what each product sums over; for the weight's gradient x is
    kept in 8 bits. weight8: the weight's 8-bit form, kept up to date by the caller; made in the
    call without one, transposed too only where x's gradient will need it. With a form of its own
    and no gradient the weight's shape alone is used: it may be on another device.
    products, weight_grad_products: matmul8's `products` for the output and x's gradient, and for
    the weight's (8: twice the rate, fewer bits in the sums; None: 16 for a float32 result, 8 for
    others; a 16-bit output whose sums cancel needs 16).

    To capture a backward pass into a HIP graph, call quantise8 and matmul8 themselves: while an
    eager graph of the same leaves lives, a capture of autograd's backward pass waits for that
    graph's stream, which a capture does not allow, and torch ends the process.
    """
    torch = B._torch()
    for t, name in ((x, "x"), (weight, "weight")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"weight must be 2-D with x's {x.shape[-1] if x.dim() else 0} elements a row")
    if x.dtype not in B.dtype_codes():
        raise ValueError("x must be float32, bfloat16 or float16")
    grads = torch.is_grad_enabled()
    if weight8 is None or (grads and weight.requires_grad):
        if weight.dtype not in B.dtype_codes():
            raise ValueError("weight must be float32, bfloat16 or float16")
        if weight.device != x.device:
            raise ValueError(f"weight must live on {x.device}")
    _check_products(products)
    _check_products(weight_grad_products)
    if weight8 is not None:
        if not isinstance(weight8, Weight8):
            raise TypeError("weight8 must be a Weight8")
        if weight8.shape != tuple(weight.shape) or weight8.direct.device != x.device:
            raise ValueError(f"weight8 must have shape {tuple(weight.shape)} and live on {x.device}")
    return _autograd_function().apply(x, weight, weight8, products, weight_grad_products, grads)
