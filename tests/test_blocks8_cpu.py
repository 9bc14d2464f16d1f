"""The 8-bit matrices, the residual norm and the rotary positions without a GPU: refusals of
the C ABI (every one before any HIP call, on fake addresses that are never dereferenced) and of
the Python entry points, the byte forms of the structs, the rules by which a product is cut, and
the oracles themselves against differences and against each other.
"""
import ctypes

import numpy as np
import pytest

from oracle import blocks8_oracle as Q
from oracle import norm_oracle as N
from oracle import rotary_oracle as R
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import add_norm as AN, binding as B, blocks8, rotary_positions as rotary

from test_abi_cpu import fake_only, lib  # noqa: F401

BASE = 1 << 40
GIB = 1 << 30
INVALID, WORKSPACE, ALIGN, ALIAS, LARGE = -1, -2, -3, -4, -6


def ptr(i):
    return None if i is None else BASE + int(i * GIB)


def blocks(i, rows=64, cols=300, tiles=0, **over):
    kb = -(-cols // 128)
    f = dict(rows=rows, cols=cols, codes=ptr(i), scales=ptr(None if i is None else i + 0.5), ld=kb * 128,
             scale_ld=-(-kb // 4) * 4, tiles=tiles, reserved=0)
    f.update(over)
    return B.Blocks8Desc(*f.values())


def quantise(lib, x=ptr(0), rows=64, cols=300, stride=300, dtype=1, direct=None, transposed=None):  # noqa: F811
    return lib.quantise8(x, rows, cols, stride, dtype, direct, transposed, None)


BAD_BLOCKS = [(dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(tiles=2), INVALID), (dict(codes=None), INVALID),
              (dict(scales=None), INVALID), (dict(ld=383), INVALID), (dict(ld=392), INVALID), (dict(ld=256), INVALID),
              (dict(scale_ld=3), INVALID), (dict(scale_ld=6), INVALID), (dict(ld=(1 << 22) + 16), LARGE),
              (dict(codes=BASE + 8), ALIGN), (dict(scales=BASE + GIB + 2), ALIGN), (dict(rows=(1 << 30) + 1), LARGE),
              (dict(cols=(1 << 22) + 1), LARGE)]


@fake_only
@pytest.mark.parametrize("over,status", BAD_BLOCKS)
def test_blocks_refusals(lib, over, status):  # noqa: F811
    bad = blocks(1, **over)
    assert quantise(lib, direct=bad) == status
    assert lib.dequantise8(bad, ptr(5), 300, 1, None) == status
    assert lib.matmul8(bad, blocks(3), ptr(6), 64, 1, 0, 0, None, 0, None) == status
    assert lib.matmul8(blocks(3), bad, ptr(6), 64, 1, 0, 0, None, 0, None) == status


@fake_only
def test_quantise_refusals(lib):  # noqa: F811
    good, turned = blocks(1), blocks(3, rows=300, cols=64)
    null = ctypes.POINTER(B.Blocks8Desc)()
    assert quantise(lib, direct=null, transposed=null) == INVALID
    assert quantise(lib, direct=good, rows=-1) == INVALID and quantise(lib, direct=good, cols=-1) == INVALID
    assert quantise(lib, direct=good, dtype=3) == INVALID and quantise(lib, direct=good, dtype=-1) == INVALID
    assert quantise(lib, x=None, direct=good) == INVALID
    assert quantise(lib, direct=good, stride=-300) == INVALID
    assert quantise(lib, direct=blocks(1, rows=63)) == INVALID and quantise(lib, direct=blocks(1, cols=299)) == INVALID
    assert quantise(lib, transposed=good) == INVALID          # not the transposed shape
    assert quantise(lib, direct=blocks(1, tiles=1), transposed=turned) == INVALID
    assert quantise(lib, x=BASE + 1, direct=good) == ALIGN and quantise(lib, x=BASE + 2, dtype=0, direct=good) == ALIGN
    assert quantise(lib, direct=blocks(0)) == ALIAS            # on x
    assert quantise(lib, direct=blocks(1, scales=ptr(1) + 128)) == ALIAS
    assert quantise(lib, direct=good, transposed=blocks(1, rows=300, cols=64)) == ALIAS
    assert quantise(lib, rows=(1 << 30) + 1, direct=good) == LARGE
    assert quantise(lib, stride=1 << 41, direct=good) == LARGE
    wide = dict(rows=1 << 30, cols=1 << 22)
    assert quantise(lib, x=BASE << 4, stride=1 << 15, direct=blocks(1, **wide, codes=BASE << 8, scales=BASE << 14), **wide) == LARGE


@fake_only
def test_dequantise_refusals(lib):  # noqa: F811
    q = blocks(1)
    assert lib.dequantise8(None, ptr(5), 300, 1, None) == INVALID
    assert lib.dequantise8(q, None, 300, 1, None) == INVALID
    assert lib.dequantise8(q, ptr(5), 300, 7, None) == INVALID and lib.dequantise8(q, ptr(5), -1, 1, None) == INVALID
    assert lib.dequantise8(q, ptr(5), 299, 1, None) == ALIAS  # rows overlap
    assert lib.dequantise8(q, ptr(1), 300, 1, None) == ALIAS
    assert lib.dequantise8(q, ptr(5) + 1, 300, 1, None) == ALIGN


@fake_only
def test_matmul_refusals(lib):  # noqa: F811
    a, b = blocks(1), blocks(2, rows=500)

    def call(a=a, b=b, c=ptr(5), ldc=500, dtype=1, products=0, ws=ptr(7), bytes_=GIB):
        return lib.matmul8(a, b, c, ldc, dtype, products, 0, ws, bytes_, None)

    assert call(a=None) == INVALID and call(b=None) == INVALID and call(c=None) == INVALID
    assert call(b=blocks(2, rows=500, cols=301)) == INVALID
    assert call(dtype=3) == INVALID and call(products=4) == INVALID and call(ldc=-1) == INVALID
    assert call(ldc=499) == ALIAS and call(c=ptr(1)) == ALIAS and call(c=ptr(2.5)) == ALIAS
    assert call(c=BASE + 1) == ALIGN
    out = ctypes.c_size_t()
    assert lib.matmul8_workspace_bytes(64, 500, 300, 1, 0, None) == INVALID
    assert lib.matmul8_workspace_bytes(-1, 500, 300, 1, 0, out) == INVALID
    assert lib.matmul8_workspace_bytes(64, 500, 300, 4, 0, out) == INVALID
    assert lib.matmul8_workspace_bytes(64, 500, 300, 1, 9, out) == INVALID
    assert lib.matmul8_workspace_bytes(64, 500, (1 << 22) + 1, 1, 0, out) == LARGE
    assert lib.matmul8_workspace_bytes(1 << 30, 1 << 30, 128, 1, 0, out) == LARGE
    # a product in parts
    m, n, k = 128, 128, 1 << 16
    assert lib.matmul8_workspace_bytes(m, n, k, 0, 0, out) == 0 and out.value >= 2 * m * n * 4
    long = dict(a=blocks(1, rows=m, cols=k), b=blocks(2, rows=n, cols=k), ldc=n, dtype=0)
    assert call(**long, ws=None) == WORKSPACE and call(**long, bytes_=out.value - 1) == WORKSPACE
    assert call(**long, ws=ptr(7) + 128) == ALIGN and call(**long, ws=ptr(1)) == ALIAS
    # nothing to do
    assert call(a=blocks(None, rows=0), c=None) == 0 and call(b=blocks(None, rows=0), c=None) == 0


def test_cuts_of_a_product(lib):  # noqa: F811
    """Parts of k: none for a product with enough tiles, partial sums for every part elsewhere,
    and with few rows as many parts as their powers' room in LDS needs."""
    def size(m, n, k, dtype=1, products=0):
        out = ctypes.c_size_t()
        assert lib.matmul8_workspace_bytes(m, n, k, dtype, products, out) == 0
        assert out.value % (m * n * 4 if m * n else 1) == 0
        return out.value // (m * n * 4) if m * n else 0

    assert size(8192, 20480, 5120) == 0 and size(1, 2048, 2048) == 0 and size(8, 30720, 5120) == 0
    assert size(2048, 2048, 65536, 0) >= 2 and size(300, 300, 40000) >= 2
    assert size(0, 5, 128) == size(5, 0, 128) == 0
    for k in (128 * 125, 128 * 126, 128 * 128, 128 * 129, 1 << 20, (1 << 22) - 5):
        parts = max(1, size(7, 60000, k))
        fours = -(-(-(-k // 128)) // 4)
        longest = max((p + 1) * fours // parts - p * fours // parts for p in range(parts))
        assert 4 * longest <= 128, (k, parts)


def add_desc(**over):
    f = dict(rows=64, cols=128, dtype=1, rdtype=0, wdtype=0, eps=1e-6, weight_offset=0.0, reserved=0)
    f.update(over)
    return B.AddNormDesc(*f.values())


def rows(i, s=128):
    return B.NormRows(ptr(i), s, 0)


def param(i):
    return B.NormParam(ptr(i), 128)


def add_forward(lib, d=None, x=rows(0), r=rows(1), w=param(2), h=rows(3), y=rows(4), q=None, rstd=ptr(9)):  # noqa: F811
    return lib.add_rms_norm_forward(d if d is not None else add_desc(), x, r, w, h, y,
                                    q if q is not None else blocks(5, 64, 128), rstd, None)


def add_backward(lib, d=None, dy=rows(0), dh=rows(1), h=rows(2), w=param(3), rstd=ptr(4), dr=rows(5), dx=rows(6),  # noqa: F811
                 dw=param(7), ws=ptr(8), bytes_=GIB):
    return lib.add_rms_norm_backward(d if d is not None else add_desc(), dy, dh, h, w, rstd, dr, dx, dw, ws, bytes_, None)


BAD_ADD = [(dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(dtype=3), INVALID), (dict(rdtype=2), INVALID),
           (dict(wdtype=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
           (dict(weight_offset=float("inf")), INVALID), (dict(cols=16385), LARGE), (dict(rows=(1 << 30) + 1), LARGE)]


@fake_only
@pytest.mark.parametrize("over,status", BAD_ADD)
def test_add_norm_descriptor_refusals(lib, over, status):  # noqa: F811
    assert add_forward(lib, add_desc(**over)) == status
    assert add_backward(lib, add_desc(**over)) == status
    assert lib.add_rms_norm_backward_workspace_bytes(add_desc(**over), ctypes.c_size_t()) == status


@fake_only
def test_add_norm_refusals(lib):  # noqa: F811
    near = 16.0 / GIB
    for bad in (None, rows(None), rows(0, -128)):
        assert add_forward(lib, x=bad) == INVALID and add_backward(lib, dy=bad) == INVALID
        assert add_forward(lib, h=bad if bad is None or bad.data is None else rows(3, -1)) == INVALID
        assert add_backward(lib, h=bad) == INVALID and add_backward(lib, dr=bad) == INVALID
    assert add_forward(lib, r=rows(None)) == INVALID                   # h without a residual
    assert add_forward(lib, q=blocks(5, 64, 127)) == INVALID and add_forward(lib, q=blocks(5, 64, 128, tiles=1)) == INVALID
    assert add_forward(lib, q=blocks(5, 64, 128, ld=120)) == INVALID and add_forward(lib, q=blocks(5, 64, 128, codes=None)) == INVALID
    assert add_forward(lib, q=blocks(5, 64, 128, codes=BASE + 4)) == ALIGN
    assert add_forward(lib, x=B.NormRows(BASE + 1, 128, 0)) == ALIGN and add_forward(lib, rstd=BASE + 9 * GIB + 2) == ALIGN
    assert add_forward(lib, w=B.NormParam(BASE + 2 * GIB + 2, 128)) == ALIGN
    assert add_forward(lib, h=rows(3, 127)) == ALIAS and add_forward(lib, y=rows(4, 0)) == ALIAS
    assert add_forward(lib, y=rows(0)) == ALIAS and add_forward(lib, y=rows(3)) == ALIAS
    assert add_forward(lib, h=rows(1 + near)) == ALIAS and add_forward(lib, h=rows(1, 256)) == ALIAS
    assert add_forward(lib, h=rows(0)) == ALIAS                        # x has another type here
    assert add_forward(lib, q=blocks(4, 64, 128)) == ALIAS and add_forward(lib, rstd=ptr(2)) == ALIAS
    assert add_forward(lib, x=rows(0, 1 << 41)) == LARGE
    assert add_backward(lib, rstd=None) == INVALID and add_backward(lib, w=None) == INVALID
    assert add_backward(lib, add_desc(rdtype=1)) == INVALID            # dx beside a dr of the same type
    assert add_backward(lib, dx=rows(5)) == ALIAS and add_backward(lib, dr=rows(1 + near)) == ALIAS
    assert add_backward(lib, dr=rows(0)) == ALIAS and add_backward(lib, dw=param(3)) == ALIAS
    many = add_desc(rows=1 << 16)
    out = ctypes.c_size_t()
    assert lib.add_rms_norm_backward_workspace_bytes(many, out) == 0 and out.value >= 2 * 128 * 4
    assert lib.add_rms_norm_backward_workspace_bytes(many, None) == INVALID
    assert add_backward(lib, many, ws=None) == WORKSPACE and add_backward(lib, many, bytes_=out.value - 1) == WORKSPACE
    assert add_backward(lib, many, ws=ptr(8) + 128) == ALIGN and add_backward(lib, many, ws=ptr(0)) == ALIAS
    for over in (dict(rows=0), dict(cols=0)):
        assert lib.add_rms_norm_forward(add_desc(**over), rows(None), rows(None), None, None, rows(None),
                                        blocks(None, over.get("rows", 64), over.get("cols", 128)), None, None) == 0
    assert add_backward(lib, add_desc(rows=0), *([rows(None)] * 3), rstd=None, dr=rows(None), dx=rows(None), dw=None) == 0


def turn_desc(**over):
    f = dict(batch=2, tokens=8, heads=4, dim=64, pairs=30, axes=3, dtype=1, layout=0, position_type=0, inverse=0)
    f.update(over)
    return B.RotaryDesc(*f.values())


def heads(i, sb=2048, st=256, sh=64):
    return B.RotaryRows(ptr(i), sb, st, sh)


def turn(lib, d=None, x=heads(0), pos=None, freq=ptr(2), axis=ptr(3), y=heads(4)):  # noqa: F811
    return lib.rotary_apply(d if d is not None else turn_desc(), x, pos if pos is not None else B.RotaryPositions(ptr(1), 24, 3),
                            freq, axis, y, None)


BAD_TURN = [(dict(batch=-1), INVALID), (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(dim=-1), INVALID),
            (dict(pairs=0), INVALID), (dict(axes=0), INVALID), (dict(pairs=33), INVALID), (dict(dtype=3), INVALID),
            (dict(layout=2), INVALID), (dict(position_type=3), INVALID), (dict(dim=1025), LARGE), (dict(heads=65537), LARGE),
            (dict(batch=1 << 20, tokens=1 << 20), LARGE), (dict(tokens=(1 << 30) + 1), LARGE)]


@fake_only
@pytest.mark.parametrize("over,status", BAD_TURN)
def test_rotary_descriptor_refusals(lib, over, status):  # noqa: F811
    assert turn(lib, turn_desc(**over)) == status


@fake_only
def test_rotary_refusals(lib):  # noqa: F811
    assert lib.rotary_apply(None, heads(0), B.RotaryPositions(ptr(1), 24, 3), ptr(2), ptr(3), heads(4), None) == INVALID
    for bad in (None, heads(None), heads(0, -1), heads(0, 2048, -1), heads(0, 2048, 256, -1)):
        assert turn(lib, x=bad) == INVALID and turn(lib, y=bad) == INVALID
    assert turn(lib, freq=None) == INVALID and turn(lib, axis=None) == INVALID
    assert turn(lib, pos=B.RotaryPositions(None, 24, 3)) == INVALID and turn(lib, pos=B.RotaryPositions(ptr(1), 24, -3)) == INVALID
    assert turn(lib, x=B.RotaryRows(BASE + 1, 2048, 256, 64)) == ALIGN
    assert turn(lib, freq=ptr(2) + 4) == ALIGN and turn(lib, axis=ptr(3) + 2) == ALIGN
    assert turn(lib, pos=B.RotaryPositions(ptr(1) + 2, 24, 3)) == ALIGN
    assert turn(lib, turn_desc(position_type=1), pos=B.RotaryPositions(ptr(1) + 4, 24, 3)) == ALIGN
    assert turn(lib, y=heads(0, 2048, 256, 128)) == ALIAS and turn(lib, y=heads(16.0 / GIB)) == ALIAS
    for over in ((2048, 256, 63), (2048, 255, 64), (2047, 256, 64), (0, 256, 64)):
        assert turn(lib, y=heads(4, *over)) == ALIAS          # heads of y overlap
    assert turn(lib, y=heads(1)) == ALIAS and turn(lib, y=heads(3)) == ALIAS
    assert turn(lib, x=heads(0, 1 << 47)) == LARGE
    for over in (dict(batch=0), dict(tokens=0), dict(heads=0)):
        assert turn(lib, turn_desc(**over), x=heads(None), y=heads(None)) == 0


def test_packed_structs_are_the_headers():
    def same(struct, packed, values):
        got = struct.from_buffer_copy(packed)
        assert [getattr(got, f) for f, _ in struct._fields_] == values and len(packed) == ctypes.sizeof(struct)

    same(B.Blocks8Desc, blocks8._pack(1, 2, 1 << 50, 4, 5, 6, 1, 0), [1, 2, 1 << 50, 4, 5, 6, 1, 0])
    same(B.AddNormDesc, AN._pack_desc(1, 2, 3, 4, 5, 0.5, 0.25, 0), [1, 2, 3, 4, 5, 0.5, 0.25, 0])
    same(B.RotaryDesc, rotary._pack_desc(*range(1, 11)), list(range(1, 11)))
    same(B.RotaryRows, rotary._pack_rows(1 << 50, 2, 3, 4), [1 << 50, 2, 3, 4])
    same(B.RotaryPositions, rotary._pack_positions(7, 2, 3), [7, 2, 3])


def test_python_refusals():
    import torch
    x = torch.zeros(4, 8)
    for call in (lambda: muon.quantise8(x), lambda: muon.add_rms_norm_forward(x), lambda: muon.add_rms_norm_backward(x, None, x, None, None),
                 lambda: muon.rotary_apply(x, torch.zeros(1, dtype=torch.int32), muon.RotaryAxes((2,), device="cpu")),
                 lambda: muon.Blocks8(torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 4, dtype=torch.uint8), 8)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: muon.quantise8([1.0]), lambda: muon.add_rms_norm_forward([1.0]), lambda: muon.matmul8(x, x),
                 lambda: muon.rotary_apply(x, x, None), lambda: muon.linear8([1.0], x), lambda: muon.Blocks8(x.tolist(), x, 8)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="elements a row"):
        muon.linear8(torch.zeros(3, 7), x)
    with pytest.raises(ValueError, match="no gradient"):
        muon.rotary(x, torch.zeros(4, 1, requires_grad=True), muon.RotaryAxes((2,), device="cpu"))


def test_rotary_axes():
    import torch
    a = muon.RotaryAxes((2, 3), base=(100.0, 10000.0), device="cpu")
    freq, axis = R.ladder((2,), 100.0)[0].tolist() + R.ladder((3,), 10000.0)[0].tolist(), [0, 0, 1, 1, 1]
    assert a.pairs == 5 and a.axes == 2 and a.axis_of_pair == tuple(axis)
    assert np.allclose(a.frequencies, freq, rtol=1e-15)
    assert torch.allclose(a._freq * 2 * np.pi, torch.tensor(freq, dtype=torch.float64), rtol=1e-15)
    mixed = muon.RotaryAxes((2, 1), frequencies=[1.0, 0.5, 0.25], axis_of_pair=[1, 0, 0], device="cpu")
    assert mixed.frequencies == (1.0, 0.5, 0.25) and mixed._axis.tolist() == [1, 0, 0]
    assert muon.RotaryAxes((0, 4), device="cpu").axis_of_pair == (1,) * 4
    for bad in (dict(sections=()), dict(sections=(0, 0)), dict(sections=(2, -1)), dict(sections=(2,), layout="other"),
                dict(sections=(2,), base=0.0), dict(sections=(2, 2), base=(1.0,)), dict(sections=(2,), frequencies=[1.0]),
                dict(sections=(2,), frequencies=[1.0, float("inf")]), dict(sections=(2,), axis_of_pair=[0, 1])):
        with pytest.raises(ValueError):
            muon.RotaryAxes(**{"device": "cpu", **bad})


def test_levels_of_tokens():
    import torch
    x = torch.zeros(3, 5, 4, 8)
    pos = torch.zeros(5, 2).expand(3, 5, 2)
    assert rotary._levels((3, 5), (x.stride(), pos.stride())) == [(3, [160, 0]), (5, [32, 2])]
    full = torch.zeros(3, 5, 2)
    assert rotary._levels((3, 5), (x.stride(), full.stride())) == [(1, [0, 0]), (15, [32, 2])]
    assert rotary._levels((), ((), ())) == [(1, [0, 0]), (1, [0, 0])]
    with pytest.raises(ValueError, match="two strides"):
        y = torch.zeros(2, 3, 5, 2, 4, 8)[:, :, :, 0]
        rotary._levels((2, 3, 5), (y.transpose(0, 1).transpose(1, 2).stride(), torch.zeros(2, 3, 5, 2).stride()))


def test_rows_at_one_stride():
    import torch

    def rows_of(t):
        # the checks ask for a GPU tensor, the arithmetic for strides
        return blocks8._rows_of(torch.Tensor._make_subclass(type("T", (torch.Tensor,), {"is_cuda": True}), t), "x")

    assert rows_of(torch.zeros(3, 5, 8)) == (15, 8, 8)
    assert rows_of(torch.zeros(6, 16)[:, :8]) == (6, 8, 16)
    assert rows_of(torch.zeros(3, 5, 16)[..., :8]) == (15, 8, 16)
    assert rows_of(torch.zeros(1, 8).expand(6, 8)) == (6, 8, 0)
    assert rows_of(torch.zeros(8)) == (1, 8, 8)
    assert rows_of(torch.zeros(0, 8)) == (0, 8, 8)
    with pytest.raises(ValueError, match="one stride"):
        rows_of(torch.zeros(4, 6, 8)[:, :3])
    with pytest.raises(ValueError, match="adjacent"):
        rows_of(torch.zeros(8, 4).t())


# ---------------------------------------------------------------- the oracles ----

def test_oracle_codes_are_the_nearest():
    """The oracle's rounding against a search over all 256 codes."""
    v = Q.e4m3_values()
    v = np.unique(v[np.isfinite(v)])
    assert v[-1] == 448.0 and len(v) == 253  # +0 and -0 are one value
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.uniform(-448, 448, 3000), rng.standard_normal(3000), rng.standard_normal(3000) * 2.0 ** -8,
                        (v[1:] + v[:-1]) / 2, v])
    got = Q.round_e4m3(x)
    gap = np.abs(x[:, None] - v[None])
    assert np.array_equal(np.abs(got - x), gap.min(1))
    ties = (v[1:] + v[:-1]) / 2
    codes = {abs(val): c & 127 for c, val in enumerate(Q.e4m3_values()) if np.isfinite(val)}
    assert all(codes[abs(r)] % 2 == 0 for r in Q.round_e4m3(ties))


def test_oracle_powers_are_the_least():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 300)) * 2.0 ** rng.integers(-60, 60, (5, 1))
    x[1, :128] = 0.0
    x[2, 5], x[2, 200] = np.inf, np.nan
    x[3, 0] = 448.0 * 2.0 ** 40
    x[3, 1:128] = 0.0
    for tiles in (False, True):
        vals, e = Q.quantise(x, tiles)
        s = Q.spread(e, x.shape, tiles).astype(float)
        fine = np.isfinite(x)
        assert (np.abs(x[fine]) <= 448 * 2.0 ** s[fine]).all()
        assert np.array_equal(np.isnan(vals), ~fine)
        assert (np.abs(vals[fine] - x[fine]) <= np.maximum(2.0 ** -4 * np.abs(x[fine]), 2.0 ** (s[fine] - 10))).all()
    e = Q.powers(x)
    assert e[1, 0] == -127 and e[3, 0] == 40
    top = np.abs(np.where(np.isfinite(x), x, 0)[0, :128]).max()
    assert top > 448 * 2.0 ** (e[0, 0] - 1)
    assert np.array_equal(Q.quantise(x.T, True)[0].T, Q.quantise(x, True)[0], equal_nan=True)


def test_oracle_residual_norm_gradient_is_the_difference():
    """dh + the RMS norm's own gradient, against differences of sum(y k) + sum(h m)."""
    rng = np.random.default_rng(3)
    x, r, k, m, w = (rng.standard_normal(s) for s in ((4, 9), (4, 9), (4, 9), (4, 9), (9,)))

    def loss():
        h = x + r
        return float((N.norm_forward(h, w, None, "rms", 1e-5, 0.5)[0][0] * k).sum() + (h * m).sum())

    _, _, rstd, _, _ = N.norm_forward(x + r, w, None, "rms", 1e-5, 0.5)
    dx, dw, _, _, _ = N.norm_backward(k, x + r, w, None, rstd, "rms", 0.5)
    d = dx[0] + m
    for arr, grad in ((x, d), (r, d), (w, dw[0])):
        for at in np.ndindex(arr.shape):
            keep = arr[at]
            arr[at] = keep + 1e-6
            up = loss()
            arr[at] = keep - 1e-6
            down = loss()
            arr[at] = keep
            assert abs((up - down) / 2e-6 - grad[at]) < 1e-7


@pytest.mark.parametrize("layout", ["halves", "adjacent"])
def test_oracle_rotation_keeps_lengths_and_its_inverse_is_the_gradient(layout):
    rng = np.random.default_rng(4)
    x, g = rng.standard_normal((5, 2, 14)), rng.standard_normal((5, 2, 14))
    pos = rng.integers(0, 1000, (5, 2))
    freq, axis = R.ladder((2, 4))
    y = R.rotate(x, pos, freq, axis, layout)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 12:], x[..., 12:])
    assert np.allclose(R.rotate(y, pos, freq, axis, layout, True), x, atol=1e-12)
    # the map is linear: <rotate(x), g> = <x, rotate back(g)>
    assert np.isclose((y * g).sum(), (x * R.rotate(g, pos, freq, axis, layout, True)).sum())
    # scores of a query and a key depend on the difference of their positions alone
    q, k = rng.standard_normal((1, 1, 12)), rng.standard_normal((1, 1, 12))

    def score(a, b):
        return (R.rotate(q, [[a, 3]], freq, axis, layout) * R.rotate(k, [[b, 9]], freq, axis, layout)).sum()

    assert np.isclose(score(7, 2), score(107, 102))
