"""The normalisation layers without a GPU: refusals of the C ABI (every one before any HIP
call, on fake addresses that are never dereferenced), refusals of the Python entry points,
the division that finds a strided row, and the oracle itself against differences.
"""
import ctypes

import numpy as np
import pytest

from oracle import norm_oracle as N
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B
from matrix_orthogonalising_optimizer_02_amd import norms

from test_abi_cpu import fake_only, lib  # noqa: F401

BASE = 1 << 40
GIB = 1 << 30


def desc(**over):
    f = dict(rows=64, cols=128, groups=4, inner=1, kind=0, dtype=1, wdtype=1, eps=1e-6, weight_offset=0.0)
    f.update(over)
    return B.NormDesc(*f.values())


def rows(i, s0=128, s1=0):
    return B.NormRows(None if i is None else BASE + int(i * GIB), s0, s1)


def param(i, stride=128):
    return B.NormParam(None if i is None else BASE + int(i * GIB), stride)


def ptr(i):
    return None if i is None else BASE + int(i * GIB)


def forward(lib, d=None, x=rows(0), w=param(1), b=param(2), y=rows(3), mean=ptr(4), rstd=ptr(5)):
    return lib.norm_forward(d if d is not None else desc(), x, w, b, y, mean, rstd, None)


def backward(lib, d=None, dy=rows(0), x=rows(1), w=param(2), mean=ptr(3), rstd=ptr(4), dx=rows(5), dw=param(6),
             db=param(7), ws=ptr(8), bytes_=GIB):
    return lib.norm_backward(d if d is not None else desc(), dy, x, w, mean, rstd, dx, dw, db, ws, bytes_, None)


BAD_DESCS = [(dict(rows=-1), -1), (dict(cols=-1), -1), (dict(groups=0), -1), (dict(groups=5), -1), (dict(inner=0), -1),
             (dict(inner=3), -1), (dict(kind=2), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(wdtype=2), -1),
             (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
             (dict(weight_offset=float("nan")), -1), (dict(cols=16385), -6), (dict(rows=(1 << 30) + 1, groups=1), -6)]
HUGE = dict(rows=1 << 30, groups=1 << 30, cols=8)  # a block a group: more threads than a launch takes


@fake_only
@pytest.mark.parametrize("over,status", BAD_DESCS)
def test_descriptor_refusals(lib, over, status):  # noqa: F811
    assert forward(lib, desc(**over)) == status
    assert backward(lib, desc(**over)) == status
    out = ctypes.c_size_t()
    assert lib.norm_backward_workspace_bytes(desc(**over), out) == status


@fake_only
def test_pointer_refusals(lib):  # noqa: F811
    null = ctypes.POINTER(B.NormDesc)()
    assert lib.norm_forward(null, rows(0), None, None, rows(3), None, None, None) == B.MUON_ERR_INVALID_ARG
    assert lib.norm_backward_workspace_bytes(null, ctypes.c_size_t()) == B.MUON_ERR_INVALID_ARG
    assert lib.norm_backward_workspace_bytes(desc(), None) == B.MUON_ERR_INVALID_ARG
    for bad in (rows(None), None, rows(0, -128)):
        assert forward(lib, x=bad) == B.MUON_ERR_INVALID_ARG
        assert forward(lib, y=bad) == B.MUON_ERR_INVALID_ARG
        for name in ("dy", "x", "dx"):
            assert backward(lib, **{name: bad}) == B.MUON_ERR_INVALID_ARG
    assert forward(lib, w=param(1, -1)) == B.MUON_ERR_INVALID_ARG
    assert backward(lib, mean=None) == B.MUON_ERR_INVALID_ARG
    assert backward(lib, rstd=None) == B.MUON_ERR_INVALID_ARG
    assert backward(lib, w=None) == B.MUON_ERR_INVALID_ARG  # dw without w
    # one byte into an element; statistics off their four bytes
    odd = B.NormRows(BASE + 1, 128, 0)
    assert forward(lib, x=odd) == B.MUON_ERR_ALIGN and backward(lib, dx=odd) == B.MUON_ERR_ALIGN
    assert forward(lib, b=B.NormParam(BASE + 2 * GIB + 1, 128)) == B.MUON_ERR_ALIGN
    assert forward(lib, rstd=BASE + 5 * GIB + 2) == B.MUON_ERR_ALIGN
    assert backward(lib, ws=BASE + 8 * GIB + 128, d=desc(rows=1 << 20)) == B.MUON_ERR_ALIGN
    assert forward(lib, x=rows(0, 1 << 41)) == B.MUON_ERR_TOO_LARGE


@fake_only
def test_more_groups_than_a_launch_takes(lib):  # noqa: F811
    far = B.NormParam(BASE << 1, 8), B.NormParam(BASE << 2, 8)
    args = dict(w=far[0], b=far[1], mean=None, rstd=None)
    assert forward(lib, desc(**HUGE), x=B.NormRows(BASE, 8, 0), y=B.NormRows(BASE << 3, 8, 0), **args) == B.MUON_ERR_TOO_LARGE
    assert backward(lib, desc(**HUGE), dy=B.NormRows(BASE, 8, 0), x=B.NormRows(BASE, 8, 0), w=far[0], mean=ptr(100), rstd=ptr(200),
                    dx=B.NormRows(BASE << 3, 8, 0), dw=B.NormParam(BASE << 4, 8), db=None) == B.MUON_ERR_TOO_LARGE


@fake_only
def test_workspace_refusals(lib):  # noqa: F811
    d = desc(rows=1 << 16, groups=1)
    out = ctypes.c_size_t()
    assert lib.norm_backward_workspace_bytes(d, out) == B.MUON_OK and out.value >= 2 * 2 * 128 * 4
    assert backward(lib, d, ws=None) == B.MUON_ERR_WORKSPACE
    assert backward(lib, d, bytes_=out.value - 1) == B.MUON_ERR_WORKSPACE


@fake_only
def test_overlap_refusals(lib):  # noqa: F811
    alias = B.MUON_ERR_ALIAS
    near = 16.0 / GIB
    assert forward(lib, y=rows(near)) == alias          # y starts inside x
    assert forward(lib, y=rows(0, 256)) == alias        # the same start, other rows
    assert forward(lib, y=rows(1)) == alias             # on the weight
    assert forward(lib, mean=ptr(5)) == alias           # on rstd
    assert forward(lib, y=rows(3, 127)) == alias        # rows of y overlap
    assert forward(lib, y=rows(3, 0)) == alias
    assert forward(lib, desc(inner=4), y=rows(3, 128, 128)) == alias
    assert forward(lib, desc(inner=4), y=rows(3, 511, 128)) == alias
    assert forward(lib, desc(inner=4), y=rows(3, 128, 16 * 128 - 1)) == alias
    assert backward(lib, dx=rows(near)) == alias and backward(lib, dx=rows(1 + near)) == alias
    assert backward(lib, dw=param(7)) == alias and backward(lib, dw=param(2)) == alias
    assert backward(lib, dw=param(6, 127)) == alias     # the groups' gradients overlap
    assert backward(lib, desc(rows=1 << 16), dx=rows(8)) == alias  # dx on the workspace


@fake_only
def test_nothing_to_do(lib):  # noqa: F811
    for over in (dict(rows=0), dict(cols=0)):
        assert forward(lib, desc(**over), x=rows(None), y=rows(None)) == B.MUON_OK
    assert backward(lib, desc(cols=0), dy=rows(None), x=rows(None), dx=rows(None)) == B.MUON_OK
    assert backward(lib, desc(rows=0), dy=rows(None), x=rows(None), dx=rows(None), mean=None, rstd=None, dw=None,
                    db=None) == B.MUON_OK


def test_python_refusals():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        muon.norm_forward(x)
    with pytest.raises(TypeError):
        muon.norm_forward([1.0])
    with pytest.raises(ValueError, match="GPU"):
        muon.norm_backward(x, x, None, None, None)
    with pytest.raises(ValueError, match="last dimension"):
        norms._row_levels(torch.zeros(8, 4).t(), "x")
    with pytest.raises(ValueError, match="two strides"):
        norms._row_levels(torch.zeros(4, 6, 8, 10)[:, :4:2, ::2], "x")
    with pytest.raises(ValueError, match="unlike"):
        norms._layout(((torch.zeros(6, 4, 9)[:, :, :8], "a"), (torch.zeros(4, 6, 8).transpose(0, 1), "b"),
                       (torch.zeros(8, 8, 9)[:, :6:2, :8], "c")))


def test_row_levels_and_layout():
    import torch
    assert norms._row_levels(torch.zeros(3, 5, 8), "x") == [(15, 8)]
    assert norms._row_levels(torch.zeros(8), "x") == []
    assert norms._row_levels(torch.zeros(7, 3, 4, 8)[:, 1], "x") == [(4, 8), (7, 96)]
    assert norms._row_levels(torch.zeros(1, 8).expand(6, 8), "x") == [(6, 0)]
    q, y = torch.zeros(7, 3, 4, 8)[:, 1], torch.zeros(7, 4, 8)
    inner, (rq, ry) = norms._layout(((q, "q"), (y, "y")))
    rq, ry = (B.NormRows.from_buffer_copy(r) for r in (rq, ry))
    assert inner == 4 and (rq.stride0, rq.stride1) == (96, 8) and (ry.stride0, ry.stride1) == (32, 8)
    assert rq.data == q.data_ptr()


def test_packed_structs_are_the_headers():
    """The byte forms of the calls' structs against the ctypes structures of the header."""
    d = B.NormDesc.from_buffer_copy(norms._pack_desc(1, 2, 3, 4, 5, 6, 7, 0.5, 0.25))
    assert [getattr(d, f) for f, _ in d._fields_] == [1, 2, 3, 4, 5, 6, 7, 0.5, 0.25]
    assert len(norms._pack_desc(1, 2, 3, 4, 5, 6, 7, 0.5, 0.25)) == ctypes.sizeof(B.NormDesc)
    r = B.NormRows.from_buffer_copy(norms._pack_rows(1 << 50, 2, 3))
    assert (r.data, r.stride0, r.stride1) == (1 << 50, 2, 3)
    p = B.NormParam.from_buffer_copy(norms._pack_param(0, 3))
    assert (p.data, p.stride) == (None, 3)
    assert norms.norm_backward_workspace_bytes(1 << 16, 128) >= 2 * 2 * 128 * 4
    with pytest.raises(B.MuonError):
        norms.norm_backward_workspace_bytes(10, 128, groups=3)


def test_division_by_the_inner_rows():
    """r / inner by the multiplier the library uses, at and around every multiple."""
    rng = np.random.default_rng(3)
    for d in [2, 3, 5, 7, 16, 40, 48, 641, 65535, 65537, 2 ** 30, 2 ** 31 - 1] + [int(v) for v in rng.integers(2, 2 ** 31, 40)]:
        shift = (d - 1).bit_length()
        mul = (((1 << shift) - d) << 32) // d + 1
        assert mul < 2 ** 32
        qs = np.unique(np.concatenate([rng.integers(0, (2 ** 31 - 1) // d + 1, 200), [0, 1, (2 ** 31 - 1) // d]]))
        for q in (int(v) for v in qs):
            for r in (q * d - 1, q * d, q * d + 1, q * d + d - 1):
                if 0 <= r < 2 ** 31:
                    assert (((r * mul) >> 32) + r) >> shift == r // d, (r, d)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_oracle_gradients_are_the_differences(kind):
    rng = np.random.default_rng(5)
    r, c, g = 6, 11, 3
    x, w, b, k = (rng.standard_normal(s) for s in ((r, c), (g, c), (g, c), (r, c)))
    _, mean, rstd, _, _ = N.norm_forward(x, w, b, kind, 1e-5, 1.0, g)
    dx, dw, db, _, _ = N.norm_backward(k, x, w, mean, rstd, kind, 1.0, g)

    def loss():
        return float((N.norm_forward(x, w, b, kind, 1e-5, 1.0, g)[0].reshape(r, c) * k).sum())

    for arr, grad in ((x, dx.reshape(r, c)), (w, dw), (b, db)):
        for at in np.ndindex(arr.shape):
            keep = arr[at]
            arr[at] = keep + 1e-6
            up = loss()
            arr[at] = keep - 1e-6
            down = loss()
            arr[at] = keep
            assert abs((up - down) / 2e-6 - grad[at]) < 1e-7 * max(1.0, abs(grad[at])) + 1e-8


def test_weight_rows_that_are_no_leading_dimensions():
    """A row a sample, a row a row of x, or one for all; a row a token of every sample would
    be taken for equal runs of rows, and is refused."""
    import torch
    x = torch.zeros(6, 10, 32)

    def groups(*shape, x=x):
        return norms._param(torch.zeros(*shape), "weight", shape[-1], None, x, (torch.float32,))[0]

    assert groups(32) == groups(1, 32) == groups(1, 1, 32) == 1
    assert groups(6, 32) == groups(6, 1, 32) == groups(6, 1, 1, 32) == 6
    assert groups(60, 32) == groups(6, 10, 32) == groups(60, 1, 32) == 60
    for bad in ((10, 32), (1, 10, 32), (12, 32), (3, 32), (2, 32), (3, 2, 32), (10, 6, 32), (6, 2, 32), (30, 1, 32)):
        with pytest.raises(ValueError, match="leading dimensions"):
            groups(*bad)
    square = torch.zeros(6, 6, 32)
    assert groups(6, 32, x=square) == 6  # a row a sample
    with pytest.raises(ValueError, match="leading dimensions"):
        groups(1, 6, 32, x=square)
    four = torch.zeros(2, 3, 10, 32)
    assert groups(2, 32, x=four) == 2 and groups(6, 32, x=four) == groups(2, 3, 32, x=four) == groups(2, 3, 1, 32, x=four) == 6
    assert groups(10, 32, x=torch.zeros(1, 10, 32)) == groups(1, 10, 32, x=torch.zeros(1, 10, 32)) == 10
    # rows that have no dimensions of their own: equal runs, as many as divide them
    assert groups(4, 32, x=torch.zeros(60, 32)) == groups(4, 1, 32, x=torch.zeros(60, 32)) == 4
