"""AdamW over many tensors and the gradient norm without a GPU: refusals of the C ABI
(before any HIP call, on fake addresses that are never dereferenced), of the Python entry
points, and the 8-bit oracle against torch's own e4m3 conversion.
"""
import ctypes

import numpy as np
import pytest

from oracle import adamw8_oracle as O8
import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B

from test_abi_cpu import fake_only, lib  # noqa: F401

BASE, GIB = 1 << 40, 1 << 30
INVALID, ALIGN, ALIAS, LARGE, WORKSPACE = (B.MUON_ERR_INVALID_ARG, B.MUON_ERR_ALIGN, B.MUON_ERR_ALIAS, B.MUON_ERR_TOO_LARGE,
                                           B.MUON_ERR_WORKSPACE)


def tensor(i=0, **over):
    p = BASE + 16 * i * GIB
    f = dict(numel=1000, w=p, copy=p + GIB, g=p + 2 * GIB, m=p + 3 * GIB, v=p + 4 * GIB, m_scale=p + 5 * GIB,
             v_scale=p + 6 * GIB, g_dtype=1, copy_dtype=1, state_bits=8, lr_scale=1.0, wd_scale=1.0)
    f.update(over)
    return B.AdamWTensor(*f.values())


def plan(lib, tensors, device=BASE + 900 * GIB, bytes_=GIB, count=None, out=None):
    arr = (B.AdamWTensor * max(len(tensors), 1))(*tensors)
    out = B.TensorPlan() if out is None else out
    return lib.adamw_multi_plan(arr, len(tensors) if count is None else count, device, bytes_, out, None)


@fake_only
@pytest.mark.parametrize("over,status", [
    (dict(numel=-1), INVALID), (dict(numel=(1 << 40) + 1), LARGE), (dict(w=None), INVALID), (dict(g=None), INVALID),
    (dict(m=None), INVALID), (dict(v=None), INVALID), (dict(m_scale=None), INVALID), (dict(v_scale=None), INVALID),
    (dict(state_bits=16), INVALID), (dict(state_bits=0), INVALID), (dict(g_dtype=3), INVALID), (dict(g_dtype=-1), INVALID),
    (dict(copy_dtype=0), INVALID), (dict(copy_dtype=5), INVALID), (dict(lr_scale=float("nan")), INVALID),
    (dict(wd_scale=float("inf")), INVALID), (dict(w=BASE + 8), ALIGN), (dict(g=BASE + 2 * GIB + 8), ALIGN),
    (dict(m=BASE + 3 * GIB + 4), ALIGN), (dict(copy=BASE + GIB + 2), ALIGN), (dict(m_scale=BASE + 5 * GIB + 2), ALIGN),
    (dict(m=BASE + 4 * GIB + 512), ALIAS), (dict(v=BASE + 16), ALIAS), (dict(g=BASE), ALIAS), (dict(copy=BASE + 3 * GIB), ALIAS),
    (dict(m_scale=BASE + 6 * GIB), ALIAS), (dict(v_scale=BASE + 900 * GIB), ALIAS), (dict(g=BASE + 900 * GIB), ALIAS)])
def test_adamw_plan_refusals(lib, over, status):  # noqa: F811
    assert plan(lib, [tensor(1), tensor(0, **over)]) == status
    out = B.TensorPlan()
    plan(lib, [tensor(0, **over)], out=out)
    assert out.kind == 0  # no plan was made


@fake_only
def test_adamw_plan_lists_and_buffers(lib):  # noqa: F811
    need = ctypes.c_size_t()
    two = (B.AdamWTensor * 2)(tensor(0), tensor(1))
    assert lib.adamw_multi_plan_bytes(two, 2, need) == B.MUON_OK and need.value > 0
    assert plan(lib, [tensor(0), tensor(1)], bytes_=need.value - 1) == WORKSPACE
    assert plan(lib, [tensor(0)], device=None) == WORKSPACE
    assert plan(lib, [tensor(0)], device=BASE + 900 * GIB + 64) == ALIGN
    assert plan(lib, [tensor(0), tensor(0)]) == ALIAS  # the same tensor twice
    assert plan(lib, [tensor(0)], count=-1) == INVALID
    assert lib.adamw_multi_plan(None, 1, BASE, GIB, B.TensorPlan(), None) == INVALID
    assert lib.adamw_multi_plan(two, 2, BASE, GIB, None, None) == INVALID
    assert lib.adamw_multi_plan_bytes(two, 2, None) == INVALID
    assert lib.adamw_multi_plan_bytes(two, -2, need) == INVALID
    big = (B.AdamWTensor * 9)(*[tensor(0, numel=1 << 40)] * 9)
    assert lib.adamw_multi_plan_bytes(big, 9, need) == LARGE
    # blocks of 4096 elements and 256 threads in a launch of less than 2^32 threads
    most = ((1 << 24) - 1) * 4096
    assert lib.adamw_multi_plan_bytes((B.AdamWTensor * 1)(tensor(0, numel=most)), 1, need) == B.MUON_OK
    assert lib.adamw_multi_plan_bytes((B.AdamWTensor * 1)(tensor(0, numel=most + 1)), 1, need) == LARGE
    assert lib.adamw_multi_plan_bytes(two, (1 << 22) - 1, need) == LARGE


@fake_only
def test_adamw_step_refusals(lib):  # noqa: F811
    hp = B.adamw_default_hparams()
    empty = B.TensorPlan()
    assert lib.adamw_multi_plan(None, 0, None, 0, empty, None) == B.MUON_OK
    assert lib.adamw_multi_step(empty, hp, 0, 0, None, None) == B.MUON_OK  # nothing to do
    none = (B.AdamWTensor * 2)(B.AdamWTensor(), B.AdamWTensor())
    skipped = B.TensorPlan()
    assert lib.adamw_multi_plan(none, 2, None, 0, skipped, None) == B.MUON_OK  # empty tensors alone
    assert lib.adamw_multi_step(skipped, hp, 0, 0, None, None) == B.MUON_OK
    assert lib.adamw_multi_step(None, hp, 0, 0, None, None) == INVALID
    assert lib.adamw_multi_step(B.TensorPlan(), hp, 0, 0, None, None) == INVALID
    assert lib.adamw_multi_step(empty, None, 0, 0, None, None) == INVALID
    assert lib.adamw_multi_step(empty, hp, -1, 0, None, None) == INVALID
    assert lib.adamw_multi_step(empty, hp, 0, 0, BASE + 2, None) == ALIGN
    for over in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(eps=1e-39), dict(lr=float("nan")),
                 dict(weight_decay=float("inf"))):
        assert lib.adamw_multi_step(empty, B.adamw_default_hparams(**over), 0, 0, None, None) == INVALID, over
    assert lib.adamw_multi_step_device(empty, hp, BASE, None, 0, None, None) == B.MUON_OK
    assert lib.adamw_multi_step_device(empty, hp, None, None, 0, None, None) == INVALID
    assert lib.adamw_multi_step_device(empty, hp, BASE + 4, None, 0, None, None) == ALIGN
    assert lib.adamw_multi_step_device(empty, hp, BASE, BASE + 2, 0, None, None) == ALIGN
    assert lib.adamw_multi_step_device(B.TensorPlan(), hp, BASE, None, 0, None, None) == INVALID
    grads = B.TensorPlan()
    assert lib.grad_norm_plan(None, 0, None, 0, grads, None) == B.MUON_OK
    assert lib.adamw_multi_step(grads, hp, 0, 0, None, None) == INVALID  # another call's plan
    assert lib.grad_norm(empty, 1.0, BASE, None, None) == INVALID
    assert lib.grad_scale(empty, BASE, None) == INVALID


def grads(lib, items, device=BASE + 900 * GIB, bytes_=GIB, out=None):
    arr = (B.GradTensor * max(len(items), 1))(*[B.GradTensor(*t, 0) for t in items])
    return lib.grad_norm_plan(arr, len(items), device, bytes_, B.TensorPlan() if out is None else out, None)


@fake_only
def test_grad_norm_refusals(lib):  # noqa: F811
    ok = (BASE, 1000, 1)
    assert grads(lib, [(None, 10, 0)]) == INVALID
    assert grads(lib, [(BASE, -1, 0)]) == INVALID
    assert grads(lib, [(BASE, 10, 3)]) == INVALID
    assert grads(lib, [(BASE, (1 << 40) + 1, 0)]) == LARGE
    assert grads(lib, [(BASE + 1, 10, 1)]) == ALIGN
    assert grads(lib, [(BASE + 2, 10, 0)]) == ALIGN
    assert grads(lib, [ok, (BASE + 1998, 10, 1)]) == ALIAS
    assert grads(lib, [ok, ok]) == ALIAS
    assert grads(lib, [(BASE + 900 * GIB, 10, 0)]) == ALIAS
    assert grads(lib, [ok], device=None) == WORKSPACE
    assert grads(lib, [ok], bytes_=16) == WORKSPACE
    assert grads(lib, [ok], device=BASE + 900 * GIB + 8) == ALIGN
    empty = B.TensorPlan()
    assert grads(lib, [], out=empty) == B.MUON_OK
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert lib.grad_norm(empty, bad, BASE, None, None) == INVALID
    assert lib.grad_norm(empty, 1.0, None, None, None) == INVALID
    assert lib.grad_norm(empty, 1.0, BASE + 2, None, None) == ALIGN
    assert lib.grad_norm(None, 1.0, BASE, None, None) == INVALID
    assert lib.grad_scale(empty, None, None) == INVALID
    assert lib.grad_scale(empty, BASE + 1, None) == ALIGN
    assert lib.grad_scale(empty, BASE, None) == B.MUON_OK


def test_python_refusals():
    import torch
    x = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        muon.AdamWMulti([x], [x])
    with pytest.raises(ValueError, match="state_bits"):
        muon.AdamWMulti([x], [x], state_bits=16)
    with pytest.raises(ValueError, match="seed"):
        muon.AdamWMulti([x], [x], seed=-1)
    with pytest.raises(ValueError, match="dtype"):
        muon.AdamWMulti([x.double()], [x])
    with pytest.raises(TypeError):
        muon.AdamWMulti([1.0], [x])
    with pytest.raises(ValueError, match="contiguous"):
        muon.GradNorm([torch.zeros(4, 4).t()])
    with pytest.raises(ValueError, match="GPU"):
        muon.GradNorm([x])
    with pytest.raises(TypeError):
        muon.GradNorm([None])


def test_oracle_decode_is_torchs_e4m3():
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = O8.decode(codes.numpy())
    assert np.array_equal(got, want, equal_nan=True)
    assert O8.VALUES[-1] == 448.0 and (np.diff(O8.VALUES) > 0).all()


def test_rounding_bits_are_spread_and_apart():
    """16-bit halves of the hash over consecutive elements: uniform in 16 buckets (chi
    squared with 15 degrees of freedom, below 50 but for one in 80000), uncorrelated
    between neighbours, halves, tensors and steps (|r| below 5 / sqrt(n))."""
    n = 1 << 16
    a, b = O8.rounding_bits(123, 7, 0, np.arange(n))
    others = [O8.rounding_bits(123, 7, 1, np.arange(n))[0], O8.rounding_bits(123, 8, 0, np.arange(n))[0],
              O8.rounding_bits(124, 7, 0, np.arange(n))[0], np.roll(a, 1), b]
    for x in (a, b):
        counts = np.bincount(x >> 12, minlength=16)
        assert ((counts - n / 16) ** 2 / (n / 16)).sum() < 50
        assert x.min() >= 0 and x.max() < 65536
    for x in others:
        assert abs(np.corrcoef(a, x)[0, 1]) < 5 / np.sqrt(n)
    far = O8.rounding_bits(123, 7, 0, np.array([5, 5 + (1 << 32)]))[0]
    assert far[0] != far[1]


def test_moved_tensors_are_found():
    import torch
    from matrix_orthogonalising_optimizer_02_amd import multi
    t = [torch.zeros(8) for _ in range(3)]
    ptrs = [x.data_ptr() for x in t]
    assert multi._moved(t, ptrs) is None and multi._moved([], []) is None
    watch = multi._Watch({"params": t[:2], "copies": t[2:]})
    watch.check()
    for i, name in ((0, r"params\[0\]"), (1, r"params\[1\]"), (2, r"copies\[0\]")):
        old = t[i].data
        t[i].data = torch.ones(8)
        assert multi._moved(t, ptrs) == i
        with pytest.raises(ValueError, match=name + " has other memory"):
            watch.check()
        t[i].data = old
        watch.check()


def test_spans_of_tensors():
    """A scalar on the first or last bytes of a tensor, between two, across an edge."""
    import torch
    from matrix_orthogonalising_optimizer_02_amd import multi
    base = torch.zeros(100)
    at = base.data_ptr()
    parts = [base[60:80], base[10:20], base[20:30], base[15:18], base[50:50], base[:0]]
    s = multi._Spans([t.data_ptr() for t in parts], [4 * t.numel() for t in parts])
    inside = [i for i in range(100) if s.touch(at + 4 * i, 4)]
    assert inside == list(range(10, 30)) + list(range(60, 80))
    assert s.touch(at + 36, 8) and not s.touch(at + 32, 8)  # an 8-byte counter across the edge
    assert s.touch(at + 4 * 29, 8) and not s.touch(at + 120, 8)
    assert s.touch(at + 38, 4) and not s.touch(at + 36, 4)
    assert not multi._Spans([], []).touch(at, 4) and not multi._Spans([0, 0], [0, 0]).touch(at, 4)
    assert s.touch(at, 400)
