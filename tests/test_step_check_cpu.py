"""muon_step's checks alone (host only): the statuses that muon_step itself gives for the
same arguments, on addresses that are never dereferenced."""
import ctypes

import pytest

from matrix_orthogonalising_optimizer_02_amd import binding as B

from test_abi_cpu import fake_only, lib  # noqa: F401

BASE, GIB = 1 << 40, 1 << 30


def matrix(i=0, **over):
    p = BASE + 8 * i * GIB
    f = dict(rows=96, cols=64, w=p, m=p + GIB, g=p + 2 * GIB)
    f.update(over)
    return B.MuonMatrix(*f.values())


def both(lib, mats, step=0, hp=None, ws=BASE + 900 * GIB, bytes_=GIB, rms=None, count=None):  # noqa: F811
    """(the check's status, the step's) for arguments that the step refuses."""
    arr = (B.MuonMatrix * max(len(mats), 1))(*mats)
    n, h = len(mats) if count is None else count, hp if hp is not None else B.default_hparams()
    check = lib.muon_step_check(arr, n, h, step, ws, bytes_, rms)
    return check, lib.muon_step(arr, n, h, step, ws, bytes_, rms, None) if check != B.MUON_OK else None


@fake_only
@pytest.mark.parametrize("step", [0, 1, 3, 4])  # refresh steps and RowNorm steps
def test_the_check_refuses_what_the_step_refuses(lib, step):  # noqa: F811
    bad = [(dict(mats=[matrix(0), matrix(1, rows=-1)]), B.MUON_ERR_INVALID_ARG),
           (dict(mats=[matrix(0, g=None)]), B.MUON_ERR_INVALID_ARG),
           (dict(mats=[matrix(0)], count=-1), B.MUON_ERR_INVALID_ARG),
           (dict(mats=[matrix(0, g=BASE + 2 * GIB + 4)]), B.MUON_ERR_ALIGN),
           (dict(mats=[matrix(0)], rms=BASE + 700 * GIB + 2), B.MUON_ERR_ALIGN),
           (dict(mats=[matrix(0)], ws=BASE + 900 * GIB + 16), B.MUON_ERR_ALIGN),
           (dict(mats=[matrix(0, rows=(1 << 30) + 1)]), B.MUON_ERR_TOO_LARGE),
           (dict(mats=[matrix(0)], ws=None), B.MUON_ERR_WORKSPACE),
           (dict(mats=[matrix(0)], bytes_=256), B.MUON_ERR_WORKSPACE),
           (dict(mats=[matrix(0), matrix(0)]), B.MUON_ERR_ALIAS),
           (dict(mats=[matrix(0, g=BASE + GIB)]), B.MUON_ERR_ALIAS),
           (dict(mats=[matrix(0)], rms=BASE + 64), B.MUON_ERR_ALIAS),
           (dict(mats=[matrix(0)], hp=B.default_hparams(eps=0.0)), B.MUON_ERR_INVALID_ARG),
           (dict(mats=[matrix(0)], hp=B.default_hparams(period_k=0)), B.MUON_ERR_INVALID_ARG),
           (dict(mats=[matrix(0)], hp=B.default_hparams(ns_steps=0)), B.MUON_ERR_INVALID_ARG)]
    for args, status in bad:
        assert both(lib, step=step, **args) == (status, status), (args.keys(), status)
    assert both(lib, [matrix(0)], step=-1) == (B.MUON_ERR_INVALID_ARG,) * 2
    assert lib.muon_step_check((B.MuonMatrix * 1)(matrix(0)), 1, None, step, BASE + 900 * GIB, GIB, None) == B.MUON_ERR_INVALID_ARG


@fake_only
def test_the_check_passes_what_is_whole(lib):  # noqa: F811
    assert both(lib, [matrix(0), matrix(1)])[0] == B.MUON_OK
    assert both(lib, [matrix(0)], step=4, rms=BASE + 700 * GIB)[0] == B.MUON_OK
    assert both(lib, [], ws=None, bytes_=0)[0] == B.MUON_OK
    need = ctypes.c_size_t()
    shape = (ctypes.c_int64 * 1)(96), (ctypes.c_int64 * 1)(64)
    assert lib.muon_workspace_bytes(*shape, 1, need) == B.MUON_OK
    assert both(lib, [matrix(0)], bytes_=need.value)[0] == B.MUON_OK
    assert both(lib, [matrix(0)], bytes_=need.value - 1)[0] == B.MUON_ERR_WORKSPACE
