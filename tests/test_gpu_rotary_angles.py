"""Rotary positions: sines and cosines that are small, where the rounding of an angle shows.

With p = 1 and q = 0 the result is the cosine and the sine. fp32 sines and cosines are off by two
units in the last place, 4 2^-24 of them, and the last addition by 2^-24; the angle itself is exact
to 2^-52 of a turn, below 2^-30 of the smallest value here.
"""
import numpy as np
import pytest

import matrix_orthogonalising_optimizer_02_amd as muon
from test_gpu_blocks8 import torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["halves", "adjacent"])
@pytest.mark.parametrize("inverse", [False, True])
def test_small_sines_and_cosines(torch_dev, layout, inverse):  # noqa: F811
    torch, dev = torch_dev
    off = np.concatenate((np.geomspace(1e-6, 0.4, 40), np.linspace(0.01, 0.49, 50)))
    turns = np.concatenate((0.5 - off / np.pi, 0.25 - off / (2 * np.pi), -0.25 + off / (3 * np.pi), 0.75 + off / 9))
    n = len(turns)
    axes = muon.RotaryAxes((n,), frequencies=2 * np.pi * turns, layout=layout, device=dev)
    x = torch.zeros(1, 1, 2 * n, device=dev)
    x[..., (slice(0, n) if layout == "halves" else slice(0, 2 * n, 2))] = 1.0
    y = muon.rotary_apply(x, torch.ones(1, 1, dtype=torch.int32, device=dev), axes, inverse=inverse)[0, 0].double().cpu().numpy()
    cos, sin = (y[:n], y[n:]) if layout == "halves" else (y[::2], y[1::2])
    # by the distance from the nearest quarter turn, so that nothing cancels
    quarter = np.rint(4 * turns)
    rest = 2 * np.pi * (turns - quarter / 4)
    c, s = np.cos(rest), np.sin(rest)
    q = quarter.astype(int) % 4
    want_c = np.choose(q, (c, -s, -c, s))
    want_s = np.choose(q, (s, c, -s, -c)) * (-1.0 if inverse else 1.0)
    for got, want in ((cos, want_c), (sin, want_s)):
        assert (np.abs(got - want) <= 5 * 2.0 ** -24 * np.abs(want)).all(), float(np.max(np.abs(got - want) / np.abs(want)) * 2.0 ** 24)
