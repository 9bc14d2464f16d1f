"""Rotary positions' checks of their arguments, on the CPU."""
import pytest

import matrix_orthogonalising_optimizer_02_amd as muon

torch = pytest.importorskip("torch")


def test_rotary_takes_tensors():
    axes = muon.RotaryAxes((2,), device="cpu")
    for x, positions in ((torch.zeros(4, 1, 8), [0, 1, 2, 3]), (torch.zeros(4, 1, 8), None), ([0.0], torch.zeros(4, 1))):
        for call in (muon.rotary, muon.rotary_apply):
            with pytest.raises(TypeError):
                call(x, positions, axes)
