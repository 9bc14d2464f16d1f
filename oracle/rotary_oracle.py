"""Plain float64 CPU oracle for rotary positions over several axes.

TEST INFRASTRUCTURE ONLY: it shares no code with the HIP library.
"""
from __future__ import annotations

import numpy as np


def ladder(sections, base=10000.0):
    """(radians per unit of position, axis) of every pair: base^(-i / n) for pair i of n."""
    freq = [base ** (-i / n) for n in sections for i in range(n)]
    return np.array(freq), np.array([a for a, n in enumerate(sections) for _ in range(n)])


def rotate(x, positions, freq, axis, layout="halves", inverse=False):
    """x [..., heads, dim], positions [..., axes]."""
    x, pos = np.asarray(x, np.float64), np.asarray(positions, np.float64)
    n = len(freq)
    angle = (pos[..., axis] * freq)[..., None, :]
    c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
    first, second = (np.arange(n), np.arange(n) + n) if layout == "halves" else (2 * np.arange(n), 2 * np.arange(n) + 1)
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., first] * s + x[..., second] * c
    return y
