"""Plain float64 CPU oracle for the normalisation layers and their gradients.

TEST INFRASTRUCTURE ONLY: it shares no code with the HIP library.

For a row x of H elements in group g (rows / groups consecutive rows a group):
  mean = sum x / H (0 for rms), rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),
  h = (x - mean) rstd, y = h (offset + w[g]) + b[g];
  a = dy (offset + w[g]), dx = rstd (a - mean(a) - h mean(a h)) (rms: without mean(a)),
  dw[g] = sum of dy h, db[g] = sum of dy.
Besides the values, each function gives the sums of magnitudes that bound what rounding
can do to them.
"""
from __future__ import annotations

import numpy as np


def _split(x, groups):
    x = np.asarray(x, np.float64)
    return x.reshape(groups, -1, x.shape[-1])


def norm_forward(x, w=None, b=None, kind="layer", eps=1e-6, offset=0.0, groups=1):
    """(y, mean, rstd, h, scale): scale is the factor offset + w, per row."""
    x = _split(x, groups)
    mean = x.mean(2) if kind == "layer" else np.zeros(x.shape[:2])
    d = x - mean[..., None]
    rstd = 1.0 / np.sqrt((d * d).mean(2) + eps)
    h = d * rstd[..., None]
    scale = np.ones((groups, 1, x.shape[2])) if w is None else offset + _split(w, groups)
    y = h * scale
    if b is not None:
        y = y + _split(b, groups)
    return y, mean, rstd, h, scale


def norm_backward(dy, x, w, mean, rstd, kind="layer", offset=0.0, groups=1):
    """(dx, dw, db, h, a) from given statistics."""
    dy, x = _split(dy, groups), _split(x, groups)
    rstd = np.asarray(rstd, np.float64).reshape(groups, -1, 1)
    d = x if kind == "rms" else x - np.asarray(mean, np.float64).reshape(groups, -1, 1)
    h = d * rstd
    a = dy * (1.0 if w is None else offset + _split(w, groups))
    dx = a - h * (a * h).mean(2, keepdims=True)
    if kind == "layer":
        dx = dx - a.mean(2, keepdims=True)
    return rstd * dx, (dy * h).sum(1), dy.sum(1), h, a
