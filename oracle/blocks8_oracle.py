"""Plain float64 CPU oracle for matrices in 8 bits with a power of two for every 128 elements.

TEST INFRASTRUCTURE ONLY: it shares no code with the HIP library.

A block (1 x 128 elements along a row, or 128 x 128) has the least power 2^e, e >= -127, with
max |x| <= 448 2^e over its finite elements; an element becomes the nearest e4m3 value (3
mantissa bits, exponents -6 .. 8, subnormals of 2^-9, largest 448, ties to even) of x 2^-e;
infinities and NaN become NaN.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_values():
    """The 256 codes' values, by the bits' meaning."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 128 else v
    return out


def round_e4m3(x):
    """x (|x| <= 448) on the grid of e4m3, ties to even."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(x), where=x != 0, out=np.full(x.shape, -6.0))), -6.0)
    step = 2.0 ** (e - 3)
    with np.errstate(invalid="ignore"):
        return np.rint(x / step) * step


def powers(x, tiles=False):
    """The exponents e [rows or row blocks, column blocks]."""
    rows, cols = x.shape
    high = BLOCK if tiles else 1
    mag = np.abs(np.asarray(x, np.float64))
    mag = np.where(np.isfinite(mag), mag, 0.0)
    mag = np.pad(mag, ((0, -rows % high), (0, -cols % BLOCK)))
    top = mag.reshape(mag.shape[0] // high, high, -1, BLOCK).max((1, 3))
    e = np.full(top.shape, -127)
    for at in np.ndindex(top.shape):
        if top[at] > 0:
            m, f = np.frexp(top[at] / 448.0)
            e[at] = max(-127, int(f) - (m == 0.5))
    return e


def spread(e, shape, tiles=False):
    """Exponents of each element."""
    s = np.repeat(e, BLOCK, 1)
    if tiles:
        s = np.repeat(s, BLOCK, 0)
    return s[:shape[0], :shape[1]]


def quantise(x, tiles=False):
    """(values, exponents): what the codes stand for, in float64."""
    x = np.asarray(x, np.float64)
    e = powers(x, tiles)
    s = 2.0 ** spread(e, x.shape, tiles).astype(np.float64)
    v = round_e4m3(np.where(np.isfinite(x), x, 0.0) / s) * s
    return np.where(np.isfinite(x), v, np.nan), e
