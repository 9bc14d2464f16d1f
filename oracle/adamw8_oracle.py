"""Plain float64 CPU oracle for AdamW with 8-bit states, and for the gradient norm.

TEST INFRASTRUCTURE ONLY: it shares no code with the HIP library.

A state of 8 bits holds e4m3 codes with a scale for every 256 consecutive elements: the
first moment m = scale code, the square root of the second u = scale code. The step runs
on these values (oracle.adamw_oracle's formula); each block's new scale is its largest
magnitude / 448, and a magnitude between two codes goes up where its fraction plus 16
random bits / 2^16 reaches 1. The bits are a hash of (seed, step, tensor, element).
"""
from __future__ import annotations

import numpy as np

from .adamw_oracle import AdamWHParams, adamw_step

BLOCK = 256
E4M3_MAX = 448.0


def decode(codes):
    """float64 values of e4m3 codes (uint8): bias 7, 3 mantissa bits, 0x7F and 0xFF NaN."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    exp, man = (c >> 3) & 15, c & 7
    mag = np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c & 128, -mag, mag)


VALUES = decode(np.arange(127))  # ascending, 0 .. 448


def mix(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x6A09E667)) & m
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85)) & m
    return x ^ (x >> np.uint64(16))


def rounding_bits(seed, step, tensor, index):
    """(bits for m, bits for u), 16 each, for an array of element indices."""
    m = 0xFFFFFFFF
    key = int(mix((int(mix((int(mix(seed & m)) + (seed >> 32)) & m)) + step) & m))
    key = int(mix((key + tensor * 0x510E527F) & m))
    index = np.asarray(index, np.uint64)
    with np.errstate(over="ignore"):
        x = (index & np.uint64(m)) * np.uint64(0x9E3779B9) + (index >> np.uint64(32)) * np.uint64(0x510E527F) \
            + np.uint64(key)
    bits = mix(x)
    return (bits & np.uint64(0xFFFF)).astype(np.int64), (bits >> np.uint64(16)).astype(np.int64)


def block_scales(x):
    """Each block's largest magnitude / 448; 0 below 1e-30, NaN where one is not finite."""
    pad = np.pad(np.abs(np.asarray(x, np.float64)).ravel(), (0, -np.size(x) % BLOCK)).reshape(-1, BLOCK)
    top = pad.max(1)
    return np.where(np.isfinite(top), np.where(top < 1e-30, 0.0, top / E4M3_MAX), np.nan)


def candidates(x, scales):
    """(lower code, upper code, fraction) of |x| / scale for finite, nonzero scales."""
    s = np.repeat(scales, BLOCK)[:np.size(x)]
    a = np.divide(np.abs(x), s, out=np.zeros(np.size(x)), where=s > 0)
    a = np.minimum(a, E4M3_MAX)
    lo = np.clip(np.searchsorted(VALUES, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    gap = VALUES[hi] - VALUES[lo]
    return lo, hi, np.divide(a - VALUES[lo], gap, out=np.zeros_like(a), where=gap > 0)


def adamw8_step(w, g, m_codes, m_scale, v_codes, v_scale, step, hp=AdamWHParams()):
    """(W, m, u): the new weight, and both states before their rounding, in float64."""
    n = np.size(w)
    m = decode(m_codes) * np.repeat(np.asarray(m_scale, np.float64), BLOCK)[:n]
    u = decode(v_codes) * np.repeat(np.asarray(v_scale, np.float64), BLOCK)[:n]
    w, m, v = adamw_step(np.ravel(w), np.ravel(g), m, u * u, step, hp)
    return w, m, np.sqrt(v)


def grad_norm(grads, max_norm):
    """(norm of each, total, clip factor)."""
    norms = np.array([np.sqrt(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads])
    total = float(np.sqrt(np.sum(norms ** 2)))
    return norms, total, min(1.0, max_norm / (total + 1e-6))
