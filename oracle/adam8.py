"""AdamW with 8-bit states, fp64 (oracle; test infrastructure).

A state holds m and r = sqrt(v), 256 elements to a scale: value = scale * F(code), F a
float with a 4-bit exponent (bias 15, subnormals) and a mantissa of 3 bits (m, and a sign
in the top bit) or 4 bits (r). The scale makes the largest magnitude of the 256 the
largest code. A magnitude y is stored as floor(its place on the code axis + dither), the
dither of element i at step t being the top bits of (a i + b t) mod 2^32.

Parity: pinned (codes enumerated; rounding of a constant averaged over the steps).
"""
from __future__ import annotations

import numpy as np

SPAN = 256
MANTISSA = {"m": 3, "v": 4}
DITHER = {"m": (0x9E3779B9, 0xC13FA9A9), "v": (0xC13FA9A9, 0x9E3779B9)}


def code_value(code, which):
    """F of magnitude codes (no sign bit)."""
    code = np.asarray(code, dtype=np.int64)
    k = MANTISSA[which]
    e, f = code >> k, (code & ((1 << k) - 1)) / 2.0 ** k
    return np.where(e == 0, f * 2.0 ** -14, 2.0 ** (e - 15.0) * (1.0 + f))


def decode(codes, scales, which):
    """m, or r."""
    codes = np.asarray(codes, dtype=np.int64).ravel()
    s = np.repeat(np.asarray(scales, dtype=np.float64), SPAN)[:codes.size]
    if which == "m":
        return np.where(codes > 127, -1.0, 1.0) * code_value(codes & 127, "m") * s
    return code_value(codes, "v") * s


def dither(n, which, t):
    """The dithers of n elements at step t, in [0, 1)."""
    a, b = DITHER[which]
    cut = 32 - 23 + MANTISSA[which]
    d = (np.arange(n, dtype=object) * a + t * b) % (1 << 32)
    return np.array([int(x) >> cut for x in d], dtype=np.float64) * 0.5 ** (32 - cut)


def places(x, which, t):
    """(place of |x| on the code axis plus its dither, scales)."""
    x = np.abs(np.asarray(x, dtype=np.float64).ravel())
    n, k = x.size, MANTISSA[which]
    pad = np.zeros((n + SPAN - 1) // SPAN * SPAN)
    pad[:n] = x
    largest = pad.reshape(-1, SPAN).max(axis=1)
    scales = largest / (2.0 - 0.5 ** k)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.nan_to_num(x / np.repeat(scales, SPAN)[:n])
        e = np.maximum(np.floor(np.log2(y)), -14.0)
    return (e + 14.0) * (1 << k) + y * 2.0 ** (k - e) + dither(n, which, t), scales


def encode(x, which, t):
    """(codes, scales)"""
    x = np.asarray(x, dtype=np.float64).ravel()
    p, scales = places(x, which, t)
    code = np.floor(p).astype(np.int64)
    if which == "m":
        return np.where(x < 0, 128, 0) + np.minimum(code, 127), scales
    return np.where(x > 0, np.clip(code, 1, 255), 0), scales
