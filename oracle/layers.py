"""Layer norm, the linear layer and 8-bit checkpoints in float64 (NumPy).

Written from the formulas, one statement per equation; the activations' tails go
through the complementary error function, so they keep their relative accuracy.
"""
import math

import numpy as np
from scipy.special import erfc

GELU_C = math.sqrt(2.0 / math.pi)
BLOCK = 32


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return z * 0.5 * erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * _sigmoid(2.0 * GELU_C * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * _sigmoid(z)
    return z


def act_slope(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * erfc(-z / math.sqrt(2.0)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        u = 2.0 * GELU_C * (z + 0.044715 * z ** 3)
        s = _sigmoid(u)
        return s + z * s * _sigmoid(-u) * 2.0 * GELU_C * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = _sigmoid(z)
        return s + z * s * _sigmoid(-z)
    return np.ones_like(z)


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) over the rows of x."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    return d * rstd[:, None] * gamma + beta, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta)"""
    dy = np.asarray(dy, dtype=np.float64)
    xh = (np.asarray(x, dtype=np.float64) - mean[:, None]) * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True)
                          - xh * (g * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def linear(x, w, bias, kind="none", residual=0.0):
    """(y, z)"""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T + bias
    return act(z, kind) + residual, z


def linear_backward_input(dy, w, kind="none", z=0.0):
    return (np.asarray(dy, np.float64) @ np.asarray(w, np.float64)) * act_slope(z, kind)


def linear_backward_weight(dy, x, kind="none"):
    dy = np.asarray(dy, np.float64)
    return dy.T @ act(x, kind), dy.sum(axis=0)


# magnitudes an e4m3 code can stand for: k / 8 * 2^-6 (k < 8), (1 + k / 8) 2^e
E4M3 = np.array([k / 8.0 * 2.0 ** -6 for k in range(8)]
                + [(1 + k / 8.0) * 2.0 ** e for e in range(-6, 9) for k in range(8)][:-1])


def _nearest_e4m3(a):
    """Nearest representable magnitude, ties to the even code."""
    hi = np.clip(np.searchsorted(E4M3, a), 1, len(E4M3) - 1)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(take_hi, E4M3[hi], E4M3[lo])


def q8_values(x, fmt):
    """The float64 values an 8-bit checkpoint of x stands for: per row and 32
    columns, the smallest power-of-two scale (at least 2^-126; 2^-124 for e4m3,
    so that its smallest step is a bf16 number) for which the block's largest
    magnitude, rounded, stays in range. A block with a NaN or an
    infinity is NaN."""
    x = np.asarray(x, dtype=np.float64)
    out = np.empty_like(x)
    most = 127.0 if fmt == "int8" else 448.0
    for i in range(x.shape[0]):
        for b in range(0, x.shape[1], BLOCK):
            v = x[i, b:b + BLOCK]
            top = np.abs(v).max()
            if not np.isfinite(top):
                out[i, b:b + BLOCK] = np.nan
                continue
            if top == 0:
                out[i, b:b + BLOCK] = 0.0
                continue
            e = max(-126 if fmt == "int8" else -124, math.frexp(top)[1] - 12)
            while True:
                a = np.abs(v) / 2.0 ** e
                # past the range a code would round to the next one up
                r = np.rint(a) if fmt == "int8" else np.where(
                    a > 464.0, 512.0, _nearest_e4m3(np.minimum(a, 448.0)))
                if r.max() <= most:
                    break
                e += 1
            out[i, b:b + BLOCK] = np.copysign(r, v) * 2.0 ** e
    return out
