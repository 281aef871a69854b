"""The join between two blocks in float64 (NumPy), with its gradient (test infrastructure).

Parity: pinned (gradients by differences of the forward form).
"""
import numpy as np


def norm(z, kind, gamma, beta, eps):
    """(N(z), mean, rstd) over the rows of z."""
    z = np.asarray(z, dtype=np.float64)
    rows, n = z.shape
    if kind == "none":
        return z, np.zeros(rows), np.ones(rows)
    mean = z.mean(axis=1) if kind == "layer" else np.zeros(rows)
    d = z - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(axis=1) / n + eps)
    return d * rstd[:, None] * gamma + beta, mean, rstd


def norm_backward(dy, z, kind, gamma, mean, rstd):
    """(dz, dgamma, dbeta)"""
    if kind == "none":
        return dy, None, None
    n = z.shape[1]
    xh = (z - mean[:, None]) * rstd[:, None]
    q = dy * gamma
    d = q - xh * ((q * xh).sum(axis=1) / n)[:, None]
    if kind == "layer":
        d = d - (q.sum(axis=1) / n)[:, None]
    return d * rstd[:, None], (dy * xh).sum(axis=0), dy.sum(axis=0)


def forward(x, b, gate, xs, bs, post, pre, eps):
    """(r, h, (mean, rstd) of both norms); post, pre: (kind, gamma, beta)."""
    u, m1, s1 = norm(b, *post, eps)
    r = xs * np.asarray(x, np.float64) + bs * gate * u
    h, m2, s2 = norm(r, *pre, eps)
    return r, h, (m1, s1, m2, s2)


def backward(dh, dr, b, r, stats, gate, xs, bs, post, pre):
    """(dx, db, dgate per element, dgamma1, dbeta1, dgamma2, dbeta2)"""
    m1, s1, m2, s2 = stats
    g2 = b2 = None
    d = np.zeros_like(b) if dr is None else dr
    if pre[0] != "none":
        t, g2, b2 = norm_backward(dh, r, pre[0], pre[1], m2, s2)
        d = d + t
    kind, gamma, beta = post
    u = b if kind == "none" else (b - m1[:, None]) * s1[:, None] * gamma + beta
    du = bs * gate * d
    db, g1, b1 = norm_backward(du, b, kind, gamma, m1, s1)
    return xs * d, db, bs * d * u, g1, b1, g2, b2
