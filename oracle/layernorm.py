"""Layer norm and its gradient in float64, and how far a float32 computation may be off.

    mean = sum_c x / cols, var = sum_c (x - mean)^2 / cols, rstd = 1 / sqrt(var + eps)
    y = (x - mean) rstd gamma + beta
    xh = (x - mean) rstd, g = dy gamma
    dx = rstd (g - mean_c(g) - xh mean_c(g xh)); dgamma = sum_r dy xh; dbeta = sum_r dy

Bounds. U = 2^-24 is half a step of float32. A sum whose longest chain of additions is D
terms is off by at most D U times the sum of the absolute values (first order); the kernel's
chains are a lane's elements (at most 32), the lanes of a wave (6 steps) and the waves of a
row (at most 16), so D = 64 covers a row sum with the roundings of its terms. The sums over
rows split the rows over lanes and workgroups; their D grows slowly with the rows. The stored
value is rounded once to its type: half a step relative to the value, ``half``, but never less
than half the type's smallest subnormal, ``tiny`` (float16: 2^-25, which is what counts below
2^-14; float32 and bfloat16 have theirs below 1e-39).
"""
import numpy as np

U = 2.0 ** -24
ROW_CHAIN = 64


def col_chain(rows):
    """Longest chain of additions of a sum over rows."""
    return 128 + rows / 256


def forward(x, gamma, beta, eps):
    """(y, mean, rstd) in float64; gamma, beta [cols] or None."""
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    mean = x.sum(1) / n
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(1) / n + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def forward_bounds(x, gamma, beta, eps, half, tiny=0.0):
    """Bounds of (y, mean, rstd); half, tiny: y's type."""
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    y, mean, rstd = forward(x, gamma, beta, eps)
    g = np.ones(n) if gamma is None else np.abs(gamma)
    b = np.zeros(n) if beta is None else np.abs(beta)
    e_mean = (ROW_CHAIN + 2) * U * np.abs(x).sum(1) / n
    d = np.abs(x - mean[:, None])
    e_var = ((ROW_CHAIN + 4) * U * (d * d).sum(1) + 2 * e_mean * d.sum(1)) / n + e_mean ** 2
    rel = 0.5 * e_var * rstd ** 2 + 4 * U                   # of rstd, first order
    rel = np.minimum(rel * 1.01 + rel * rel, 1e300)
    e_y = (g[None, :] * rstd[:, None] * (e_mean[:, None] + U * d)
           + g[None, :] * d * (rstd * (rel + 3 * U))[:, None] + U * (np.abs(y) + b[None, :]))
    return (e_y * (1 + 2 * half) + half * np.abs(y) + tiny + 1e-30, e_mean + U * np.abs(mean),
            rel * rstd)


def backward(dy, x, mean, rstd, gamma):
    """(dx, dgamma, dbeta) in float64 from the statistics that the forward kept."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    n = x.shape[1]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy if gamma is None else dy * gamma
    m1, m2 = g.sum(1, keepdims=True) / n, (g * xh).sum(1, keepdims=True) / n
    dx = np.asarray(rstd, np.float64)[:, None] * (g - m1 - xh * m2)
    return dx, (dy * xh).sum(0), dy.sum(0)


def backward_bounds(dy, x, mean, rstd, gamma, half, half_p, tiny=0.0, tiny_p=0.0):
    """Bounds of (dx, dgamma, dbeta); half, tiny: dx's type, half_p, tiny_p: the parameters'."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rows, n = x.shape
    rs = np.asarray(rstd, np.float64)[:, None]
    xh = np.abs((x - np.asarray(mean, np.float64)[:, None]) * rs)
    g = np.abs(dy if gamma is None else dy * gamma)
    dx, dgamma, dbeta = backward(dy, x, mean, rstd, gamma)
    e1 = (ROW_CHAIN + 3) * U * g.sum(1, keepdims=True) / n
    e2 = (ROW_CHAIN + 6) * U * (g * xh).sum(1, keepdims=True) / n
    m1, m2 = g.sum(1, keepdims=True) / n, (g * xh).sum(1, keepdims=True) / n
    e = np.abs(rs) * (4 * U * g + e1 + 3 * U * m1 + xh * e2 + 7 * U * xh * m2) + 2 * U * np.abs(dx)
    d = col_chain(rows)
    e_dg, e_db = (d + 3) * U * (np.abs(dy) * xh).sum(0), d * U * np.abs(dy).sum(0)
    return (e * (1 + 2 * half) + half * np.abs(dx) + tiny + 1e-30,
            e_dg * (1 + 2 * half_p) + half_p * np.abs(dgamma) + tiny_p + 1e-30,
            e_db * (1 + 2 * half_p) + half_p * np.abs(dbeta) + tiny_p + 1e-30)
