"""The activation between two linears in float64, its gradient, and what its 8-bit tiles stand
for.

Bounds (U = 2^-24): a value v of a tile with scale s is coded as the nearest e4m3 value to
v m, where m s is 1 up to 6 U (both factors within 2 units of 2 U, and the product's rounding):
the code times s is within half a step of v, 2^-4 |v| or, below the normal range (2^-6), 2^-10 s.
The logistic function of z carries the roundings of its argument, 4 of |z| each, and 8 more.
Where it is below 2^-126 (exp(-z) leaves float32, or its reciprocal would be subnormal, which the
hardware flushes) it may be taken as 0: it is then off by its whole value, less than 2^-126, and
act by |x| times that, act' = s (1 + x (1 - s) z') by at most (1 + |x z'|) times that.
"""
import numpy as np

U = 2.0 ** -24
FLUSH = 2.0 ** -126
ROOT = np.sqrt(2 / np.pi)
BLOCK, TOP, FLOOR = 128, 448.0, 1e-12


def argument(x, act):
    """What the logistic function is taken of."""
    return x if act == "silu" else 2 * ROOT * (x + 0.044715 * x ** 3) if act == "gelu" else 0 * x


def logistic(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def act(x, kind):
    return np.maximum(x, 0.0) if kind == "relu" else x * logistic(argument(x, kind))


def dact(x, kind):
    """(act', the magnitude of the terms it is added from, what a flushed logistic takes)."""
    if kind == "relu":
        return (x > 0) * 1.0, (x > 0) * 1.0, 0 * x
    s = logistic(argument(x, kind))
    dz = 1.0 if kind == "silu" else 2 * ROOT * (1 + 3 * 0.044715 * x * x)
    return s + x * s * (1 - s) * dz, s + np.abs(x * s * dz), FLUSH * (1 + np.abs(x * dz))


def rel(x, kind):
    """Relative error of act(x)."""
    return 0 * x if kind == "relu" else (8 * np.abs(argument(x, kind)) + 16) * U


def forward(h, kind, gated):
    """(a, bound of float32's errors in it)."""
    if not gated:
        a = act(h, kind)
        return a, np.abs(a) * rel(h, kind) + FLUSH * (1 + np.abs(h))
    c = h.shape[1] // 2
    a = act(h[:, :c], kind) * h[:, c:]
    flushed = FLUSH * (1 + np.abs(h[:, :c] * h[:, c:]))
    return a, np.abs(a) * (rel(h[:, :c], kind) + 2 * U) + flushed


def backward(da, h, kind, gated):
    """(dh, bound of float32's errors in it)."""
    c = da.shape[1]
    g = h[:, :c]
    d, mag, lost = dact(g, kind)
    far = (8 * np.abs(argument(g, kind)) + 40) * U
    if not gated:
        return da * d, np.abs(da) * (mag * far + lost) + FLUSH
    u = h[:, c:]
    return (np.concatenate([da * u * d, da * act(g, kind)], 1),
            np.concatenate([np.abs(da * u) * (mag * far + lost),
                            np.abs(da * act(g, kind)) * (rel(g, kind) + 6 * U)
                            + np.abs(da * g) * FLUSH], 1) + FLUSH)


def scales(v):
    """Scales of the 1x128 tiles along the rows of v."""
    m = np.abs(v).reshape(v.shape[0], -1, BLOCK).max(2)
    return np.maximum(m, FLOOR) / TOP


def scale_bound(v, err):
    """How far a tile's scale may be off, with ``err`` the bound of v."""
    return scales(v) * 8 * U + np.abs(err).reshape(v.shape[0], -1, BLOCK).max(2) / TOP * (1 + 1e-6)


def value_bound(v, err, scale):
    """How far code times scale may be from v."""
    s = np.repeat(scale, BLOCK, axis=1)
    return (np.abs(v) + err) * (2.0 ** -4 + 16 * U) + err + s * 2.0 ** -10 * (1 + 16 * U)
