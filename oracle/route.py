"""The router of an expert block in float64: softmax, topk choices, counts, losses, gradient.

Bounds (U = 2^-24, one float32 rounding; the hardware's exponential, logarithm and reciprocal
are within 2 of them): an exponential exp(d) is taken as 2^(d log2 e), whose argument carries
the roundings of d, of log2 e and of the product, 3 |d| U together; with D the row's range of
finite logits a softmax term is off by at most (3 D + 4) U, a sum of them over the experts by
that and a rounding for each of at most 20 steps, the quotient by both and 4 more.
"""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -120          # products of small exponentials may leave float32's normal range


def forward(logits, topk, normalize=True, valid=None):
    """(idx, weights, lse, counts, losses, p) of float64 logits [tokens, experts]."""
    x = np.asarray(logits, np.float64)
    tokens, experts = x.shape
    valid = tokens if valid is None else valid
    idx = np.full((tokens, topk), -1, np.int64)
    w = np.zeros((tokens, topk))
    lse = np.zeros(tokens)
    p = np.zeros((tokens, experts))
    for t in range(valid):
        row = x[t]
        live = row > -np.inf
        if not live.any():
            lse[t] = -np.inf
            continue
        top = row.max()
        ex = np.where(live, np.exp(row - top), 0.0)
        p[t] = ex / ex.sum()
        lse[t] = top + np.log(ex.sum())
        order = sorted(np.flatnonzero(live).tolist(), key=lambda e: (-row[e], e))[:topk]
        idx[t, :len(order)] = order
        w[t, :len(order)] = p[t, order]
        if normalize:
            v = np.exp(row[order] - row[order[0]])
            w[t, :len(order)] = v / v.sum()
    counts = np.bincount(idx[idx >= 0].ravel(), minlength=experts)
    losses = np.zeros(2)
    if valid:
        losses[0] = experts / (valid * topk) * (counts * p[:valid].sum(0)).sum() / valid
        finite = np.where(np.isfinite(lse[:valid]), lse[:valid], 0.0)
        losses[1] = (finite ** 2).sum() / valid
    return idx, w, lse, counts, losses, p


def spread(logits):
    """The largest range of a row's finite logits."""
    x = np.asarray(logits, np.float64)
    hi = np.where(np.isfinite(x), x, -np.inf).max(1, initial=-np.inf)
    lo = np.where(np.isfinite(x), x, np.inf).min(1, initial=np.inf)
    ok = np.isfinite(hi) & np.isfinite(lo)
    return float((hi - lo)[ok].max()) if ok.any() else 0.0


def forward_bounds(logits, weights, lse, losses):
    d = spread(logits)
    tokens = np.asarray(logits).shape[0]
    term = (3 * d + 4) * U
    w = weights * (2 * term + 24 * U) + TINY
    # top + log(total): the total's own relative error, the logarithm's and the addition's
    finite = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    l = term + 24 * U + 8 * U + 2 * U * (finite + np.log(512.0))
    # a lane adds its tokens one by one, then lanes, waves and workgroups
    adds = tokens / 16 + 300
    b = losses[0] * (2 * term + (30 + adds) * U) + TINY
    z = losses[1] * (adds + 10) * U + 2 * float((finite * l).max(initial=0.0)) + TINY
    return w, l, np.array([b, z])


def backward(logits, lse, idx, weights, counts, dweights, dlosses, normalize=True, valid=None):
    """(dlogits, magnitude of the sums it is made of)."""
    x = np.asarray(logits, np.float64)
    tokens, experts = x.shape
    topk = idx.shape[1]
    valid = tokens if valid is None else valid
    d, mag = np.zeros_like(x), np.zeros_like(x)
    if not valid:
        return d, mag
    db, dz = (0.0, 0.0) if dlosses is None else (float(v) for v in dlosses)
    A, B = db * experts / (valid ** 2 * topk), dz * 2 / valid
    c = np.asarray(counts, np.float64)
    for t in range(valid):
        if lse[t] == -np.inf:
            continue
        p = np.exp(x[t] - lse[t])
        pc = (p * c).sum()
        d[t] = p * (A * (c - pc) + B * lse[t])
        mag[t] = p * (abs(A) * (c + pc) + abs(B * lse[t]))
        if dweights is None:
            continue
        kept = [j for j in range(topk) if idx[t, j] >= 0]
        dot = sum(weights[t, j] * dweights[t, j] for j in kept)
        dabs = sum(abs(weights[t, j] * dweights[t, j]) for j in kept)
        if not normalize:
            d[t] -= p * dot
            mag[t] += p * dabs
        for j in kept:
            e = idx[t, j]
            d[t, e] += weights[t, j] * (dweights[t, j] - (dot if normalize else 0.0))
            mag[t, e] += weights[t, j] * (abs(dweights[t, j]) + (dabs if normalize else 0.0))
    return d, mag


def backward_bound(logits, lse, d, mag, half, tiny):
    """``half``: half a step of the output type, relative; ``tiny``: half its smallest step."""
    x = np.asarray(logits, np.float64)
    away = np.abs(np.where(np.isfinite(x), x, 0.0) - np.where(np.isfinite(lse), lse, 0.0)[:, None])
    far = float(np.where(np.isfinite(x), away, 0.0).max(initial=0.0))
    err = mag * (3 * far + 90) * U + TINY
    return err + half * (np.abs(d) + err) + tiny
