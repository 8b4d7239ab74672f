"""Tokens sorted by expert and back, pair by pair in Python integers and float64.

Pair t * topk + j of expert_idx [tokens, topk] goes to expert idx (outside [0, experts): to
none). An expert's rows keep the pairs' order and are padded to a multiple of ``multiple``.

Bounds (U = 2^-24): a token's sum over its choices is a chain of topk products and additions;
the dot product of a row runs over lanes that each add cols / 256 pieces of at most 8 elements,
6 steps of a wave and 4 waves.
"""
import numpy as np

U = 2.0 ** -24


def rows_of(tokens, topk, experts, multiple):
    """Rows that hold any routing: the worst case is found by trying the number of experts
    that get a pair, each with one row more than a whole multiple where pairs last."""
    n = tokens * topk
    best = 0
    for used in range(1, min(experts, n) + 1):
        # `used` experts with one pair each; the remaining pairs fill whole multiples
        best = max(best, (used + (n - used) // multiple) * multiple)
    return best


def sort(expert_idx, experts, multiple, rows):
    idx = np.asarray(expert_idx)
    bins = [[] for _ in range(experts)]
    for i, e in enumerate(idx.reshape(-1).tolist()):
        if 0 <= e < experts:
            bins[e].append(i)
    slot = np.full(idx.size, -1, np.int32)
    source = np.full(rows, -1, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    at = 0
    for e, b in enumerate(bins):
        for r, i in enumerate(b):
            slot[i] = at + r
            source[at + r] = i
        at += (len(b) + multiple - 1) // multiple * multiple
        offsets[e + 1] = at
    return (slot.reshape(idx.shape), source, np.array([len(b) for b in bins], np.int32), offsets)


def _kept(slot):
    for t in range(slot.shape[0]):
        for j in range(slot.shape[1]):
            if slot[t, j] >= 0:
                yield t, j, int(slot[t, j])


def dispatch(x, slot, rows):
    xs = np.zeros((rows, x.shape[1]), x.dtype)
    for t, _, r in _kept(slot):
        xs[r] = x[t]
    return xs


def combine(ys, slot, weights):
    """(y, bound before the last rounding); weights None: 1."""
    ys = np.asarray(ys, np.float64)
    y = np.zeros((slot.shape[0], ys.shape[1]))
    mag = np.zeros_like(y)
    for t, j, r in _kept(slot):
        v = ys[r] if weights is None else float(weights[t, j]) * ys[r]
        y[t] += v
        mag[t] += np.abs(v)
    return y, (slot.shape[1] + 1) * U * mag


def combine_bwd(dy, ys, slot, weights, rows):
    """(dys, dw, bound of dw)."""
    dy, ys = np.asarray(dy, np.float64), np.asarray(ys, np.float64)
    cols = dy.shape[1]
    dys, dw, mag = np.zeros((rows, cols)), np.zeros(slot.shape), np.zeros(slot.shape)
    for t, j, r in _kept(slot):
        dys[r] = float(weights[t, j]) * dy[t]
        dw[t, j] = (dy[t] * ys[r]).sum()
        mag[t, j] = np.abs(dy[t] * ys[r]).sum()
    return dys, dw, (8 * np.ceil(cols / 256) + 24) * U * mag + 1e-30
