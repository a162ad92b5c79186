"""CPU oracle for the balance loss, its counts and the gradient of the router's
logits, in float64.  TEST INFRASTRUCTURE ONLY: shares no code with the product
path.  Definitions: include/moe_balance.h; pinned by
tests/test_oracle_balance_pins.py (closed forms, differences).
"""
from __future__ import annotations

import numpy as np


def log_scores(x):
    """log sigmoid(x), exact to float64 in every range."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return np.where(x >= 0, -np.log1p(np.exp(-np.abs(x))), x - np.log1p(np.exp(-np.abs(x))))


def normalised(ls):
    """exp(ls) / sum over the last axis; zero where every entry is -infinity."""
    m = ls.max(axis=-1, keepdims=True) if ls.shape[-1] else np.zeros(ls.shape[:-1] + (1,))
    none = np.isneginf(m)
    with np.errstate(invalid="ignore"):
        z = np.exp(ls - np.where(none, 0.0, m))
    t = z.sum(axis=-1, keepdims=True)
    return np.where(none, 0.0, z / np.where(none, 1.0, t))


def sequences(M, seq_offsets, mask):
    off = [0, M] if seq_offsets is None else list(seq_offsets)
    live = np.ones(M, bool) if mask is None else np.asarray(mask) != 0
    for b in range(len(off) - 1):
        t = np.arange(off[b], off[b + 1])
        yield b, t[live[t]]


def balance(x, ids, coef, seq_offsets=None, mask=None):
    """(loss, counts [B, E], tokens [B + 1], shares [B, E])."""
    x = np.asarray(x, dtype=np.float64)
    (M, E), k = x.shape, ids.shape[1]
    B = 1 if seq_offsets is None else len(seq_offsets) - 1
    counts, tokens, shares = np.zeros((B, E), np.int64), np.zeros(B + 1, np.int64), np.zeros((B, E))
    total = 0.0
    for b, t in sequences(M, seq_offsets, mask):
        if t.size == 0:
            continue
        picks = ids[t].ravel()
        counts[b] = np.bincount(picks[(picks >= 0) & (picks < E)], minlength=E)
        tokens[b] = t.size
        shares[b] = normalised(log_scores(x[t])).mean(axis=0)
        total += E / (k * t.size) * (counts[b] * shares[b]).sum()
    tokens[B] = (tokens[:B] > 0).sum()
    return (coef * total / tokens[B] if tokens[B] else 0.0), counts, tokens, shares


def weights(x, ids):
    """Routing weights s / sum s over a token's kept picks (dropped: 0)."""
    x = np.asarray(x, dtype=np.float64)
    E = x.shape[1]
    ok = (ids >= 0) & (ids < E)
    ls = np.where(ok, np.take_along_axis(log_scores(x), np.clip(ids, 0, E - 1).astype(np.int64), 1), -np.inf)
    return normalised(ls)


def backward(x, ids, coef, grad_loss=1.0, grad_w=None, counts=None, seq_offsets=None, mask=None):
    """(gradient [M, E], scale [M, E] of the terms that were added up)."""
    x = np.asarray(x, dtype=np.float64)
    (M, E), k = x.shape, ids.shape[1]
    grad, size = np.zeros((M, E)), np.zeros((M, E))
    seqs = list(sequences(M, seq_offsets, mask))
    filled = sum(t.size > 0 for _, t in seqs)
    for b, t in seqs:
        if t.size == 0:
            continue
        p, rest = normalised(log_scores(x[t])), np.exp(log_scores(-x[t]))  # p, 1 - s
        if counts is not None:
            g = grad_loss * coef * E / (k * t.size ** 2 * filled)
            c = counts[b].astype(np.float64)
            mean = (p * c).sum(axis=1, keepdims=True)
            grad[t] += g * p * rest * (c - mean)
            size[t] += abs(g) * p * rest * (c + mean)
        if grad_w is not None:
            w = weights(x[t], ids[t])
            ok = (ids[t] >= 0) & (ids[t] < E)
            at = np.clip(ids[t], 0, E - 1).astype(np.int64)
            gw = np.where(ok, grad_w[t].astype(np.float64), 0.0)
            mean = (gw * w).sum(axis=1, keepdims=True)
            big = (np.abs(gw) * w).sum(axis=1, keepdims=True)
            for j in range(k):
                r = np.take_along_axis(rest, at[:, j:j + 1], 1)[:, 0]
                np.add.at(grad, (t, at[:, j]), w[:, j] * r * (gw[:, j] - mean[:, 0]) * ok[:, j])
                np.add.at(size, (t, at[:, j]), w[:, j] * r * (np.abs(gw[:, j]) + big[:, 0]) * ok[:, j])
    return grad, size


U = 2.0 ** -24  # half a step of FP32, relative


def score_bound(xmax):
    """Relative error of an FP32 sigmoid(x) with |x| <= xmax: the argument
    x log2(e) is rounded twice (1.5 U |x| after the exponential), and the
    exponential (2 U), 1 + u, the reciprocal (2 U) and a product follow."""
    return (1.5 * xmax + 6) * U


def share_bound(xmax, E, tokens):
    """Relative error of a mean share: the score and its row total carry
    score_bound each, the total's sum E / 64 + 8 additions, the division one
    rounding, the sum over a sequence's tokens one a token, the result one."""
    return 2 * score_bound(xmax) + (E / 64 + 8 + 2 + tokens + 1) * U


def grad_bound(xmax, E):
    """Relative to the terms' sizes: scores, slopes and totals (four times
    score_bound), the two wave sums (E / 64 + 8 each) and ten roundings."""
    return 4 * score_bound(xmax) + (2 * (E / 64 + 8) + 10) * U


FLUSH = 2.0 ** -64  # scores flushed to zero beside a total of 2^-60 or more
