"""CPU oracle for the experts' 16-bit products, the gated activation and the mix of
the outputs.  TEST INFRASTRUCTURE ONLY: shares no code with the product path.

Everything in float64, row by row.  Metadata: row r < npp of expert eob[r // block]
holds slot sid[r]; a slot outside [0, M k) marks a padding row.
Parity status: pinned by tests/test_oracle_experts_pins.py.
"""
from __future__ import annotations

import numpy as np


def _live(sid, npp, routes):
    return [r for r in range(npp) if 0 <= sid[r] < routes]


def _row(r, s, k, by_tokens):
    return s // k if by_tokens else r


def product(x, w, sid, eob, npp, M, k, block, by_tokens):
    """(y [npp, N], the same sums of magnitudes)."""
    y, mag = np.zeros((npp, w.shape[1])), np.zeros((npp, w.shape[1]))
    for r in _live(sid, npp, M * k):
        v, m = x[_row(r, int(sid[r]), k, by_tokens)], w[eob[r // block]]
        y[r] = m @ v
        mag[r] = np.abs(m) @ np.abs(v)
    return y, mag


def product_dx(dy, w, sid, eob, npp, M, k, block):
    dx, mag = np.zeros((npp, w.shape[2])), np.zeros((npp, w.shape[2]))
    for r in _live(sid, npp, M * k):
        m = w[eob[r // block]]
        dx[r] = dy[r] @ m
        mag[r] = np.abs(dy[r]) @ np.abs(m)
    return dx, mag


def product_dw(dy, x, E, sid, eob, npp, M, k, block, by_tokens):
    dw, mag = np.zeros((E, dy.shape[1], x.shape[1])), np.zeros((E, dy.shape[1], x.shape[1]))
    rows = [[] for _ in range(E)]
    for r in _live(sid, npp, M * k):
        rows[eob[r // block]].append(r)
    for e, rs in enumerate(rows):
        if rs:
            src = [_row(r, int(sid[r]), k, by_tokens) for r in rs]
            dw[e] = dy[rs].T @ x[src]
            mag[e] = np.abs(dy[rs]).T @ np.abs(x[src])
    return dw, mag


def sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def swiglu(a):
    half = a.shape[1] // 2
    g, u = a[:, :half], a[:, half:]
    return g * sigmoid(g) * u


def swiglu_backward(a, dh):
    half = a.shape[1] // 2
    g, u = a[:, :half], a[:, half:]
    s = sigmoid(g)
    return np.concatenate([dh * u * (s + g * s * (1.0 - s)), dh * g * s], axis=1)


def slot_rows(sid, npp, M, k):
    rows = np.full(M * k, -1, dtype=np.int32)
    for r in _live(sid, npp, M * k):
        rows[sid[r]] = r
    return rows.reshape(M, k)


def combine(y, rows, weights):
    """(out [M, N], the same sums of magnitudes)."""
    M, k = rows.shape
    out, mag = np.zeros((M, y.shape[1])), np.zeros((M, y.shape[1]))
    for t in range(M):
        for j in range(k):
            if 0 <= rows[t, j] < y.shape[0]:
                v = 1.0 if weights is None else weights[t, j]
                out[t] += v * y[rows[t, j]]
                mag[t] += np.abs(v * y[rows[t, j]])
    return out, mag


def combine_backward(dout, rows, weights, y, capacity):
    """(dy [capacity, N], dweights [M, k], its sums of magnitudes)."""
    M, k = rows.shape
    dy = np.zeros((capacity, dout.shape[1]))
    dv, mag = np.zeros((M, k)), np.zeros((M, k))
    for t in range(M):
        for j in range(k):
            r = rows[t, j]
            if 0 <= r < capacity:
                dy[r] = (1.0 if weights is None else weights[t, j]) * dout[t]
                if y is not None:
                    dv[t, j] = dout[t] @ y[r]
                    mag[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return dy, dv, mag
