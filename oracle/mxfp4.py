"""CPU oracle for 4-bit microscaled rows and their grouped product.
TEST INFRASTRUCTURE ONLY: shares no code with the product path.

Format: a row of K values is padded with zeros to Kp, a multiple of 128, in
blocks of 32.  A block's scale byte X stands for 2^(X - 127) (255: NaN block),
each value for a level 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign.

Parity status: the published microscaling format (block of 32, E2M1 codes, E8M0
scales, scale exponent = floor(log2 of the largest magnitude) - 2); pinned by
tests/test_oracle_mxfp4_pins.py.
"""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def padded(K: int) -> int:
    return -(-K // 128) * 128


def quantize(x: np.ndarray):
    """x [R, K] (any float type, taken exactly) -> codes [R, Kp/2], scales
    [R, Kp/32] (uint8), values [R, K] (float64)."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    Kp = padded(K)
    v = np.zeros((R, Kp))
    v[:, :K] = x
    v = v.reshape(R, Kp // 32, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.abs(v).max(axis=2)
    ex = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)  # frexp: top = f 2^n with f in [.5, 1)
    ex = np.maximum(ex, -127)
    a = np.ldexp(np.abs(v), -ex[:, :, None])
    dist = np.abs(a[..., None] - LEVELS)
    lo = dist.argmin(axis=-1)
    hi = 7 - dist[..., ::-1].argmin(axis=-1)
    idx = np.where(lo % 2 == 0, lo, hi)              # on a tie the even code
    code = idx + 8 * np.signbit(v)
    code = np.where(bad[:, :, None], 0, code).reshape(R, Kp).astype(np.uint8)
    X = np.where(bad, 255, ex + 127).astype(np.uint8)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes, X, decode(codes, X)[:, :K]


def decode(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Packed rows [..., Kp/2], [..., Kp/32] -> float64 [..., Kp]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[:-1] + (codes.shape[-1] * 2,))
    mag = np.where(c >= 8, -LEVELS[c & 7], LEVELS[c & 7])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return mag * np.repeat(s, 32, axis=-1)


def product(xc, xs, wc, ws, sorted_ids, expert_of_block, num_post_pad, M, k, block, in_order=False):
    """y [num_post_pad, N] float64 and sum |x||w| of the same shape."""
    N = wc.shape[1]
    y = np.zeros((num_post_pad, N))
    ab = np.zeros((num_post_pad, N))
    s = np.asarray(sorted_ids[:num_post_pad], dtype=np.int64)
    r = np.arange(num_post_pad)
    e = np.asarray(expert_of_block, dtype=np.int64)[r // block]
    ok = (s >= 0) & (s < M * k)
    for ex in np.unique(e[ok]):
        sel = np.nonzero(ok & (e == ex))[0]
        src = sel if in_order else s[sel] // k
        xa, wa = decode(xc[src], xs[src]), decode(wc[ex], ws[ex])
        y[sel] = xa @ wa.T
        ab[sel] = np.abs(xa) @ np.abs(wa).T
    return y, ab


def tolerance(y, ab, Kp, bf16: bool):
    """FP32 sums of Kp exact products in any order, each addition off by at most
    one unit in the last place of a partial sum (2^-23, covering an adder that
    truncates), then half a step of y's type."""
    acc = Kp * 2.0 ** -23 * ab
    return acc + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(y) + acc)
