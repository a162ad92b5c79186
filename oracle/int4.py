"""CPU oracle for 4-bit weights with group scales and their matrix-vector products.
TEST INFRASTRUCTURE ONLY: shares no code with the product path.

Format: a row of K weights is padded with zeros to Kp, a multiple of 128, in groups
of 32, 64 or 128 columns; weight = scale * (code - 8).  The scale is the FP32 quotient
of the group's largest magnitude and 7, rounded to the scales' 16-bit type; a code is
8 plus the FP32 quotient of weight and scale, rounded to the nearest integer, ties to
even, at most 7 in magnitude.  Parity status: pinned by tests/test_oracle_int4_pins.py.
"""
from __future__ import annotations

import numpy as np


def padded(K: int) -> int:
    return -(-K // 128) * 128


def to_half(x: np.ndarray, kind: str) -> np.ndarray:
    """float32 values rounded to "bf16" or "f16" (nearest even), as float32."""
    x = np.asarray(x, dtype=np.float32)
    if kind == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float32)
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def quantize(w: np.ndarray, group: int, kind: str):
    """w [R, K] float32 -> codes [R, Kp / 2] uint8, scales [R, Kp / group] float32."""
    w = np.asarray(w, dtype=np.float32)
    R, K = w.shape
    Kp = padded(K)
    v = np.zeros((R, Kp), dtype=np.float32)
    v[:, :K] = w
    v = v.reshape(R, Kp // group, group)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        scale = to_half(np.abs(v).max(axis=2) / np.float32(7), kind)
        bad = ~(np.isfinite(v).all(axis=2) & np.isfinite(scale))
        q = np.rint(v / scale[:, :, None])
        q = np.where(bad[:, :, None] | (scale == 0)[:, :, None], 0.0, np.clip(q, -7, 7)).astype(np.int64) + 8
    q = q.reshape(R, Kp // 2, 2)
    return (q[:, :, 0] | (q[:, :, 1] << 4)).astype(np.uint8), np.where(bad, np.float32(np.nan), scale)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [..., Kp / 2], scales [..., Kp / group] -> weights [..., Kp] float64."""
    q = np.empty(codes.shape[:-1] + (codes.shape[-1] * 2,))
    q[..., 0::2] = codes & 15
    q[..., 1::2] = codes >> 4
    group = q.shape[-1] // scales.shape[-1]
    return (q - 8.0) * np.repeat(scales.astype(np.float64), group, axis=-1)


def matvec(x, w, ids):
    """x [M, K] or [M, k, K], w [E, N, >= K], ids [M, k] -> p [M, k, N] float64."""
    M, k = ids.shape
    K = x.shape[-1]
    p = np.zeros((M, k, w.shape[1]))
    for t in range(M):
        for j in range(k):
            if 0 <= ids[t, j] < w.shape[0]:
                p[t, j] = w[ids[t, j], :, :K] @ (x[t] if x.ndim == 2 else x[t, j])
    return p


def silu_gate(p):
    half = p.shape[-1] // 2
    g, u = p[..., :half], p[..., half:]
    return g / (1.0 + np.exp(-g)) * u
