"""Pins of oracle/int4.py: values by hand, every code and scale against a search."""
import numpy as np
import pytest

from oracle import int4 as orc


def test_by_hand():
    w = np.zeros((1, 40), dtype=np.float32)
    w[0, :5] = [7.0, -7.0, 2.5, -3.5, 0.4]  # scale 1: ties to even
    w[0, 32] = -14.0                        # scale 2
    codes, scales = orc.quantize(w, 32, "bf16")
    assert scales.tolist() == [[1.0, 2.0, 0.0, 0.0]]
    q = orc.values(codes, scales)[0]
    assert q[:5].tolist() == [7.0, -7.0, 2.0, -4.0, 0.0] and q[32] == -14.0 and not q[33:].any()
    assert codes[0, 0] == 15 | (1 << 4) and codes.shape == (1, 64)


@pytest.mark.parametrize("kind,bits", [("bf16", 8), ("f16", 11)])
def test_nearest(kind, bits):
    rng = np.random.default_rng(1)
    w = (rng.normal(size=(6, 200)) * 10.0 ** rng.integers(-3, 3, size=(6, 1))).astype(np.float32)
    codes, scales = orc.quantize(w, 64, kind)
    q = orc.values(codes, scales)[:, :200]
    s = np.repeat(scales, 64, axis=1)[:, :200].astype(np.float64)
    best = np.min(np.abs(w[:, :, None] - s[:, :, None] * np.arange(-7, 8)), axis=2)
    assert np.all(np.abs(w - q) <= best + 1e-6 * s)
    top = np.abs(np.pad(w, ((0, 0), (0, 56))).reshape(6, 4, 64)).max(axis=2)
    assert np.all(np.abs(scales - top / 7) <= 2.0 ** -bits * top / 7 * 1.001)


def test_not_finite():
    w = np.ones((1, 128), dtype=np.float32)
    w[0, 3], w[0, 40] = np.inf, np.nan
    codes, scales = orc.quantize(w, 32, "f16")
    assert np.isnan(scales[0, :2]).all() and (codes[0, :32] == 0x88).all() and scales[0, 2] > 0
    big, s = orc.quantize(np.full((1, 128), 3e38, dtype=np.float32), 128, "f16")  # no finite scale
    assert np.isnan(s).all() and (big == 0x88).all()


def test_matvec_by_hand():
    w = np.zeros((2, 2, 128))
    w[0, :, :2], w[1, :, :2] = [[1, 2], [3, 4]], [[-1, 0], [0, 1]]
    x = np.array([[1.0, 10.0]])
    assert orc.matvec(x, w, np.array([[1, 0, 5]])).tolist() == [[[-1, 10], [21, 43], [0, 0]]]
    y = orc.matvec(np.array([[[1.0, 10.0], [2.0, 0.0], [1.0, 1.0]]]), w, np.array([[1, 0, -1]]))
    assert y.tolist() == [[[-1, 10], [2, 6], [0, 0]]]
    assert np.allclose(orc.silu_gate(np.array([0.0, 1.0, 5.0, 3.0])), [0.0, 3.0 / (1 + np.exp(-1.0))])
