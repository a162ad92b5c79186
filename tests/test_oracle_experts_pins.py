"""Pins of oracle/experts.py: small integer cases by hand, gradients against
central differences of the forward functions."""
import numpy as np

from oracle import experts as orc

# two experts, blocks of 2, three tokens with two picks; slot 3 is dropped; row 3 is padding
SID = np.array([0, 2, 4, 6, 1, 5, 6, 6], dtype=np.int32)
EOB = np.array([0, 0, 1], dtype=np.int32)
NPP, M, K2, BLOCK = 6, 3, 2, 2


def test_product_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    w = np.array([[[1.0, 0.0], [1.0, 1.0]], [[0.0, -1.0], [2.0, 0.0]]])
    y, mag = orc.product(x, w, SID, EOB, NPP, M, K2, BLOCK, True)
    assert y.tolist() == [[1, 3], [3, 7], [5, 11], [0, 0], [-2, 2], [-6, 10]]
    assert mag.tolist() == [[1, 3], [3, 7], [5, 11], [0, 0], [2, 2], [6, 10]]


def test_slot_rows_by_hand():
    assert orc.slot_rows(SID, NPP, M, K2).tolist() == [[0, 4], [1, -1], [2, 5]]


def test_combine_by_hand():
    y = np.arange(12.0).reshape(6, 2)
    rows = np.array([[0, 4], [1, -1], [2, 6]])
    out, _ = orc.combine(y, rows, np.array([[1.0, 0.5], [2.0, 9.0], [1.0, 9.0]]))
    assert out.tolist() == [[4.0, 5.5], [4.0, 6.0], [4.0, 5.0]]
    assert orc.combine(y, rows, None)[0].tolist() == [[8.0, 10.0], [2.0, 3.0], [4.0, 5.0]]


def _layer(x, w1, w2, v):
    a, _ = orc.product(x, w1, SID, EOB, NPP, M, K2, BLOCK, True)
    y, _ = orc.product(orc.swiglu(a), w2, SID, EOB, NPP, M, K2, BLOCK, False)
    return a, y, orc.combine(y, orc.slot_rows(SID, NPP, M, K2), v)[0]


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, w1, w2 = rng.normal(size=(M, 4)), rng.normal(size=(2, 6, 4)), rng.normal(size=(2, 4, 3))
    v, g = rng.normal(size=(M, K2)), rng.normal(size=(M, 4))
    a, y, _ = _layer(x, w1, w2, v)
    rows = orc.slot_rows(SID, NPP, M, K2)
    dy, dv, _ = orc.combine_backward(g, rows, v, y, NPP)
    dw2, _ = orc.product_dw(dy, orc.swiglu(a), 2, SID, EOB, NPP, M, K2, BLOCK, False)
    da = orc.swiglu_backward(a, orc.product_dx(dy, w2, SID, EOB, NPP, M, K2, BLOCK)[0])
    dw1, _ = orc.product_dw(da, x, 2, SID, EOB, NPP, M, K2, BLOCK, True)
    dx = orc.combine(orc.product_dx(da, w1, SID, EOB, NPP, M, K2, BLOCK)[0], rows, None)[0]
    for t, grad in ((x, dx), (w1, dw1), (w2, dw2), (v, dv)):
        for i in np.ndindex(t.shape):
            keep, h = t[i], 1e-5
            t[i] = keep + h
            up = (_layer(x, w1, w2, v)[2] * g).sum()
            t[i] = keep - h
            down = (_layer(x, w1, w2, v)[2] * g).sum()
            t[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7, i
