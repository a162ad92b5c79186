"""Pins of the 4-bit rows' oracle: hand-made blocks, ties, limits, products."""
import numpy as np

from oracle import mxfp4 as om


def block(vals):
    x = np.zeros((1, 32))
    x[0, :len(vals)] = vals
    return x


def test_levels_survive_and_pack_low_half_first():
    vals = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.5, -6]
    codes, X, v = om.quantize(block(vals))
    assert X[0, 0] == 127 and np.array_equal(v[0, :10], vals)
    assert codes[0, 0] == 0x10 and codes[0, 3] == 0x76 and codes[0, 4] == 0xF9
    assert codes.shape == (1, 64) and X.shape == (1, 4) and not codes[0, 16:].any() and not X[0, 1:].any()


def test_ties_go_to_the_even_code():
    v = om.quantize(block([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7.99]))[2]
    assert v[0, :9].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6]


def test_scale_is_the_largest_exponent_less_two():
    for top, X in ((1.0, 125), (1.999, 125), (2.0, 126), (2.0 ** 127, 252), (2.0 ** -125, 0), (2.0 ** -140, 0)):
        assert om.quantize(block([top]))[1][0, 0] == X, top


def test_a_bad_value_poisons_its_block_only():
    x = np.ones((1, 64))
    x[0, 3] = np.inf
    codes, X, v = om.quantize(x)
    assert X[0].tolist() == [255, 125, 0, 0] and not codes[0, :16].any()
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_rounding_is_within_half_a_level():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 160))
    v = om.quantize(x)[2]
    top = np.abs(x.reshape(50, 5, 32)).max(2).repeat(32, 1)
    # the widest gap is 4..6 and the cut at 6 loses under 2 of a block maximum in [4, 8)
    assert (np.abs(v - x) <= top / 4 * 1.0 + 1e-12).all()


def test_product_matches_a_loop():
    rng = np.random.default_rng(1)
    xc, xs, xv = om.quantize(rng.standard_normal((3, 40)))
    wc, ws, wv = om.quantize(rng.standard_normal((2 * 5, 40)))
    wv = wv.reshape(2, 5, 40)
    sid = np.array([0, 2, 6, 6, 1, 6, 6, 6])
    y, _ = om.product(xc, xs, wc.reshape(2, 5, -1), ws.reshape(2, 5, -1), sid, np.array([0, 1]), 8, 3, 2, 4)
    for r, (s, e) in enumerate(zip(sid, [0] * 4 + [1] * 4)):
        want = np.zeros(5) if s == 6 else np.array([(xv[s // 2] * wv[e, n]).sum() for n in range(5)])
        np.testing.assert_allclose(y[r], want, rtol=1e-13, atol=1e-13)
