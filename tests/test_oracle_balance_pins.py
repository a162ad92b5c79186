"""Pins of the balance loss's oracle: closed forms, and its gradient against
central differences of the loss and of the routing weights."""
import numpy as np
import pytest

from oracle import balance as ob


def test_even_routing_has_loss_coef():
    # equal logits and equal counts: every share 1 / E, count M k / E
    ids = np.arange(12).reshape(6, 2) % 4
    loss, counts, tokens, shares = ob.balance(np.full((6, 4), 0.3), ids, 0.5)
    assert abs(loss - 0.5) < 1e-15 and (counts == 3).all() and tokens.tolist() == [6, 1] and np.allclose(shares, .25)


def test_empty_and_masked_sequences_do_not_count():
    rng = np.random.default_rng(0)
    x, ids = rng.standard_normal((5, 3)), rng.integers(0, 3, (5, 2))
    mask = np.array([1, 1, 0, 0, 1])
    x[2] = np.nan
    loss, counts, tokens, _ = ob.balance(x, ids, 1.0, [0, 2, 2, 4, 5], mask)
    assert tokens.tolist() == [2, 0, 0, 1, 2] and np.isfinite(loss) and counts.sum() == 6
    assert ob.balance(x, ids, 1.0, None, np.zeros(5))[0] == 0.0


def test_far_rows_are_normalised():
    p = ob.normalised(ob.log_scores(np.array([[-1e4, -1e4 + np.log(3.0), -np.inf], [-np.inf] * 3])))
    np.testing.assert_allclose(p, [[0.25, 0.75, 0], [0, 0, 0]], atol=1e-12)


@pytest.mark.parametrize("seed", range(3))
def test_gradient_against_differences(seed):
    rng = np.random.default_rng(seed)
    M, E, k = 7, 6, 3
    x = rng.standard_normal((M, E)) * 2
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(M)])
    ids[1, 0] = -1
    gw = rng.standard_normal((M, k))
    off, mask = [0, 3, 3, 7], np.array([1, 1, 1, 1, 0, 1, 1])

    def total(z):
        loss = ob.balance(z, ids, 0.7, off, mask)[0]
        return 1.3 * loss + (gw * ob.weights(z, ids) * mask[:, None]).sum()

    counts = ob.balance(x, ids, 0.7, off, mask)[1]
    g, _ = ob.backward(x, ids, 0.7, 1.3, gw, counts, off, mask)
    for t in range(M):
        for e in range(E):
            h = 1e-5
            a, b = x.copy(), x.copy()
            a[t, e] += h
            b[t, e] -= h
            # differences: h^2 times a third derivative of order one, and 1e-16 / h
            assert abs((total(a) - total(b)) / (2 * h) - g[t, e]) < 1e-8
