"""Pins of the adapter oracle: merged weights, scaling, rows without an adapter."""
import numpy as np

from oracle.lora import lora


def make(R, k, n, rank, na, seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((R, k)), g.standard_normal((na, rank, k)),
            g.standard_normal((na, n, rank)), g.integers(-1, na, R), g.standard_normal((R, n)),
            g.standard_normal(na))


def test_equals_the_merged_weight():
    x, a, b, ids, base, s = make(9, 24, 17, 8, 3)
    w = np.random.default_rng(1).standard_normal((17, 24))
    y, mag, bad = lora(x, a, b, ids, x @ w.T, s)
    for r in range(9):
        m = w + (s[ids[r]] * b[ids[r]] @ a[ids[r]] if ids[r] >= 0 else 0)
        np.testing.assert_allclose(y[r], m @ x[r], rtol=1e-9, atol=1e-12)
    assert not bad and (mag >= np.abs(y) - 1e-9).all()


def test_no_adapter_bad_ids_and_rank_one():
    x, a, b, _, base, s = make(4, 8, 5, 8, 2)
    y, _, bad = lora(x, a, b, [-1, -1, -1, -1], base, s)
    assert np.array_equal(y, base) and not bad
    y, _, bad = lora(x, a, b, [-1, 2, -5, 0], base, s)
    assert np.array_equal(y[:3], base[:3]) and bad and not np.array_equal(y[3], base[3])
    a1 = np.zeros((1, 8, 8))
    b1 = np.zeros((1, 5, 8))
    a1[0, 3], b1[0, :, 3] = 1.0, np.arange(5)
    y, _, _ = lora(x, a1, b1, [0] * 4)
    np.testing.assert_allclose(y, x.sum(1)[:, None] * np.arange(5)[None])
