"""Pins of the paged cache's oracle: bookkeeping invariants, hand examples, and attention against closed
forms and the ring oracle."""
import numpy as np
import pytest

from oracle.attn import window_attn
from oracle.numerics import round_bf16
from oracle.paged import attend, plan, turned


def fresh(R, max_pages, pages, seed=0):
    free = np.random.default_rng(seed).permutation(pages)
    return np.full((R, max_pages), -7), np.zeros(R, int), free, pages


def test_plan_by_hand():
    table, held, free, n = np.full((2, 3), -7), np.zeros(2, int), np.array([4, 3, 2, 1, 0]), 5
    p = plan([0, 0], [3, 5], 4, table, held, free, n, 9)
    assert p["held"].tolist() == [1, 2] and p["n_free"] == 2 and not p["bad"]
    assert p["table"][0, 0] == 0 and p["table"][1, :2].tolist() == [1, 2] and p["table"][1, 2] == -7
    assert p["row_start"].tolist() == [0, 3, 8]
    assert p["slots"].tolist() == [0, 1, 2, 4, 5, 6, 7, 8, -1]
    assert p["pos"].tolist() == [0, 1, 2, 0, 1, 2, 3, 4, -1]


@pytest.mark.parametrize("seed", range(5))
def test_plan_keeps_every_page_once_and_turns_back(seed):
    g = np.random.default_rng(seed)
    R, ps, pages = 7, 4, 60
    table, held, free, n = fresh(R, 12, pages, seed)
    lens = np.zeros(R, int)
    for _ in range(12):
        new = g.integers(0, 5, R)
        p = plan(lens, new, ps, table, held, free, n, int(new.sum()))
        assert not p["bad"]
        mine = [int(i) for r in range(R) for i in p["table"][r, :p["held"][r]]]
        left = p["free_ids"][:p["n_free"]].tolist()
        assert sorted(mine + left) == list(range(pages))
        assert len(set(p["slots"].tolist())) == int(new.sum())
        q = plan(lens, np.zeros(R, int), ps, p["table"], p["held"], p["free_ids"], p["n_free"], 0)
        if all(held == -(-lens // ps)):                   # nothing but the new rows' pages moved
            assert q["free_ids"][:q["n_free"]].tolist() == free[:n].tolist()
        lens = np.minimum(lens + g.integers(0, new + 1), 12 * ps - 5)
        table, held, free, n = p["table"], p["held"], p["free_ids"], p["n_free"]


def test_plan_reports_what_is_wrong():
    table, held, free, n = fresh(3, 4, 5)
    p = plan([0, 0, 0], [8, 16, 1], 4, table, held, free, n, 25)
    assert p["bad"] and p["held"].tolist() == [2, 0, 0]   # 2, then 4 of 3, then counted behind those
    assert (p["table"][1] == -1).all() and (p["slots"][8:] == -1).all() and p["n_free"] == 3
    assert plan([-1, 0, 0], [1, 1, 1], 4, table, held, free, n, 3)["slots"].tolist()[0] == -1
    assert plan([0, 0, 0], [17, 1, 1], 4, table, held, free, n, 19)["held"].tolist() == [0, 1, 1]
    p = plan([0, 0, 0], [1, 1, 1], 4, table, held, free, 6, 3)
    assert p["bad"] and p["n_free"] == 6 and p["held"].tolist() == [0, 0, 0]
    assert plan([0, 0, 0], [1, 1, 1], 4, table, held, free, n, 2)["bad"]


def test_attend_closed_forms():
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((1, 2, 8)), g.standard_normal((5, 1, 8)), g.standard_normal((5, 1, 8))
    out, lse, _ = attend(q, np.tile(k[:1], (5, 1, 1)), v, 4)
    np.testing.assert_allclose(out[0, 0], v[:, 0].mean(0), rtol=1e-12)
    np.testing.assert_allclose(lse[0, 1], k[0, 0] @ q[0, 1] / np.sqrt(8) + np.log(5), rtol=1e-12)
    out, _, _ = attend(q, k, v, 4, window=0)
    np.testing.assert_allclose(out[0, 1], v[4, 0])
    out, lse, _ = attend(q, k[4:], v[4:], 0, tree=[0])
    assert not out.any() and np.isneginf(lse).all()


def test_attend_a_chain_is_a_tree_and_rows_are_requests_of_their_own():
    g = np.random.default_rng(1)
    n, length = 4, 9
    q, k, v = g.standard_normal((n, 4, 8)), *g.standard_normal((2, length + n, 2, 8))
    for window in (-1, 0, 2, 6, 50):
        a = attend(q, k, v, length, window=window)
        b = attend(q, k, v, length, tree=[(2 << j) - 1 for j in range(n)], window=window)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
        for j in range(n):
            c = attend(q[j:j + 1], k[:length + j + 1], v[:length + j + 1], length + j, window=window)
            np.testing.assert_allclose(c[0][0], a[0][j], rtol=1e-12)
            np.testing.assert_allclose(c[1][0], a[1][j], rtol=1e-12)


def test_attend_joins_by_its_log_sums():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((1, 2, 8)), *g.standard_normal((2, 12, 2, 8))
    y, lse, _ = attend(q, k, v, 11)
    parts = [attend(q, k[a:b], v[a:b], b - a - 1) for a, b in ((0, 5), (5, 12))]
    w = [np.exp(p[1] - lse) for p in parts]
    np.testing.assert_allclose(sum(w), 1.0, rtol=1e-12)
    np.testing.assert_allclose(sum(x[..., None] * p[0] for x, p in zip(w, parts)), y, rtol=1e-9,
                               atol=1e-12)


def test_attend_is_the_ring_oracle():
    g = np.random.default_rng(3)
    H, D, W, p = 2, 8, 5, 9
    q, kn, vn = g.standard_normal((3, 1, H, D))
    kr, vr = round_bf16(g.standard_normal((2, 1, 16, H, D)))
    terms = {}
    _, k2, v2 = window_attn(q, kn, vn, [p], kr, vr, W, terms=terms)
    qt, pair = turned(q, [p])
    kt, _ = turned(kn, [p])
    assert np.array_equal(round_bf16(kt[0]), k2[0, p])
    y, _, t = attend(qt, k2[0, :p + 1], v2[0, :p + 1], p, window=W)
    np.testing.assert_allclose(y.reshape(1, -1), terms["out_exact"], rtol=1e-12)
    np.testing.assert_allclose(t["abs_out"].reshape(1, -1), terms["abs_out"], rtol=1e-12)
    np.testing.assert_allclose(np.hypot(qt[..., :4], qt[..., 4:]), pair[..., :4], rtol=1e-12)


def test_plan_leaves_out_pages_that_are_none():
    table, held, free, n = fresh(3, 4, 12)
    p = plan([8, 8, 0], [0, 0, 0], 4, table, held, free, n, 0)
    t = p["table"]
    given = t[0, :2].tolist() + t[1, :2].tolist()
    t[0, 1] = 12
    q = plan([0, 0, 0], [0, 0, 0], 4, t, p["held"], p["free_ids"], p["n_free"], 0)
    assert q["bad"] and q["n_free"] == 11 and q["held"].tolist() == [0, 0, 0]
    assert q["free_ids"][8:11].tolist() == [given[3], given[2], given[0]]
