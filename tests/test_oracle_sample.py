"""Pins of the sampling oracle: hand examples, closed forms and invariants."""
import numpy as np
import pytest

from oracle.sample import accept_sampled, draw, filtered, sample


def test_hand_example_of_every_filter():
    x = np.log([8.0, 4.0, 2.0, 1.0, 1.0])
    np.testing.assert_allclose(filtered(x)[0], np.array([8, 4, 2, 1, 1]) / 16)
    np.testing.assert_allclose(filtered(x, top_k=2)[0], np.array([8, 4, 0, 0, 0]) / 12)
    np.testing.assert_allclose(filtered(x, top_p=0.6)[0], np.array([8, 4, 0, 0, 0]) / 12)
    np.testing.assert_allclose(filtered(x, top_k=3, top_p=0.5)[0], np.array([8, 0, 0, 0, 0]) / 8)
    np.testing.assert_allclose(filtered(x, min_p=0.2)[0], np.array([8, 4, 2, 0, 0]) / 14)
    np.testing.assert_allclose(filtered(x, temperature=0.5)[0], np.array([64, 16, 4, 1, 1]) / 86)
    np.testing.assert_allclose(filtered(x, top_k=4)[0], np.array([8, 4, 2, 1, 0]) / 15)  # tie: id 3


def test_ties_go_to_the_lower_mapped_id():
    dist, _ = filtered(np.zeros(4), top_k=2, id_map=[7, 1, 9, 3])
    np.testing.assert_allclose(dist, [0, 0.5, 0, 0.5])


def test_temperature_zero_and_edges():
    x = np.array([1.0, 3.0, 3.0, -np.inf, np.nan])
    assert filtered(x, temperature=0)[0].tolist() == [0, 1, 0, 0, 0]
    assert filtered(x, top_p=0.0)[0].tolist() == [0, 1, 0, 0, 0]
    assert filtered(x, min_p=1.0)[0].tolist() == [0, 0.5, 0.5, 0, 0]
    assert filtered(np.array([np.inf, 0, np.inf]))[0].tolist() == [0.5, 0, 0.5]
    assert filtered(np.full(3, -np.inf))[0] is None
    ids, probs, _ = sample(np.full((1, 3), -np.inf), [0.5])
    assert ids[0] == -1 and not probs.any()


@pytest.mark.parametrize("bad", [dict(temperature=[-1.0]), dict(temperature=[np.inf]),
                                 dict(top_p=[np.nan]), dict(min_p=[np.nan])])
def test_bad_parameters_draw_nothing(bad):
    assert sample(np.zeros((1, 4)), [0.5], **bad)[0][0] == -1
    assert sample(np.zeros((1, 4)), [1.0])[0][0] == -1


def test_evenly_spaced_numbers_give_every_token_its_share():
    dist = np.array([0.125, 0.25, 0.0, 0.5, 0.125])
    got = np.bincount([draw(dist, (i + 0.5) / 64)[0] for i in range(64)], minlength=5)
    assert got.tolist() == [8, 16, 0, 32, 8]


def test_accept_by_hand():
    p = np.array([[[0.5, 0.5, 0.0], [0.25, 0.5, 0.25], [0.0, 0.0, 1.0]]])
    q = np.array([[[1.0, 0.0, 0.0], [0.5, 0.25, 0.25]]])
    d = [[0, 0]]
    # 0.4 < 0.5 keeps the first; 0.6 * 0.5 >= 0.25 turns the second down: the rest of p - q is id 1
    assert [v[0] for v in accept_sampled(p, q, d, [2], [[0.4, 0.6]], [0.9])[:3]] == [1, 1, 1.0]
    # the first turned down: p - q = (-, 0.5, 0)
    assert [v[0] for v in accept_sampled(p, q, d, [2], [[0.5, 0.0]], [0.0])[:3]] == [0, 1, 1.0]
    # both kept: the row behind them
    assert [v[0] for v in accept_sampled(p, q, d, [2], [[0.0, 0.0]], [0.0])[:3]] == [2, 2, 1.0]
    # one asked and kept: the next row is p's second
    assert [v[0] for v in accept_sampled(p, q, d, [1], [[0.0, 0.0]], [0.3])[:3]] == [1, 1, 0.5]
    # equal rows never turn a draft down, except at u q == p = 0; then p itself is drawn from
    e = np.array([[[0.5, 0.5, 0.0], [1.0, 0.0, 0.0]]])
    assert accept_sampled(e, e[:, :1], [[2]], [1], [[0.5]], [0.5])[1][0] == 1


def test_accept_is_distributed_as_p():
    """Over a fine grid of (draft, u, u_next) the token at the first position has p's shares."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    got = np.zeros(3)
    m = 60
    for d in range(3):
        for i in range(m):
            for j in range(m):
                k, nxt, _, _, _ = accept_sampled(np.stack([p, p])[None], q[None, None], [[d]], [1],
                                                 [[(i + 0.5) / m]], [(j + 0.5) / m])
                got[d if k[0] else nxt[0]] += q[d] / m / m
    np.testing.assert_allclose(got, p, atol=2.0 / m)


def test_accept_through_a_subset_map_and_bad_streams():
    p = np.array([[[0.2, 0.3, 0.5], [1.0, 0.0, 0.0]]])
    q = np.array([[[0.75, 0.25]]])          # of tokens 2 and 0
    q_map = [1, -1, 0]
    k, nxt, prob, _, _ = accept_sampled(p, q, [[2]], [1], [[0.7]], [0.0], q_map)
    assert (k[0], nxt[0]) == (0, 1) and prob[0] == 1.0   # only token 1 has p above q
    for bad in (dict(n_asked=[2]), dict(drafts=[[3]]), dict(u=[[1.0]]), dict(u_next=[-0.1])):
        a = dict(drafts=[[2]], n_asked=[1], u=[[0.5]], u_next=[0.5])
        a.update(bad)
        assert accept_sampled(p, q, q_map=q_map, **a)[4][0]
