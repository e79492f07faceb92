"""tfd_paged_attn where values are not ordinary numbers: infinite keys and values that rows see.

Where only some elements of a value vector are infinite, all other elements, and all other rows, come from
the same products in the same order as without them, so they are equal bit by bit."""
import numpy as np
import pytest
import torch

from helpers import assert_bf16_rounding, need_gpu, np32
from oracle.paged import attend
from paged_cases import Case

pytestmark = pytest.mark.gpu


def place(c, r, t):
    """Page and place in it of request r's token t."""
    return int(c.table[r, t // c.page]), t % c.page


def rows_of(c, got, r):
    """Request r's outputs [n][q_heads][dim]."""
    a, b = c.row_start[r], c.row_start[r + 1]
    return got[0][a:b, :c.q_heads * c.dim].float().cpu().numpy().reshape(b - a, c.q_heads, c.dim)


def check_infinite_values(c, r, t, seen_by=None, **kw):
    """Every third element of token t's values +inf, every third -inf: they reach the rows that see the token
    (seen_by, or by causal order), and change nothing else."""
    ref = c.run(**kw)
    page, at = place(c, r, t)
    keep = c.cache.v[page, at].clone()
    c.cache.v[page, at, :, 0::3] = float("inf")
    c.cache.v[page, at, :, 1::3] = float("-inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = c.run(**kw, st=st)
    torch.cuda.synchronize()
    c.cache.v[page, at] = keep
    assert st.item() == 0
    n, length = int(c.new[r]), int(c.lens[r])
    want = rows_of(c, ref, r).copy()
    assert np.isfinite(want).all()
    for j in range(n) if seen_by is None else seen_by:
        if seen_by is not None or t <= length + j:
            want[j, :, 0::3], want[j, :, 1::3] = np.inf, -np.inf
    x = rows_of(c, got, r)
    assert np.array_equal(x, want), (t, np.argwhere(x != want)[:4], x[x != want][:4])
    other = np.ones(c.rows, bool)
    other[c.row_start[r]:c.row_start[r + 1]] = False
    assert torch.equal(got[0][other], ref[0][other]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,heads", [(4, 1), (2, 2), (8, 1)])
def test_infinite_values_that_some_rows_see(q_heads, heads, dim):
    """New tokens on both sides of a tile's end: rows that see one tile, and rows that see two."""
    need_gpu()
    c = Case([125, 40], [4, 2], q_heads, heads, dim, 16)
    for t in (126, 127, 128):
        check_infinite_values(c, 0, t)


@pytest.mark.parametrize("k", [150, 153, 156, 157, 158, 161])
def test_infinite_values_that_some_rows_see_in_pieces(k):
    """The same where the unit is cut at several places, with two tiles and more a piece."""
    need_gpu()
    c = Case([128 * k + 125], [4], 8, 2, 128, 64)
    for t in (1, 2, 3):
        check_infinite_values(c, 0, 128 * k + 125 + t)


@pytest.mark.parametrize("dim", [64, 128])
def test_infinite_values_left_of_some_rows_windows(dim):
    need_gpu()
    c = Case([140], [4], 4, 1, dim, 16)
    check_infinite_values(c, 0, 127, seen_by=[0], window=13)
    check_infinite_values(c, 0, 128, seen_by=[0, 1], window=13)
    check_infinite_values(c, 0, 129, seen_by=[0, 1, 2], window=13)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,q_heads,heads,tokens", [([0], [1], 1, 1, [0]), ([300], [4], 4, 1, [5, 200, 300]),
                                                           ([300, 9], [4, 4], 16, 2, [0, 127, 300]),
                                                           ([9000], [1], 4, 1, [0, 4444, 8999, 9000])])
def test_infinite_values_that_all_rows_see(lens, new, q_heads, heads, tokens, dim):
    """The weights enter as two parts, of which the low one is zero or negative: inf times it is not added."""
    need_gpu()
    c = Case(lens, new, q_heads, heads, dim, 16)
    for t in tokens:
        check_infinite_values(c, 0, t)


def many_rows(dim, **kw):
    """Requests of up to 32 rows of 8 query heads a key head, enough of them for units of 64 rows."""
    g = np.random.default_rng(dim)
    new = np.full(24, 32)
    new[[3, 11, 17]] = 19, 1, 0
    return Case(g.integers(0, 260, 24), new, 16, 2, dim, 16, tid=880, **kw)


@pytest.mark.parametrize("dim", [64, 128])
def test_infinite_values_in_units_of_64_rows(dim):
    need_gpu()
    c = many_rows(dim)
    for r, t in ((0, 0), (5, int(c.lens[5]) + 9), (20, int(c.lens[20]) + 31), (22, int(c.lens[22]))):
        check_infinite_values(c, r, t)


def check_infinite_keys(c, r, t):
    """One element of a cached token's keys infinite: rows and heads whose score is -inf do without the token, in
    the others it is +inf, and the softmax NaN."""
    kw = dict(norm=False, rope=False, gamma=False)
    ref = c.run(**kw)
    page, at = place(c, r, t)
    for d, bad in ((0, float("inf")), (c.dim - 1, float("-inf"))):
        keep = c.cache.k[page, at].clone()
        c.cache.k[page, at, :, d] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.run(**kw, st=st)
        torch.cuda.synchronize()
        c.cache.k[page, at] = keep
        assert st.item() == 0
        a, b = c.row_start[r], c.row_start[r + 1]
        other = np.ones(c.rows, bool)
        other[a:b] = False
        assert torch.equal(got[0][other], ref[0][other]) and torch.equal(got[1][other], ref[1][other])
        q = np32(c.q)[a:b]
        k, v = (np.delete(x, t, 0) for x in c.tokens(r))
        sc = 1.0 / np.sqrt(c.dim)
        y, ls, m = attend(q, k, v, int(c.lens[r]) - 1, scale=sc)
        without = np.sign(q[:, :, d]) * np.sign(bad) < 0
        assert without.any() and not without.all()
        x, l = rows_of(c, got, r), np32(got[1])[a:b]
        assert np.isnan(x[~without]).all() and np.isnan(l[~without]).all()
        # the tolerances of paged_cases, for the tokens that are left
        part, tok = 2.0 ** -16 + 2.0 ** -18, len(k) + 1
        err = 1.01 * (part * m["dev_a"] + 2.0 ** -20 * m["dev"]) + \
            (2.0 ** -16 + 2.0 ** -17 + 2.0 ** -23 * tok / 8) * m["abs_out"]
        assert_bf16_rounding(x[without], y[without], err[without], f"token {t}")
        lim = 2 * part * m["a"] + 2.0 ** -20 + 2.0 ** -24 * tok + 2.0 ** -23 * np.abs(ls)
        assert (np.abs(l - ls) <= lim)[without].all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,q_heads,heads,tokens", [([2], [4], 4, 1, [0, 1]), ([300], [4], 4, 1, [5, 200]),
                                                           ([300, 9], [4, 4], 16, 2, [0, 127, 299]),
                                                           ([9000], [2], 8, 1, [0, 4444])])
def test_infinite_keys(lens, new, q_heads, heads, tokens, dim):
    need_gpu()
    c = Case(lens, new, q_heads, heads, dim, 16)
    for t in tokens:
        check_infinite_keys(c, 0, t)


def test_infinite_keys_in_units_of_64_rows():
    need_gpu()
    c = many_rows(64)
    r = int(np.argmax(c.lens * (c.new == 32)))
    for t in (0, int(c.lens[r]) - 1):
        check_infinite_keys(c, r, t)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [0, 260])
def test_rows_whose_scores_are_all_minus_infinity(lens, dim):
    need_gpu()
    c = Case([lens], [1], 8, 2, dim, 16)
    c.cache.k[:, :, :, 3] = float("inf")
    c.q[0, :, 3] = -c.q[0, :, 3].abs()
    out, lse = c.run(norm=False, rope=False, gamma=False)
    torch.cuda.synchronize()
    assert not out[0, :8 * dim].any() and torch.isneginf(lse[0]).all()
