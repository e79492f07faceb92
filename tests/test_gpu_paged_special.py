"""tfd_paged_attn where values are not ordinary numbers: infinite keys and values that rows see, value scales far
apart and beyond what is served, and what is reported and what is not.

Where only some elements of a value vector are infinite, all other elements, and all other rows, come from
the same products in the same order as without them, so they are equal bit by bit."""
import numpy as np
import pytest
import torch

from helpers import assert_bf16_rounding, need_gpu, np32
from oracle.paged import attend
from paged_cases import Case
from speculative_decoding_draft_row_gb300 import tfd

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


def scaled_values(c, f):
    """Value scales times f [pages][heads][page], also in what the oracle reads."""
    c.cache.v_scales.mul_(f)
    codes = c.cache.v.view(torch.float8_e4m3fn).double()
    c.kv[1] = (codes * c.cache.v_scales.double().transpose(1, 2)[..., None]).cpu().numpy()


def by_token(c, exponent):
    """2^exponent(token) at each token of request 0, 1 elsewhere."""
    f = torch.ones_like(c.cache.v_scales)
    for t in range(int(c.lens[0] + c.new[0])):
        page, at = place(c, 0, t)
        f[page, :, at] = 2.0 ** exponent(t)
    return f


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,q_heads,heads", [([700], [2], 4, 2), ([600], [6], 8, 1), ([9000], [1], 4, 1)])
@pytest.mark.parametrize("what", ["rising", "falling", "by turns", "all large"])
def test_e4m3_scales_far_apart(what, lens, new, q_heads, heads, dim):
    """From 2^-95 to 2^79.6, tile by tile: what a weight is relative to the largest one is far from what its
    probability is, and every probability counts in the sum."""
    need_gpu()
    c = Case(lens, new, q_heads, heads, dim, 16, "e4m3")
    n = lens[0]
    scaled_values(c, by_token(c, {
        "rising": lambda t: -86 if t < n // 2 else 87, "falling": lambda t: 87 if t < n // 2 else -86,
        "by turns": lambda t: 87 if t // 128 % 3 == 1 else -86, "all large": lambda t: 87}[what]))
    c.check()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [2.0 ** 81, 2.0 ** 112, 2.0 ** 127, -2.0 ** 90, float("inf"), float("nan")])
def test_e4m3_scales_beyond_what_is_served(bad, dim):
    """NaN for the rows that see such a value, and for no others."""
    need_gpu()
    c = Case([45, 200], [6, 4], 4, 2, dim, 16, "e4m3")
    ref = c.run()
    page, at = place(c, 0, 45 + 3)
    c.cache.v_scales[page, :, at] = bad
    got = c.run()
    torch.cuda.synchronize()
    others = [0, 1, 2, 6, 7, 8, 9]
    assert torch.equal(got[0][others], ref[0][others]) and torch.equal(got[1][others], ref[1][others])
    assert torch.isnan(got[0][3:6, :4 * dim]).all() and torch.isnan(got[1][3:6]).all()


def test_the_largest_e4m3_scale_that_is_served():
    """One value scale 2^88 times the others. Weights enter as f16 numbers exp2(s - reference + 7), s with the
    scale in it and the reference at most the largest s; rounding one is off by at most half of f16's smallest step,
    2^-25, where it is not by 2^-11 of itself, and its four parts leave up to 3 2^-24 of one below 2^-12 (over all f16
    numbers). So beside the tolerances of paged_cases an output may be off by
    (2^-25 + 3 2^-24) 2^-7 max_j(p_j s_j) sum_j |code_j|: most of it in elements where that token's code is zero."""
    need_gpu()
    c = Case([400], [3], 4, 2, 128, 16, "e4m3")
    page, at = place(c, 0, 77)
    f = torch.ones_like(c.cache.v_scales)
    f[page, :, at] = 2.0 ** 80 / c.cache.v_scales[page, :, at]
    scaled_values(c, f)
    assert (c.cache.v_scales[page, :, at] == 2.0 ** 80).all()
    got = c.run(norm=False, rope=False, gamma=False)
    torch.cuda.synchronize()
    k, v = c.tokens(0)
    q, sc = np32(c.q)[:3].astype(float), 1.0 / np.sqrt(128)
    t = np.arange(403)
    scales = np32(c.cache.v_scales)[c.table[0, t // 16], :, t % 16].astype(float)
    y, ls, m = attend(q, k, v, 400, scale=sc)
    part = 2.0 ** -16 + 2.0 ** -18
    err = 1.01 * (part * m["dev_a"] + (2.0 ** -20 + 2.0 ** -23 * m["a_most"][..., None]) * m["dev"]) + \
        (2.0 ** -11 + 2.0 ** -17 + 2.0 ** -23 * 403 / 8) * m["abs_out"]
    for j in range(3):
        for i in range(4):
            n, h = 401 + j, i // 2
            p = np.exp(sc * k[:n, h] @ q[j, i] - ls[j, i])
            err[j, i] += 7 * 2.0 ** -32 * (p * scales[:n, h]).max() * np.abs(v[:n, h] / scales[:n, h, None]).sum(0)
    assert_bf16_rounding(rows_of(c, got, 0), y, err)
    lim = 2 * part * m["a"] + 2.0 ** -23 * m["a_most"] + 2.0 ** -20 + 2.0 ** -24 * 403 + 2.0 ** -23 * (80 + np.abs(ls))
    assert (np.abs(np32(got[1])[:3] - ls) <= lim).all()


def test_positions_that_no_rotation_uses_are_not_judged():
    """A row that sees nothing, in a request without tokens: its depth is -1, its position nobody's."""
    need_gpu()
    c = Case([0, 30], [3, 2], 2, 1, 64, 16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(tree=[0, 0b010, 0b110, 1, 3, 0, 0], rope=False)
    ref = c.run(**kw)
    got = c.run(**kw, pos=[0, 0, 1, 30, 31, 0, 0], st=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    c.run(**kw, pos=[-1] * 7, st=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    c.run(tree=kw["tree"], pos=[0, 0, 0, -1, 0, 0, 0], st=st)
    torch.cuda.synchronize()
    assert st.item() == tfd.ERR_DEVICE_DATA


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,q_heads,heads", [([1500], [4], 128, 32), ([3000, 700], [2, 1], 64, 32),
                                                    ([2500], [8], 64, 16)])
@pytest.mark.parametrize("spread", [2.0, 4.0, 8.0])
def test_e4m3_weights_above_their_reference(spread, lens, new, q_heads, heads, dim):
    """Scores so far apart that a tile's largest often passes the reference by some powers of two, and fewer than
    move it: what is left of such a weight after two parts, times 2^8, is an f16 number as well."""
    need_gpu()
    c = Case(lens, new, q_heads, heads, dim, 16, "e4m3", q_std=spread)
    c.check(norm=False)
