"""GPU parity of tfd_paged_attn against the oracle (tolerances: ``paged_cases``)."""
import numpy as np
import pytest
import torch

from helpers import need_gpu, np32
from paged_cases import Case, i32, random_tree
from speculative_decoding_draft_row_gb300 import tfd

pytestmark = pytest.mark.gpu

FMT = ["bf16", "e4m3"]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,heads", [(1, 1), (4, 4), (8, 2), (7, 1), (32, 2), (20, 1)])
def test_one_token_a_request(q_heads, heads, dim, fmt):
    need_gpu()
    Case([0, 1, 15, 16, 63, 64, 127, 300], [1] * 8, q_heads, heads, dim, 16, fmt).check()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_heads,heads,new", [(2, 2, 5), (8, 2, 6), (4, 1, 32), (12, 2, 3), (14, 2, 32),
                                               (3, 3, 17)])
def test_windows_of_rows(q_heads, heads, new, dim, fmt):
    """Requests with 0 to `new` rows, in any order; units of 16 rows and of 32, whole and in part."""
    need_gpu()
    c = Case([40, 3, 129, 0, 77, 258], [new, 1, 0, new, max(1, new // 2), new], q_heads, heads, dim, 24,
             fmt)
    c.check()


@pytest.mark.parametrize("layout", ["hnd", "both"])
@pytest.mark.parametrize("page", [1, 5, 8, 100, 1024])
@pytest.mark.parametrize("fmt", FMT)
def test_pages_and_layouts(page, layout, fmt):
    need_gpu()
    Case([0, 190, 31, 99], [3, 2, 4, 1], 6, 3, 128, page, fmt, layout).check()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("window", [0, 1, 3, 15, 64, 200, 511, 100000])
def test_sliding_windows(window, fmt):
    need_gpu()
    Case([0, 700, 66, 12, 64], [4, 6, 1, 2, 6], 4, 2, 128, 16, fmt).check(window=window)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("window", [-1, 2, 40])
def test_trees_and_rows_that_see_nothing(window, fmt):
    need_gpu()
    g = np.random.default_rng(5)
    c = Case([70, 0, 5, 0], [32, 20, 6, 3], 8, 2, 64, 16, fmt)
    words = np.zeros(c.rows, np.uint32)
    for r, n in enumerate([32, 20, 6]):
        words[c.row_start[r]:c.row_start[r + 1]] = random_tree(n, g)
    words[7] = 0                                          # sees the cached tokens alone
    words[c.row_start[1] + 4] = 0                         # nothing cached, nothing seen
    words[c.row_start[2] + 1] |= 0xFFFFFF00               # bits past the rows
    words[c.row_start[3]:c.row_start[4]] = [0, 0, 0]      # a request that sees nothing at all
    got = c.check(tree=words, window=window)
    row = c.row_start[1] + 4
    assert not got[0][row, :512].any() and torch.isneginf(got[1][row]).all()


@pytest.mark.parametrize("norm,rope,gamma,scale", [(False, False, False, 0.0), (True, False, True, 0.3),
                                                   (False, True, False, 0.02), (True, True, False, 1.0)])
@pytest.mark.parametrize("fmt", FMT)
def test_each_step_and_scales(norm, rope, gamma, scale, fmt):
    need_gpu()
    c = Case([130, 20], [3, 5], 8, 4, 128, 16, fmt, q_std=0.7)
    c.check(norm=norm, rope=rope, gamma=gamma, scale=scale)


def test_given_positions():
    need_gpu()
    c = Case([33, 70], [4, 2], 4, 2, 64, 16)
    c.check(pos=[2000000000, 0, 7, 100000, 70, 71, 0, 0])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("lens,new,q_heads,heads,dim", [([9000], 1, 4, 1, 128), ([5000, 1], 7, 8, 2, 64),
                                                        ([20000], 2, 1, 1, 64)])
def test_long_contexts_in_pieces(lens, new, q_heads, heads, dim, fmt):
    """A unit spread over many blocks, joined: twice the same bits, on the same workspace."""
    need_gpu()
    c = Case(lens, [new] * len(lens), q_heads, heads, dim, 64, fmt)
    a = c.check()
    b = c.run()
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FMT)
def test_many_requests(fmt):
    """More requests than threads that add up their lengths; the results of a request do not depend on
    the others but for the place of its cuts."""
    need_gpu()
    g = np.random.default_rng(9)
    lens, new = g.integers(0, 150, 700), g.integers(0, 4, 700)
    Case(lens, new, 2, 1, 64, 16, fmt, tid=830).check(requests=list(range(0, 700, 23)) + [699])


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("q_heads,heads,dim,new", [(12, 3, 128, 1), (12, 3, 64, 4), (8, 2, 128, 7),
                                                   (16, 2, 64, 32)])
def test_many_units_a_block(q_heads, heads, dim, new, fmt):
    """Units of all lengths, several a block and cut anywhere: rows in one piece, two and more."""
    need_gpu()
    g = np.random.default_rng(new)
    lens = np.concatenate([g.integers(0, 400, 150), g.integers(1000, 6000, 6), g.integers(0, 200, 100)])
    c = Case(lens, np.where(g.random(256) < 0.1, 0, new), q_heads, heads, dim, 16, fmt, tid=850)
    got = c.check(requests=list(range(3, 150, 29)) + [151, 154] + [200, 255])
    again = c.run()
    torch.cuda.synchronize()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests,new,q_heads,heads", [(40, 20, 16, 2), (2, 20, 16, 2), (1, 3, 40, 1), (300, 1, 5, 5)])
def test_units_of_each_size(requests, new, q_heads, heads, dim):
    """Many rows a head with and without units for the SMs, one unit of rows between 64 and 128, one row a unit."""
    need_gpu()
    g = np.random.default_rng(requests)
    c = Case(g.integers(100, 600, requests), [new] * requests, q_heads, heads, dim, 16, tid=870)
    c.check(requests=sorted({0, requests // 2, requests - 1}))


def test_one_request_is_the_same_beside_others():
    """The sums of a unit that no cut divides do not depend on the other requests."""
    need_gpu()
    c = Case([300, 180, 260], [2, 1, 2], 4, 2, 128, 16)
    got = c.run()
    for r in range(3):
        a, b = c.row_start[r], c.row_start[r + 1]
        out = tfd.tfd_paged_attn(c.q[a:b], c.cache, i32(c.table[r:r + 1]), i32(c.lens[r:r + 1]), i32([0, b - a]),
                                 2, q_gamma=c.gamma)[0]
        torch.cuda.synchronize()
        x, y = np32(out), np32(got[0])[a:b, :512]
        # cut differently, the sums' order differs: neighbouring bf16 values at most
        assert (np.abs(x - y) <= 2.0 ** -7 * np.abs(y) + 1e-6).all()


def test_scores_far_apart_and_masked_maxima():
    """A hidden token with the largest score, and one seen token that outweighs all others."""
    need_gpu()
    c = Case([100], [3], 2, 1, 64, 16)
    k = c.cache.k.view(-1, 64)
    at = [int(c.table[0, t // 16]) * 16 + t % 16 for t in range(103)]
    k[at[50]] *= 30.0
    k[at[102]] *= 1000.0                                  # the last new token: rows 0 and 1 do not see it
    c.kv[0] = np32(c.cache.k)
    c.check(norm=False, rope=False, gamma=False, scale=1.0)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("what", ["inf", "nan"])
def test_infinities_in_tokens_that_a_row_does_not_see(what, fmt):
    """A new token with an infinite or NaN key and value reaches the rows that see it, and no others."""
    need_gpu()
    c = Case([45, 200], [6, 4], 4, 2, 128, 16, fmt)
    ref = c.run()
    bad = float(what)
    t = 45 + 3                                            # row 3 of request 0
    page, at = int(c.table[0, t // 16]), t % 16
    if fmt == "bf16":
        c.cache.k[page, at], c.cache.v[page, at] = bad, bad
    else:
        c.cache.k_scales[page, :, at], c.cache.v_scales[page, :, at] = bad, bad
    got = c.run()
    torch.cuda.synchronize()
    see = [3, 4, 5]
    others = [0, 1, 2, 6, 7, 8, 9]
    # weights multiplied by hand and by the tensor cores may round to neighbouring values
    a, b = got[0][others].float(), ref[0][others].float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-6).all()
    assert torch.equal(got[0][6:10], ref[0][6:10]) and torch.equal(got[1][others], ref[1][others])
    assert torch.isnan(got[0][see][:, :512]).any(1).all()


def test_infinite_values_left_of_a_sliding_window():
    need_gpu()
    c = Case([90], [4], 2, 1, 128, 16)
    ref = c.run(window=20)
    t = 70                                                # row 0 sees it, rows 1 to 3 do not
    page, at = int(c.table[0, t // 16]), t % 16
    c.cache.v[page, at] = float("inf")
    got = c.run(window=20)
    torch.cuda.synchronize()
    # the exact weights by hand differ from the products' by less than a rounding
    d = (got[0][1:4, :256].float() - ref[0][1:4, :256].float()).abs()
    assert (d <= 2.0 ** -7 * ref[0][1:4, :256].float().abs() + 1e-6).all()
    assert torch.isposinf(got[0][0, :256]).all()


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dim", [64, 128])
def test_left_of_the_window_nothing_is_read(dim, fmt):
    """NaN codes and scales there, and pages given back, in the middle of a tile."""
    need_gpu()
    tree = [0b0001, 0b0011, 0b0001, 0b1001, 0, 0]         # row 2 is seen by nobody
    for words, low in ((tree, 289), (None, 290)):
        c = Case([390], [4], 4, 2, dim, 16, fmt)
        kw = dict(tree=words, window=100)
        ref = c.run(**kw)
        for t in list(range(low)) + [392] * (words is not None):
            page, at = int(c.table[0, t // 16]), t % 16
            if fmt == "bf16":
                c.cache.k[page, at] = c.cache.v[page, at] = float("nan")
            else:
                c.cache.k_scales[page, :, at] = c.cache.v_scales[page, :, at] = float("nan")
                if t < low:
                    c.cache.k[page, at], c.cache.v[page, at] = 0x7F, 0xFF if t & 1 else 0x7F
        c.table[0, :low // 16] = [-1, 10 ** 6] * (low // 32)
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.run(**kw, st=st)
        torch.cuda.synchronize()
        assert st.item() == 0
        assert torch.isfinite(ref[0].float()).all()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("fmt", FMT)
def test_two_graphs_on_one_workspace(fmt):
    """Captured apart, replayed in turn on one stream: each finds the counters at zero."""
    need_gpu()
    a = Case([5000, 70], [4, 4], 8, 2, 128, 16, fmt, tid=860)
    b = Case([900, 2500, 3], [3, 0, 4], 8, 2, 128, 16, fmt, tid=861)
    want = [c.run(max_new=4) for c in (a, b)]
    b.ws = a.ws
    graphs, outs = [], []
    for c in (a, b):
        args = (c.q, c.cache, i32(c.table), i32(c.lens), i32(c.row_start), 4)
        out = torch.full_like(want[len(outs)][0], 7.0)
        outs.append((out, args))
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            tfd.tfd_paged_attn(*args, q_gamma=c.gamma, out=out[:, :8 * 128], ws=a.ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        outs[i][0].fill_(7.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[i][0])


def test_growing_scores():
    """Every tile's scores are far above the last one's: the reference moves tile by tile, and back never."""
    need_gpu()
    for fmt in FMT:
        c = Case([1200], [3], 2, 1, 128, 16, fmt)
        f = np.repeat(1.0 + 3.0 * np.arange(10), 128)[:1203]
        at = [int(c.table[0, t // 16]) * 16 + t % 16 for t in range(1203)]
        if fmt == "bf16":
            k = c.cache.k.view(-1, 128)
            k[at] = (k[at].float() * torch.tensor(f, device="cuda")[:, None]).bfloat16()
            c.kv[0] = np32(c.cache.k)
        else:
            page, off = [a // 16 for a in at], [a % 16 for a in at]
            c.cache.k_scales[page, 0, off] *= torch.tensor(f, device="cuda", dtype=torch.float32)
            codes = c.cache.k.view(torch.float8_e4m3fn).float()
            c.kv[0] = (codes.double() * c.cache.k_scales.double().transpose(1, 2)[..., None]).cpu().numpy()
        c.check(gamma=False)


@pytest.mark.parametrize("what", ["tiny", "huge", "mixed", "negative", "zero"])
def test_e4m3_scales_of_any_size(what):
    need_gpu()
    c = Case([300, 20], [2, 1], 4, 2, 64, 16, "e4m3")
    g = torch.Generator(device="cuda").manual_seed(1)
    r = torch.rand(c.cache.v_scales.shape, generator=g, device="cuda")
    f = dict(tiny=1e-25, huge=1e12, mixed=1.0, negative=-1.0, zero=0.0)[what]
    v = c.cache.v_scales
    v.mul_(f if what != "mixed" else torch.exp2(torch.floor(24 * r - 12)))
    if what == "zero":
        v[torch.isnan(v)] = 0.0
    codes = c.cache.v.view(torch.float8_e4m3fn).double()
    c.kv[1] = (codes * v.double().transpose(1, 2)[..., None]).cpu().numpy()
    got = c.check()
    if what == "zero":
        assert not got[0][:3, :256].any()


def test_infinite_queries_stay_in_their_rows():
    need_gpu()
    c = Case([45], [5], 4, 2, 64, 16)
    kw = dict(norm=False, rope=False, gamma=False)
    ref = c.run(**kw)
    c.q[2, 1, 5] = float("inf")
    got = c.run(**kw)
    torch.cuda.synchronize()
    keep = torch.ones((5, 4), dtype=torch.bool)
    keep[2, 1] = False
    a, b = (t[0][:5, :256].view(5, 4, 64).cpu() for t in (got, ref))
    assert torch.equal(a[keep], b[keep]) and torch.isnan(a[2, 1]).all()


@pytest.mark.parametrize("fmt", FMT)
def test_bad_pages_are_reported_and_not_seen(fmt):
    need_gpu()
    c = Case([100, 50], [2, 1], 2, 1, 64, 16, fmt)
    good = c.run()
    for bad in (-1, 10 ** 6, 2 ** 31 - 1):
        c2 = c.table[0, 2]
        c.table[0, 2] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.run(st=st)
        torch.cuda.synchronize()
        assert st.item() == tfd.ERR_DEVICE_DATA
        assert torch.isfinite(got[0].float()).all()
        # the other request reads its own pages (its cuts may fall elsewhere only with the lengths)
        assert torch.equal(got[0][2], good[0][2])
        assert (got[1][:2] < good[1][:2]).all()           # 16 tokens fewer
        c.table[0, 2] = c2


def test_bad_requests_are_left_as_they_were():
    need_gpu()
    for change in ("len", "long", "rows", "back", "past"):
        c = Case([30, 40, 50], [2, 2, 2], 2, 1, 64, 16)
        good = c.run()
        if change == "len":
            c.lens[1] = -5
        elif change == "long":
            c.lens[1] = c.table.shape[1] * 16
        elif change == "rows":                            # more rows than max_new
            c.row_start = np.array([0, 2, 5, 7])
        elif change == "back":
            c.row_start = np.array([0, 2, 1, 3])
        else:
            c.row_start = np.array([0, 2, 4, 9])          # behind the last row
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.run(st=st, max_new=2)
        torch.cuda.synchronize()
        assert st.item() == tfd.ERR_DEVICE_DATA, change
        assert torch.equal(got[0][:1], good[0][:1])
        bad = slice(4, 6) if change == "past" else slice(2, 4)
        if change in ("len", "long", "past"):
            assert (got[0][bad] == 7).all() and (got[1][bad] == 7).all(), change


def test_negative_positions_count_as_zero():
    need_gpu()
    c = Case([30], [2], 2, 1, 64, 16)
    a = c.run(pos=[0, 5, 0, 0])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = c.run(pos=[-3, 5, 0, 0], st=st)
    torch.cuda.synchronize()
    assert st.item() == tfd.ERR_DEVICE_DATA and torch.equal(a[0], b[0])


def test_no_rows_at_all():
    need_gpu()
    c = Case([30, 4], [0, 0], 2, 1, 64, 16)
    got = c.run()
    torch.cuda.synchronize()
    assert (got[0] == 7).all() and (got[1] == 7).all()


def test_shared_pages_and_cache_behind_2_to_the_32_elements():
    """Two requests whose tables name the same pages, the pages at the far end of a large cache."""
    need_gpu()
    pages, page, heads, dim = 16500, 256, 16, 64
    k, v = (torch.empty((pages, page, heads, dim), dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in (k, v):
        t[-2:] = torch.randn((2, page, heads, dim), generator=g, device="cuda")
    q = torch.randn((2, heads, dim), generator=g, device="cuda").bfloat16()
    table = i32([[pages - 1, pages - 2]] * 2)
    kw = dict(norm=False, rope=False, want_lse=True)
    far = tfd.tfd_paged_attn(q, tfd.KvPages(k, v), table, i32([400, 400]), i32([0, 1, 2]), 1, **kw)
    near = tfd.tfd_paged_attn(q, tfd.KvPages(k[-2:].clone(), v[-2:].clone()), i32([[1, 0]] * 2),
                              i32([400, 400]), i32([0, 1, 2]), 1, **kw)
    torch.cuda.synchronize()
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])


def test_on_another_stream_captured_and_replayed():
    need_gpu()
    c = Case([900, 33, 5], [1, 4, 2], 8, 2, 128, 16)
    ref = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lens, start, table = i32(c.lens), i32(c.row_start), i32(c.table)
    out, lse = torch.zeros_like(ref[0][:, :1024]).contiguous(), torch.zeros_like(ref[1])
    ws = torch.zeros_like(c.ws)
    torch.cuda.synchronize()

    def call(stream=None):
        tfd.tfd_paged_attn(c.q, c.cache, table, lens, start, 4, q_gamma=c.gamma, out=out, lse=lse, ws=ws,
                           stream=stream)
    call(side)
    torch.cuda.synchronize()
    assert torch.equal(out[:7], ref[0][:7, :1024])
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for shorter in (0, 100, 0):                           # other lengths in the same graph
        lens[0] = 900 - shorter
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:7], ref[0][:7, :1024]) == (shorter == 0)


def test_without_lse_and_allocating():
    need_gpu()
    c = Case([70], [2], 4, 2, 64, 16)
    ref = c.run()
    out, lse = tfd.tfd_paged_attn(c.q, c.cache, i32(c.table), i32(c.lens), i32(c.row_start), 2,
                                  q_gamma=c.gamma)
    torch.cuda.synchronize()
    assert lse is None and torch.equal(out[:2], ref[0][:2, :256])


def of_64_rows(dim, seed=0):
    """Requests of up to 32 rows of 8 query heads a key head, enough of them for units of 64 rows."""
    g = np.random.default_rng(seed)
    new = np.full(24, 32)
    new[[3, 11, 17]] = 19, 1, 0
    return Case(g.integers(0, 260, 24), new, 16, 2, dim, 16, tid=880 + seed)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [-1, 2, 40, 300])
def test_trees_and_windows_in_units_of_64_rows(window, dim):
    need_gpu()
    g = np.random.default_rng(6)
    c = of_64_rows(dim, seed=1)
    c.lens[8] = 0
    words = np.zeros(c.rows, np.uint32)
    for r, n in enumerate(c.new):
        if n:
            words[c.row_start[r]:c.row_start[r + 1]] = random_tree(int(n), g)
    words[c.row_start[5] + 7] = 0                         # sees the cached tokens alone
    words[c.row_start[8] + 4] = 0                         # nothing cached, nothing seen
    words[c.row_start[9] + 1] = 1 << 1 | 1 << 30          # itself and a later row
    got = c.check(tree=words, window=window, requests=[3, 5, 8, 9, 11, 23])
    row = c.row_start[8] + 4
    assert not got[0][row, :16 * dim].any() and torch.isneginf(got[1][row]).all()
    c.check(window=window, requests=[3, 5, 8, 11, 22])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("what", ["inf", "nan"])
def test_tokens_that_are_not_finite_in_units_of_64_rows(what, dim):
    """Edited in a tile by four groups at once; only the rows that see such a token know of it."""
    need_gpu()
    c = of_64_rows(dim, seed=2)
    ref = c.run()
    for r, j, key in ((5, 9, False), (6, 31, True), (20, 16, True)):
        t = int(c.lens[r]) + j
        page, at = int(c.table[r, t // 16]), t % 16
        keep = c.cache.k[page, at].clone(), c.cache.v[page, at].clone()
        c.cache.v[page, at] = float(what)
        if key:
            c.cache.k[page, at] = float(what)
        got = c.run()
        torch.cuda.synchronize()
        c.cache.k[page, at], c.cache.v[page, at] = keep
        see = np.zeros(c.rows, bool)
        see[c.row_start[r] + j:c.row_start[r + 1]] = True
        assert torch.equal(got[0][~see], ref[0][~see]) and torch.equal(got[1][~see], ref[1][~see])
        x = got[0][see][:, :16 * dim].float()
        assert torch.isposinf(x).all() if what == "inf" and not key else torch.isnan(x).all()
