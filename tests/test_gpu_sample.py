"""GPU parity of tfd_sample against the oracle.

Tolerances. A weight is within 2^-38 relative and 2^-44 (of the largest) absolute of the exact one,
so a row's running masses are within DRAW_TOL(n) = 2^-37 + n * 2^-43 of the exact ones, relative to
the total (which is at least the largest weight). A row whose oracle margin is above that has the
oracle's token; below it, a neighbour of the border is as good. A probability carries the
hardware's 2^x (2^-22 at most) with its correction, the total's conversion, a division and a product
(2^-24 each, two for the correction), and its total DRAW_TOL: PROB_REL = 2.5 * 2^-22 relative, plus
2^-44 absolute at the cut."""
import numpy as np
import pytest
import torch

from helpers import need_gpu
from oracle.sample import sample as oracle_sample
from speculative_decoding_draft_row_gb300 import tfd

pytestmark = pytest.mark.gpu

PROB_REL, PROB_ABS = 2.5 * 2.0 ** -22, 2.0 ** -44


def draw_tol(n):
    return 2.0 ** -37 + n * 2.0 ** -43


def logits(rows, n, seed, std=2.5):
    rng = np.random.default_rng([0, 90, seed])
    x = rng.standard_normal((rows, n), dtype=np.float32) * np.float32(std)
    for r in range(rows):
        at = rng.integers(0, n, 8)
        x[r, at] += rng.random(8, dtype=np.float32) * 9
    return x


def settings(rows, mode, seed):
    rng = np.random.default_rng([0, 91, seed])
    s = dict(temperature=rng.choice(np.array([0.3, 0.7, 1.0, 1.6], np.float32), rows))
    if mode in ("top_k", "all", "mixed"):
        s["top_k"] = rng.choice(np.array([1, 2, 20, 50, 700], np.int32), rows)
    if mode in ("top_p", "all", "mixed"):
        s["top_p"] = rng.choice(np.array([0.1, 0.8, 0.9, 0.99], np.float32), rows)
    if mode in ("min_p", "all", "mixed"):
        s["min_p"] = rng.choice(np.array([0.01, 0.05, 0.2], np.float32), rows)
    if mode == "mixed":
        for k, off in (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0), ("temperature", 0.0)):
            s[k][rng.random(rows) < 0.4] = off
    u = rng.random(rows, dtype=np.float32)
    return s, np.minimum(u, np.float32(1 - 2.0 ** -24))


def dev(s):
    return {k: torch.from_numpy(v).cuda() for k, v in s.items()}


def run(x, u, s, dtype=torch.float32, probs=True, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    xg = torch.from_numpy(x).cuda().to(dtype)
    ids, prob, pr = tfd.tfd_sample(xg, torch.from_numpy(u).cuda(), want_probs=probs,
                                   dev_status=st, **dev(s), **kw)
    torch.cuda.synchronize()
    return (ids.cpu().numpy(), prob.cpu().numpy(), None if pr is None else pr.cpu().numpy(),
            st.item(), xg.double().cpu().numpy())


def check(got, x64, u, s, id_map=None, need=0.9):
    ids, prob, probs, st, _ = got
    assert st == 0
    oi, op, margin = oracle_sample(x64, u, id_map=id_map, **s)
    clear = margin > draw_tol(x64.shape[1])
    assert clear.mean() >= need
    assert np.array_equal(ids[clear], oi[clear])
    col = oi if id_map is None else np.array([int(np.flatnonzero(np.asarray(id_map) == i)[0])
                                              if i >= 0 else 0 for i in oi])
    for r in np.flatnonzero(clear):
        want = op[r, col[r]] if oi[r] >= 0 else 0.0
        assert abs(prob[r] - want) <= PROB_REL * want
        if probs is not None:
            d = np.abs(probs[r] - op[r])
            assert (d <= PROB_REL * op[r] + PROB_ABS).all(), (r, d.max())


@pytest.mark.parametrize("mode", ["none", "top_k", "top_p", "min_p", "all", "mixed"])
@pytest.mark.parametrize("rows,n,dtype", [
    (1, 1, torch.float32), (3, 2, torch.bfloat16), (5, 31, torch.float32),
    (2, 4096, torch.float32), (7, 4097, torch.bfloat16), (40, 5003, torch.float32),
    (3, 50021, torch.bfloat16), (4, 163840, torch.float32)])
def test_against_the_oracle(rows, n, dtype, mode):
    need_gpu()
    x = logits(rows, n, n + rows)
    s, u = settings(rows, mode, n)
    got = run(x, u, s, dtype)
    # few columns: a bf16 row may have its border on an exact tie, so fewer rows are clear
    check(got, got[4], u, s, need=0.5 if n < 100 else 0.9)


@pytest.mark.parametrize("dtype,n", [(torch.float32, 1 << 20), (torch.bfloat16, 1 << 20),
                                     (torch.float32, 700001)])
def test_the_longest_rows(dtype, n):
    need_gpu()
    x = logits(2, n, 5)
    s, u = settings(2, "all", 6)
    got = run(x, u, s, dtype)
    check(got, got[4], u, s, need=0.0)
    s, u = settings(2, "none", 6)
    got = run(x, u, s, dtype)
    check(got, got[4], u, s, need=0.0)


def test_many_rows_equal_the_same_rows_alone():
    """Another launch shape (blocks a row) gives the same bits."""
    need_gpu()
    x = logits(160, 20011, 7)
    s, u = settings(160, "mixed", 8)
    ids, prob, probs, _, _ = run(x, u, s)
    for r in (0, 3, 77, 159):
        one = {k: v[r:r + 1].copy() for k, v in s.items()}
        i1, p1, pr1, _, _ = run(x[r:r + 1], u[r:r + 1], one)
        assert i1[0] == ids[r] and p1[0] == prob[r] and np.array_equal(pr1[0], probs[r])


@pytest.mark.parametrize("n", [5, 300, 4096, 70000])
def test_equal_logits(n):
    """Every weight the same: counts decide, ties to the lower id; the list of undecided columns
    overflows and is split by ids."""
    need_gpu()
    rows = 6
    x = np.full((rows, n), -1.25, np.float32)
    half = np.float32(0.5)
    s = dict(top_k=np.array([0, n // 2, 1, 0, 0, n // 2], np.int32),
             top_p=np.array([1, 1, 1, half, half, half], np.float32),
             min_p=np.array([0, 0, 0, 0, 1, 0], np.float32))
    u = np.array([0.5, 0.0, 0.9, 0.75, 0.0, 0.999], np.float32)
    ids, prob, probs, st, _ = run(x, u, s)
    a, b = max(1, n // 2), -(-n // 2)
    kept = [n, a, 1, b, b, -(-a // 2)]
    if n // 2 == 0:
        kept[1], kept[5] = n, b
    for r in range(rows):
        assert ids[r] == int(np.float64(u[r]) * kept[r])
        assert (probs[r] > 0).sum() == kept[r] and (probs[r][:kept[r]] > 0).all()
        np.testing.assert_allclose(probs[r][:kept[r]], 1.0 / kept[r], rtol=PROB_REL)
    assert st == 0


def test_ties_by_mapped_id():
    need_gpu()
    n = 9001
    rng = np.random.default_rng(3)
    id_map = rng.permutation(n).astype(np.int32)
    x = np.zeros((2, n), np.float32)
    x[1, ::3] = 1.0
    s = dict(top_k=np.array([1000, 1500], np.int32))
    u = np.array([0.3, 0.8], np.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, _, probs = tfd.tfd_sample(torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda(),
                                   id_map=torch.from_numpy(id_map).cuda(), want_probs=True,
                                   dev_status=st, **dev(s))
    probs = probs.cpu().numpy()
    oi, op, _ = oracle_sample(x, u, id_map=id_map, **s)
    for r in range(2):
        assert np.array_equal(probs[r] > 0, op[r] > 0)
        assert ids[r].item() == oi[r]


def test_masked_rows_nan_and_infinities():
    need_gpu()
    n = 6007
    x = logits(8, n, 11)
    x[0] = -np.inf                                   # nothing left
    x[1] = np.nan
    x[2, 1:] = -np.inf                               # one left
    x[3, ::2] = np.nan                               # NaN has no mass
    x[4, [5, 17, 900]] = np.inf                      # these share it
    x[5, :] = np.finfo(np.float32).min               # the type's lowest value is a value
    x[6, 100:] = np.finfo(np.float32).min
    x[7, :] = -np.inf
    x[7, n - 1] = -3e38
    u = np.array([0.5, 0.5, 0.99, 0.25, 0.5, 0.5, 0.7, 0.0], np.float32)
    for mode in ("none", "top_k", "top_p", "all"):
        s, _ = settings(8, mode, 12)
        got = run(x, u, s)
        check(got, x.astype(np.float64), u, s, need=0.5)
        ids = got[0]
        assert ids[0] == -1 and ids[1] == -1 and ids[2] == 0 and ids[7] == n - 1
        assert got[1][0] == 0 and not got[2][:2].any()
        if mode == "none":
            assert ids[4] == 17


def test_extreme_settings():
    need_gpu()
    n = 3001
    x = logits(9, n, 13)
    s = dict(temperature=np.array([0, 1e-6, 1e-39, 1e30, 3e38, 1, 1, 1, 100], np.float32),
             top_k=np.array([0, 0, 0, 0, 0, n, n + 5, -3, 0], np.int32),
             top_p=np.array([1, 1, 0.9, 1, 1, 2.0, 0.0, -1.0, 0.9], np.float32),
             min_p=np.array([0, 0, 0, 0, 0, -1, 0, 0, 5.0], np.float32))
    u = np.array([0.9, 0.9, 0.5, 0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.9, 0.9, 0.9], np.float32)
    ids, prob, probs, st, _ = run(x, u, s)
    top = x.argmax(1)
    for r in (0, 1, 2, 6, 7, 8):
        assert ids[r] == top[r] and prob[r] == 1.0 and probs[r].sum() == 1.0
    assert ids[3] == 0                               # u = 0: the first column with mass
    assert ids[4] == n - 1                           # all but equal weights: the last one
    oi, _, margin = oracle_sample(x[5:6], u[5:6])
    assert ids[5] == oi[0] and margin[0] > draw_tol(n)
    assert st == 0


def test_bad_settings_set_the_status_and_leave_the_other_rows():
    need_gpu()
    n, rows = 5001, 8
    x = logits(rows, n, 14)
    good = dict(temperature=np.full(rows, 0.8, np.float32), top_p=np.full(rows, 0.9, np.float32),
                min_p=np.full(rows, 0.01, np.float32))
    u = np.full(rows, 0.4, np.float32)
    ref = run(x, u, good)
    bad = {k: v.copy() for k, v in good.items()}
    ub = u.copy()
    bad["temperature"][:3] = [-1.0, np.nan, np.inf]
    bad["top_p"][3] = np.nan
    bad["min_p"][4] = np.nan
    ub[5:7] = [1.0, np.nan]
    ids, prob, probs, st, _ = run(x, ub, bad)
    assert st == tfd.ERR_DEVICE_DATA
    assert (ids[:7] == -1).all() and not prob[:7].any() and not probs[:7].any()
    assert ids[7] == ref[0][7] and np.array_equal(probs[7], ref[2][7])


def test_strides_columns_and_what_lies_beyond():
    """Rows at odd strides, ids and probabilities in a column of a larger array, a distribution in
    the middle of one: nothing else is written."""
    need_gpu()
    rows, n = 5, 4999
    x = logits(rows, n, 15)
    s, u = settings(rows, "all", 16)
    ref = run(x, u, s)
    for dtype, pad in ((torch.float32, 3), (torch.bfloat16, 5)):
        wide = torch.full((rows, n + pad), float("nan"), dtype=dtype, device="cuda")
        wide[:, :n] = torch.from_numpy(x).cuda().to(dtype)
        ids = torch.full((rows, 4), -7, dtype=torch.int32, device="cuda")
        prob = torch.full((rows, 4), -7.0, device="cuda")
        probs = torch.full((rows, 3, n + 2), -7.0, device="cuda")
        out = probs.view(rows, -1)[:, :n] if dtype == torch.float32 else probs[:, 0, :n]
        tfd.tfd_sample(wide, torch.from_numpy(u).cuda(), ids=ids[:, 2], prob=prob[:, 2],
                       probs=out, n=n, **dev(s))
        if dtype == torch.float32:
            assert np.array_equal(ids[:, 2].cpu().numpy(), ref[0])
            assert np.array_equal(out.cpu().numpy(), ref[2])
        else:
            oi, _, margin = oracle_sample(wide[:, :n].double().cpu().numpy(), u, **s)
            clear = margin > draw_tol(n)
            assert np.array_equal(ids[:, 2].cpu().numpy()[clear], oi[clear])
        assert (ids[:, [0, 1, 3]] == -7).all() and (prob[:, [0, 1, 3]] == -7).all()
        assert (probs[:, 1:] == -7).all() and (probs[:, 0, n:] == -7).all()


def test_even_numbers_give_every_token_its_share():
    need_gpu()
    m, n = 4096, 257
    x = np.repeat(logits(1, n, 17, std=1.0), m, 0)
    u = ((np.arange(m) + 0.5) / m).astype(np.float32)
    ids, _, probs, _, _ = run(x, u, {})
    got = np.bincount(ids, minlength=n)
    assert (np.diff(ids) >= 0).all()
    assert (np.abs(got - probs[0].astype(np.float64) * m) <= 1.0 + 1e-3).all()


def test_captured_replayed_and_on_two_streams():
    need_gpu()
    rows, n = 4, 30011
    xs = [torch.from_numpy(logits(rows, n, 20 + i)).cuda() for i in range(2)]
    s, u = settings(rows, "all", 21)
    sd, ud = dev(s), torch.from_numpy(u).cuda()
    ref = [tfd.tfd_sample(x, ud, want_probs=True, **sd) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    probs = torch.zeros((rows, n), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tfd.tfd_sample(x, ud, ids=ids, probs=probs, **sd)
    for i in (0, 1, 0):
        x.copy_(xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, ref[i][0]) and torch.equal(probs, ref[i][2])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = [tfd.tfd_sample(xs[i % 2], ud, want_probs=True, stream=streams[i % 2], **sd)
           for i in range(8)]
    torch.cuda.synchronize()
    for i, o in enumerate(out):
        assert torch.equal(o[0], ref[i % 2][0]) and torch.equal(o[2], ref[i % 2][2])


def test_binding_refuses_wrong_tensors():
    need_gpu()
    x = torch.zeros((2, 64), device="cuda")
    u = torch.zeros(2, device="cuda")
    for bad in (dict(logits=x.half()), dict(logits=x.t()), dict(u=u[:1]), dict(u=u.double()),
                dict(top_k=u), dict(temperature=u.cpu()), dict(n=65),
                dict(probs=torch.zeros((2, 63), device="cuda"))):
        a = dict(logits=x, u=u)
        a.update(bad)
        with pytest.raises(ValueError):
            tfd.tfd_sample(**a)
    with pytest.raises(tfd.TfdError):
        tfd.tfd_sample(x, u, probs=x)                # overlaps the logits
