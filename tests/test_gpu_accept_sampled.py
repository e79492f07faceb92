"""GPU parity of tfd_accept_sampled against the oracle: kept counts and histograms exact, the next
token equal wherever the oracle's margin exceeds the integer sums' error: each column is rounded to
a multiple of 2^-43, p and q both, so a running mass is within n * 2^-43 of the exact one; divided
by the total mass. Its probability carries that, two conversions and a division (2^-22 relative)."""
import numpy as np
import pytest
import torch

from helpers import need_gpu
from oracle.accept import accept as oracle_accept
from oracle.sample import accept_sampled as oracle_accept_sampled
from speculative_decoding_draft_row_gb300 import tfd

pytestmark = pytest.mark.gpu


def make(S, W, n, seed, nq=None, near=0.7):
    rng = np.random.default_rng([0, 95, seed])
    lp = rng.standard_normal((S, W + 1, n)) * 2.5
    lq = lp[:, :W] + near * rng.standard_normal((S, W, n))

    def soft(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    q_map = None
    if nq is not None:
        cols = rng.permutation(n)[:nq]
        q_map = np.full(n, -1, np.int32)
        q_map[cols] = np.arange(nq)
        lq = lq[:, :, cols]
    p, q = soft(lp), soft(lq)
    c = np.cumsum(q.astype(np.float64), -1)
    j = (c <= rng.random((S, W, 1)) * c[..., -1:]).sum(-1).clip(max=c.shape[-1] - 1)
    drafts = (j if nq is None else cols[j]).astype(np.int32)
    asked = rng.integers(0, W + 1, S).astype(np.int32)
    asked[::2] = W
    u, un = rng.random((S, W), dtype=np.float32), rng.random(S, dtype=np.float32)
    return p, q, drafts, asked, u, un, q_map


def run(p, q, d, asked, u, un, q_map=None, hist=True, **kw):
    W = d.shape[1]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ah = torch.full((W,), 3, dtype=torch.int64, device="cuda")
    kh = torch.full((W,), 1, dtype=torch.int64, device="cuda")
    t = [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (p, q, d, asked, u, un)]
    qm = None if q_map is None else torch.from_numpy(q_map).cuda()
    k, nx, pr = tfd.tfd_accept_sampled(*t, q_map=qm, asked_hist=ah if hist else None,
                                       kept_hist=kh if hist else None, dev_status=st, **kw)
    torch.cuda.synchronize()
    return (k.cpu().numpy(), nx.cpu().numpy(), pr.cpu().numpy(), ah.cpu().numpy() - 3,
            kh.cpu().numpy() - 1, st.item())


def check(got, args):
    p, q, d, asked, u, un, q_map = args
    k, nx, pr, ah, kh, st = got
    ok, onx, opr, margin, bad = oracle_accept_sampled(p, q, d, asked, u, un, q_map)
    assert np.array_equal(k, ok)
    W, n = d.shape[1], p.shape[2]
    want = oracle_accept(np.zeros((len(ok), W)), np.where(bad, -1, asked),
                         (np.arange(W)[None] >= ok[:, None]).astype(int))
    assert np.array_equal(ah, want[1]) and np.array_equal(kh, want[2])
    assert st == (tfd.ERR_DEVICE_DATA if bad.any() else 0)
    clear = 0
    for s in range(len(ok)):
        if onx[s] < 0:
            assert nx[s] == -1 and pr[s] == 0
            continue
        # mass of the distribution drawn from, before it is normalised
        m = ok[s]
        qr = np.zeros(n)
        if m < asked[s]:
            qr = q[s, m].astype(np.float64) if q_map is None else \
                np.where(q_map >= 0, q[s, m][np.maximum(q_map, 0)], 0).astype(np.float64)
        r = np.maximum(p[s, m].astype(np.float64) - qr, 0)
        tol = n * 2.0 ** -43 / (r.sum() or p[s, m].sum())
        if margin[s] > tol:
            assert nx[s] == onx[s]
            assert abs(pr[s] - opr[s]) <= 2.0 ** -22 * opr[s] + 2 * tol
            clear += 1
    assert clear >= 0.5 * (onx >= 0).sum()


@pytest.mark.parametrize("S,W,n,nq", [
    (1, 1, 1, None), (1, 1, 4096, None), (3, 2, 7, None), (4, 5, 163840, None),
    (9, 4, 31999, None), (40, 3, 2051, None), (200, 2, 513, None), (3, 4, 5001, 1200),
    (2, 512, 33, None), (5, 3, 100003, 32000)])
def test_against_the_oracle(S, W, n, nq):
    need_gpu()
    a = make(S, W, n, S + n, nq)
    check(run(*a), a)


@pytest.mark.parametrize("near", [0.0, 0.05, 3.0])
def test_near_and_far_drafts(near):
    """Equal rows keep every draft; rows far apart turn nearly all down."""
    need_gpu()
    a = make(12, 4, 3001, 7, near=near)
    got = run(*a)
    check(got, a)
    if near == 0.0:
        assert np.array_equal(got[0], a[3])


def test_equal_rows_with_a_draft_of_no_mass():
    """p == q and a draft without mass in either is turned down: the next token comes from p."""
    need_gpu()
    p = np.zeros((2, 2, 300), np.float32)
    p[:, :, 5], p[:, :, 250] = 0.5, 0.5
    q = p[:, :1].copy()
    args = (p, q, np.array([[7], [5]], np.int32), np.array([1, 1], np.int32),
            np.array([[0.25], [0.5]], np.float32), np.array([0.5, 0.49], np.float32), None)
    k, nx, pr, _, _, st = run(*args)
    assert k.tolist() == [0, 1] and nx.tolist() == [250, 5] and pr.tolist() == [0.5, 0.5]


def test_one_hot_rows_are_the_greedy_accept():
    need_gpu()
    S, W, n = 8, 4, 1000
    rng = np.random.default_rng(5)
    want, d = rng.integers(0, n, (S, W + 1)), rng.integers(0, n, (S, W))
    d = np.where(rng.random((S, W)) < 0.7, want[:, :W], d).astype(np.int32)
    p = np.eye(n, dtype=np.float32)[want]
    q = np.eye(n, dtype=np.float32)[d]
    asked = np.full(S, W, np.int32)
    u, un = rng.random((S, W), dtype=np.float32), rng.random(S, dtype=np.float32)
    k, nx, pr, _, _, _ = run(p, q, d, asked, u, un)
    ok = oracle_accept(d, asked, want[:, :W])[0]
    assert np.array_equal(k, ok) and np.array_equal(nx, want[np.arange(S), ok])
    assert (pr == 1).all()


def test_bad_streams_empty_rows_and_values_out_of_range():
    need_gpu()
    S, W, n = 8, 3, 777
    p, q, d, asked, u, un, _ = make(S, W, n, 9)
    asked[:] = W
    asked[0], asked[1] = W + 1, -1
    d[2, 1], d[3, 2] = n, -1
    u[4, 0] = 1.0
    un[5] = np.nan
    p[6] = 0.0                                        # no mass at all
    p[7, 0, :5], q[7, 0, 5:9] = np.nan, -1.0
    a = (p, q, d, asked, u, un, None)
    got = run(*a)
    check(got, a)
    assert (got[1][:7] == -1).all() and (got[0][:6] == 0).all()
    # what lies behind the asked drafts is not looked at
    asked[2], asked[3], asked[4] = 1, 2, 0
    a = (p, q, d, asked, u, un, None)
    got = run(*a)
    check(got, a)
    assert (got[1][2:5] >= 0).all()


def test_strided_rows_and_no_histograms():
    need_gpu()
    S, W, n = 5, 3, 1003
    a = make(S, W, n, 21)
    ref = run(*a)
    p = torch.full((S, W + 1, n + 6), 0.5, device="cuda")
    q = torch.full((S, W, n + 1), 0.5, device="cuda")
    p[:, :, :n], q[:, :, :n] = torch.from_numpy(a[0]).cuda(), torch.from_numpy(a[1]).cuda()
    t = [torch.from_numpy(v).cuda() for v in a[2:6]]
    k, nx, pr = tfd.tfd_accept_sampled(p[:, :, :n], q[:, :, :n], *t)
    assert np.array_equal(k.cpu().numpy(), ref[0]) and np.array_equal(nx.cpu().numpy(), ref[1])
    assert np.array_equal(pr.cpu().numpy(), ref[2])


def test_sampled_rows_then_accept_captured():
    """Drafts drawn by tfd_sample, the target's rows filtered by it, the accept: one graph."""
    need_gpu()
    S, W, n = 4, 3, 20011
    rng = np.random.default_rng(31)
    lt = torch.from_numpy(rng.standard_normal((S * (W + 1), n), dtype=np.float32) * 3).cuda()
    ld = (lt.view(S, W + 1, n)[:, :W] + 0.3).contiguous()
    ld += 0.5 * torch.from_numpy(rng.standard_normal((S, W, n), dtype=np.float32)).cuda()
    f = dict(dtype=torch.float32, device="cuda")
    ud, ut = torch.rand((W, S), **f), torch.rand(S * (W + 1), **f)
    u, un = torch.rand((S, W), **f), torch.rand(S, **f)
    tp, tpt = torch.full((S,), 0.9, **f), torch.full((S * (W + 1),), 0.9, **f)
    drafts = torch.zeros((S, W), dtype=torch.int32, device="cuda")
    q, p = torch.zeros((S, W, n), **f), torch.zeros((S, W + 1, n), **f)
    asked = torch.full((S,), W, dtype=torch.int32, device="cuda")
    k, nx = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))

    def step():
        for t in range(W):
            tfd.tfd_sample(ld[:, t], ud[t], top_p=tp, ids=drafts[:, t], probs=q[:, t])
        tfd.tfd_sample(lt, ut, top_p=tpt, probs=p.view(-1, n))
        tfd.tfd_accept_sampled(p, q, drafts, asked, u, un, n_kept=k, next_ids=nx)

    step()
    torch.cuda.synchronize()
    first = [v.clone() for v in (drafts, q, p, k, nx)]
    ok, onx, _, margin, _ = oracle_accept_sampled(p.cpu().numpy(), q.cpu().numpy(),
                                                  drafts.cpu().numpy(), asked.cpu().numpy(),
                                                  u.cpu().numpy(), un.cpu().numpy())
    assert np.array_equal(k.cpu().numpy(), ok)
    clear = margin > 1e-7
    assert np.array_equal(nx.cpu().numpy()[clear], onx[clear])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for v in (drafts, q, p, k, nx):
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    for v, w in zip((drafts, q, p, k, nx), first):
        assert torch.equal(v, w)
