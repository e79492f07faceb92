"""tfd_sample on its less travelled ways: a top_k too long for the list with other filters behind it, a
top-p border among very small weights, lists that overflow on unequal logits, and the longest rows.

Tolerances are those of test_gpu_sample.py. A row counts as clear where the oracle's margin is above
draw_tol(n): rows are chosen so that most are."""
import itertools

import numpy as np
import pytest
import torch

from helpers import need_gpu
from speculative_decoding_draft_row_gb300 import tfd
from test_gpu_sample import PROB_REL, check, dev, logits, run

pytestmark = pytest.mark.gpu


def uniform(rows, seed):
    u = np.random.default_rng([0, 93, seed]).random(rows, dtype=np.float32)
    return np.minimum(u, np.float32(1 - 2.0 ** -24))


def combine(n, ks, ps, mps):
    c = [(k, p, mp) for k, p, mp in itertools.product(ks, ps, mps) if k < n]
    return dict(temperature=np.full(len(c), 0.9, np.float32),
                top_k=np.array([k for k, _, _ in c], np.int32),
                top_p=np.array([p for _, p, _ in c], np.float32),
                min_p=np.array([m for _, _, m in c], np.float32))


@pytest.mark.parametrize("n,dtype", [(1800, torch.float32), (5003, torch.float32),
                                     (50021, torch.bfloat16), (163840, torch.float32)])
def test_a_long_top_k_before_top_p_and_min_p(n, dtype):
    """top_k above the list's 1024: its border and top-p's come from the row's histogram."""
    need_gpu()
    s = combine(n, [1025, 1500, 4000, 20000], [1.0, 0.5, 0.9, 0.999], [0.0, 1e-3, 1e-6])
    rows = len(s["top_k"])
    x, u = logits(rows, n, 51), uniform(rows, n)
    got = run(x, u, s, dtype)
    check(got, got[4], u, s)


@pytest.mark.parametrize("n", [50021, 163840])
@pytest.mark.parametrize("equal", [False, True])
def test_top_p_ends_among_weights_below_2_to_minus_20(n, equal):
    """One large column and many small ones that together hold a few percent of the mass. At n = 163840
    a small one is w = 1 / (40 n) = 1.5e-7 of the mass, draw_tol(n) 1.9e-8: a margin, even over
    [0, w / 2], is above it in (1 - 2 * 1.9e-8 / 1.5e-7) = 0.75 of all cases, and a row has two, so
    fewer than elsewhere are clear (the oracle says 4 of the 6)."""
    need_gpu()
    tail = np.float32(-np.log(n * 40.0))                 # together about 1/40 of the large one's
    rng = np.random.default_rng([0, 94, n])
    x = np.full((6, n), tail, np.float32)
    if not equal:
        x += (0.3 * rng.standard_normal(x.shape)).astype(np.float32)
    x[np.arange(6), rng.integers(0, n, 6)] = 0
    assert tail * np.log2(np.e) < -20.5
    s = dict(top_p=np.array([0.98, 0.985, 0.99, 0.999, 0.98, 0.98], np.float32),
             min_p=np.array([0, 0, 0, 0, 1e-9, 1e-5], np.float32))
    u = np.array([0.98, 0.995, 0.5, 0.999, 0.9975, 0.3], np.float32)
    got = run(x, u, s)
    check(got, got[4], u, s, need=0.6)


@pytest.mark.parametrize("n", [20000, 163840])
def test_more_unequal_logits_in_a_bin_than_the_list_holds(n):
    """Far more than 1024 columns close under the largest, beside a region far below that stretches the
    bins: the short list overflows, and the histogram's bin is split by keys."""
    need_gpu()
    rng = np.random.default_rng([0, 95, n])
    s = combine(n, [0, 50, 900, 3000], [1.0, 0.3, 0.9], [0.0, 0.9999])
    rows = len(s["top_k"])
    x = (5 + 1e-3 * rng.random((rows, n))).astype(np.float32)
    x[:, n // 2:] = -20 - rng.random((rows, n - n // 2)).astype(np.float32)
    u = uniform(rows, n)
    got = run(x, u, s)
    check(got, got[4], u, s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_histograms_of_the_longest_rows(dtype):
    need_gpu()
    n = 1 << 20
    s = dict(top_p=np.array([0.3, 0.9, 0.99, 1, 1, 0.9, 0.9, 1], np.float32),
             top_k=np.array([0, 0, 0, 2000, 100000, 2000, 100000, 0], np.int32),
             temperature=np.full(8, 0.5, np.float32))
    x, u = logits(8, n, 61), uniform(8, 62)
    got = run(x, u, s, dtype)
    check(got, got[4], u, s, need=0.7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
def test_the_largest_sums(dtype, shift):
    """2^20 equal weights sum to 2^63 exactly; counts decide. Rows that start off a 16-byte boundary
    have a column or more above 65536 in a block."""
    need_gpu()
    n = 1 << 20
    half = np.float32(0.5)
    k = np.array([0, 0, 2000, 2000, 600000, 0], np.int32)
    p = np.array([1, half, 1, half, half, 1], np.float32)
    u = np.array([1 - 2.0 ** -24, 0.75, 0.999, 0.25, 0.5, 0.0], np.float32)
    kept = [n, n // 2, 2000, 1000, 300000, n]
    rows = len(k)
    buf = torch.full((rows, n + 8), float("nan"), dtype=dtype, device="cuda")
    x = buf[:, shift:shift + n]
    x.fill_(3.25)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, prob, probs = tfd.tfd_sample(x, torch.from_numpy(u).cuda(), want_probs=True, dev_status=st,
                                      **dev(dict(top_k=k, top_p=p)))
    torch.cuda.synchronize()
    assert st.item() == 0
    for r in range(rows):
        assert ids[r].item() == int(np.float64(u[r]) * kept[r])
        assert (probs[r] > 0).sum().item() == kept[r] and (probs[r, :kept[r]] > 0).all()
        assert abs(prob[r].item() * kept[r] - 1) <= PROB_REL


def test_captured_behind_copies_and_between_joined_streams():
    """A draw whose predecessors in the graph are a copy and another stream's kernel waits for both."""
    need_gpu()
    rows, n = 4, 30011
    xs = [torch.from_numpy(logits(rows, n, 70 + i)).cuda() for i in range(3)]
    s = dev(dict(top_k=np.array([0, 50, 20, 2000], np.int32),
                 top_p=np.array([0.9, 0.8, 1, 1], np.float32)))
    u = [torch.from_numpy(uniform(rows, 71 + i)).cuda() for i in range(3)]
    ref = [tfd.tfd_sample(x, v, want_probs=True, **s) for x, v in zip(xs, u)]
    src, usrc = xs[0].clone(), u[0].clone()
    x, v = torch.zeros_like(src), torch.zeros_like(usrc)
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    probs, copy = torch.zeros((rows, n), device="cuda"), torch.zeros((rows, n), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            v.copy_(usrc)
        x.copy_(src)
        main.wait_stream(side)
        tfd.tfd_sample(x, v, ids=ids, probs=probs, **s)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            copy.copy_(probs)
        main.wait_stream(side)
    for i in (0, 1, 2, 0):
        src.copy_(xs[i])
        usrc.copy_(u[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, ref[i][0]) and torch.equal(probs, ref[i][2])
        assert torch.equal(copy, probs)
