"""GPU parity of tfd_page_plan: every table, stack, slot and position equal to the oracle's."""
import numpy as np
import pytest
import torch

from helpers import need_gpu
from oracle.paged import plan as oracle_plan
from speculative_decoding_draft_row_gb300 import tfd

pytestmark = pytest.mark.gpu


class State:
    def __init__(self, R, max_pages, pages, page, ldt=None, seed=0):
        self.page = page
        self.table = np.full((R, ldt or max_pages), -7, np.int32)[:, :max_pages]
        self.held = np.zeros(R, np.int32)
        self.free = np.random.default_rng(seed).permutation(pages).astype(np.int32)
        self.n_free = np.array([pages], np.int32)
        self.on_gpu()

    def on_gpu(self):
        wide = torch.from_numpy(np.ascontiguousarray(self.table.base if self.table.base is not None
                                                     else self.table)).cuda()
        self.d = [wide[:, :self.table.shape[1]]] + [torch.from_numpy(x.copy()).cuda() for x in
                                                     (self.held, self.free, self.n_free)]

    def round(self, lens, new, rows, stream=None, bad=False):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = tfd.tfd_page_plan(i32(lens), i32(new), self.page, *self.d, rows=rows or None,
                                dev_status=st)
        torch.cuda.synchronize()
        ex = oracle_plan(lens, new, self.page, self.table, self.held, self.free, self.n_free[0], rows)
        assert ex["bad"] == bad and st.item() == (tfd.ERR_DEVICE_DATA if bad else 0)
        for name, t in zip(("row_start", "slots", "pos"), got):
            if t is not None:
                assert np.array_equal(t.cpu().numpy(), ex[name]), name
        for name, t in zip(("table", "held", "free_ids"), self.d):
            assert np.array_equal(t.cpu().numpy(), ex[name]), name
        assert self.d[3].item() == ex["n_free"]
        self.table[:] = ex["table"]
        self.held, self.free, self.n_free = ex["held"], ex["free_ids"], np.array([ex["n_free"]])
        return ex


@pytest.mark.parametrize("R,page,most", [(1, 16, 40), (4, 16, 600), (33, 1, 30), (511, 24, 90),
                                         (512, 16, 90), (513, 16, 90), (1500, 7, 60), (8192, 64, 200)])
def test_rounds_of_growing_and_turned_down_rows(R, page, most):
    need_gpu()
    g = np.random.default_rng(R)
    max_pages = -(-(most + 40) // page) + 1
    s = State(R, max_pages, R * max_pages, page, ldt=max_pages + 3, seed=R)
    lens = g.integers(0, most, R)
    lens[0] = 0
    for i in range(5):
        new = g.integers(0, 33, R)
        new[g.random(R) < 0.2] = 0
        rows = int(new.sum())
        s.round(lens, new, rows + (0 if i else 9))
        lens = np.minimum(lens + g.integers(0, new + 1), most)
        if i == 2:                                        # some requests end
            gone = g.random(R) < 0.3
            lens[gone] = 0
            s.round(lens, np.zeros(R, int), 0)
    s.round(np.zeros(R, int), np.zeros(R, int), 3)
    assert s.n_free[0] == R * max_pages


@pytest.mark.parametrize("R", [3, 700])
def test_prompts_and_the_stack_as_it_was(R):
    need_gpu()
    s = State(R, 600, 600 * R, 8, seed=5)
    lens = np.arange(R) * 3 % 50
    new = np.full(R, 2)
    new[R // 2] = 4700
    s.round(lens, np.zeros(R, int), 0)
    before = s.free.copy(), s.n_free[0]
    s.round(lens, new, int(new.sum()))
    s.round(lens, np.zeros(R, int), 0)
    assert s.n_free[0] == before[1]
    assert np.array_equal(s.free[:before[1]], before[0][:before[1]])


@pytest.mark.parametrize("R", [6, 600])
def test_pages_run_out(R):
    """A request whose missing pages are not there gets none, and neither do those counted behind it."""
    need_gpu()
    s = State(R, 8, R, 4)
    new = np.full(R, 1)
    new[2], new[4] = 20, 4
    s.round(np.zeros(R, int), new, int(new.sum()), bad=True)
    s.round(np.zeros(R, int), new, int(new.sum()), bad=True)
    s.round(np.zeros(R, int), np.zeros(R, int), 0)
    assert s.n_free[0] == R


def test_bad_lengths_counts_and_stacks():
    need_gpu()
    def state():
        return State(4, 4, 16, 4)
    state().round([-1, 0, 0, 0], [1, 1, 1, 1], 4, bad=True)
    state().round([0, 0, 0, 0], [1, -3, 1, 1], 4, bad=True)
    state().round([0, 13, 0, 0], [1, 4, 1, 1], 8, bad=True)
    state().round([0, 0, 0, 0], [2, 2, 2, 2], 5, bad=True)   # more rows than asked for
    for held in (-1, 5):
        s = state()
        s.held[2] = held
        s.on_gpu()
        s.round([3, 3, 3, 3], [1, 1, 1, 1], 4, bad=True)
    for n_free in (-1, 17):
        s = state()
        s.n_free[0] = n_free
        s.on_gpu()
        s.round([0, 0, 0, 0], [1, 0, 0, 1], 2, bad=True)
    s = state()                                           # pages given back to a full stack
    s.held[:] = 2
    s.table[:] = 3
    s.on_gpu()
    s.round([4, 4, 4, 9], [0, 0, 0, 0], 0, bad=True)
    s = state()                                           # a page that is none
    s.free[-1] = 16
    s.on_gpu()
    s.round([0, 0, 0, 0], [1, 1, 1, 1], 4, bad=True)


def test_captured_and_replayed_on_another_stream():
    """Lengths on the GPU: rounds replayed from one graph, each from what the last one left."""
    need_gpu()
    R, page = 5, 4
    s = State(R, 30, 90, page)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, new = torch.zeros(R, **i32), torch.full((R,), 3, **i32)
    start, slots, pos = torch.zeros(R + 1, **i32), torch.zeros(20, **i32), torch.zeros(20, **i32)
    kept = torch.tensor([0, 1, 2, 3, 1], **i32)

    def step():
        tfd.tfd_page_plan(lens, new, page, *s.d, row_start=start, slots=slots, pos=pos)
        lens.add_(kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for _ in range(10):
            graph.replay()
    torch.cuda.synchronize()
    ln = np.zeros(R, int)
    for _ in range(11):
        ex = oracle_plan(ln, [3] * R, page, s.table, s.held, s.free, s.n_free[0], 20)
        s.table[:], s.held, s.free = ex["table"], ex["held"], ex["free_ids"]
        s.n_free = np.array([ex["n_free"]])
        ln = ln + kept.cpu().numpy()
    for name, t in zip(("table", "held", "free_ids", "n_free", "slots", "pos"),
                       [*s.d, slots, pos]):
        assert np.array_equal(t.cpu().numpy().reshape(-1), np.asarray(ex[name]).reshape(-1)), name


@pytest.mark.parametrize("R,page", [(6, 4), (512, 1), (600, 4)])
def test_pages_that_are_none_do_not_come_back(R, page):
    """Ids outside the cache in what requests give back are reported and left out of the stack: the pages that are
    there move as ever, in the same call too, and later requests get pages that are some."""
    need_gpu()
    s = State(R, 40, 40 * R, page, seed=R)
    new = np.full(R, 20)
    s.round(np.zeros(R, int), new, int(new.sum()))
    had = s.held.copy()
    s.table[2, 1], s.table[2, int(had[2]) - 1], s.table[R - 1, 0] = -3, 10 ** 6, 40 * R
    s.n_free = s.n_free.astype(np.int32)
    s.on_gpu()
    lens, new = np.full(R, 20), np.full(R, 10)            # the others grow meanwhile
    lens[[1, 2, R - 1]], new[[1, 2, R - 1]] = 0, 0
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    st = i32([0])
    got = tfd.tfd_page_plan(i32(lens), i32(new), page, *s.d, rows=int(new.sum()), dev_status=st)
    torch.cuda.synchronize()
    ex = oracle_plan(lens, new, page, s.table, s.held, s.free, s.n_free[0], int(new.sum()))
    assert ex["bad"] and st.item() == tfd.ERR_DEVICE_DATA
    for name, t in zip(("row_start", "slots", "pos"), got):
        assert np.array_equal(t.cpu().numpy(), ex[name]), name
    table, held, free, n_free = (t.cpu().numpy() for t in s.d)
    assert n_free[0] == ex["n_free"]
    assert np.array_equal(free[:n_free[0]], ex["free_ids"][:n_free[0]])   # what stands behind is of no meaning
    assert np.array_equal(table, ex["table"]) and np.array_equal(held, ex["held"])
    s.table[:], s.held, s.free, s.n_free = table, held, free, n_free
    mine = np.concatenate([free[:n_free[0]]] + [table[r, :held[r]] for r in range(R)])
    assert len(set(mine.tolist())) == len(mine) == 40 * R - 3 and mine.min() >= 0 and mine.max() < 40 * R
    s.round(np.zeros(R, int), np.full(R, 37), 37 * R)     # and a round that is sound
    s.round(np.zeros(R, int), np.zeros(R, int), 0)
    assert s.n_free[0] == 40 * R - 3


@pytest.mark.parametrize("R,new,max_pages", [(512, 2, 40), (32, 32, 40), (41, 25, 60), (513, 1, 30), (1, 1024, 300),
                                             (1, 1025, 300), (512, 1, 4), (409, 1, 5), (410, 1, 5)])
def test_sizes_around_one_block(R, new, max_pages):
    """Rounds of about 1024 rows, about 512 requests, and pages given back without rows, about 2048 that can move."""
    need_gpu()
    s = State(R, max_pages, R * max_pages, 4, seed=R + new)
    lens, n = np.arange(R) % 7, np.full(R, new)
    lens[n + lens > 4 * max_pages] = 0
    s.round(lens, np.zeros(R, int), 0)
    for i in range(3):
        s.round(lens, n, R * new + (i == 1))
        s.round(lens, np.zeros(R, int), 0)
    s.round(np.zeros(R, int), np.zeros(R, int), 0)
    assert s.n_free[0] == R * max_pages
