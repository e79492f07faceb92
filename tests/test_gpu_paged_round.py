"""The paged cache's calls together: rounds of plan, append and attend with drafts turned down between them,
against the oracle's cache; and the draft pass over pages."""
import numpy as np
import pytest
import torch

from helpers import assert_bf16_rounding, need_gpu, np32
from oracle.paged import attend, turned
from oracle.quant import quant_fp8_row
from paged_cases import i32
from speculative_decoding_draft_row_gb300 import tfd
from speculative_decoding_draft_row_gb300.draft_pass import DraftPass
from synth import inputs

pytestmark = pytest.mark.gpu


def empty_cache(pages, page, heads, dim, fmt):
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    k, v = (torch.full((pages, page, heads, dim), float("nan"), device="cuda").to(dt)
            if fmt == "bf16" else torch.full((pages, page, heads, dim), 0x7F, dtype=dt, device="cuda")
            for _ in range(2))
    sc = [torch.full((pages, heads, page), float("nan"), device="cuda") for _ in range(2)] \
        if fmt != "bf16" else [None, None]
    return tfd.KvPages(k, v, *sc)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_rounds_of_verify_windows(fmt):
    """Prompts, then rounds of 4 rows of which 1 to 4 are kept; nothing is read back in between. The rows
    of the last round, over what the GPU's cache holds, against the oracle over the rows kept."""
    need_gpu()
    R, hq, H, D, page, n, rounds = 3, 4, 2, 64, 8, 4, 6
    g = np.random.default_rng(11)
    prompt = np.array([21, 3, 40])
    kept = g.integers(1, n + 1, (rounds, R))
    most = int(prompt.max()) + n * rounds
    max_pages, pages = -(-most // page), 40
    cache = empty_cache(pages, page, H, D, fmt)
    table, held = torch.full((R, max_pages), -1, dtype=torch.int32, device="cuda"), i32([0] * R)
    free, n_free = i32(g.permutation(pages)), i32([pages])
    ws = tfd.zeroed_workspace(tfd.tfd_paged_attn_workspace(n, hq, H, D))
    st = i32([0])
    lens = i32([0] * R)
    kept_d = i32(kept)
    mine = [([], []) for _ in range(R)]                   # the rows kept

    def rows_of(count, tid):
        return [inputs.normal_bf16((count, h, D), 1.0, tid + i) for i, h in enumerate((hq, H, H))]

    def step(new, rows, q, k, v):
        start, slots, pos = tfd.tfd_page_plan(lens, i32(new), page, table, held, free, n_free, rows=rows,
                                              dev_status=st)
        tfd.tfd_paged_append(k.cuda(), v.cuda(), slots, pos, cache, dev_status=st)
        if q is None:
            return None
        return tfd.tfd_paged_attn(q.cuda(), cache, table, lens, start, n, ws=ws, dev_status=st)[0]

    total = int(prompt.sum())
    _, k, v = rows_of(total, 1000)
    step(prompt, total, None, k, v)
    at = 0
    for r in range(R):
        mine[r][0].extend(np32(k)[at:at + prompt[r]])
        mine[r][1].extend(np32(v)[at:at + prompt[r]])
        at += prompt[r]
    lens += i32(prompt)
    for i in range(rounds):
        q, k, v = rows_of(R * n + 1, 1010 + 5 * i)        # a row more than are planned
        out = step([n] * R, R * n + 1, q, k, v)
        lens += kept_d[i]
        for r in range(R):
            keep = n if i == rounds - 1 else kept[i][r]
            mine[r][0].extend(np32(k)[r * n:r * n + keep])
            mine[r][1].extend(np32(v)[r * n:r * n + keep])
    torch.cuda.synchronize()
    assert st.item() == 0
    tab = table.cpu().numpy()
    for r in range(R):
        k, v = (np.stack(x) for x in mine[r])
        tokens = len(k)
        kx, pair = turned(k, range(tokens))
        t = np.arange(tokens)
        where = tab[r, t // page], t % page
        if fmt == "bf16":
            ks, vs = (np32(x)[where] for x in (cache.k, cache.v))
            assert_bf16_rounding(ks, kx, 2.0 ** -18 * pair, "keys")
            assert np.array_equal(vs, v)
        else:
            ks, vs = (np32(x.view(torch.float8_e4m3fn))[where] *
                      np32(s).transpose(0, 2, 1)[where].astype(np.float64)[..., None]
                      for x, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)))
            assert (np.abs(ks - kx) <= 2.0 ** -4 * np.abs(kx) + np.abs(kx).max() * 2.0 ** -17).all()
        length = tokens - n
        qx, mag = turned(np32(q)[r * n:r * n + n], range(length, tokens))
        y, _, t = attend(qx, ks, vs, length, mag=mag)
        err = 1.01 * (2.0 ** -15 * t["dev_a"] + (2.0 ** -20 + 2.0 ** -23 * t["a_most"][..., None]) *
                      t["dev"]) + (2.0 ** -15 if fmt == "bf16" else 2.0 ** -11 + 2.0 ** -17) * t["abs_out"]
        assert_bf16_rounding(np32(out)[r * n:r * n + n].reshape(y.shape), y, err, f"request {r}")


S, H, D, HIDDEN, INNER, VOCAB, STEPS = 3, 4, 128, 256, 96, 2500, 4


def build(paged, k_ring=None, v_ring=None, window=-1):
    wo = quant_fp8_row(inputs.linear(HIDDEN, H * D, 700).float().numpy())
    w2 = quant_fp8_row(inputs.linear(HIDDEN, INNER, 701).float().numpy())
    head = inputs.normal_bf16((VOCAB, HIDDEN), 0.2, 702)
    return DraftPass(torch.from_numpy(wo[0]).cuda(), torch.from_numpy(wo[1]).cuda(),
                     torch.from_numpy(w2[0]).cuda(), torch.from_numpy(w2[1]).cuda(), head.cuda(),
                     tfd.W_BF16, None, k_ring, v_ring, window, STEPS, paged=paged)


def pages_of(lens, kv_heads, page=16, fmt="bf16"):
    pages = sum(-(-(ln + STEPS) // page) for ln in lens) + 3
    k, v = (inputs.normal_bf16((pages, page, kv_heads, D), 1.0, 710 + i).cuda() for i in range(2))
    width = max(-(-(ln + STEPS) // page) for ln in lens)
    table, held, at = np.full((S, width), -1), [], 0
    for r, ln in enumerate(lens):
        need = -(-ln // page)
        table[r, :need] = np.arange(at, at + need)
        held.append(need)
        at += need
    free = np.concatenate([np.arange(at, pages), [-1] * at])
    return dict(cache=tfd.KvPages(k, v), table=i32(table), held=i32(held), free_ids=i32(free),
                n_free=i32([pages - at]))


def load(dp, pos0, kv_heads, seed=0):
    make = lambda h, i: [inputs.normal_bf16((S, h, D), 1.0, 730 + 3 * t + i + seed) for t in range(STEPS)]
    us = [inputs.normal_bf16((S, INNER), 1.0, 760 + t) for t in range(STEPS)]
    qs, ks, vs = make(H, 0), make(kv_heads, 1), make(kv_heads, 2)
    dp.load(qs, ks, vs, us, pos0, inputs.normal_bf16((S, HIDDEN), 1.0, 770).cuda(),
            np.array([4, 3, 4], np.int32), np.zeros((S, STEPS), np.int32))
    return qs, ks, vs


@pytest.mark.parametrize("kv_heads", [4, 1])
@pytest.mark.parametrize("window", [-1, 31])
def test_pass_over_pages_step_by_step(kv_heads, window):
    need_gpu()
    lens = [700, 33, 0]
    p = pages_of(lens, kv_heads)
    dp = build(p, window=window)
    qs, ks, vs = load(dp, lens, kv_heads)
    for t in range(STEPS):
        dp.step_attn(t)
        torch.cuda.synchronize()
        tab = p["table"].cpu().numpy()
        for r in range(S):
            n = lens[r] + t + 1
            where = tab[r, np.arange(n) // 16], np.arange(n) % 16
            k, v = np32(p["cache"].k)[where], np32(p["cache"].v)[where]
            assert np.array_equal(v[-1], np32(vs[t][r]))
            kx, pair = turned(np32(ks[t][r:r + 1]), [n - 1])
            assert_bf16_rounding(k[-1:], kx, 2.0 ** -18 * pair, "key")
            qx, mag = turned(np32(qs[t][r:r + 1]), [n - 1])
            y, _, m = attend(qx, k, v, n - 1, window=window, mag=mag)
            err = 1.01 * (2.0 ** -15 * m["dev_a"] + 2.0 ** -20 * m["dev"]) + 2.0 ** -15 * m["abs_out"]
            assert_bf16_rounding(np32(dp.attn[r]).reshape(y[0].shape), y[0], err[0], f"step {t} row {r}")
    assert dp.status.item() == 0


def test_pass_over_pages_replayed_and_turned_down():
    """A captured pass equals the eager one, and a pass that starts again where the last one began gives
    the same results on the same pages."""
    need_gpu()
    lens = [60, 15, 31]
    results = []
    for capture in (False, True):
        p = pages_of(lens, 2)
        dp = build(p)
        load(dp, lens, 2)
        if capture:
            dp.capture()
        for _ in range(3):
            dp.resid.copy_(inputs.normal_bf16((S, HIDDEN), 1.0, 770))
            dp.run()
            torch.cuda.synchronize()
            results.append((dp.drafts.clone(), dp.draft_vals.clone(), dp.attn.clone(),
                            p["table"].clone(), p["held"].clone(), p["n_free"].clone()))
        assert dp.status.item() == 0
        assert p["held"].tolist() == [-(-(n + STEPS) // 16) for n in lens]
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


def test_pass_over_pages_is_the_pass_over_rings():
    """The same context in a ring and in pages: the attention of every step within both tolerances."""
    need_gpu()
    ring, window, pos0 = 40, 31, [33, 34, 35]
    kr, vr = (inputs.normal_bf16((S * ring, H, D), 1.0, 703 + i).reshape(S, ring, H, D).cuda()
              for i in range(2))
    p = pages_of(pos0, H)
    tab = p["table"].cpu().numpy()
    for r in range(S):
        for t in range(pos0[r]):
            for ours, its in ((p["cache"].k, kr), (p["cache"].v, vr)):
                ours[int(tab[r, t // 16]), t % 16] = its[r, t % ring]
    a, b = build(None, kr.clone(), vr.clone(), window), build(p, window=window)
    for dp in (a, b):
        load(dp, pos0, H)
    for t in range(STEPS):
        a.step_attn(t)
        b.step_attn(t)
        torch.cuda.synchronize()
        x, y = np32(a.attn), np32(b.attn)
        # a rounding each (2^-8 of the value), and the two computations' errors (far below 2^-8 of the scale)
        assert (np.abs(x - y) <= 2.0 ** -7 * np.abs(x) + 2.0 ** -10).all()


def test_rings_and_pages_are_not_mixed():
    need_gpu()
    p = pages_of([5, 5, 5], 2)
    with pytest.raises(ValueError):
        build(p, k_ring=torch.zeros((S, 8, H, D), dtype=torch.bfloat16, device="cuda"))
    a, b = build(p), build(None, *(torch.zeros((S, 8, H, D), dtype=torch.bfloat16, device="cuda")
                                   for _ in range(2)), window=7)
    assert a.launches() == b.launches() + 2 * STEPS
