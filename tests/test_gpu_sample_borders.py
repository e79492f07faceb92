"""tfd_sample where a row's filters meet: top-k and top-p resolved one after the other on one short list.
Every block of a row's cluster resolves them for itself, and all have to find the same border.

Tolerances are those of test_gpu_sample.py."""
import numpy as np
import pytest
import torch

from helpers import need_gpu
from speculative_decoding_draft_row_gb300 import tfd
from test_gpu_sample import check, dev, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n", [(1, 4096), (4, 163840), (16, 50021), (96, 30011)])
@pytest.mark.parametrize("k", [2, 20, 50, 100])
def test_top_p_after_top_k_on_a_short_list_repeats_bit_for_bit(rows, n, k):
    """The mass that top-k leaves is read by every thread before top-p's border replaces it."""
    need_gpu()
    x = logits(rows, n, 31 * rows + k)
    rng = np.random.default_rng([0, 92, rows, k])
    s = dict(temperature=np.full(rows, 0.8, np.float32), top_k=np.full(rows, k, np.int32),
             top_p=rng.choice(np.array([0.3, 0.8, 0.95], np.float32), rows))
    u = np.minimum(rng.random(rows, dtype=np.float32), np.float32(1 - 2.0 ** -24))
    xg, ug, sd = torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda(), dev(s)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, prob, probs = tfd.tfd_sample(xg, ug, want_probs=True, dev_status=st, **sd)
    torch.cuda.synchronize()
    got = (ids.cpu().numpy(), prob.cpu().numpy(), probs.cpu().numpy(), st.item(), None)
    check(got, x.astype(np.float64), u, s)
    other = [torch.full_like(ids, -5), torch.empty_like(prob), torch.empty_like(probs)]
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        tfd.tfd_sample(xg, ug, ids=other[0], prob=other[1], probs=other[2], **sd)
        differ += (other[0] != ids).sum() + (other[1] != prob).sum() + (other[2] != probs).sum()
        other[0].fill_(-5)
    assert differ.item() == 0


@pytest.mark.parametrize("temperature", [1e4, 1e5, 1e6, 1e7])
def test_min_p_beside_top_p_at_high_temperatures(temperature):
    """Nearly equal weights: min_p just below 1 cuts a few columns off from where top_p does, on
    either side, and the stricter of the two decides. Weights are within 2^-38 of the exact ones;
    rows whose cuts lie nearer than 2^-36 to a column are left out."""
    need_gpu()
    n = 4096
    x0 = logits(1, n, 41)[0]
    t = np.float32(temperature)
    w = np.sort(np.exp((x0.astype(np.float64) - float(x0.max())) / float(t)))[::-1]
    incl = np.cumsum(w)
    below = np.unique(np.round(np.geomspace(1, (1 - w[-1]) * 2.0 ** 24, 60)))
    mp, tp, kept = [], [], []
    for m in below:
        cut = np.float32(1 - m * 2.0 ** -24)
        j = int((w >= np.float64(cut)).sum())
        for d in (-40, -10, -3, -1, 1, 3, 10, 40):
            i = j - d                                # top_p keeps i columns, min_p j
            if not 2 <= i < n or np.abs(w - np.float64(cut)).min() < 2.0 ** -36:
                continue
            p = np.float32((incl[i - 1] - 0.5 * w[i - 1]) / incl[-1])
            mp.append(cut)
            tp.append(p)
            kept.append(min(max(j, 1), i))
    rows = len(mp)
    assert rows > 30
    s = dict(temperature=np.full(rows, t), min_p=np.array(mp), top_p=np.array(tp))
    u = np.full(rows, 0.5, np.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    xg = torch.from_numpy(x0).cuda().repeat(rows, 1)
    _, _, probs = tfd.tfd_sample(xg, torch.from_numpy(u).cuda(), want_probs=True, dev_status=st,
                                 **dev(s))
    torch.cuda.synchronize()
    got = (probs > 0).sum(1).cpu().numpy()
    assert st.item() == 0 and np.array_equal(got, np.array(kept)), \
        [(i, got[i], kept[i]) for i in np.flatnonzero(got != np.array(kept))[:20]]
