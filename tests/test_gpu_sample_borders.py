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
