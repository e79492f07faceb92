"""Failure detection of tfd_paged_attn's bounded waits, without a GPU fault: in the build of
test_gpu_timeout.py the scores' products are not announced, so the waits for them run out (about a
second). The call reports TFD_ERR_TIMEOUT, its products and copies have ended before its memory is given
back, and the other calls on the cache compute on the same context."""
import json
import os
import subprocess
import sys

import pytest

from helpers import need_gpu
from test_gpu_timeout_lora import ROOT, stalled_library

pytestmark = pytest.mark.gpu

CHILD = r"""
import json, sys, torch
sys.path.insert(0, sys.argv[1])
from speculative_decoding_draft_row_gb300 import tfd
torch.cuda.set_device(0)
out = {}
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
for name, fmt, heads, dim, new in (("one", 0, 2, 128, 1), ("window", 0, 2, 128, 8), ("tree", 0, 1, 64, 32),
                                   ("e4m3", 1, 2, 128, 1)):
    shape = (40, 16, heads, dim)
    if fmt:
        sc = [torch.ones((40, heads, 16), device="cuda") for _ in range(2)]
        cache = tfd.KvPages(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)), *sc)
    else:
        cache = tfd.KvPages(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.ones((new, 4 * heads, dim), dtype=torch.bfloat16, device="cuda")
    tfd.tfd_paged_attn(q, cache, i32([list(range(40))]), i32([640 - new]), i32([0, new]), new, dev_status=st)
    torch.cuda.synchronize()
    out[name] = int(st.item())
st = torch.zeros(1, dtype=torch.int32, device="cuda")
k = torch.ones((3, 2, 128), dtype=torch.bfloat16, device="cuda")
cache = tfd.KvPages(*(torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
tfd.tfd_paged_append(k, k, i32([5, 9, 63]), None, cache, norm=False, rope=False, dev_status=st)
torch.cuda.synchronize()
out["after"] = [int(st.item()), float(cache.k.float().sum())]
print(json.dumps(out))
"""


def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable():
    need_gpu()
    env = dict(os.environ, TFD_LIBRARY=stalled_library())
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    for name in ("one", "window", "tree", "e4m3"):
        assert out[name] == 6, out                        # TFD_ERR_TIMEOUT
    assert out["after"] == [0, 3.0 * 2 * 128], out
