"""Failure detection of tfd_paged_attn's bounded waits in its form for units of 64 rows (test_gpu_timeout_paged.py
has the others): four softmax groups wait for scores that are not announced, and the call ends and reports."""
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
R, heads = 24, 2                                          # 192 units: more than half the SMs
for dim in (64, 128):
    cache = tfd.KvPages(*(torch.zeros((20, 16, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    st = i32([0])
    q = torch.ones((32 * R, 8 * heads, dim), dtype=torch.bfloat16, device="cuda")
    tfd.tfd_paged_attn(q, cache, i32([list(range(20))] * R), i32([288] * R), i32([32 * r for r in range(R + 1)]), 32,
                       dev_status=st)
    torch.cuda.synchronize()
    out[str(dim)] = int(st.item())
x = torch.ones((4, 100), device="cuda")
out["after"] = float((x @ x.T).sum())
print(json.dumps(out))
"""


def test_waits_in_units_of_64_rows_run_out_and_are_reported():
    need_gpu()
    env = dict(os.environ, TFD_LIBRARY=stalled_library())
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out == {"64": 6, "128": 6, "after": 1600.0}, out   # TFD_ERR_TIMEOUT
