"""Failure detection of tfd_lora's bounded waits, without a GPU fault: in the build of test_gpu_timeout.py
the prompts' form does not announce that its first products are complete, so its waits run out (about
a second). The call reports TFD_ERR_TIMEOUT, its products have ended before its tensor memory is given
back, and the next calls compute."""
import json
import os
import subprocess
import sys

import pytest

from helpers import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys, torch
sys.path.insert(0, sys.argv[1])
from speculative_decoding_draft_row_gb300 import tfd
torch.cuda.set_device(0)
out = {}

def call(R, k, n, rank):
    g = torch.Generator().manual_seed(R)
    x = torch.randn((R, k), generator=g).bfloat16().cuda()
    a = (torch.randn((1, rank, k), generator=g) / k ** 0.5).bfloat16().cuda()
    b = torch.randn((1, n, rank), generator=g).bfloat16().cuda()
    ids = torch.zeros(R, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = tfd.tfd_lora(x, a, b, ids, out_mode=tfd.OUT_F32, dev_status=st)
    torch.cuda.synchronize()
    ref = (x.float() @ a[0].float().T) @ b[0].float().T
    return int(st.item()), float((y - ref).abs().max() / ref.abs().max())

torch.backends.cuda.matmul.allow_tf32 = False
for rank in (16, 64, 128):
    out[f"prompt {rank}"] = call(300, 1024, 512, rank)[0]
out["few rows"] = call(16, 1024, 512, 16)
print(json.dumps(out))
"""


def stalled_library():
    from speculative_decoding_draft_row_gb300 import build
    path = os.path.join(build.BUILD_DIR, "stall")
    lib = os.path.join(path, "libtfd.so")
    if os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib)
                                   for d in build._deps()):
        return lib
    return build.build_library(extra_flags=["-DTFD_TEST_STALL_EXCHANGE=1"], build_dir=path)


def test_a_wait_that_runs_out_is_reported_and_the_context_stays_usable():
    need_gpu()
    env = dict(os.environ, TFD_LIBRARY=stalled_library())
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    timeout = 6  # TFD_ERR_TIMEOUT
    for rank in (16, 64, 128):
        assert out[f"prompt {rank}"] == timeout, out
    status, error = out["few rows"]
    assert status == 0 and error < 1e-5, out
