"""The host's choice of blocks a cluster, against made-up answers of the runtime (host_launch.cu)."""
import os
import subprocess

from speculative_decoding_draft_row_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_cluster_sizes_that_cannot_be_placed_are_left_out(tmp_path):
    exe = str(tmp_path / "host_launch")
    subprocess.run([build.nvcc_path(), *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I",
                    build.CSRC, os.path.join(HERE, "host_launch.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
