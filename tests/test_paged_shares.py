"""How the paged attention's work is shared out in the launches that there are (CPU: a host program walks all shares)."""
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_key_of_a_lane_is_taken_once():
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "paged_shares_check")
        subprocess.run([nvcc, "-std=c++17", "--expt-relaxed-constexpr", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "attention_backward_02_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "paged_shares_check.cu"), "-o", exe], check=True, capture_output=True, timeout=600)
        f = subprocess.run([exe], check=True, capture_output=True, text=True, timeout=300).stdout.split()
    got = dict(zip(f[::2], map(int, f[1::2])))
    assert got["batches"] == 12000 and got["pieces"] > 10 ** 6
    for k in ("holes", "twice", "empty", "slot", "chain", "heavy"):
        assert got[k] == 0, got
