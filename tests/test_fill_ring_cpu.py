"""Bookkeeping of the ring that feeds the layer norm's gradient, on the CPU
(tests/fill_ring_check.cu: host code, nothing touches CUDA)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_copies_on_their_way_are_waited_for(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "fill_ring_check")
    csrc = os.path.join(ROOT, "first_order_linear_gb300", "csrc")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-diag-suppress", "1886", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    "-gencode", "arch=compute_103a,code=sm_103a", os.path.join(ROOT, "tests", "fill_ring_check.cu"),
                    "-o", exe], check=True, capture_output=True, timeout=600)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and "ring ok" in out.stdout, out.stdout
