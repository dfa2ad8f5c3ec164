"""The gated scan's gradient where a row is cut into segments by its second
rule (half of the SMs idle in clusters, long rows) and where the segments are
doubled, at both alignments, with ends of episodes next to the segments'
borders and a length that ends inside one, against the 64-bit reference; one
case of each in the index-check build."""
import os
import subprocess
import sys

import pytest
import torch

from first_order_linear_gb300 import _lib, rlca
from oracle import trunk_ref as ref
from tests.test_trunk_gpu import SCAN, U, _close, _norm_close, half_step, steps_problem

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _lib_and_status(cuda_lib):
    yield
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 1) == _lib.RLCA_OK and st.value == 0


def check_long_row(T, D, dtype, length=None, seed=0):
    d = steps_problem(1, T, D, dtype, seed=seed, ends=0.0)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    # segments are whole multiples of 64 steps: ends at the last step of one, the first and the second of the next, at a
    # tenth of the multiples
    gen = torch.Generator().manual_seed(seed)
    ends = torch.zeros(1, T, dtype=torch.uint8)
    for at in range(64, T - 1, 64):
        if torch.rand((), generator=gen).item() < 0.1:
            ends[0, at + int(torch.randint(-1, 2, (), generator=gen))] = 1
    d["terminated"] = ends.cuda()
    if length is not None:
        d["lengths"] = torch.tensor([length], dtype=torch.int32, device="cuda")
        for v in (d["x"], d["gate"], dh):
            v[:, length:] = float("nan")
    k = SCAN[dtype] * U
    tol = 1e-6 if dtype is torch.float32 else 2.4e-3
    h, last = rlca.rlca_gated_scan(**d)
    want_h, want_last, bh, bl = ref.gated_scan(**d)
    _close(h, want_h, k * bh + half_step(dtype) * (want_h.abs() + k * bh), "h")
    _close(last, want_last, k * bl + U * want_last.abs(), "last")
    _norm_close(h, want_h, tol, "h")
    args = (dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"], d["lengths"])
    dx, dgate, d_state = rlca.rlca_gated_scan_backward(*args, d_last=d_last)
    want = ref.gated_scan_backward(*args, d_last)
    for name, got, w, b in (("dx", dx, want[0], want[3]), ("dgate", dgate, want[1], want[4])):
        _close(got, w, k * b + half_step(dtype) * (w.abs() + k * b), name)
        _norm_close(got, w, tol, name)
    _close(d_state, want[2], k * want[5] + U * want[2].abs(), "d_state")


# 12 blocks of 64 channels: doubled; 16 blocks, rows on 16-byte boundaries and not: the second rule; one block: doubled,
# hundreds of segments
CASES = [(13000, 768, None), (13000, 768, 9999), (8300, 1024, None), (8300, 1000, 8111), (8300, 1001, None),
         (20001, 64, 15000)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,D,length", CASES)
def test_long_rows_in_segments(T, D, length, dtype):
    check_long_row(T, D, dtype, length, seed=T + D)


SCRIPT = r"""
import ctypes as C, sys
sys.path.insert(0, ROOT)
import torch
from first_order_linear_gb300 import _lib, build
build.build()
lib = _lib.load()
assert lib.rlca_index_checks() == 1, "not the index-check build"
from tests import test_trunk_segments_gpu as t
for dtype in (torch.float32, torch.bfloat16):
    t.check_long_row(13000, 768, dtype, 9999)
    t.check_long_row(8300, 1001, dtype)
st = C.c_uint(0)
assert lib.rlca_device_status(C.byref(st), 0) == 0 and st.value == 0
print("clean")
"""


def test_long_rows_run_clean_in_the_index_check_build():
    env = dict(os.environ, RLCA_LIBRARY="checked")
    res = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + SCRIPT], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=900)
    assert res.returncode == 0 and "clean" in res.stdout, res.stdout[-2000:] + res.stderr[-4000:]
