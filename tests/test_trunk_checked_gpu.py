"""The operators of a recurrent policy's trunk in the index-check build: a
fresh process runs their tests' cases on librlca_checked.so, whose calls wait
for their kernels and fail when one recorded an index outside its array or a
wait that gave up."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import ctypes as C, sys
sys.path.insert(0, ROOT)
import torch
from first_order_linear_gb300 import _lib, build
build.build()
lib = _lib.load()
assert lib.rlca_index_checks() == 1, "not the index-check build"
from tests import test_trunk_gpu as t
for dtype in (torch.float32, torch.bfloat16):
    for E, T, D in t.SCAN_SIZES:
        for kw in (dict(time_major=True, fused=True), dict(shift=True, lengths=[T, 0, T // 2, 1])):
            t.check_scan(E, T, D, dtype, seed=T, **kw)
    for E, T, D in ((3000, 12, 64), (2500, 11, 61)):
        t.check_scan(E, T, D, dtype, seed=T, lengths=[T, 0, 3])
    for N, D in t.RMS_SIZES:
        for kw in (dict(), dict(strided=True), dict(shift=True, residual=False)):
            t.check_rms(N, D, dtype, seed=N, **kw)
st = C.c_uint(0)
assert lib.rlca_device_status(C.byref(st), 0) == 0 and st.value == 0
print("clean")
"""


def test_trunk_operators_run_clean_in_the_index_check_build():
    env = dict(os.environ, RLCA_LIBRARY="checked")
    res = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + SCRIPT], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=900)
    assert res.returncode == 0 and "clean" in res.stdout, res.stdout[-2000:] + res.stderr[-4000:]
