"""The policy-update operators in the index-check build: a fresh process runs
their tests' cases of ragged, masked, strided, unaligned and many-piece sizes
on librlca_checked.so, whose calls wait for their kernels and fail when one
recorded an index outside its array or a wait that gave up."""
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
from tests import test_policy_gpu as t
for dtype in (torch.float32, torch.bfloat16):
    for N, D, V in ((1, 64, 2), (8, 100, 1003), (37, 200, 1003), (129, 136, 256), (300, 96, 4097), (513, 320, 1537)):
        for kw in (dict(), dict(mask=0.4, junk=True), dict(strided=True), dict(shift=True)):
            t.check_head(N, D, V, dtype, seed=N, **kw)
    t.check_head(3000, 40, 70001, dtype, seed=3, mask=0.2)
    for N, D in ((1, 1), (33, 32), (64, 257), (100, 1001), (300, 4096), (17, 8192), (3, 20000)):
        t.check_norm(N, D, dtype, seed=N)
t.check_clip(t.grads_of([1, 3, 8, 17, 1000, 32769, 100001], seed=1), 1.0)
st = C.c_uint(0)
assert lib.rlca_device_status(C.byref(st), 0) == 0 and st.value == 0
print("clean")
"""


def test_policy_operators_run_clean_in_the_index_check_build():
    env = dict(os.environ, RLCA_LIBRARY="checked")
    res = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + SCRIPT], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=900)
    assert res.returncode == 0 and "clean" in res.stdout, res.stdout[-2000:] + res.stderr[-4000:]
