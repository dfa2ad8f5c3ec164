"""The index-check build over the paths of the policy-update operators that
tests/test_policy_index_check.py does not reach: every count of few rows,
vocabularies in several pieces, all variants of the layer norm and its gradient
(registers at both alignments, the ring, rows too long for either), and clipping
at odd starts, in place, over more tensors than one launch holds."""
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
    for N in (1, 2, 3, 4, 5, 8, 9, 16, 17):
        for D, V in ((1, 3), (129, 300), (512, 2501)):
            for kw in (dict(), dict(mask=0.4, junk=True), dict(strided=True), dict(shift=True)):
                t.check_head(N, D, V, dtype, seed=N, **kw)
    for N, D in t.NORM_SIZES:
        for kw in (dict(), dict(strided=True), dict(shift=True)):
            if N * D < 2000000:
                t.check_norm(N, D, dtype, seed=N, **kw)
t.check_head(40, 512, 100003, torch.float32, seed=1, mask=0.3)
t.check_head(70, 1001, 280001, torch.bfloat16, seed=2)
t.check_head(8192, 512, 66001, torch.bfloat16, seed=3, mask=0.2)
sizes = [1, 3, 8, 17, 1000, 4096, 32768, 32769, 100001, 1 << 20]
for shift in (False, True):
    t.check_clip(t.grads_of(sizes, seed=1, shift=shift), 1.0)
    g = t.grads_of(sizes, seed=2, shift=shift)
    t.check_clip(g, 1.0, out=g)
    g = t.grads_of(sizes, seed=2, shift=shift)
    t.check_clip(g, 1.0, out=t.grads_of(sizes, seed=3, shift=not shift))
t.check_clip(t.grads_of([(k * 37) % 61 for k in range(2500)], seed=3), 1.0)
st = C.c_uint(0)
assert lib.rlca_device_status(C.byref(st), 0) == 0 and st.value == 0
print("clean")
"""


def test_policy_operators_run_clean_on_all_their_paths():
    env = dict(os.environ, RLCA_LIBRARY="checked")
    res = subprocess.run([sys.executable, "-c", "ROOT = %r\n" % ROOT + SCRIPT], cwd=ROOT, env=env, capture_output=True,
                         text=True, timeout=900)
    assert res.returncode == 0 and "clean" in res.stdout, res.stdout[-2000:] + res.stderr[-4000:]
