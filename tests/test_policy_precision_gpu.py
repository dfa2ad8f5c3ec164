"""What the policy head's arithmetic is claimed to reach, in the 2-norm
relative to 64 bits: bounds 1.4 to 2 times what it does reach, where

* logits in one accumulator over the width give 4.3e-7 (1024) to 3.5e-6 (8192)
  in the log-probabilities, in groups of 1024 instead of 512 4e-7;
* float32 operands as two bfloat16 planes instead of three give 1.1e-6 in the
  log-probabilities and 5e-6 in the gradients (computed by
  tests/test_policy_precision_cpu.py).

The bounds of tests/test_policy_gpu.py are the worst that single elements may
be off by, which these sums of many errors of either sign stay far below."""
import pytest
import torch

from first_order_linear_gb300 import rlca
from oracle import policy_ref as ref
from tests.test_policy_gpu import DT, head_inputs

pytestmark = pytest.mark.gpu

STATS = {"bf16": (3e-7, 3e-7, 5e-7), "f32": (1.5e-7, 9e-8, 2e-7)}


def far(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1024, 2048, 4095, 4096, 8192])
def test_statistics(cuda_lib, D, dtype):
    h, w, tok, _, _ = head_inputs(512, D, 4001, DT[dtype], D)
    want = ref.token_logprob(h, w, tok)[:3]
    got = rlca.rlca_token_logprob(h, w, tok)
    errs = [far(a, b) for a, b in zip(got, want)]
    assert all(e <= b for e, b in zip(errs, STATS[dtype])), errs


# bfloat16: results rounded once are 1.65e-3 off; up to 128 rows dz adds
# nothing to that, beyond its own rounding adds as much (1.65e-3 sqrt(2))
@pytest.mark.parametrize("N,D,dtype,bound", [(512, 1024, "f32", 1.1e-6), (512, 2048, "f32", 1.1e-6), (2, 4000, "f32", 1.1e-6),
                                             (128, 1024, "bf16", 1.8e-3), (512, 1024, "bf16", 2.6e-3)])
def test_gradients(cuda_lib, N, D, dtype, bound):
    h, w, tok, g, e = head_inputs(N, D, 4001, DT[dtype], D)
    _, lse, ent, _ = (t.float() for t in ref.token_logprob(h, w, tok))
    got = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, entropy=ent, d_entropy=e)
    want = ref.token_logprob_backward(h, w, tok, lse, g, ent, e)[:2]
    errs = [far(a, b) for a, b in zip(got, want)]
    assert all(x <= bound for x in errs), errs
