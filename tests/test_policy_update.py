"""The policy update of examples/policy_update.py, which runs the operators
together, against 64-bit automatic differentiation of the same loss."""
import os
import sys

import pytest
import torch

from tests import parity  # noqa: F401  (the repository's root on sys.path)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def _reference(b, advantages, entropy_bonus, max_norm):
    names = ("trunk", "norm_weight", "norm_bias", "head")
    leaf = {k: b[k].double().requires_grad_() for k in names}
    x = torch.nn.functional.layer_norm(leaf["trunk"], leaf["trunk"].shape[1:], leaf["norm_weight"], leaf["norm_bias"])
    logq = torch.log_softmax(x @ leaf["head"].t(), 1)
    part = b["tokens"] >= 0
    logp = logq.gather(1, b["tokens"].clamp(min=0).long()[:, None])[:, 0]
    entropy = -(logq.exp() * logq).sum(1)
    loss = -((advantages.reshape(-1).double() * logp + entropy_bonus * entropy) * part).sum() / part.sum()
    grads = torch.autograd.grad(loss, [leaf[k] for k in names])
    norm = torch.sqrt(sum((g * g).sum() for g in grads))
    scale = min(1.0, max_norm / (norm.item() + 1e-6))
    return dict(zip(names, [g * scale for g in grads])), norm, logp * part


# float32: every sum in float32, the products to 24 bits: relative error of a
# gradient well below 1e-4 in the 2-norm.  bfloat16: the normalised rows, dz,
# the gradient of the rows and the results are each rounded to 8 bits (2^-9
# in the mean each, a few of them in a row)
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 2.0 ** -6)])
@pytest.mark.parametrize("E,T,D,V", [(3, 17, 40, 301), (8, 64, 256, 2000)])
def test_policy_update(cuda_lib, E, T, D, V, dtype, tol):
    import policy_update as ex
    from first_order_linear_gb300 import rlca
    b = ex.synthetic(E, T, D, V, seed=E, dtype=dtype)
    out = ex.policy_update(**b, entropy_bonus=0.02, max_norm=0.05)
    _, adv = rlca.rlca_vtrace(b["rewards"], b["values"], out["logp"].view(E, T), b["behaviour_logp"], b["terminated"],
                              bootstrap=b["bootstrap"])
    want, norm, logp = _reference(b, adv, 0.02, 0.05)
    assert abs(out["norm"].item() - norm.item()) <= tol * norm.item()
    assert (out["logp"].double() - logp).abs().max() <= (1e-4 if dtype == torch.float32 else 0.1)
    for k, w in want.items():
        far = (out[k].double() - w).norm() / w.norm()
        assert far <= tol, (k, far.item())
