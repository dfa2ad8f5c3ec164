"""Long sums of the policy head's gradient: their error does not grow with
their length."""
import math

import pytest
import torch

from first_order_linear_gb300 import rlca
from oracle import policy_ref as ref
from tests.test_policy_gpu import DT, check_head, head_inputs

pytestmark = pytest.mark.gpu


def one_signed(N, D, V, dtype, seed):
    """Rows whose gradients add up without cancelling: positive hidden rows,
    and token 0 taken by all, so that every other token's dz is negative.
    Columns and tokens differ in size, so the results lie all over their
    type's steps."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    h = (0.5 + torch.rand((N, D), generator=gen, device="cuda")) * 2.0 ** torch.rand(D, generator=gen, device="cuda")
    w = torch.randn((V, D), generator=gen, device="cuda") / math.sqrt(D)
    tok = torch.zeros(N, dtype=torch.int32, device="cuda")
    g = (0.5 + torch.rand(N, generator=gen, device="cuda")) / N
    return h.to(dtype), w.to(dtype), tok, g


def exact(h, w, g, rows=1 << 18):
    """lse and d_weight in 64 bits, d_weight of tokens 1 on."""
    lse, dw = [], 0
    for hc, gc in zip(h.split(rows), g.split(rows)):
        z = hc.double() @ w.double().t()
        s = torch.logsumexp(z, 1)
        lse.append(s)
        dw = dw + (-gc.double()[:, None] * torch.exp(z - s[:, None])[:, 1:]).t() @ hc.double()
    return torch.cat(lse), dw


def test_weight_gradient_of_millions_of_bfloat16_rows():
    """The mean over the entries of d_weight's distance from the rounded exact
    results.  A sum of one sign loses about 2e-7 of itself at each of the
    tensor cores' steps of 16 rows: restarted at least every 256 steps, 2.6e-5
    on average.  An entry that far off is rounded to the neighbouring
    bfloat16, at most 2^-7 away, with probability 2.6e-5 / 2^-8 = 0.7%: in
    the mean of 4032 a standard deviation of at most 1e-5, of which four
    are allowed.  Without restarts the sum would be 1% off."""
    N, D, V = 3_000_001, 64, 64
    h, w, tok, g = one_signed(N, D, V, torch.bfloat16, 1)
    lse, dw0 = exact(h, w, g)
    _, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse.float(), g, want_d_hidden=False)
    bias = ((dw[1:].double() - dw0.bfloat16().double()) / dw0).mean().item()
    assert abs(bias) <= 2.6e-5 + 4e-5, bias


def test_probabilities_of_wide_bfloat16_rows():
    """Logits of 16 that add up from 65536 terms of one sign: an accumulator
    restarted every 64 steps loses 6.4e-6 of them on average, 1e-4 in the
    exponent of p and so of every dz; as much again is allowed.  One
    accumulator for all 4096 steps would make it 6.6e-3."""
    N, D, V = 64, 65536, 300
    h, _, tok, g = one_signed(N, D, V, torch.bfloat16, 3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    w = ((0.75 + 0.5 * torch.rand((V, D), generator=gen, device="cuda")) * (16.0 / h.float().sum(1).mean())).bfloat16()
    lse, dw0 = exact(h, w, g)
    _, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse.float(), g, want_d_hidden=False)
    bias = ((dw[1:].double() - dw0.bfloat16().double()) / dw0).mean().item()
    assert abs(bias) <= 2e-4, bias


@pytest.mark.parametrize("D", [1024, 4096, 5000])
def test_probabilities_of_bfloat16_rows_of_any_width(D):
    """The same where one accumulator takes all columns, where a few do, and
    at an odd number of them: the error does not depend on the width."""
    N, V = 64, 300
    h, _, tok, g = one_signed(N, D, V, torch.bfloat16, 3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    w = ((0.75 + 0.5 * torch.rand((V, D), generator=gen, device="cuda")) * (16.0 / h.float().sum(1).mean())).bfloat16()
    lse, dw0 = exact(h, w, g)
    _, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse.float(), g, want_d_hidden=False)
    bias = ((dw[1:].double() - dw0.bfloat16().double()) / dw0).mean().item()
    assert abs(bias) <= 2e-4, bias


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(300, 300), (9000, 300), (8000, 20000), (9000, 20000)])
def test_short_and_long_sums_in_every_pairing(N, V, dtype):
    """d_hidden's sums over V tokens (two halves at 8000 rows and more) and
    d_weight's over N rows, each within one accumulator of 128 steps (8192
    terms) or beyond, together in a launch and alone: right, and the same bits
    either way."""
    *_, dh, dw = check_head(N, 64, V, DT[dtype], seed=N + V, mask=0.1)
    h, w, tok, g, e = head_inputs(N, 64, V, DT[dtype], N + V, mask=0.1)
    _, lse0, ent0, _ = ref.token_logprob(h, w, tok)
    kw = dict(entropy=ent0.float(), d_entropy=e)
    only_h = rlca.rlca_token_logprob_backward(h, w, tok, lse0.float(), g, want_d_weight=False, **kw)[0]
    only_w = rlca.rlca_token_logprob_backward(h, w, tok, lse0.float(), g, want_d_hidden=False, **kw)[1]
    assert torch.equal(only_h, dh) and torch.equal(only_w, dw)
