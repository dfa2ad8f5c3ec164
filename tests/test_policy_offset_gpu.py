"""Logits with a large offset that all tokens of a row share: it cancels in
the log-probabilities, the entropies and dz, and so must its rounding.

The operands hold few bits (multiples of 1/8 and powers of two), so every
product and every partial sum, the logits themselves and their differences are
exact in float32, and what is tested is what the statistics and dz make of
them.  Bounds, with u = 2^-23:

* e = 2^(c2 (z - max)) is off by (4 + |c2 (z - max)|) u of itself (the function's
  two units, two roundings in front of it), of which the terms that matter
  have |c2 (z - max)| < 30; a sum of V of them by (4 sqrt(V) + 32) u more:
  together `rel`;
* logp by rel + 4 u |logp|, the entropy by rel (1 + E_p |z - max| / temperature),
  lse by rel + u |lse|: none but lse, whose own size it is, by anything that
  grows with the offset;
* dz, from the lse and entropy given, by (8 + 2 |log p|) u of its terms, whose
  contraction adds (4 sqrt(K) + 32) u, and for bfloat16 one rounding of the
  result (2^-8) and, from 129 rows on, one of dz.
"""
import math

import pytest
import torch

from first_order_linear_gb300 import rlca
from oracle import policy_ref as ref

pytestmark = pytest.mark.gpu

U, R = 2.0 ** -23, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def offset_inputs(N, V, offset, dtype, seed, D=64):
    """h [N, D], w [V, D], tokens: logits = offset + multiples of 1/8 within about +-8."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    h = torch.randint(-2, 3, (N, D), generator=gen, device="cuda").float()
    w = torch.randint(-2, 3, (V, D), generator=gen, device="cuda").float() / 8
    scale = 2.0 ** int(math.log2(abs(offset)) / 2) if offset else 1.0
    h[:, 0], w[:, 0] = scale, offset / scale
    assert torch.equal(w[:, 0].bfloat16().float(), w[:, 0])
    z = h.double() @ w.double().t()
    # half of the tokens taken are the likeliest of their row
    tok = torch.randint(0, V, (N,), generator=gen, device="cuda")
    tok[::2] = z.argmax(1)[::2]
    return h.to(dtype), w.to(dtype), tok.to(torch.int32), z


OFFSETS = [0.0, -304.0, 4096.0, -16384.0]
# few rows (their own kernel), tensor-core tiles, several of them, and a last one cut short
SIZES = [(1, 300), (3, 2001), (13, 515), (40, 1003), (200, 4097)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 2.0])
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("N,V", SIZES)
def test_statistics_do_not_feel_a_common_offset(cuda_lib, N, V, offset, temperature, dtype):
    h, w, tok, z = offset_inputs(N, V, offset, DT[dtype], N + V)
    logp, lse, ent = (t.double() for t in rlca.rlca_token_logprob(h, w, tok, temperature=temperature))
    x = z / temperature
    lse0 = torch.logsumexp(x, 1)
    logq = x - lse0[:, None]
    p = logq.exp()
    logp0, ent0 = logq.gather(1, tok.long()[:, None])[:, 0], -(p * logq).sum(1)
    below = (p * (x.amax(1, keepdim=True) - x)).sum(1)
    rel = (4 + 30 + 4 * math.sqrt(V) + 32) * U
    assert ((logp - logp0).abs() <= rel + 4 * U * logp0.abs()).all(), (logp - logp0).abs().max().item()
    assert ((ent - ent0).abs() <= rel * (1 + below)).all(), (ent - ent0).abs().max().item()
    assert ((lse - lse0).abs() <= rel + U * lse0.abs()).all(), (lse - lse0).abs().max().item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.0])
@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("N,V", SIZES)
def test_gradients_do_not_feel_a_common_offset(cuda_lib, N, V, offset, temperature, dtype):
    # the factor that is multiplied with the logits is 1 / temperature in
    # float32: the reference takes its exact inverse
    exact_t = 1.0 / float(torch.tensor(1.0 / temperature, dtype=torch.float32).double())
    h, w, tok, z = offset_inputs(N, V, offset, DT[dtype], N + V)
    x = z / exact_t
    lse = torch.logsumexp(x, 1).float()
    logq = x - torch.logsumexp(x, 1)[:, None]
    ent = -(logq.exp() * logq).sum(1).float()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    g, e = (torch.randn(N, generator=gen, device="cuda") / N for _ in range(2))
    dh, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, entropy=ent, d_entropy=e, temperature=exact_t)
    dh0, dw0, *_ = ref.token_logprob_backward(h, w, tok, lse, g, ent, e, exact_t)
    # dz's terms, each with its own relative error
    logq32 = x - lse.double()[:, None]
    p, gd, ed = logq32.exp(), g.double().abs()[:, None], e.double().abs()[:, None]
    taken = torch.zeros_like(p).scatter_(1, tok.long()[:, None], 1.0)
    err = (8 + 2 * logq32.abs()) * U * p * (gd + ed * (logq32.abs() + ent.double()[:, None])) + 4 * U * gd * taken
    mag = p * (gd + ed * (logq32 + ent.double()[:, None]).abs()) + gd * taken
    rd, out = ((R if N > 128 else R * R), R) if dtype == "bf16" else (0.0, U)
    for got, want, left, right, K, name in ((dh, dh0, (err, mag), w.double().abs(), V, "d_hidden"),
                                            (dw, dw0, (err.t(), mag.t()), h.double().abs(), N, "d_weight")):
        tol = (left[0] + (rd + (4 * math.sqrt(K) + 32) * U) * left[1]) @ right / exact_t + out * want.abs()
        over = (got.double() - want).abs() - tol
        assert over.max().item() <= 0, (name, over.max().item(), tol.reshape(-1)[over.argmax()].item())
