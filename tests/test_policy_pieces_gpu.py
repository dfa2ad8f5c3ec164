"""The policy head where the vocabulary is worked through in several pieces,
where a CTA pair has several tiles of many ring turns each, and with logits
that are not finite, or huge, in rows that take part.

A piece ends where its packed weight or its dz would pass a limit.  Each case
states how many pieces it is, computed from the limits in the source, so that a
raised limit shows here."""
import os
import re

import pytest
import torch

from first_order_linear_gb300 import rlca
from tests.test_policy_gpu import DT, check_head, head_inputs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def limit(name):
    with open(os.path.join(ROOT, "first_order_linear_gb300", "csrc", "k_head.cu")) as f:
        m = re.search(rf"constexpr int64_t {name} = int64_t\((\d+)\) << (\d+);", f.read())
    return int(m[1]) << int(m[2])


def up(a, b):
    return -(-a // b) * b


def pieces(N, D, V, dtype, backward, packed):
    """as the plan in k_head.cu divides V"""
    planes = 1 if dtype == "bf16" else 3
    tiles = piece = up(V, 256) // 256
    if packed:
        piece = min(piece, max(1, limit("kPackBytes") // (2 * planes * up(D, 8) * 256)))
    if backward:
        piece = min(piece, max(1, limit("kPieceBytes") // (2 * planes * up(N, 256) * 256)))
    return -(-tiles // piece)


def whole_sums(N, D):
    """d_hidden has enough tiles for every pair of 152 SMs: its sums are not
    split, and the last piece adds the stored ones and writes the results"""
    return (up(N, 256) // 256) * (up(D, 256) // 256) > 152 // 2 // 2


@pytest.mark.parametrize("N,D,V,dtype,packed,fwd,bwd,kw", [
    # packed weights in several pieces, in both directions; few rows: d_hidden's sums are split
    (40, 512, 100003, "f32", True, 2, 2, dict(mask=0.3, junk=True)),
    (9, 1001, 150001, "bf16", True, 2, 2, dict(temperature=0.7)),
    (70, 1001, 280001, "bf16", True, 3, 3, dict()),
    # dz in several pieces, d_hidden's sums whole
    (8192, 512, 66001, "bf16", False, 1, 2, dict(mask=0.2)),
    (8192, 512, 66001, "bf16", True, 1, 2, dict(shift=True)),
    (8000, 513, 140001, "bf16", True, 1, 3, dict(mask=0.2, junk=True)),
    (8192, 512, 22501, "f32", True, 1, 2, dict(mask=0.2)),
])
def test_several_pieces(cuda_lib, N, D, V, dtype, packed, fwd, bwd, kw):
    assert (pieces(N, D, V, dtype, False, packed), pieces(N, D, V, dtype, True, packed)) == (fwd, bwd)
    assert N < 1000 or whole_sums(N, D)
    check_head(N, D, V, DT[dtype], seed=N + V, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_tiles_of_many_ring_turns(cuda_lib, dtype):
    """6 x 24 tiles on 76 pairs, 33 stages each on a ring of 6."""
    check_head(1500, 2100, 6000, DT[dtype], seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 60, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite_stays_apart(cuda_lib, N, bad, dtype):
    """Its results are NaN, and so is every sum it takes part in (d_weight);
    the other rows' results keep their bits."""
    h, w, tok, g, e = head_inputs(N, 96, 700, DT[dtype], N)
    logp, lse, ent = rlca.rlca_token_logprob(h, w, tok)
    dh, _ = rlca.rlca_token_logprob_backward(h, w, tok, lse, g, entropy=ent, d_entropy=e)
    row, keep = N // 2, torch.arange(N, device="cuda") != N // 2
    h2 = h.clone()
    h2[row, 5] = bad
    got = rlca.rlca_token_logprob(h2, w, tok)
    for a, b in zip(got, (logp, lse, ent)):
        assert torch.isnan(a[row]) and torch.equal(a[keep], b[keep])
    dh2, dw2 = rlca.rlca_token_logprob_backward(h2, w, tok, got[1], g, entropy=got[2], d_entropy=e)
    assert torch.equal(dh2[keep], dh[keep]) and torch.isnan(dh2[row]).all() and torch.isnan(dw2).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 60, 300])
@pytest.mark.parametrize("size", [2.0 ** 13, 2.0 ** 33, 2.0 ** 100])
def test_huge_logits(cuda_lib, N, size, dtype):
    """Rows whose likeliest token is far ahead of all others: probability 1,
    entropy 0, the others' log-probabilities minus the distance; where the
    likeliest is taken the gradients vanish, elsewhere they are those of one
    token against another."""
    D = V = 64  # w = size times the identity: z = size h
    gen = torch.Generator(device="cuda")
    gen.manual_seed(N)
    h = torch.stack([torch.randperm(V, generator=gen, device="cuda") for _ in range(N)]).to(DT[dtype])
    w = (size * torch.eye(V, device="cuda")).to(DT[dtype])
    z = h.double() * w[0, 0].double()
    best = h.float().argmax(1)
    tok = best.clone()
    tok[1::2] = h.float().argmin(1)[1::2]
    tok = tok.to(torch.int32)
    logp, lse, ent = rlca.rlca_token_logprob(h, w, tok)
    top = z.amax(1)
    logp0 = z.gather(1, tok.long()[:, None])[:, 0] - top
    assert ((lse.double() - top).abs() <= 2e-7 * top).all()
    assert ((logp.double() - logp0).abs() <= 2e-7 * logp0.abs() + 1e-6).all() and (ent.abs() <= 1e-6).all()
    g, e = torch.ones(N, device="cuda"), torch.ones(N, device="cuda")
    # (the saved lse is the largest logit rounded to float32: in the exponent
    # its rounding would count, so that the logits are exact in it here)
    lse_exact = top.float()
    assert torch.equal(lse_exact.double(), top)
    dh, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse_exact, g, entropy=ent.clamp(min=0) * 0, d_entropy=e)
    hot = torch.zeros(N, V, dtype=torch.float64, device="cuda")
    dz = hot.scatter(1, tok.long()[:, None], 1.0) - hot.scatter(1, best[:, None], 1.0)
    assert torch.allclose(dh.double(), dz @ w.double(), rtol=1e-2 if dtype == "bf16" else 1e-5, atol=1e-5 * size)
    assert torch.allclose(dw.double(), dz.t() @ h.double(), rtol=1e-2 if dtype == "bf16" else 1e-5, atol=1e-3)
