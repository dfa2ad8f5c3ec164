"""A launch that lasts longer than any one of its waits may (0.2 s): the waits
of a healthy kernel cover a few stages each, so it leaves the status word 0
and its results are right."""
import ctypes as C
import math

import pytest
import torch

from first_order_linear_gb300 import _lib, rlca

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def status(lib, clear=0):
    st = C.c_uint(0)
    assert lib.rlca_device_status(C.byref(st), clear) == 0
    return st.value


def test_scoring_in_one_launch_of_over_a_fifth_of_a_second(cuda_lib):
    """The weight is read in place, so the vocabulary is one launch: 2 N D V flop
    at no more than 2.4 PFLOP/s, the tensor cores' rate at their highest clock, last over 0.25 s."""
    N, D, V = 290_000, 8192, 131072
    assert 2 * N * D * V / 2.4e15 > 0.25
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    w = torch.randn(V, D, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(2.0 / math.sqrt(D))
    h = torch.randn(N, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    tok = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    assert status(cuda_lib, clear=1) == 0
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    logp, lse, entropy = rlca.rlca_token_logprob(h, w, tok)
    end.record()
    torch.cuda.synchronize()
    assert begin.elapsed_time(end) > 250.0
    assert status(cuda_lib) == 0

    # rows of the first, a middle and the last tiles against 64 bits.  A logit
    # is off by at most (4 sqrt(D) + 32) U times the sum of its terms'
    # magnitudes, a log-probability by twice that and a few roundings, the
    # entropy by that times its sensitivity 1 + |lse| + |entropy|
    rows = torch.cat([torch.arange(a, a + 12, device="cuda") for a in (0, N // 2, N - 12)])
    at = tok[rows].long()
    z = torch.cat([h[rows].double() @ part.double().t() for part in w.split(8192)], 1)
    scale = torch.cat([(h[rows].double().abs() @ part.double().abs().t()).amax(1, keepdim=True)
                       for part in w.split(8192)], 1).amax(1)
    lse0 = torch.logsumexp(z, 1)
    logq = z - lse0[:, None]
    logp0, ent0 = logq.gather(1, at[:, None])[:, 0], -(logq.exp() * logq).sum(1)
    tol = 2 * (4 * math.sqrt(D) + 32) * U * scale + 8 * U * (1 + lse0.abs() + logp0.abs())
    assert ((lse[rows] - lse0).abs() <= tol).all()
    assert ((logp[rows] - logp0).abs() <= tol).all()
    assert ((entropy[rows] - ent0).abs() <= tol * (1 + lse0.abs() + ent0.abs())).all()


def test_float32_gradient_of_sixteen_million_rows(cuda_lib):
    """One tile of d_weight is six products over all rows: 1.5 million steps
    of one CTA pair, of which each wait covers 128 at most."""
    from tests.test_policy_sums_gpu import exact, one_signed
    N, D, V = 16_000_001, 8, 20
    h, w, tok, g = one_signed(N, D, V, torch.float32, 2)
    lse, dw0 = exact(h, w, g)
    assert status(cuda_lib, clear=1) == 0
    _, dw = rlca.rlca_token_logprob_backward(h, w, tok, lse.float(), g, want_d_hidden=False)
    torch.cuda.synchronize()
    assert status(cuda_lib) == 0
    # 32 steps of the tensor cores' sums at 2e-7 of one sign each, on average
    # over them 3.2e-6; 31,251 partial sums added with errors of either sign,
    # of 2^-25 / sqrt(3) each: 3e-6, of which four are allowed; 2e-6 for dz
    assert ((dw[1:].double() - dw0) / dw0).abs().max().item() <= 3.2e-6 + 1.2e-5 + 2e-6
