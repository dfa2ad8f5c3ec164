"""A projection that takes the norm's result in 8 bits, as its layout is meant:
a group of 128 columns at a time, q_g @ w_g.t() with the rows' scales of that
group as one column, summed over the groups.

A value read back is half a step of e4m3 off at most: 2^-4 of it, or 2^-10 of
its scale below e4m3's normal range (where a step is 2^-9); y itself and its
division by the scale some 40 units of 2^-24 more.  A sum over D columns adds
that up against |w|; float32 products and sums add (D + 4) 2^-24 of their
magnitude."""
import pytest
import torch

from first_order_linear_gb300 import rlca
from oracle import trunk_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,D,OUT", [(1, 128, 8), (33, 1024, 96), (40, 1000, 33), (7, 4096, 64), (64, 257, 5)])
def test_product_of_rows_in_8_bits(cuda_lib, N, D, OUT, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = (n(N, D) * (1.0 + 20.0 * (torch.rand(D, generator=gen, device="cuda") < 0.02))).to(dtype)
    r, w = n(N, D).to(dtype), (1.0 + 0.1 * n(D)).to(dtype)
    into = n(OUT, D) / D ** 0.5
    y, total, _, (q, scale), _ = rlca.rlca_rms_norm(x, w, r, want_y=False, want_y8=True)
    assert y is None
    got = torch.zeros(N, OUT, device="cuda")
    for g, (qg, wg) in enumerate(zip(q.float().split(ref.GROUP, 1), into.split(ref.GROUP, 1))):
        got += (qg.double() @ wg.double().t()).float() * scale[:, g:g + 1]
    exact, _ = ref.rms_norm(total, w, 1e-6)
    want = exact @ into.double().t()
    wide = ref.scales(exact).repeat_interleave(ref.GROUP, 1)[:, :D]
    off = (2.0 ** -4 + (D / 32 + 48) * U) * exact.abs() + 1.01 * 2.0 ** -10 * wide
    bound = off @ into.double().abs().t() + (D + 4) * U * (exact.abs() @ into.double().abs().t())
    assert ((got.double() - want).abs() <= bound).all()
    # and on average far less: independent roundings of 2^-4 / sqrt(3) at most
    far = ((got.double() - want).norm() / want.norm()).item()
    assert N * OUT < 256 or far <= 2.0 ** -4, far
