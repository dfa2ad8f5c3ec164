"""What the precision bounds of tests/test_policy_precision_gpu.py can tell
apart, computed on the CPU: float32 operands as three bfloat16 planes with the
six products down to 2^-16 stay well inside the float32 bounds, and fail them
with a plane, or the products of one order, left out."""
import math

import torch

from oracle import policy_ref as ref
from tests.test_policy_precision_gpu import STATS, far

# plane pairs by the order of their products
ORDERS = {0: [(0, 0)], 1: [(0, 1), (1, 0)], 2: [(0, 2), (2, 0), (1, 1)]}


def planes(v):
    out, rest = [], v
    for _ in range(3):
        p = rest.float().bfloat16().double()
        out.append(p)
        rest = rest - p
    return out


def product(a, b, orders):
    """a @ b.t() of the planes' products; sums in 64 bits"""
    pa, pb = planes(a), planes(b)
    return sum(pa[i] @ pb[j].t() for o in orders for i, j in ORDERS[o])


def errors(orders, N=64, D=1024, V=4001):
    gen = torch.Generator()
    gen.manual_seed(0)
    w = torch.randn(V, D, generator=gen) * (2.0 / math.sqrt(D))
    taken = torch.randint(0, V, (N,), generator=gen)
    h = torch.randn(N, D, generator=gen) + 2.0 * torch.rand((N, 1), generator=gen) * w[taken]
    tok, g, e = taken.to(torch.int32), torch.randn(N, generator=gen) / N, 0.1 * torch.randn(N, generator=gen) / N
    logp0, lse0, ent0, _ = ref.token_logprob(h, w, tok)
    z = product(h.double(), w.double(), orders)
    lse = torch.logsumexp(z, 1)
    logq = z - lse[:, None]
    logp, ent = logq.gather(1, taken[:, None])[:, 0], -(logq.exp() * logq).sum(1)
    lse32, ent32 = lse0.float(), ent0.float()
    logq = z - lse32.double()[:, None]
    dz = -logq.exp() * (g.double()[:, None] + e.double()[:, None] * (logq + ent32.double()[:, None]))
    dz.scatter_add_(1, taken[:, None], g.double()[:, None])
    dh = product(dz, w.double().t(), orders)
    dw = product(dz.t(), h.double().t(), orders)
    dh0, dw0, *_ = ref.token_logprob_backward(h, w, tok, lse32, g, ent32, e)
    return [far(logp, logp0), far(lse, lse0), far(ent, ent0)], [far(dh, dh0), far(dw, dw0)]


def test_three_planes_are_inside_the_bounds():
    stats, grads = errors([0, 1, 2])
    assert all(x <= 0.5 * b for x, b in zip(stats, STATS["f32"])), stats
    assert all(x <= 0.55e-6 for x in grads), grads


def test_two_planes_are_outside():
    for orders in ([0, 1], [0]):
        stats, grads = errors(orders)
        assert all(x > 1.4 * b for x, b in zip(stats, STATS["f32"])), (orders, stats)
        assert all(x > 2.2e-6 for x in grads), (orders, grads)

