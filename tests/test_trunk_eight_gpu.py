"""Rows in 8 bits, bit by bit: the scale is the group's maximum times the
float32 next to 1 / 448, a value is multiplied by the float32 next to 1 / scale
and goes to the nearest e4m3 -- as the same operations give on the host.  No
tolerance: a value next to a border of two steps goes where its product says."""
import pytest
import torch

from first_order_linear_gb300 import _lib, rlca

pytestmark = pytest.mark.gpu

GROUP = 128


@pytest.fixture(autouse=True)
def _lib_and_status(cuda_lib):
    yield
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 1) == _lib.RLCA_OK and st.value == 0


def eight(v):
    """The rows of v (float32, on the host) in 8 bits, as bytes and scales."""
    n, d = v.shape
    groups = -(-d // GROUP)
    wide = torch.zeros(n, groups * GROUP)
    wide[:, :d] = v
    wide = wide.view(n, groups, GROUP)
    scale = (wide.abs().amax(2) * (torch.tensor(1.0) / 448.0)).clamp(min=2.0 ** -126)
    q = (wide * (1.0 / scale)[..., None]).clamp(-448.0, 448.0).view(n, -1)[:, :d]
    return q.to(torch.float8_e4m3fn).view(torch.uint8), scale


def _values(n, d, dtype, seed):
    """Rows with a few large columns, and rows whose values over their maximum are few-digit fractions: ratios that lie on
    borders of two steps, or next to them."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=gen) * (1.0 + 20.0 * (torch.rand(d, generator=gen) < 0.01))
    some = torch.arange(n) % 4 == 1
    top = torch.randint(1, 128, (n, 1), generator=gen).float()
    x[some] = (torch.randint(-64, 65, (n, d), generator=gen) / 64.0 * top)[some]
    x *= torch.exp2(torch.randint(-60, 60, (n, 1), generator=gen).float())
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,D", [(400, 64), (300, 1001), (300, 1024), (500, 392), (100, 4096), (30, 8192), (20, 8200),
                                 (9, 20000), (2000, 130)])
def test_values_are_the_nearest_to_their_products(N, D, dtype):
    x = _values(N, D, dtype, N + D)
    w = torch.ones(D, dtype=dtype)
    # (without a residual total is x; ones as weights; eps lost next to rows this large or small would not matter: total8)
    y, _, _, y8, total8 = rlca.rlca_rms_norm(x.cuda(), w.cuda(), want_y8=True, want_total8=True)
    q, scale = eight(x.float())
    assert torch.equal(total8[1].cpu(), scale)
    off = (total8[0].cpu().view(torch.uint8) != q).sum().item()
    assert off == 0, f"{off} of {q.numel()} values of total in 8 bits"
    if dtype is torch.float32:  # (y itself is at hand only where its storage does not round it)
        q, scale = eight(y.cpu())
        assert torch.equal(y8[1].cpu(), scale)
        off = (y8[0].cpu().view(torch.uint8) != q).sum().item()
        assert off == 0, f"{off} of {q.numel()} values of y in 8 bits"


@pytest.mark.parametrize("D", [256, 300, 8200, 16390])
def test_the_ends_of_the_range(D):
    """Groups whose scale is the least one, groups of values no smaller than it, and of float32's largest."""
    x = torch.randn(6, D)
    x[0] *= 2.0 ** -126 / 4
    x[1] *= 2.0 ** -118
    x[2] = torch.where(torch.arange(D) % 2 == 0, 3.0e38, -1.7e38)
    x[3] *= 2.0 ** 120
    x[4, ::7] = 0.0
    x[5] = -0.0
    _, _, _, _, (got, got_scale) = rlca.rlca_rms_norm(x.cuda(), torch.ones(D, device="cuda"), want_y=False, want_total8=True)
    q, scale = eight(x)
    assert torch.equal(got_scale.cpu(), scale) and torch.equal(got.cpu().view(torch.uint8), q)


def test_calls_repeat_themselves():
    """The same call gives the same bits, with other calls between and with outputs in other places."""
    n, d = 4096, 4096
    x, r = (torch.randn(n, d, device="cuda").bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(d, device="cuda")).bfloat16()
    first = rlca.rlca_rms_norm(x, w, r, want_y8=True, want_total8=True)
    kept = []
    for _ in range(4):
        rlca.rlca_rms_norm(r, w, x, want_total8=True)
        again = rlca.rlca_rms_norm(x, w, r, want_y8=True, want_total8=True)
        kept.append(again)
        for a, b in ((first[0], again[0]), (first[1], again[1]), (first[2], again[2]), (first[3][1], again[3][1]),
                     (first[4][1], again[4][1]), (first[3][0].view(torch.uint8), again[3][0].view(torch.uint8)),
                     (first[4][0].view(torch.uint8), again[4][0].view(torch.uint8))):
            assert torch.equal(a, b)
