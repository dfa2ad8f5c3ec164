"""Gradients of gates that are shut or nearly so, each relative to itself.

sigma(g) is e^-|g| there, and dgate and d_state are proportional to it.  Errors
in units u = 2^-24: the exponential of bfloat16 gates 2 + 1.2 |g| last places
(2 u each) off at most, the sum with 1, the reciprocal and the product 4 u
together, so sigma and 1 - sigma 8 + 2.4 |g| u each; of float32 gates 10 u.  A
step adds its gate's error, three operations, and the same composed in another
order: k = 2 (8 + 2.4 |g| + 3) u, times the magnitudes that the reference adds
up.  A channel is held to its own magnitudes alone, and then to half a step of
its type.
"""
import pytest
import torch

from first_order_linear_gb300 import _lib, rlca
from oracle import trunk_ref as ref
from tests.test_trunk_gpu import U, half_step, steps_problem

pytestmark = pytest.mark.gpu

TINIEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133}  # the spacing next to 0


@pytest.fixture(autouse=True)
def _lib_and_status(cuda_lib):
    yield
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 1) == _lib.RLCA_OK and st.value == 0


def _within(got, want, k, bound, what):
    bound = k * bound
    half = half_step(got.dtype)
    far = (got.double() - want).abs() - (bound + half * (want.abs() + bound) + TINIEST[got.dtype])
    worst = ((got.double() - want).abs() / want.abs().clamp(min=1e-300)).max().item()
    assert not torch.isnan(got).any() and far.max().item() <= 0, f"{what}: {worst:.2e} of a value off"


SHUT = [-8.0, -9.5, -11.0, -12.5, -14.0, -15.5, -17.0, -20.0, -25.0, -30.0, -50.0, -80.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("time_major", [False, True])
@pytest.mark.parametrize("E,T,D", [(5, 1, 96), (5, 1, 61), (3, 7, 64), (2, 200, 96), (2, 200, 61), (1, 900, 64),
                                   (1, 2300, 40), (1, 2301, 33), (2500, 11, 64), (2500, 11, 61)])
def test_gradients_of_shut_gates(E, T, D, time_major, dtype):
    d = steps_problem(E, T, D, dtype, seed=E + T + D, ends=0.02, time_major=time_major)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    # every other channel at one of the gates above from step to step, the others open
    steps = torch.arange(E * T, device="cuda").view(d["gate"].shape[:2])[..., None] + torch.arange(D, device="cuda")
    shut = torch.tensor(SHUT, device="cuda").to(dtype)[steps % len(SHUT)]
    d["gate"][..., 0::2] = shut[..., 0::2]
    k = 2 * (8 + 2.4 * 80 + 3) * U if dtype is torch.bfloat16 else 26 * U
    own = slice(0, None, 2)
    want_h, want_last, bh, bl = ref.gated_scan(**d)
    h, last = rlca.rlca_gated_scan(**d)
    _within(h[..., own], want_h[..., own], k, bh[..., own], "h")
    _within(last[..., own], want_last[..., own], k, bl[..., own], "last")
    args = (dh, d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"])
    dx, dgate, d_state = rlca.rlca_gated_scan_backward(*args, d_last=d_last, time_major=time_major)
    want = ref.gated_scan_backward(*args, None, d_last, time_major)
    for name, got, w, b in (("dx", dx, want[0], want[3]), ("dgate", dgate, want[1], want[4]),
                            ("d_state", d_state, want[2], want[5])):
        _within(got[..., own], w[..., own], k, b[..., own], name)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 300])
def test_gates_beyond_what_their_exponential_holds(T, dtype):
    """sigma of a gate below -87 is below 2^-125: what passes is no more than that, and the gradients are finite."""
    d = steps_problem(2, T, 64, dtype, seed=T, ends=0.0)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    d["gate"][..., 0::4], d["gate"][..., 1::4], d["gate"][..., 2::4] = -100.0, -3.0e38, -float("inf")
    h, last = rlca.rlca_gated_scan(**d)
    shut = torch.arange(64, device="cuda") % 4 != 3
    assert torch.equal(h[..., shut], d["x"][..., shut])
    dx, dgate, d_state = rlca.rlca_gated_scan_backward(dh, d["x"], d["gate"], h, state=d["state"], d_last=d_last)
    most = 2.0 ** -125 * 64 * (dh.float().abs().max() + d_last.abs().max()).item()
    assert dgate[..., shut].abs().max().item() <= most and d_state[..., shut].abs().max().item() <= most
    assert torch.isfinite(dx).all() and torch.isfinite(dgate).all() and torch.isfinite(d_state).all()
