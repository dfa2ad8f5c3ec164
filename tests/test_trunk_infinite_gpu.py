"""Values that are not finite stay what the recurrence makes of them, however
a row is shared out: an infinite state or candidate stays infinite (a product
of gates that vanishes meets no infinity), its opposite beside it makes NaN, up
to the end of the episode.  The reference walks the steps in 64 bits."""
import pytest
import torch

from first_order_linear_gb300 import _lib, rlca
from oracle import trunk_ref as ref
from tests.test_trunk_gpu import SCAN, U, _close, half_step, steps_problem

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _lib_and_status(cuda_lib):
    yield
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 1) == _lib.RLCA_OK and st.value == 0


def _same(got, want, bound, what):
    """Where the reference is not finite, the same infinity or NaN; elsewhere within the bound."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN at {(torch.isnan(got) != torch.isnan(want)).sum().item()} places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities"
    _close(got[fine], want[fine], bound[fine], what)


# walked step by step in vectors and not, by tiles, in clusters, in segments; aligned rows and others
SIZES = [(4, 7, 64), (4, 7, 61), (3000, 40, 64), (300, 200, 64), (5, 300, 96), (5, 300, 61), (1, 900, 64), (1, 1100, 61),
         (1, 5000, 64), (1, 5000, 61), (2, 2999, 40)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ends", [0.0, 0.003])
@pytest.mark.parametrize("E,T,D", SIZES)
def test_not_finite_values(E, T, D, ends, dtype):
    # gates about sigma = 0.1: their products vanish in float32 within 50 steps
    d = steps_problem(E, T, D, dtype, seed=T + D, ends=ends, bias=0.0)
    dh, d_last = d.pop("dh"), d.pop("d_last")
    d["gate"] -= 2.0
    good = dict(d, x=d["x"].clone(), state=d["state"].clone())
    d["state"][:, 0], d["state"][:, 1], d["state"][:, 2] = INF, -INF, NAN
    d["x"][:, T // 3, 4], d["x"][:, T // 2, 5] = INF, -INF
    d["x"][:, T // 3, 7], d["x"][:, T - 1, 7] = INF, -INF
    d["state"][:, 9], d["x"][:, T // 2, 9] = INF, -INF
    k = SCAN[dtype] * U
    h, last = rlca.rlca_gated_scan(**d)
    want_h, want_last, bh, bl = ref.gated_scan(**d)
    _same(h, want_h, k * bh + half_step(dtype) * (want_h.abs() + k * bh), "h")
    _same(last, want_last, k * bl + U * want_last.abs(), "last")

    h, _ = rlca.rlca_gated_scan(**good)
    d_last[:, 0], d_last[:, 1], d_last[:, 2] = INF, -INF, NAN
    dh[:, T // 3, 4], dh[:, T // 2, 5] = INF, -INF
    dh[:, T // 3, 7], dh[:, 0, 7] = INF, -INF
    d_last[:, 9], dh[:, T // 2, 9] = INF, -INF
    args = (dh, good["x"], good["gate"], h, good["terminated"], good["truncated"], good["state"])
    dx, dgate, d_state = rlca.rlca_gated_scan_backward(*args, d_last=d_last)
    want = ref.gated_scan_backward(*args, None, d_last)
    for name, got, w, b in (("dx", dx, want[0], want[3]), ("dgate", dgate, want[1], want[4])):
        _same(got, w, k * b + half_step(dtype) * (w.abs() + k * b), name)
    _same(d_state, want[2], k * want[5] + U * want[2].abs(), "d_state")
