"""Calls of the trunk's operators as programs make them: two at once on two
streams, captured with a workspace of the caller's and replayed while others
run, and the widest and narrowest sizes."""
import pytest
import torch

from first_order_linear_gb300 import _lib, rlca
from tests.test_trunk_gpu import check_rms, check_scan, steps_problem

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib_and_status(cuda_lib):
    yield
    import ctypes as C
    st = C.c_uint(0)
    assert cuda_lib.rlca_device_status(C.byref(st), 1) == _lib.RLCA_OK and st.value == 0


# one row in segments, rows in clusters, rows of a CTA each, steps; unaligned rows
SCANS = [(1, 6000, 64), (2, 1500, 256), (40, 300, 320), (3, 5, 100), (2, 3100, 61)]


def _all(d):
    """A scan, its gradient, and a norm with its gradient over the same elements."""
    scan = {k: v for k, v in d.items() if k not in ("dh", "d_last")}
    h, last = rlca.rlca_gated_scan(**scan)
    grads = rlca.rlca_gated_scan_backward(d["dh"], d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"],
                                          d_last=d["d_last"])
    rows, width = h.reshape(-1, h.shape[2]), h.shape[2]
    w = torch.ones(width, dtype=h.dtype, device="cuda")
    y, total, rstd, y8, t8 = rlca.rlca_rms_norm(rows, w, grads[0].reshape(-1, width), want_y8=True, want_total8=True)
    dx, dw = rlca.rlca_rms_norm_backward(y, t8, w, rstd, d_total=total)
    return [h, last, *grads, y, total, rstd, y8[0].view(torch.uint8), y8[1], t8[0].view(torch.uint8), t8[1], dx, dw]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_streams_at_once(dtype):
    problems = [steps_problem(*s, dtype, seed=i) for i, s in enumerate(SCANS)]
    want = [_all(d) for d in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for turn in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                order = problems if k == 0 else problems[::-1]
                got[k].append([_all(d) for d in order])
    torch.cuda.synchronize()
    for k in range(2):
        for results in got[k]:
            for a, b in zip(results if k == 0 else results[::-1], want):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_captured_call_with_its_own_workspace_beside_others():
    d = steps_problem(1, 6000, 64, torch.bfloat16, seed=1)
    scan = {k: v for k, v in d.items() if k not in ("dh", "d_last")}
    need = [rlca.rlca_workspace_size(e, 1, 6000, 64, _lib.RLCA_BF16, d["x"].device)
            for e in (_lib.RLCA_EST_GATED_SCAN, _lib.RLCA_EST_GATED_SCAN_BACKWARD)]
    assert min(need) > 0
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in need]
    h, last = rlca.rlca_gated_scan(**scan)
    args = (d["dh"], d["x"], d["gate"], h, d["terminated"], d["truncated"], d["state"])
    grads = rlca.rlca_gated_scan_backward(*args, d_last=d["d_last"])
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gh, gl = rlca.rlca_gated_scan(**scan, workspace=ws[0])
        gg = rlca.rlca_gated_scan_backward(*args, d_last=d["d_last"], workspace=ws[1])
    others = []
    for _ in range(10):
        with torch.cuda.stream(side):
            graph.replay()
        others.append(rlca.rlca_gated_scan(**scan))
    torch.cuda.synchronize()
    assert torch.equal(gh, h) and torch.equal(gl, last) and all(torch.equal(a, b) for a, b in zip(gg, grads))
    assert all(torch.equal(a, h) and torch.equal(b, last) for a, b in others)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_widest_and_the_narrowest(dtype):
    check_scan(1, 1, 1 << 20, dtype, seed=1)
    check_scan(2, 70, 100003, dtype, seed=2)
    check_scan(1, 3000, 1, dtype, seed=3)
    check_scan(5000, 2, 1, dtype, seed=4)
    check_rms(2, 300001, dtype, seed=5)
    check_rms(3, 131072, dtype, seed=6, residual=False)
    check_rms(70000, 1, dtype, seed=7)
