"""A workspace shares no memory with what a call reads: kernels write to it
before others of the same call have read their inputs.  Host checks of the C
entry points, on fake pointers that nothing reads."""
import ctypes as C

import pytest

from first_order_linear_gb300 import _lib, build

INV = _lib.RLCA_ERR_INVALID_ARG
P = [C.c_void_p(0x10000000 * (i + 1)) for i in range(20)]
WS = P[19]


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def _at(p, offset):
    return C.c_void_p(p.value + offset)


# arguments up to the workspace, which inputs it may not share, and their bytes
E, T, D = 3, 5, 8
N = E * T
SCAN = dict(x=P[0], gate=P[1], term=P[2], trunc=P[3], state=P[4], len=P[5], h=P[6], last=P[7], E=E, T=T, D=D, xs=D, gs=D,
            flags=0)
SCAN_BYTES = dict(x=4 * N * D, gate=4 * N * D, term=N, trunc=N, state=4 * E * D, len=4 * E)
GRAD = dict(dh=P[0], x=P[1], gate=P[2], h=P[3], term=P[4], trunc=P[5], state=P[6], len=P[7], dl=P[8], dx=P[9], dg=P[10],
            ds=P[11], E=E, T=T, D=D, dhs=D, xs=D, gs=D, hs=D, dxs=D, dgs=D, flags=0)
GRAD_BYTES = dict(dh=4 * N * D, x=4 * N * D, gate=4 * N * D, h=4 * N * D, term=N, trunc=N, state=4 * E * D, len=4 * E,
                  dl=4 * E * D)
RMS = dict(dy=P[0], dt=P[1], total=P[2], t8=None, t8s=None, w=P[5], rstd=P[6], dx=P[7], dw=P[8], N=N, D=D, dys=D, dts=D,
           ts=D, flags=0)
RMS_BYTES = dict(dy=4 * N * D, dt=4 * N * D, total=4 * N * D, w=4 * D, rstd=4 * N)
RMS8 = dict(RMS, total=None, t8=P[3], t8s=P[4])
RMS8_BYTES = dict(dy=4 * N * D, t8=N * D, t8s=4 * N)


@pytest.mark.parametrize("call,args,sizes", [("rlca_gated_scan", SCAN, SCAN_BYTES), ("rlca_gated_scan_backward", GRAD, GRAD_BYTES),
                                             ("rlca_rms_norm_backward", RMS, RMS_BYTES),
                                             ("rlca_rms_norm_backward", RMS8, RMS8_BYTES)])
def test_a_workspace_on_an_input_is_refused(lib, call, args, sizes):
    for name, size in sizes.items():
        for a in (dict(args, **{name: WS}),                                # its first bytes
                  dict(args, **{name: _at(WS, 4096 - 4)}),                 # its last
                  dict(args, **{name: _at(WS, -(size - 4) // 4 * 4)})):    # the input's last
            assert getattr(lib, call)(*a.values(), WS, 4096, None) == INV, name


def test_an_output_in_an_inputs_place_keeps_the_workspace_apart(lib):
    """last in the state's buffer and d_state in d_last's: the workspace overlaps neither."""
    a = dict(SCAN, state=WS, last=WS)
    assert lib.rlca_gated_scan(*a.values(), WS, 4096, None) == INV
    a = dict(GRAD, dl=WS, ds=WS)
    assert lib.rlca_gated_scan_backward(*a.values(), WS, 4096, None) == INV
