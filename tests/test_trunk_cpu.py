"""The operators of a recurrent policy's trunk without a GPU: the 64-bit
reference against differences of its own forward pass and against a rollout cut
in two, and the refusals of the C entry points and of the Python binding (none
of these calls reaches the device)."""
import ctypes as C
import math

import pytest
import torch

from first_order_linear_gb300 import _lib, build, rlca
from oracle import trunk_ref as ref

INV, OK = _lib.RLCA_ERR_INVALID_ARG, _lib.RLCA_OK
BF = _lib.RLCA_BF16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def _problem(E, T, D, seed=0):
    torch.manual_seed(seed)
    n = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    return dict(x=n(E, T, D), gate=n(E, T, D), terminated=(torch.rand(E, T) < 0.2).to(torch.uint8),
                truncated=(torch.rand(E, T) < 0.1).to(torch.uint8), state=n(E, D),
                lengths=torch.tensor([T, 0, 1, T - 2][:E], dtype=torch.int32))


# central differences at h = 1e-5 in 64 bits: truncation h^2 times a third
# derivative of order 1 (1e-10), rounding 1e-16 / h (1e-11), times sums of
# tens of terms
DIFF_TOL = 1e-7


def test_gated_scan_gradient_against_differences():
    E, T, D = 4, 9, 3
    p = _problem(E, T, D)
    dh, dl = torch.randn(E, T, D, dtype=torch.float64), torch.randn(E, D, dtype=torch.float64)

    def value(**k):
        h, last, _, _ = ref.gated_scan(**dict(p, **k))
        return ((h * dh).sum() + (last * dl).sum()).item()

    h = ref.gated_scan(**p)[0]
    got = ref.gated_scan_backward(dh, p["x"], p["gate"], h, p["terminated"], p["truncated"], p["state"], p["lengths"], dl)
    for name, grad in zip(("x", "gate", "state"), got):
        for seed in range(3):
            torch.manual_seed(seed)
            d = torch.randn_like(p[name])
            diff = (value(**{name: p[name] + 1e-5 * d}) - value(**{name: p[name] - 1e-5 * d})) / 2e-5
            assert abs(diff - (grad * d).sum().item()) < DIFF_TOL, name
    real = torch.arange(T)[None, :] < p["lengths"][:, None]
    assert got[0][~real].abs().max() == 0 and got[1][~real].abs().max() == 0


def test_gated_scan_of_a_rollout_cut_in_two():
    p = _problem(3, 12, 4, seed=5)
    del p["lengths"]
    h, last, _, _ = ref.gated_scan(**p)
    state, parts = p["state"], []
    for lo, hi in ((0, 5), (5, 12)):
        cut = {k: p[k][:, lo:hi] for k in ("x", "gate", "terminated", "truncated")}
        part, state, _, _ = ref.gated_scan(state=state, **cut)
        parts.append(part)
    assert torch.equal(torch.cat(parts, 1), h) and torch.equal(state, last)
    tm = {k: (v if k == "state" else v.transpose(0, 1)) for k, v in p.items()}
    assert torch.equal(ref.gated_scan(time_major=True, **tm)[0].transpose(0, 1), h)


def test_rms_norm_gradient_against_differences():
    torch.manual_seed(1)
    n = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    x, r, w, dy, dt = n(4, 9), n(4, 9), n(9), n(4, 9), n(4, 9)

    def value(xx, ww):
        return ((ref.rms_norm(xx + r, ww, 1e-6)[0] * dy).sum() + ((xx + r) * dt).sum()).item()

    _, rstd = ref.rms_norm(x + r, w, 1e-6)
    dx, dw, _, _ = ref.rms_norm_backward(dy, x + r, w, rstd, dt)
    for seed in range(3):
        torch.manual_seed(seed)
        a, c = torch.randn_like(x), torch.randn_like(w)
        assert abs((value(x + 1e-5 * a, w) - value(x - 1e-5 * a, w)) / 2e-5 - (dx * a).sum().item()) < DIFF_TOL
        assert abs((value(x, w + 1e-5 * c) - value(x, w - 1e-5 * c)) / 2e-5 - (dw * c).sum().item()) < DIFF_TOL


def test_rows_in_8_bits_of_the_reference():
    v = torch.tensor([[0.0] * 128 + [1.0, -448.0, math.nan]])
    assert torch.equal(ref.scales(v), torch.tensor([[2.0 ** -126, 1.0]], dtype=torch.float64))
    assert ref.read_back(torch.ones(1, 131), torch.tensor([[2.0, 3.0]])).sum() == 128 * 2 + 3 * 3


# ---- refusals of the C entry points -----------------------------------------
# fake pointers, never dereferenced: every call fails its checks
P = [C.c_void_p(0x10000000 * (i + 1)) for i in range(16)]


def _at(k, offset):
    return C.c_void_p(P[k].value + offset)


def _rms(lib, **k):
    a = dict(x=P[0], res=P[1], w=P[2], total=P[3], y=P[4], y8=P[5], y8s=P[6], t8=P[7], t8s=P[8], rstd=P[9], N=4, D=8,
             xs=8, rs=8, eps=1e-6, flags=0)
    a.update(k)
    return lib.rlca_rms_norm(*a.values(), None)


def test_rms_norm_refusals(lib):
    assert _rms(lib, N=0, x=None) == OK and _rms(lib, D=0, x=None) == OK
    for bad in (dict(N=-1), dict(D=-1), dict(N=1 << 31), dict(D=(1 << 30) + 1), dict(x=None), dict(w=None), dict(xs=7),
                dict(rs=7), dict(xs=(1 << 31) + 1), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan),
                dict(flags=0x1), dict(flags=0x40), dict(total=None), dict(res=None), dict(y8=None), dict(y8s=None),
                dict(t8=None), dict(t8s=None), dict(y=P[0]), dict(total=P[0]), dict(y=P[1]), dict(y8=P[2]),
                dict(t8=P[5]), dict(rstd=_at(4, 4 * 31)), dict(y8s=P[8]), dict(x=_at(0, 2)), dict(y=_at(4, 1)),
                dict(t8s=_at(8, 2)),
                # the residual's own buffer only where it lies as the output does
                dict(total=P[1], rs=16), dict(total=_at(1, 4)),
                dict(res=None, total=None, y=None, y8=None, y8s=None, t8=None, t8s=None, rstd=None)):
        assert _rms(lib, **bad) == INV, bad
    assert _rms(lib, xs=100, y=_at(0, 4 * 307)) == INV       # the last row counts its own width
    assert _rms(lib, flags=BF, y=_at(0, 2 * 31)) == INV      # 2-byte elements


def _rms_grad(lib, **k):
    a = dict(dy=P[0], dt=P[1], total=P[2], t8=None, t8s=None, w=P[5], rstd=P[6], dx=P[7], dw=P[8], N=4, D=8, dys=8,
             dts=8, ts=8, flags=0, ws=None, wsb=0)
    a.update(k)
    return lib.rlca_rms_norm_backward(*a.values(), None)


def test_rms_norm_backward_refusals(lib):
    assert _rms_grad(lib, D=0, dy=None) == OK
    for bad in (dict(N=-1), dict(dy=None), dict(total=None), dict(w=None), dict(rstd=None), dict(t8=P[3], t8s=P[4]),
                dict(total=None, t8=P[3]), dict(total=None, t8s=P[4]), dict(dys=7), dict(dts=7), dict(ts=7),
                dict(flags=0x1), dict(dx=None, dw=None), dict(dx=P[0]), dict(dx=P[1]), dict(dw=P[7]), dict(dx=P[5]),
                dict(dx=_at(7, 2)), dict(dw=_at(8, 1)), dict(total=None, t8=P[3], t8s=_at(4, 2))):
        assert _rms_grad(lib, **bad) == INV, bad


def _scan(lib, **k):
    a = dict(x=P[0], gate=P[1], term=P[2], trunc=None, state=P[4], len=P[5], h=P[6], last=P[7], E=3, T=5, D=8, xs=8, gs=8,
             flags=0, ws=None, wsb=0)
    a.update(k)
    return lib.rlca_gated_scan(*a.values(), None)


def test_gated_scan_refusals(lib):
    assert _scan(lib, E=0, x=None) == OK and _scan(lib, D=0, x=None) == OK
    assert _scan(lib, T=0, x=None, gate=None, h=None, last=None) == OK
    for bad in (dict(E=-1), dict(T=-1), dict(D=-1), dict(E=1 << 16, T=1 << 15), dict(x=None), dict(gate=None),
                dict(h=None), dict(xs=7), dict(gs=0), dict(flags=0x2), dict(flags=0x10), dict(h=P[0]), dict(h=P[4]),
                dict(last=P[1]), dict(last=P[6]), dict(ws=P[6], wsb=64), dict(last=_at(4, 4)), dict(last=P[5]), dict(h=P[2]),
                dict(x=_at(0, 1)), dict(state=_at(4, 2)), dict(len=_at(5, 1))):
        assert _scan(lib, **bad) == INV, bad


def _scan_grad(lib, **k):
    a = dict(dh=P[0], x=P[1], gate=P[2], h=P[3], term=P[4], trunc=None, state=P[5], len=P[6], dl=P[7], dx=P[8], dg=P[9],
             ds=P[10], E=3, T=5, D=8, dhs=8, xs=8, gs=8, hs=8, dxs=8, dgs=8, flags=0, ws=None,
             wsb=0)
    a.update(k)
    return lib.rlca_gated_scan_backward(*a.values(), None)


def test_gated_scan_backward_refusals(lib):
    assert _scan_grad(lib, E=0, x=None) == OK and _scan_grad(lib, T=0, dh=None, ds=None) == OK
    for bad in (dict(E=-1), dict(T=-1), dict(dh=None), dict(x=None), dict(gate=None), dict(h=None), dict(dx=None),
                dict(dg=None), dict(dhs=7), dict(xs=7), dict(gs=7), dict(hs=7), dict(dxs=7), dict(dgs=7),
                dict(flags=0x4), dict(dx=P[0]), dict(dg=P[1]), dict(dx=P[3]), dict(dg=P[8]), dict(ds=P[5]),
                dict(ds=_at(7, 4)), dict(ws=P[9], wsb=64), dict(dx=P[7]), dict(dx=_at(8, 2)),
                # parts of one matrix's rows that share a column, or lie at different strides
                dict(dxs=15, dgs=15, dg=_at(8, 32)), dict(dxs=16, dgs=17, dg=_at(8, 32)),
                dict(dxs=16, dgs=16, dg=_at(8, 36)), dict(dxs=16, dgs=16, dg=_at(8, 28))):
        assert _scan_grad(lib, **bad) == INV, bad


def test_rms_workspace_size_refusals(lib):
    out = C.c_size_t(1)
    q = lambda *a: lib.rlca_workspace_size(_lib.RLCA_EST_RMS_NORM_BACKWARD, *a, C.byref(out))  # noqa: E731
    assert q(-1, 8, 0, 0) == INV and q(4, 8, 0, _lib.RLCA_TIME_MAJOR) == INV
    assert q(0, 8, 0, 0) == OK and out.value == 0


@pytest.mark.parametrize("estimator", [_lib.RLCA_EST_GATED_SCAN, _lib.RLCA_EST_GATED_SCAN_BACKWARD])
def test_gated_scan_workspace_size_refusals(lib, estimator):
    out = C.c_size_t(1)
    q = lambda *a: lib.rlca_workspace_size(estimator, *a, C.byref(out))  # noqa: E731
    assert q(4, 8, -1, 0) == INV and q(1 << 16, 1 << 15, 8, 0) == INV and q(4, 8, 8, _lib.RLCA_MULTIPASS) == INV
    assert q(4, 0, 8, _lib.RLCA_TIME_MAJOR | BF) == OK and out.value == 0
    assert lib.rlca_workspace_size(estimator + 2, 4, 8, 8, 0, C.byref(out)) == INV


# ---- refusals of the Python binding ------------------------------------------

def _f(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refusals():
    bf, e4 = torch.bfloat16, torch.float8_e4m3fn
    rms, rms_grad = rlca.rlca_rms_norm, rlca.rlca_rms_norm_backward
    scan, scan_grad = rlca.rlca_gated_scan, rlca.rlca_gated_scan_backward
    x, pair = _f(4, 200), (_f(4, 200).to(e4), _f(4, 2))
    s = _f(2, 3, 8)
    u8, i32 = torch.uint8, torch.int32
    cases = [
        (TypeError, lambda: rms(_f(4, 8, dtype=torch.float16), _f(8))),
        (TypeError, lambda: rms(_f(4, 8), _f(8, dtype=bf))),
        (ValueError, lambda: rms(_f(4, 8), _f(7))),
        (ValueError, lambda: rms(_f(4, 8), _f(8), _f(4, 9))),
        (TypeError, lambda: rms(_f(4, 8), _f(8), _f(4, 8, dtype=bf))),
        (ValueError, lambda: rms(_f(4, 8), _f(8), total=_f(4, 8))),            # no residual: total is x
        (TypeError, lambda: rms(x, _f(200), y8=pair[0])),
        (TypeError, lambda: rms(x, _f(200), y8=(x, pair[1]))),
        (ValueError, lambda: rms(x, _f(200), total8=(pair[0], _f(4, 1)))),
        (ValueError, lambda: rms(_f(1, 8).expand(4, 8), _f(8))),
        (ValueError, lambda: rms(_f(4, 8), _f(8))),                            # not on a CUDA device
        (TypeError, lambda: rms_grad(x, (x, pair[1]), _f(200), _f(4))),
        (ValueError, lambda: rms_grad(x, (pair[0], _f(4, 3)), _f(200), _f(4))),
        (ValueError, lambda: rms_grad(x, pair, _f(200), _f(5))),
        (ValueError, lambda: rms_grad(x, pair, _f(200), _f(4), d_total=_f(4, 199))),
        (ValueError, lambda: rms_grad(x, pair, _f(200), _f(4), want_dx=False, want_dweight=False)),
        (ValueError, lambda: rms_grad(x, pair, _f(200), _f(4))),
        (TypeError, lambda: scan(_f(2, 3, 8, dtype=torch.float64), s)),
        (TypeError, lambda: scan(s, _f(2, 3, 8, dtype=bf))),
        (ValueError, lambda: scan(s, _f(2, 4, 8))),
        (ValueError, lambda: scan(_f(6, 8), _f(6, 8))),
        (ValueError, lambda: scan(_f(2, 8, 3).transpose(1, 2), s)),            # channels not contiguous
        (ValueError, lambda: scan(_f(2, 5, 8)[:, :3], s)),                     # rows not at one stride
        (ValueError, lambda: scan(_f(1, 1, 8).expand(2, 3, 8), s)),
        (TypeError, lambda: scan(s, s, _f(2, 3))),
        (ValueError, lambda: scan(s, s, torch.zeros(3, 2, dtype=u8))),
        (TypeError, lambda: scan(s, s, state=_f(2, 8, dtype=bf))),
        (ValueError, lambda: scan(s, s, state=_f(3, 8))),
        (TypeError, lambda: scan(s, s, lengths=torch.zeros(2, dtype=torch.int64))),
        (ValueError, lambda: scan(s, s, lengths=torch.zeros(3, dtype=i32))),
        (ValueError, lambda: scan(s, s, h=_f(2, 3, 16)[..., :8])),
        (ValueError, lambda: scan(s, s)),
        (ValueError, lambda: scan_grad(_f(2, 3, 7), s, s, s)),
        (ValueError, lambda: scan_grad(s, s, s, _f(2, 4, 8))),
        (TypeError, lambda: scan_grad(s, s, s, s, d_last=_f(2, 8, dtype=bf))),
        (TypeError, lambda: scan_grad(s, s, s, s, dx=_f(2, 3, 8, dtype=bf))),
        (ValueError, lambda: scan_grad(s, s, s, s)),
    ]
    for k, (err, call) in enumerate(cases):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {k} was not refused")
