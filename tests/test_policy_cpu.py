"""The policy-update operators without a GPU: the 64-bit reference against
differences of its own forward pass, and the refusals of the C entry points
and of the Python binding (none of these calls reaches the device)."""
import ctypes as C
import math

import pytest
import torch

from first_order_linear_gb300 import _lib, build, rlca
from oracle import policy_ref as ref

INV, UNS, OK = _lib.RLCA_ERR_INVALID_ARG, _lib.RLCA_ERR_UNSUPPORTED, _lib.RLCA_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


# ---- the reference against differences -------------------------------------

def _directional(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


# central differences at h = 1e-5 in 64 bits: truncation h^2 times a third
# derivative of order 1 (1e-10), rounding 1e-16 / h (1e-11), times sums of
# tens of terms
DIFF_TOL = 1e-7


@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_token_logprob_gradient_against_differences(temperature):
    torch.manual_seed(0)
    N, D, V = 5, 7, 11
    h, w = torch.randn(N, D, dtype=torch.float64), torch.randn(V, D, dtype=torch.float64)
    tok = torch.tensor([3, 0, -1, 10, 11], dtype=torch.int32)
    g, e = torch.randn(N, dtype=torch.float64), torch.randn(N, dtype=torch.float64)

    def value(hh, ww):
        logp, _, ent, _ = ref.token_logprob(hh, ww, tok, temperature)
        return (logp * g + ent * e).sum().item()

    _, lse, ent, _ = ref.token_logprob(h, w, tok, temperature)
    dh, dw = ref.token_logprob_backward(h, w, tok, lse, g, ent, e, temperature)[:2]
    for seed in range(3):
        torch.manual_seed(seed)
        a, b = torch.randn_like(h), torch.randn_like(w)
        assert abs(_directional(lambda v: value(v, w), h, a) - (dh * a).sum().item()) < DIFF_TOL
        assert abs(_directional(lambda v: value(h, v), w, b) - (dw * b).sum().item()) < DIFF_TOL
    assert dh[2].abs().max() == 0 and dh[4].abs().max() == 0


def test_layer_norm_gradient_against_differences():
    torch.manual_seed(1)
    x, dy = torch.randn(4, 9, dtype=torch.float64), torch.randn(4, 9, dtype=torch.float64)
    w, b = torch.randn(9, dtype=torch.float64), torch.randn(9, dtype=torch.float64)

    def value(xx, ww, bb):
        return (ref.layer_norm(xx, ww, bb, 1e-5)[0] * dy).sum().item()

    _, mean, rstd = ref.layer_norm(x, w, b, 1e-5)
    dx, dw, db = ref.layer_norm_backward(dy, x, w, mean, rstd)
    for seed in range(3):
        torch.manual_seed(seed)
        a, c = torch.randn_like(x), torch.randn_like(w)
        assert abs(_directional(lambda v: value(v, w, b), x, a) - (dx * a).sum().item()) < DIFF_TOL
        assert abs(_directional(lambda v: value(x, v, b), w, c) - (dw * c).sum().item()) < DIFF_TOL
        assert abs(_directional(lambda v: value(x, w, v), b, c) - (db * c).sum().item()) < DIFF_TOL


# ---- refusals of the C entry points -----------------------------------------
# fake pointers, never dereferenced: every call fails its checks
P = [C.c_void_p(0x10000000 * (i + 1)) for i in range(16)]


def _norm(lib, **k):
    a = dict(x=P[0], w=P[1], b=None, y=P[2], mean=P[3], rstd=P[4], N=4, D=8, xs=8, eps=1e-5, flags=0)
    a.update(k)
    return lib.rlca_layer_norm(*a.values(), None)


def test_layer_norm_refusals(lib):
    assert _norm(lib, N=0, x=None, w=None, y=None) == OK
    assert _norm(lib, D=0, x=None, w=None, y=None) == OK
    for bad in (dict(N=-1), dict(D=-1), dict(x=None), dict(w=None), dict(y=None), dict(xs=7), dict(eps=-1.0),
                dict(eps=math.inf), dict(eps=math.nan), dict(flags=0x1), dict(flags=0x40),
                dict(y=P[0]), dict(mean=P[2]), dict(rstd=C.c_void_p(P[2].value + 4 * 31)), dict(y=P[1])):
        assert _norm(lib, **bad) == INV, bad
    # the last row of a strided input counts only its own width
    assert _norm(lib, xs=100, y=C.c_void_p(P[0].value + 4 * 302)) == INV


def _norm_grad(lib, **k):
    a = dict(dy=P[0], x=P[1], w=P[2], mean=P[3], rstd=P[4], dx=P[5], dw=P[6], db=P[7], N=4, D=8, ds=8, xs=8, flags=0,
             ws=None, wsb=0)
    a.update(k)
    return lib.rlca_layer_norm_backward(*a.values(), None)


def test_layer_norm_backward_refusals(lib):
    assert _norm_grad(lib, D=0, dy=None) == OK
    for bad in (dict(N=-1), dict(dy=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None), dict(ds=7),
                dict(xs=0), dict(flags=0x2), dict(dx=None, dw=None, db=None), dict(dx=P[0]), dict(dx=P[1]),
                dict(db=P[6]), dict(dw=P[3])):
        assert _norm_grad(lib, **bad) == INV, bad


def _head(lib, **k):
    a = dict(h=P[0], w=P[1], tok=P[2], logp=P[3], lse=P[4], ent=P[5], N=4, D=8, V=16, hs=8, wst=8, it=1.0, flags=0,
             ws=None, wsb=0)
    a.update(k)
    return lib.rlca_token_logprob(*a.values(), None)


def _head_grad(lib, **k):
    a = dict(h=P[0], w=P[1], tok=P[2], lse=P[3], ent=P[4], g=P[5], e=P[6], dh=P[7], dw=P[8], N=4, D=8, V=16, hs=8,
             wst=8, it=1.0, flags=0, ws=None, wsb=0)
    a.update(k)
    return lib.rlca_token_logprob_backward(*a.values(), None)


def test_token_logprob_refusals(lib):
    assert _head(lib, N=0, h=None) == OK
    assert _head_grad(lib, N=0, h=None, dw=None) == OK
    common = [dict(N=-1), dict(D=0), dict(V=0), dict(h=None), dict(w=None), dict(tok=None), dict(lse=None),
              dict(hs=7), dict(wst=7), dict(it=math.nan), dict(it=math.inf), dict(it=0.0),
              dict(it=-1.0), dict(flags=0x10)]
    for bad in common + [dict(logp=None), dict(logp=P[0]), dict(lse=P[3]), dict(ent=P[2])]:
        assert _head(lib, **bad) == INV, bad
    for bad in common + [dict(g=None), dict(ent=None), dict(e=None), dict(dh=None, dw=None), dict(dh=P[0]),
                         dict(dw=P[1]), dict(dw=P[7])]:
        assert _head_grad(lib, **bad) == INV, bad
    for big in (dict(D=_lib.RLCA_MAX_HEAD_DIM + 1, hs=1 << 20, wst=1 << 20), dict(N=_lib.RLCA_MAX_HEAD_ROWS + 1),
                dict(V=_lib.RLCA_MAX_HEAD_ROWS + 1)):
        assert _head(lib, **big) == UNS and _head_grad(lib, **big) == UNS


def _clip(lib, grads, outs, sizes, dtypes, max_norm=1.0, eps=1e-6, norm=P[15], count=None, ws=None, wsb=0):
    n = len(grads)
    arr = lambda t, v: None if v is None else (t * n)(*v)  # noqa: E731
    return lib.rlca_clip_grads(arr(C.c_void_p, grads), arr(C.c_void_p, outs), arr(C.c_int64, sizes),
                               arr(C.c_uint32, dtypes), n if count is None else count, max_norm, eps, norm, ws, wsb, None)


def test_clip_refusals(lib):
    g, o = [P[0].value, P[1].value], [P[2].value, P[3].value]
    for kw in (dict(count=-1), dict(norm=None), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=-1.0),
               dict(norm=P[0]), dict(norm=P[2])):
        assert _clip(lib, g, o, [4, 4], [0, 0], **kw) == INV, kw
    assert _clip(lib, g, o, [4, -1], [0, 0]) == INV
    assert _clip(lib, g, o, [4, 4], [0, 1]) == INV
    assert _clip(lib, [P[0].value, None], o, [4, 4], [0, 0]) == INV
    assert _clip(lib, g, [P[2].value, None], [4, 4], [0, 0]) == INV
    assert _clip(lib, g, [P[0].value + 4, P[3].value], [4, 4], [0, 0]) == INV       # part overlap within a pair
    assert _clip(lib, [P[0].value + 1, P[1].value], o, [4, 4], [_lib.RLCA_BF16, 0]) == INV  # not on an element boundary


def test_workspace_size_refusals(lib):
    out = C.c_size_t(1)
    q = lambda *a: lib.rlca_workspace_size(*a, C.byref(out))  # noqa: E731
    assert q(_lib.RLCA_EST_TOKEN_LOGPROB, 0, 8, 16, 0) == OK and out.value == 0
    assert q(_lib.RLCA_EST_TOKEN_LOGPROB, 4, 0, 16, 0) == INV
    assert q(_lib.RLCA_EST_TOKEN_LOGPROB_BACKWARD, 4, 8, 0, 0) == INV
    assert q(_lib.RLCA_EST_TOKEN_LOGPROB, 4, 8, 16, _lib.RLCA_TIME_MAJOR) == INV
    assert q(_lib.RLCA_EST_TOKEN_LOGPROB, 4, _lib.RLCA_MAX_HEAD_DIM + 1, 16, 0) == UNS
    assert q(_lib.RLCA_EST_LAYER_NORM_BACKWARD, -1, 8, 0, 0) == INV
    assert q(_lib.RLCA_EST_CLIP_GRADS, 0, 1, 0, 0) == OK and out.value == 0


# ---- refusals of the Python binding ------------------------------------------

def _f(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def _tok(n):
    return torch.zeros(n, dtype=torch.int32)


def test_binding_refusals():
    bf = torch.bfloat16
    norm, grad = rlca.rlca_layer_norm, rlca.rlca_layer_norm_backward
    head, head_grad, clip = rlca.rlca_token_logprob, rlca.rlca_token_logprob_backward, rlca.rlca_clip_grads
    cases = [
        (TypeError, lambda: norm(_f(4, 8, dtype=torch.float64), _f(8))),
        (TypeError, lambda: norm(_f(4, 8), _f(8, dtype=bf))),
        (ValueError, lambda: norm(_f(4, 8), _f(7))),
        (ValueError, lambda: norm(_f(32), _f(32))),
        (ValueError, lambda: norm(_f(8, 4).t(), _f(8))),                       # columns contiguous
        (ValueError, lambda: norm(_f(1, 8).expand(4, 8), _f(8))),              # rows overlap
        (ValueError, lambda: norm(_f(4, 8), _f(8), y=_f(4, 9))),
        (ValueError, lambda: norm(_f(4, 8), _f(8))),                           # not on a CUDA device
        (ValueError, lambda: grad(_f(4, 7), _f(4, 8), _f(8), _f(4), _f(4))),
        (TypeError, lambda: grad(_f(4, 8), _f(4, 8), _f(8), _f(4, dtype=bf), _f(4))),
        (ValueError, lambda: grad(_f(4, 8), _f(4, 8), _f(8), _f(4), _f(4), want_dx=False, want_dweight=False,
                                  want_dbias=False)),
        (ValueError, lambda: grad(_f(4, 8), _f(4, 8), _f(8), _f(4), _f(4))),
        (TypeError, lambda: head(_f(4, 8), _f(16, 8), torch.zeros(4, dtype=torch.int64))),
        (TypeError, lambda: head(_f(4, 8), _f(16, 8, dtype=bf), _tok(4))),
        (ValueError, lambda: head(_f(4, 8), _f(16, 9), _tok(4))),
        (ValueError, lambda: head(_f(4, 8), _f(8), _tok(4))),
        (ValueError, lambda: head(_f(4, 8), _f(16, 8), _tok(5))),
        (ValueError, lambda: head(_f(4, 8), _f(16, 8), _tok(4), temperature=0.0)),
        (ValueError, lambda: head(_f(4, 8), _f(16, 8), _tok(4))),
        (ValueError, lambda: head_grad(_f(4, 8), _f(16, 8), _tok(4), _f(4), _f(4), entropy=_f(4))),
        (ValueError, lambda: head_grad(_f(4, 8), _f(16, 8), _tok(4), _f(4), _f(5))),
        (ValueError, lambda: head_grad(_f(4, 8), _f(16, 8), _tok(4), _f(4), None)),
        (ValueError, lambda: head_grad(_f(4, 8), _f(16, 8), _tok(4), _f(4), _f(4), want_d_hidden=False,
                                       want_d_weight=False)),
        (ValueError, lambda: head_grad(_f(4, 8), _f(16, 8), _tok(4), _f(4), _f(4))),
        (ValueError, lambda: clip([], 1.0)),
        (TypeError, lambda: clip([_f(4, dtype=torch.float16)], 1.0)),
        (ValueError, lambda: clip([_f(8, 4).t()], 1.0)),
        (ValueError, lambda: clip([_f(4)], 1.0, out=[_f(4), _f(4)])),
        (TypeError, lambda: clip([_f(4)], 1.0, out=[_f(4, dtype=bf)])),
        (ValueError, lambda: clip([_f(4)], 1.0)),
    ]
    for k, (err, call) in enumerate(cases):
        with pytest.raises(err):
            call()
            raise AssertionError(f"case {k} was not refused")
