"""64-bit results of the operators of a recurrent policy's trunk, from their
definitions, in plain torch on whatever device the inputs are on.

Inputs of any float type are widened first; nothing is narrowed.  Beside the
results, the functions return the magnitudes that a rounding-error bound
needs: the same recurrences and sums over absolute values, and over the errors
that one relative error per operation leaves.
"""
from __future__ import annotations

import torch

GROUP = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126


def _steps(x, gate, terminated, truncated, lengths, time_major):
    """Time first: x and gate where a row takes part (0 elsewhere), which
    steps take part, and for t = 0 .. T whether the state before step t counts."""
    x, gate = x.double(), gate.double()
    if not time_major:
        x, gate = x.transpose(0, 1), gate.transpose(0, 1)
    T, E, _ = x.shape
    dev = x.device
    real = torch.ones((T, E), dtype=torch.bool, device=dev)
    if lengths is not None:
        real = torch.arange(T, device=dev)[:, None] < lengths[None, :]
    cut = torch.zeros((T, E), dtype=torch.bool, device=dev)
    for f in (terminated, truncated):
        if f is not None:
            cut |= (f if time_major else f.t()) != 0
    keep = torch.ones((T + 1, E), dtype=torch.bool, device=dev)
    keep[1:] = ~(cut & real)
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    x, gate = (torch.where(real[..., None], v, zero) for v in (x, gate))
    return x, torch.sigmoid(gate), torch.sigmoid(-gate), real, keep


def _order(v, time_major):
    return v if time_major else v.transpose(0, 1)


def gated_scan(x, gate, terminated=None, truncated=None, state=None, lengths=None, time_major=False):
    """(h, last, bound_h, bound_last): the bounds accumulate, for every step
    that a value passes through, the magnitude it has there."""
    x, a, na, real, keep = _steps(x, gate, terminated, truncated, lengths, time_major)
    T, E, D = x.shape
    v = torch.zeros((E, D), dtype=torch.float64, device=x.device) if state is None else state.double()
    m, s = v.abs(), torch.zeros_like(v)
    h, bound = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(T):
        on, k = real[t][:, None], keep[t][:, None]
        v, m, s = (torch.where(k, y, torch.zeros_like(y)) for y in (v, m, s))
        nv, nm = a[t] * v + na[t] * x[t], a[t] * m + na[t] * x[t].abs()
        ns = a[t] * s + nm
        v, m, s = (torch.where(on, new, old) for new, old in ((nv, v), (nm, m), (ns, s)))
        h[t], bound[t] = torch.where(on, v, torch.zeros_like(v)), torch.where(on, s, torch.zeros_like(s))
    k = keep[T][:, None]
    v, s = (torch.where(k, y, torch.zeros_like(y)) for y in (v, s))
    return _order(h, time_major), v, _order(bound, time_major), s


def gated_scan_backward(dh, x, gate, h, terminated=None, truncated=None, state=None, lengths=None, d_last=None,
                        time_major=False):
    """(dx, dgate, d_state, bound_dx, bound_dgate, bound_state)."""
    x, a, na, real, keep = _steps(x, gate, terminated, truncated, lengths, time_major)
    T, E, D = x.shape
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    dh, h = _order(dh.double(), time_major), _order(h.double(), time_major)
    first = torch.zeros((E, D), dtype=torch.float64, device=x.device) if state is None else state.double()
    u = torch.zeros_like(first) if d_last is None else d_last.double()
    u = torch.where(keep[T][:, None], u, zero)
    mu, su = u.abs(), torch.zeros_like(u)
    dx, dgate, bx, bg = (torch.zeros_like(x) for _ in range(4))
    for t in range(T - 1, -1, -1):
        on, k = real[t][:, None], keep[t][:, None]
        g = torch.where(on, dh[t], zero)
        G, M = g + u, g.abs() + mu
        S = su + M
        before = torch.where(k, h[t - 1] if t > 0 else first, zero)
        dx[t] = torch.where(on, na[t] * G, zero)
        dgate[t] = torch.where(on, a[t] * na[t] * G * (before - x[t]), zero)
        bx[t] = torch.where(on, na[t] * S, zero)
        bg[t] = torch.where(on, a[t] * na[t] * S * (before.abs() + x[t].abs()), zero)
        nu, nm = torch.where(k, a[t] * G, zero), torch.where(k, a[t] * M, zero)
        ns = torch.where(k, a[t] * S, zero) + nm
        # (a step that takes no part hands on what it got, or nothing behind a flag)
        u, mu, su = (torch.where(on, new, torch.where(k, old, zero)) for new, old in ((nu, u), (nm, mu), (ns, su)))
    return tuple(_order(v, time_major) for v in (dx, dgate)) + (u,) + tuple(_order(v, time_major) for v in (bx, bg)) + (su,)


def scales(v):
    """The scales of v's groups of columns [N, ceil(D / 128)]; NaN does not count."""
    v = torch.nan_to_num(v.double().abs(), nan=0.0, posinf=float("inf"))
    amax = torch.stack([g.amax(1) for g in torch.split(v, GROUP, 1)], 1)
    return (amax / E4M3_MAX).clamp(min=TINY)


def read_back(q, scale):
    """The values that rows in 8 bits stand for."""
    return q.double() * scale.double().repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def rms_norm(total, weight, eps):
    """(y, rstd)"""
    total = total.double()
    rstd = 1.0 / torch.sqrt((total * total).mean(1) + eps)
    return total * rstd[:, None] * weight.double(), rstd


def rms_norm_backward(dy, total, weight, rstd, d_total=None):
    """(dx, dweight, bound_along, bound_weight): the bounds are the sums of
    absolute values behind mean(g s) and dweight."""
    dy, s = dy.double(), total.double() * rstd.double()[:, None]
    g = dy * weight.double()
    dx = rstd.double()[:, None] * (g - s * (g * s).mean(1, keepdim=True))
    if d_total is not None:
        dx = dx + d_total.double()
    return dx, (dy * s).sum(0), (g * s).abs().mean(1, keepdim=True), (dy * s).abs().sum(0)
