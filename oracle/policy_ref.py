"""64-bit results of the policy-update operators, from their definitions, in
plain torch on whatever device the inputs are on.

Inputs of any float type are widened first; nothing is narrowed.  Beside the
results, :func:`token_logprob` and :func:`token_logprob_backward` return the
magnitudes that a rounding-error bound needs: sums of absolute values along
the same contractions.
"""
from __future__ import annotations

import torch


def _part(tokens, V):
    return (tokens >= 0) & (tokens < V)


def _clean(hidden, part):
    # rows that take no part may hold anything
    return torch.where(part[:, None], hidden.double(), torch.zeros((), dtype=torch.float64, device=hidden.device))


def _logits(hidden, weight, temperature):
    return hidden @ weight.double().t() / temperature


def token_logprob(hidden, weight, tokens, temperature=1.0):
    """(logp, lse, entropy, scale): scale[i] = max_j sum_k |h_ik w_jk| / temperature."""
    part = _part(tokens, weight.shape[0])
    h = _clean(hidden, part)
    z = _logits(h, weight, temperature)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    entropy = -(torch.special.xlogy(p, p)).sum(1)
    at = torch.where(part, tokens, torch.zeros_like(tokens)).long()
    logp = z.gather(1, at[:, None])[:, 0] - lse
    scale = (h.abs() @ weight.double().abs().t()).amax(1) / temperature
    zero = torch.zeros_like(lse)
    return tuple(torch.where(part, v, zero) for v in (logp, lse, entropy, scale))


def token_logprob_backward(hidden, weight, tokens, lse, d_logp, entropy=None, d_entropy=None, temperature=1.0):
    """(d_hidden, d_weight, bound_hidden, bound_weight, root_hidden,
    root_weight); the bounds contract the magnitudes of dz's terms with those
    of the other operand, the roots are the square roots of the same
    contractions of squares."""
    part = _part(tokens, weight.shape[0])
    h, w = _clean(hidden, part), weight.double()
    zero = torch.zeros(hidden.shape[0], dtype=torch.float64, device=hidden.device)

    def rows(v):
        return zero if v is None else torch.where(part, v.double(), zero)

    g, e, s, ent = rows(d_logp), rows(d_entropy), rows(lse), rows(entropy)
    logq = _logits(h, weight, temperature) - s[:, None]
    p = torch.where(part[:, None], torch.exp(logq), zero[:, None])
    logq = torch.where(part[:, None], logq, zero[:, None])
    taken = torch.zeros_like(p)
    at = torch.where(part, tokens, torch.zeros_like(tokens)).long()
    taken.scatter_(1, at[:, None], part.double()[:, None])
    dz = (g[:, None] * (taken - p) - e[:, None] * p * (logq + ent[:, None])) / temperature
    mag = (g.abs()[:, None] * (taken + p) + e.abs()[:, None] * p * (logq.abs() + ent.abs()[:, None])) / temperature
    squares = mag * mag
    return (dz @ w, dz.t() @ h, mag @ w.abs(), mag.t() @ h.abs(), torch.sqrt(squares @ (w * w)),
            torch.sqrt(squares.t() @ (h * h)))


def layer_norm(x, weight, bias, eps):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None] * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """(dx, dweight, dbias) from the given statistics."""
    dy, xh = dy.double(), (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy * weight.double()
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def clip_grads(grads, max_norm, eps=1e-6):
    """(clipped, norm, scale)."""
    total = sum((g.double() ** 2).sum() for g in grads) if grads else torch.zeros((), dtype=torch.float64)
    norm = torch.sqrt(total)
    scale = min(1.0, max_norm / (float(norm) + eps)) if bool(torch.isfinite(norm)) else 1.0
    return [g.double() * scale for g in grads], norm, scale
