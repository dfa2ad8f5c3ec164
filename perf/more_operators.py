"""The operators of a recurrent token policy's trunk, as measured cases: listed sizes, drawn sizes, inputs, one pass,
the work a pass cannot do without, and 64-bit results.

A layer of such a trunk normalises its residual stream by the root mean square -- adding the last layer's output on the
way, and leaving its result in 8 bits for an 8-bit product --, projects it to candidates and gates, and mixes the
steps of each rollout by a gated linear recurrence that starts anew behind an episode's end.  Training needs the
gradients of both, the norm's from activations kept in 8 bits; acting needs the recurrence one token at a time.
``own`` selects whether :func:`run` computes them in plain 32-bit torch operations or through this package.
"""
import math

import torch

own = False

_DTYPES = {"bfloat16": torch.bfloat16, "float32": torch.float32}
_GROUP = 128  # columns of a row that share a scale in 8 bits
_E4M3_MAX = 448.0
_TINY = 2.0 ** -126


# ---- cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # a chunk of a prompt appended to one sequence's state while serving
        dict(name="scan-chunk", op="scan", envs=1, steps=512, dim=2048, dtype="bfloat16", time_major=False, ends=0.0,
             padded=False),
        # a rollout batch of a float32 policy: odd sizes, time-major, episodes end inside, rollouts of several lengths
        dict(name="scan-rollouts", op="scan", envs=37, steps=515, dim=1001, dtype="float32", time_major=True, ends=0.01,
             padded=True),
        # one very long sequence: few rows, so the steps have to be shared out
        dict(name="scan-long", op="scan", envs=1, steps=65536, dim=4096, dtype="bfloat16", time_major=False, ends=0.0,
             padded=False),
        # the gradient over the rollout batch
        dict(name="scan-grad-rollouts", op="scan_backward", envs=37, steps=515, dim=1001, dtype="float32",
             time_major=True, ends=0.01, padded=True),
        # the gradient over a training batch of packed documents
        dict(name="scan-grad-batch", op="scan_backward", envs=32, steps=4096, dim=2048, dtype="bfloat16",
             time_major=False, ends=0.001, padded=False),
        # acting: one new token of a few sequences, and of many environments
        dict(name="step-few", op="scan", envs=8, steps=1, dim=1024, dtype="bfloat16", time_major=False, ends=0.0,
             padded=False),
        dict(name="step-many", op="scan", envs=1024, steps=1, dim=4096, dtype="bfloat16", time_major=False, ends=0.0,
             padded=False),
        # the norm in front of an 8-bit product, for a few sequences' new tokens
        dict(name="rms-few-rows", op="rms", rows=8, dim=1024, dtype="bfloat16", residual=True, eight=True, keep=False),
        # ragged rows in float32, the stream kept in 8 bits
        dict(name="rms-ragged", op="rms", rows=5001, dim=1001, dtype="float32", residual=True, eight=False, keep=True),
        # a long training batch: 8-bit output, the stream kept in 8 bits
        dict(name="rms-long", op="rms", rows=65536, dim=4096, dtype="bfloat16", residual=True, eight=True, keep=True),
        # the gradients of the last two from the kept stream
        dict(name="rms-grad-ragged", op="rms_backward", rows=5001, dim=1001, dtype="float32", residual=True, keep=True),
        dict(name="rms-grad-long", op="rms_backward", rows=32768, dim=4096, dtype="bfloat16", residual=True, keep=True),
    ]


def _log_uniform(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 64:
        n = (n + 31) // 64 * 64  # half of the larger sizes are whole multiples, the others odd as drawn
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_backward", "scan_backward", "step", "rms", "rms", "rms_backward", "rms_backward"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op == "step":
        return dict(op="scan", envs=_log_uniform(rng, 1, 1024), steps=1, dim=_log_uniform(rng, 32, 4096), dtype=dtype,
                    time_major=rng.random() < 0.5, ends=rng.choice([0.0, 0.1]), padded=False)
    if op in ("scan", "scan_backward"):
        while True:
            case = dict(op=op, envs=_log_uniform(rng, 1, 256), steps=_log_uniform(rng, 2, 65536),
                        dim=_log_uniform(rng, 32, 4096), dtype=dtype, time_major=rng.random() < 0.5,
                        ends=rng.choice([0.0, 0.001, 0.01, 0.1]), padded=rng.random() < 0.4)
            if work(case)["bytes"] <= (1.6e9 if op == "scan" else 3.2e9):
                return case
    while True:
        case = dict(op=op, rows=_log_uniform(rng, 1, 65536), dim=_log_uniform(rng, 32, 8192), dtype=dtype,
                    residual=rng.random() < 0.7, keep=rng.random() < 0.6)
        if op == "rms":
            case["eight"] = rng.random() < 0.5
        if work(case)["bytes"] <= (2.1e9 if op == "rms" else 9.0e8):
            return case


# ---- inputs --------------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    state, dtype, d = dict(op=case["op"]), _DTYPES[case["dtype"]], case["dim"]
    if case["op"] in ("rms", "rms_backward"):
        n = case["rows"]
        # a few columns of a residual stream are much larger than the others
        x = normal(n, d) * (1.0 + 20.0 * (torch.rand(d, generator=gen, device="cuda") < 0.01))
        weight = (1.0 + 0.1 * normal(d)).to(dtype)
        if case["op"] == "rms":
            state.update(x=x.to(dtype), weight=weight, residual=normal(n, d).to(dtype) if case["residual"] else None,
                         eps=1e-6, eight=case["eight"], keep=case["keep"])
        else:
            total = x.to(dtype)
            rstd = torch.rsqrt((total.float() * total.float()).mean(1) + 1e-6)
            state.update(total=_eight(total.float()) if case["keep"] else total, weight=weight, rstd=rstd,
                         dy=normal(n, d).to(dtype), d_total=normal(n, d).to(dtype) if case["residual"] else None)
        return state

    e, t = case["envs"], case["steps"]
    shape = (t, e) if case["time_major"] else (e, t)
    # candidates and gates are the two halves of one projection's rows; channels forget at rates of their own
    both = normal(*shape, 2 * d)
    both[..., d:] += 6.0 * torch.rand(d, generator=gen, device="cuda")
    both = both.to(dtype)
    ended = (torch.rand(shape, generator=gen, device="cuda") < case["ends"]).to(torch.uint8) if case["ends"] else None
    lengths = torch.randint(0, t + 1, (e,), generator=gen, device="cuda", dtype=torch.int32) if case["padded"] else None
    state.update(x=both[..., :d], gate=both[..., d:], terminated=ended, lengths=lengths, state=0.5 * normal(e, d),
                 time_major=case["time_major"])
    if case["op"] == "scan_backward":
        h, _ = _scan(state)
        grads = torch.zeros_like(both)
        state.update(h=h, dh=normal(*shape, d).to(dtype), d_last=normal(e, d), dx=grads[..., :d], dgate=grads[..., d:])
    return state


# ---- the plain forms -----------------------------------------------------------------------------------------

def _rows_first(s, *names):
    """The named [E, T, ...] tensors with the rows first."""
    swap = (lambda v: v.transpose(0, 1)) if s["time_major"] else (lambda v: v)
    return [None if s[k] is None else swap(s[k]) for k in names]


def _gates(s):
    """Rows first: candidates, gates, 1 - gates, which steps keep the state before them, and which exist."""
    x, gate, ended = _rows_first(s, "x", "gate", "terminated")
    e, t, _ = x.shape
    real = torch.ones((e, t), dtype=torch.bool, device=x.device)
    if s["lengths"] is not None:
        real = torch.arange(t, device=x.device)[None, :] < s["lengths"][:, None]
    keep = torch.ones((e, t + 1), dtype=torch.bool, device=x.device)  # [:, t]: whether the state goes on behind step t - 1
    if ended is not None:
        keep[:, 1:] = ~((ended != 0) & real)
    zero = torch.zeros((), device=x.device)
    x, gate = (torch.where(real[..., None], v.float(), zero) for v in (x, gate))
    a, other = 1.0 / (1.0 + torch.exp(-gate)), 1.0 / (1.0 + torch.exp(gate))
    return x, a, other, keep, real


def _affine(p, q):
    """v_t = p_t v_{t-1} + q_t along dimension 1 from v_{-1} = 0, by doubling: (products of p, v)."""
    step, steps = 1, p.shape[1]
    while step < steps:
        q = torch.cat((q[:, :step], q[:, step:] + p[:, step:] * q[:, :-step]), 1)
        p = torch.cat((p[:, :step], p[:, step:] * p[:, :-step]), 1)
        step *= 2
    return p, q


def _scan(s):
    x, a, other, keep, real = _gates(s)
    p = torch.where(real[..., None], a, torch.ones_like(a)) * keep[:, :-1, None]
    p, q = _affine(p, torch.where(real[..., None], other * x, torch.zeros_like(x)))
    h = q + p * s["state"][:, None, :]
    last = h[:, -1] * keep[:, -1, None]
    h = torch.where(real[..., None], h, torch.zeros_like(h)).to(s["x"].dtype)
    return (h.transpose(0, 1).contiguous() if s["time_major"] else h), last


def _scan_backward(s):
    x, a, other, keep, real = _gates(s)
    h, dh = _rows_first(s, "h", "dh")
    on, zero = real[..., None], torch.zeros((), device=x.device)
    before = torch.cat((s["state"][:, None, :], h[:, :-1].float()), 1) * keep[:, :-1, None]
    # u_t, what step t hands to the state before it, from the last step to the first
    p = torch.where(on, a, torch.ones_like(a)) * keep[:, :-1, None]
    dh = torch.where(on, dh.float(), zero)
    end = (s["d_last"] * keep[:, -1, None])[:, None, :]
    p, q = (v.flip(1) for v in _affine(p.flip(1), (p * dh).flip(1)))
    u = q + p * end
    grad = dh + torch.cat((u[:, 1:], end), 1)
    dx = torch.where(on, other * grad, zero)
    dgate = torch.where(on, a * other * grad * (before - x), zero)
    dx, dgate = ((v.transpose(0, 1) if s["time_major"] else v).to(s["x"].dtype) for v in (dx, dgate))
    return dx.contiguous(), dgate.contiguous(), u[:, 0]


def _eight(v):
    """The rows of v in 8 bits: values and the scales of their groups of columns."""
    n, d = v.shape
    groups = -(-d // _GROUP)
    padded = torch.zeros((n, groups * _GROUP), device=v.device)
    padded[:, :d] = v
    padded = padded.view(n, groups, _GROUP)
    scale = (padded.abs().amax(2) / _E4M3_MAX).clamp(min=_TINY)
    q = (padded / scale[..., None]).clamp(-_E4M3_MAX, _E4M3_MAX).view(n, -1)[:, :d]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def _from_eight(pair):
    q, scale = pair
    return q.float() * scale.repeat_interleave(_GROUP, 1)[:, :q.shape[1]]


def _rms(s):
    total = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    wide = total.float()
    rstd = torch.rsqrt((wide * wide).mean(1) + s["eps"])
    y = wide * rstd[:, None] * s["weight"].float()
    return (None if s["eight"] else y.to(total.dtype), total, rstd, _eight(y) if s["eight"] else None,
            _eight(wide) if s["keep"] else None)


def _rms_backward(s):
    total = _from_eight(s["total"]) if isinstance(s["total"], tuple) else s["total"].float()
    dy, w = s["dy"].float(), s["weight"].float()
    xh = total * s["rstd"][:, None]
    g = dy * w
    dx = (g - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["d_total"] is not None:
        dx = dx + s["d_total"].float()
    return dx.to(s["dy"].dtype), (dy * xh).sum(0).to(s["weight"].dtype)


# ---- one pass ------------------------------------------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if own:
        from first_order_linear_gb300 import rlca
        if op == "scan":
            h, last = rlca.rlca_gated_scan(s["x"], s["gate"], s["terminated"], state=s["state"], lengths=s["lengths"],
                                           time_major=s["time_major"])
            return {"h": h, "last": last}
        if op == "scan_backward":
            dx, dgate, d_state = rlca.rlca_gated_scan_backward(
                s["dh"], s["x"], s["gate"], s["h"], s["terminated"], state=s["state"], lengths=s["lengths"],
                d_last=s["d_last"], dx=s["dx"], dgate=s["dgate"], time_major=s["time_major"])
            return {"dx": dx, "dgate": dgate, "d_state": d_state}
        if op == "rms":
            y, total, rstd, y8, total8 = rlca.rlca_rms_norm(s["x"], s["weight"], s["residual"], eps=s["eps"],
                                                            want_y=not s["eight"], want_y8=s["eight"],
                                                            want_total8=s["keep"])
            return {"y": y, "total": total, "rstd": rstd, "y8": y8, "total8": total8}
        dx, dweight = rlca.rlca_rms_norm_backward(s["dy"], s["total"], s["weight"], s["rstd"], d_total=s["d_total"])
        return {"dx": dx, "dweight": dweight}
    if op == "scan":
        return dict(zip(("h", "last"), _scan(s)))
    if op == "scan_backward":
        return dict(zip(("dx", "dgate", "d_state"), _scan_backward(s)))
    if op == "rms":
        return dict(zip(("y", "total", "rstd", "y8", "total8"), _rms(s)))
    return dict(zip(("dx", "dweight"), _rms_backward(s)))


# ---- what a pass cannot do without ---------------------------------------------------------------------------

def work(case):
    size, d = 2 if case["dtype"] == "bfloat16" else 4, case["dim"]
    if case["op"] in ("rms", "rms_backward"):
        n, r = case["rows"], int(case["residual"])
        eight = d + 4 * -(-d // _GROUP)  # a row in 8 bits
        if case["op"] == "rms":  # reads x and the residual, writes the total and the result, maybe keeps the total
            row = d * size * (1 + 2 * r) + (eight if case["eight"] else d * size) + (eight if case["keep"] else 0)
            return {"bytes": n * (row + 4) + d * size, "flops": (5 + r + 4 * case["eight"] + 4 * case["keep"]) * n * d}
        row = d * size * (2 + r) + (eight if case["keep"] else d * size)
        return {"bytes": n * (row + 4) + 2 * d * size, "flops": (9 + r + case["keep"]) * n * d}
    e, t = case["envs"], case["steps"]
    # the mean length of a padded batch's rollouts is half the steps: the other half is only written, as zeros
    real = e * t * d * (0.5 if case["padded"] else 1.0)
    rows = (e * t if case["ends"] else 0) + (4 * e if case["padded"] else 0)
    if case["op"] == "scan":
        return {"bytes": 2 * real * size + e * t * d * size + 8 * e * d + rows, "flops": 10 * real}
    return {"bytes": 4 * real * size + 2 * e * t * d * size + 12 * e * d + rows, "flops": 18 * real}


# ---- 64-bit results ------------------------------------------------------------------------------------------

def _exact_scan(s, backward):
    """One step after the other, time first; a step's own equations and nothing else."""
    first = (lambda v: v) if s["time_major"] else (lambda v: v.transpose(0, 1))
    x, gate = first(s["x"]).double(), first(s["gate"]).double()
    steps, envs, dim = x.shape
    a = torch.sigmoid(gate)
    if s["lengths"] is None:
        inside = torch.ones((steps, envs, 1), dtype=torch.float64, device="cuda")
    else:
        inside = (torch.arange(steps, device="cuda")[:, None] < s["lengths"][None, :]).double()[..., None]
    on = torch.ones((steps + 1, envs, 1), dtype=torch.float64, device="cuda")
    if s["terminated"] is not None:
        on[1:] -= (first(s["terminated"]) != 0).double()[..., None] * inside
    factor = on[:-1] * (1.0 - inside + inside * a)
    if not backward:
        b = (inside * x).sub_(inside * x * a)
        out, v = torch.empty_like(x), s["state"].double()
        for k in range(steps):
            v = torch.addcmul(b[k], factor[k], v, out=out[k])
        last = out[-1] * on[-1]
        out.mul_(inside)
        return {"h": out if s["time_major"] else out.transpose(0, 1), "last": last}
    grad = first(s["dh"]).double() * inside
    v = s["d_last"].double() * on[-1]
    for k in range(steps - 1, -1, -1):
        grad[k] += v
        v = factor[k] * grad[k]
    previous = torch.cat((s["state"].double()[None], first(s["h"])[:-1].double())) * on[:-1]
    dx = grad * (1.0 - a) * inside
    dgate = dx * a * (previous - x)
    if not s["time_major"]:
        dx, dgate = dx.transpose(0, 1), dgate.transpose(0, 1)
    return {"dx": dx, "dgate": dgate, "d_state": v}


def _exact_eight(v):
    """Scales, and the values over their scales before they are rounded."""
    pieces = torch.split(v, _GROUP, dim=1)
    scale = torch.stack([torch.linalg.vector_norm(p, ord=float("inf"), dim=1) for p in pieces], 1) / _E4M3_MAX
    scale = torch.maximum(scale, torch.full_like(scale, _TINY))
    return torch.cat([p / scale[:, k:k + 1] for k, p in enumerate(pieces)], 1), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("scan", "scan_backward"):
        return _exact_scan(s, case["op"] == "scan_backward")
    w = s["weight"].double()
    if case["op"] == "rms":
        total = s["x"].double()
        if s["residual"] is not None:
            total = (total + s["residual"].double()).to(s["x"].dtype).double()
        rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(total, dim=1).square() / total.shape[1] + s["eps"])
        y = total * rstd[:, None] * w
        return {"y": None if s["eight"] else y, "total": total, "rstd": rstd, "y8": _exact_eight(y) if s["eight"] else None,
                "total8": _exact_eight(total) if s["keep"] else None}
    if isinstance(s["total"], tuple):
        q, scale = s["total"]
        total = torch.cat([p.double() * scale[:, k:k + 1].double() for k, p in enumerate(torch.split(q, _GROUP, dim=1))], 1)
    else:
        total = s["total"].double()
    dy, rstd = s["dy"].double(), s["rstd"].double()
    g, xh = dy * w, total * rstd[:, None]
    along = torch.einsum("nd,nd->n", g, xh) / total.shape[1]
    dx = rstd[:, None] * torch.addcmul(g, xh, along[:, None], value=-1.0)
    if s["d_total"] is not None:
        dx += s["d_total"].double()
    return {"dx": dx, "dweight": torch.einsum("nd,nd->d", dy, xh)}
