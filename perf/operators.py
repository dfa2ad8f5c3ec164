"""The operators of a token-level policy update, as measured cases: listed sizes, drawn sizes, inputs, one pass,
the work a pass cannot do without, and 64-bit results.

Policies over a vocabulary of tokens train on the advantages that the credit-assignment scans produce.  Around the
scans such an update runs the final layer norm, the policy head -- log-probabilities of the taken tokens and the
policy's entropy, straight from the hidden rows -- the gradients of both, and the clipping of all gradients by their
global norm.  ``own`` selects whether :func:`run` computes them in plain 32-bit torch operations or through this
package.
"""
import math

import torch

own = False

_DTYPES = {"bfloat16": torch.bfloat16, "float32": torch.float32}
_SEQ = 512  # rows are laid out as sequences of this length; the first part of each is a prompt that takes no part


# ---- cases ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token of one sequence, scored while serving: latency, the head's weights are read once
        dict(name="logprob-one-token", op="logprob", rows=1, dim=1024, vocab=32768, dtype="bfloat16", masked=0.0,
             temperature=1.0),
        # scoring a rollout batch whose prompts take no part; an odd vocabulary
        dict(name="logprob-rollout", op="logprob", rows=6001, dim=2048, vocab=49999, dtype="bfloat16", masked=0.4,
             temperature=0.7),
        # the largest scoring batch: every row takes part, a large vocabulary
        dict(name="logprob-long", op="logprob", rows=8192, dim=4096, vocab=131072, dtype="bfloat16", masked=0.0,
             temperature=1.0),
        # a small policy's update step: odd sizes everywhere, launch latency counts
        dict(name="logprob-grad-small", op="logprob_backward", rows=37, dim=200, vocab=1003, dtype="bfloat16",
             masked=0.0, temperature=1.0),
        # a policy trained in float32
        dict(name="logprob-grad-float32", op="logprob_backward", rows=1024, dim=1024, vocab=32768, dtype="float32",
             masked=0.25, temperature=1.0),
        # the largest update: gradients of the hidden rows and of a large head
        dict(name="logprob-grad-long", op="logprob_backward", rows=4096, dim=4096, vocab=131072, dtype="bfloat16",
             masked=0.25, temperature=1.0),
        # the final norm of a few sequences' new tokens
        dict(name="norm-few-rows", op="norm", rows=8, dim=1024, dtype="bfloat16"),
        # the final norm of a long training batch
        dict(name="norm-long", op="norm", rows=65536, dim=4096, dtype="bfloat16"),
        # its backward pass, ragged rows in float32
        dict(name="norm-grad-ragged", op="norm_backward", rows=5001, dim=1001, dtype="float32"),
        # its backward pass over a long training batch
        dict(name="norm-grad-long", op="norm_backward", rows=32768, dim=4096, dtype="bfloat16"),
        # clipping the gradients of a small policy: a few tensors of a few thousand elements
        dict(name="clip-small", op="clip", layers=2, dim=63, vocab=257, dtype="float32", scale=1e-1),
        # clipping the gradients of a large policy: 50 tensors, 1.3 G elements, matrices in bfloat16, norms in float32
        dict(name="clip-large", op="clip", layers=6, dim=4096, vocab=32768, dtype="bfloat16", scale=1e-3),
    ]


def _log_uniform(rng, lo, hi):
    while True:
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if rng.random() < 0.5 and n >= 64:
            n = (n + 31) // 64 * 64  # half of the larger sizes are whole multiples, the others odd as drawn
        if lo <= n <= hi and n != 3072:
            return n


def draw(rng):
    op = rng.choice(["logprob", "logprob", "logprob_backward", "logprob_backward", "norm", "norm_backward", "clip"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op in ("logprob", "logprob_backward"):
        cap = 2.0e12 if dtype == "float32" else 8.0e12
        while True:
            case = dict(op=op, rows=_log_uniform(rng, 1, 8192), dim=_log_uniform(rng, 64, 4096),
                        vocab=_log_uniform(rng, 300, 131072), dtype=dtype,
                        masked=rng.choice([0.0, 0.0, 0.25, 0.4, 0.75]), temperature=rng.choice([1.0, 1.0, 0.7, 1.3]))
            if work(case)["flops"] <= cap:
                return case
    if op in ("norm", "norm_backward"):
        while True:
            case = dict(op=op, rows=_log_uniform(rng, 1, 65536), dim=_log_uniform(rng, 32, 8192), dtype=dtype)
            if work(case)["bytes"] <= 8.0e8:
                return case
    while True:
        case = dict(op=op, layers=rng.randint(1, 7), dim=_log_uniform(rng, 16, 4096),
                    vocab=_log_uniform(rng, 100, 65536), dtype=dtype, scale=rng.choice([1e-3, 1e-2, 1e-6]))
        if case["dim"] != 768 and work(case)["bytes"] <= 4.0e9:
            return case


# ---- inputs --------------------------------------------------------------------------------------------------

def _prompt(case):
    """Rows of each whole or partial sequence that take no part, and how many rows of all take part."""
    rows, off = case["rows"], case["masked"]
    lengths = [min(_SEQ, rows - at) for at in range(0, rows, _SEQ)]
    return [int(off * n) for n in lengths], rows - sum(int(off * n) for n in lengths)


def _shapes(case):
    """Gradient tensors of a decoder-shaped policy: (shape, type); vectors are float32."""
    d, v, t = case["dim"], case["vocab"], case["dtype"]
    layer = [((d, d), t)] * 4 + [((4 * d, d), t), ((d, 4 * d), t), ((d,), "float32"), ((d,), "float32")]
    return [((v, d), t)] + layer * case["layers"] + [((d,), "float32")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    op, state = case["op"], dict(op=case["op"])
    dtype = _DTYPES[case["dtype"]]
    if op in ("logprob", "logprob_backward"):
        n, d, v = case["rows"], case["dim"], case["vocab"]
        weight = (normal(v, d) * (2.0 / math.sqrt(d))).to(dtype)
        taken = torch.randint(0, v, (n,), generator=gen, device="cuda")
        # rows lean towards the token taken, some a little and some so far that it is the likeliest
        lean = 2.0 * torch.rand((n, 1), generator=gen, device="cuda")
        hidden = (normal(n, d) + lean * weight[taken].float()).to(dtype)
        tokens = taken.to(torch.int32)
        for i, off in enumerate(_prompt(case)[0]):
            tokens[i * _SEQ:i * _SEQ + off] = -1
        state.update(hidden=hidden, weight=weight, tokens=tokens, temperature=case["temperature"])
        if op == "logprob_backward":
            logp, lse, entropy = _logprob(hidden, weight, tokens, case["temperature"])
            count = max(1, _prompt(case)[1])
            # the policy gradient's factors: minus the advantage over the rows, and a small entropy bonus
            state.update(lse=lse, entropy=entropy, d_logp=-normal(n) / count,
                         d_entropy=torch.full((n,), -0.01 / count, device="cuda"))
    elif op in ("norm", "norm_backward"):
        n, d = case["rows"], case["dim"]
        x = (1.5 * normal(n, d) + 0.5 * normal(n, 1)).to(dtype)
        weight, bias = (1.0 + 0.1 * normal(d)).to(dtype), (0.1 * normal(d)).to(dtype)
        state.update(x=x, weight=weight, bias=bias, eps=1e-5)
        if op == "norm_backward":
            _, mean, rstd = _norm(x, weight, bias, 1e-5)
            state.update(dy=normal(n, d).to(dtype), mean=mean, rstd=rstd)
    else:
        grads = [(normal(*shape) * case["scale"]).to(_DTYPES[t]) for shape, t in _shapes(case)]
        state.update(grads=grads, out=[torch.empty_like(g) for g in grads], max_norm=1.0)
    return state


# ---- the plain forms -----------------------------------------------------------------------------------------

def _logits(hidden, weight, temperature):
    return (hidden.float() @ weight.float().t()) * (1.0 / temperature)


def _logprob(hidden, weight, tokens, temperature):
    part = (tokens >= 0) & (tokens < weight.shape[0])
    z = _logits(hidden, weight, temperature)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1)
    lse = top[:, 0] + torch.log(total)
    entropy = lse - e.mul_(z).sum(1) / total
    at = torch.where(part, tokens, torch.zeros_like(tokens)).long()
    logp = z.gather(1, at[:, None])[:, 0] - lse
    zero = torch.zeros_like(lse)
    return torch.where(part, logp, zero), torch.where(part, lse, zero), torch.where(part, entropy, zero)


def _logprob_backward(s):
    hidden, weight, tokens = s["hidden"], s["weight"], s["tokens"]
    part = (tokens >= 0) & (tokens < weight.shape[0])
    at = torch.where(part, tokens, torch.zeros_like(tokens)).long()
    zero = torch.zeros_like(s["d_logp"])
    d_logp, d_entropy = torch.where(part, s["d_logp"], zero), torch.where(part, s["d_entropy"], zero)
    logq = _logits(hidden, weight, s["temperature"]).sub_(s["lse"][:, None])
    p = torch.exp(logq)
    dz = logq.add_(s["entropy"][:, None]).mul_(-d_entropy[:, None]).sub_(d_logp[:, None]).mul_(p)
    dz = torch.where(part[:, None], dz, torch.zeros_like(dz))
    dz.scatter_add_(1, at[:, None], d_logp[:, None])
    dz.mul_(1.0 / s["temperature"])
    return (dz @ weight.float()).to(hidden.dtype), (dz.t() @ hidden.float()).to(weight.dtype)


def _norm(x, weight, bias, eps):
    x32 = x.float()
    mean = x32.mean(1)
    centred = x32 - mean[:, None]
    rstd = torch.rsqrt((centred * centred).mean(1) + eps)
    return (centred * rstd[:, None] * weight.float() + bias.float()).to(x.dtype), mean, rstd


def _norm_backward(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    return dx.to(s["x"].dtype), (dy * xhat).sum(0).to(s["weight"].dtype), dy.sum(0).to(s["weight"].dtype)


def _clip(grads, max_norm, eps=1e-6):
    squares = torch.stack([torch.sum(torch.square(g.float())) for g in grads])
    norm = torch.sqrt(squares.sum())
    one = torch.ones_like(norm)
    scale = torch.where(torch.isfinite(norm), torch.minimum(one, max_norm / (norm + eps)), one)
    return [(g.float() * scale).to(g.dtype) for g in grads], norm


# ---- one pass ------------------------------------------------------------------------------------------------

def run(state):
    s, op = state, state["op"]
    if own:
        from first_order_linear_gb300 import rlca
        if op == "logprob":
            logp, lse, entropy = rlca.rlca_token_logprob(s["hidden"], s["weight"], s["tokens"],
                                                         temperature=s["temperature"])
            return {"logp": logp, "lse": lse, "entropy": entropy}
        if op == "logprob_backward":
            d_hidden, d_weight = rlca.rlca_token_logprob_backward(
                s["hidden"], s["weight"], s["tokens"], s["lse"], s["d_logp"], entropy=s["entropy"],
                d_entropy=s["d_entropy"], temperature=s["temperature"])
            return {"d_hidden": d_hidden, "d_weight": d_weight}
        if op == "norm":
            y, mean, rstd = rlca.rlca_layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"])
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "norm_backward":
            dx, dweight, dbias = rlca.rlca_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
            return {"dx": dx, "dweight": dweight, "dbias": dbias}
        clipped, norm = rlca.rlca_clip_grads(s["grads"], s["max_norm"], out=s["out"])
        return {"grads": clipped, "norm": norm}
    if op == "logprob":
        logp, lse, entropy = _logprob(s["hidden"], s["weight"], s["tokens"], s["temperature"])
        return {"logp": logp, "lse": lse, "entropy": entropy}
    if op == "logprob_backward":
        d_hidden, d_weight = _logprob_backward(s)
        return {"d_hidden": d_hidden, "d_weight": d_weight}
    if op == "norm":
        y, mean, rstd = _norm(s["x"], s["weight"], s["bias"], s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dx, dweight, dbias = _norm_backward(s)
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    clipped, norm = _clip(s["grads"], s["max_norm"])
    return {"grads": clipped, "norm": norm}


# ---- what a pass cannot do without ---------------------------------------------------------------------------

def work(case):
    op, size = case["op"], 2 if case["dtype"] == "bfloat16" else 4
    if op in ("logprob", "logprob_backward"):
        n, d, v, part = case["rows"], case["dim"], case["vocab"], _prompt(case)[1]
        read = (part * d + v * d) * size + 4 * n
        if op == "logprob":  # one product: the logits
            return {"bytes": read + 12 * n, "flops": 2 * part * d * v}
        # three products: the logits, which are not kept, and the two gradients
        return {"bytes": read + 16 * n + (n * d + v * d) * size, "flops": 6 * part * d * v}
    if op == "norm":
        n, d = case["rows"], case["dim"]
        return {"bytes": 2 * n * d * size + 2 * d * size + 8 * n, "flops": 8 * n * d}
    if op == "norm_backward":
        n, d = case["rows"], case["dim"]
        return {"bytes": 3 * n * d * size + 3 * d * size + 8 * n, "flops": 14 * n * d}
    total = sum(math.prod(shape) * (2 if t == "bfloat16" else 4) for shape, t in _shapes(case))
    count = sum(math.prod(shape) for shape, _ in _shapes(case))
    return {"bytes": 2 * total + 4, "flops": 3 * count}


# ---- 64-bit results ------------------------------------------------------------------------------------------

def _exact_logprob(s, backward):
    hidden, weight = s["hidden"].double(), s["weight"].double().requires_grad_(backward)
    tokens, temperature = s["tokens"].long(), s["temperature"]
    n, v = hidden.shape[0], weight.shape[0]
    results = [torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(3)]
    d_hidden, d_weight = torch.zeros_like(hidden), torch.zeros_like(weight)
    rows = torch.nonzero((tokens >= 0) & (tokens < v))[:, 0]
    step = max(1, min(2048, (1 << 28) // v))
    for chunk in torch.split(rows, step):
        if not len(chunk):
            continue
        h = hidden[chunk].requires_grad_(backward)
        z = torch.matmul(h, weight.t()) / temperature
        logq = torch.log_softmax(z, dim=1)
        logp = torch.gather(logq, 1, tokens[chunk][:, None]).squeeze(1)
        entropy = -(logq.exp() * logq).sum(dim=1)
        if backward:
            value = (logp * s["d_logp"].double()[chunk] + entropy * s["d_entropy"].double()[chunk]).sum()
            gh, gw = torch.autograd.grad(value, [h, weight])
            d_hidden[chunk] = gh
            d_weight += gw
        else:
            for to, value in zip(results, (logp, torch.logsumexp(z, dim=1), entropy)):
                to[chunk] = value
    return {"d_hidden": d_hidden, "d_weight": d_weight} if backward else dict(zip(("logp", "lse", "entropy"), results))


def exact(case, seed):
    if case["op"] in ("logprob", "logprob_backward") and work(case)["flops"] > 1.1e13:
        return None
    s, op = prepare(case, seed), case["op"]
    if op in ("logprob", "logprob_backward"):
        return _exact_logprob(s, op == "logprob_backward")
    if op in ("norm", "norm_backward"):
        x, w, b = (s[k].double().requires_grad_() for k in ("x", "weight", "bias"))
        if op == "norm":
            with torch.no_grad():
                y = torch.nn.functional.layer_norm(x, (x.shape[1],), w, b, s["eps"])
                var, mean = torch.var_mean(x, dim=1, correction=0)
                return {"y": y, "mean": mean, "rstd": 1.0 / torch.sqrt(var + s["eps"])}
        # the statistics are inputs of the backward pass; the normalised rows they give are differentiated through
        y = torch.nn.functional.layer_norm(x, (x.shape[1],), w, b, s["eps"])
        dx, dweight, dbias = torch.autograd.grad(y, [x, w, b], s["dy"].double())
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    total = sum(torch.dot(g.double().reshape(-1), g.double().reshape(-1)) for g in s["grads"])
    norm = torch.sqrt(total)
    scale = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return {"grads": [g.double() * scale for g in s["grads"]], "norm": norm}
