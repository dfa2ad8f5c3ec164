"""The operators of a recurrent policy's trunk together, as one update and one
step of acting use them, against 64-bit differentiation of the same network."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _rms(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w


def _network(d):
    """Normalised rows and last states in 64 bits."""
    x, delta, lasts = d["embedded"], 0, []
    E, T, D = x.shape
    for p, state in zip(d["layers"], d["states"]):
        x = x + delta
        both = _rms(x, p["norm"]) @ p["into"].t()
        a, h, hs = torch.sigmoid(both[..., D:]), state, []
        for t in range(T):
            if t > 0:
                h = h * (d["terminated"][:, t - 1] == 0)[:, None]
            h = a[:, t] * h + (1 - a[:, t]) * both[:, t, :D]
            hs.append(h)
        lasts.append(h * (d["terminated"][:, T - 1] == 0)[:, None])
        delta = torch.stack(hs, 1) @ p["out"].t()
    return _rms(x + delta, d["norm"]), lasts


def _reference(batch):
    """Results of the update by automatic differentiation in 64 bits."""
    def wide(v):
        if isinstance(v, list):
            return [wide(x) for x in v]
        if isinstance(v, dict):
            return {k: wide(x) for k, x in v.items()}
        return v.double().requires_grad_() if v.is_floating_point() else v

    d = wide(batch)
    x, lasts = _network(d)
    V = d["head"].shape[0]
    part = (d["tokens"] >= 0) & (d["tokens"] < V)
    logq = torch.log_softmax(x.reshape(-1, x.shape[2]) @ d["head"].t(), 1)
    logp = logq.gather(1, d["tokens"].clamp(min=0).long()[:, None])[:, 0] * part
    (-(d["advantages"] * logp)).sum().backward()
    return dict(logp=logp.detach(), states=[s.detach() for s in lasts], embedded=d["embedded"].grad, norm=d["norm"].grad,
                head=d["head"].grad, layers=[{k: v.grad for k, v in p.items()} for p in d["layers"]])


def _each(got, want, path=""):
    if isinstance(want, dict):
        for k in want:
            yield from _each(got[k], want[k], f"{path}.{k}")
    elif isinstance(want, list):
        for k, (g, w) in enumerate(zip(got, want)):
            yield from _each(g, w, f"{path}[{k}]")
    else:
        yield path, got, want


# float32: products of width 64 to 96 and sums over 300 rows, a dozen operators deep, each a few units of 6e-8 off:
# below 1e-5.  The stream kept in 8 bits is half a step, 2^-4, of a value off at most, so are the products of it that
# a weight gradient of a norm sums, and what the stream's gradient takes along it; the two last count both.
# bfloat16: every operator rounds its result by 2^-8 at most, some 30 in a row.
@pytest.mark.parametrize("dtype,eight,tol", [(torch.float32, False, 1e-5), (torch.float32, True, 2.0 ** -3),
                                             (torch.bfloat16, False, 0.12)])
def test_update_against_64_bit_differentiation(cuda_lib, dtype, eight, tol):
    import recurrent_policy as example
    for E, T, D, V, layers in ((3, 100, 64, 301, 2), (1, 40, 96, 50, 3)):
        matmul = torch.backends.cuda.matmul.allow_tf32
        torch.backends.cuda.matmul.allow_tf32 = False
        try:
            batch = example.synthetic(E, T, D, V, layers, seed=T, dtype=dtype)
            got = example.update(**batch, keep_in_8_bits=eight)
        finally:
            torch.backends.cuda.matmul.allow_tf32 = matmul
        want = _reference(batch)
        for path, g, w in _each(got, want):
            far = ((g.double() - w).norm() / w.norm().clamp(min=1e-30)).item()
            limit = tol if path.startswith((".embedded", ".layers", ".norm")) or dtype != torch.float32 else 1e-5
            assert far <= limit, f"{path}: {far:.2e} off ({E}, {T}, {D})"


def test_acting_token_by_token_equals_the_scan(cuda_lib):
    """A rollout one token at a time, states moved on in place, against the forward pass over all its steps."""
    import recurrent_policy as example
    E, T, D = 5, 12, 64
    batch = example.synthetic(E, T, D, 50, 2, seed=3, dtype=torch.float32)
    x, lasts, _ = example.forward(batch["embedded"], batch["layers"], batch["norm"], torch.zeros_like(batch["terminated"]),
                                  batch["states"])
    states = [s.clone() for s in batch["states"]]
    rows = [example.act(batch["embedded"][:, t].contiguous(), batch["layers"], batch["norm"], states) for t in range(T)]
    far = (torch.stack(rows, 1).reshape(E * T, D) - x).norm() / x.norm()
    assert far.item() <= 1e-5
    for s, last in zip(states, lasts):
        assert ((s - last).norm() / last.norm()).item() <= 1e-5


def test_example_runs(cuda_lib, capsys):
    import recurrent_policy as example
    argv, sys.argv = sys.argv, ["recurrent_policy.py", "--envs", "2", "--steps", "33", "--dim", "128", "--layers", "2",
                                "--vocab", "500"]
    try:
        example.main()
    finally:
        sys.argv = argv
    assert "ms an update" in capsys.readouterr().out
