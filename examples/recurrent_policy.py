"""One update of a recurrent token policy's trunk, end to end through the library.

The trunk is a stack of layers over a residual stream of rows [E * T, D]; each

    adds the last layer's output to the stream and normalises it   (rlca_rms_norm)
    projects it to candidates and gates, one product
    mixes the steps of each rollout                                 (rlca_gated_scan)
    projects the result back to the stream

and a last norm and a head (rlca_token_logprob) follow.  Rollouts start from
the state the last update left and start anew behind an episode's end.  The
stream is kept in 8 bits for the norms' gradients.  The products are the
caller's: here torch.matmul.

    python examples/recurrent_policy.py [--envs 16] [--steps 256] [--dim 1024] [--layers 4] [--vocab 32768]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from first_order_linear_gb300 import rlca  # noqa: E402


def forward(embedded, layers, norm, terminated, states, *, keep_in_8_bits=True):
    """``embedded`` [E, T, D]; ``layers``: dicts of norm [D], into [2 D, D] and
    out [D, D]; ``states``: a [E, D] float32 a layer.  Returns the normalised
    rows [E * T, D], the states to go on with and what the backward pass needs."""
    E, T, D = embedded.shape
    stream, delta, saved, lasts = embedded.reshape(E * T, D), None, [], []
    for p, state in zip(layers, states):
        y, stream, rstd, _, kept = rlca.rlca_rms_norm(stream if delta is None else delta, p["norm"],
                                                      None if delta is None else stream, want_total8=keep_in_8_bits)
        both = (y @ p["into"].t()).view(E, T, 2 * D)
        h, last = rlca.rlca_gated_scan(both[..., :D], both[..., D:], terminated, state=state)
        delta = h.view(E * T, D) @ p["out"].t()
        saved.append((y, stream if kept is None else kept, rstd, both, h, state))
        lasts.append(last)
    x, stream, rstd, _, kept = rlca.rlca_rms_norm(delta, norm, stream, want_total8=keep_in_8_bits)
    return x, lasts, (saved, stream if kept is None else kept, rstd)


def backward(dx, layers, norm, terminated, saved):
    """Gradients of :func:`forward` for ``dx``: of the embedded rows [E, T, D],
    of each layer's parameters and of the last norm."""
    saved, total, rstd = saved
    d_stream, d_norm = rlca.rlca_rms_norm_backward(dx, total, norm, rstd)
    grads = []
    for p, (y, total, rstd, both, h, state) in zip(reversed(layers), reversed(saved)):
        E, T, D = h.shape
        d_out = d_stream.t() @ h.view(E * T, D)
        dh = (d_stream @ p["out"]).view(E, T, D)
        d_both = torch.empty_like(both)
        rlca.rlca_gated_scan_backward(dh, both[..., :D], both[..., D:], h, terminated, state=state, dx=d_both[..., :D],
                                      dgate=d_both[..., D:], want_d_state=False)
        d_both = d_both.view(E * T, 2 * D)
        d_into = d_both.t() @ y
        d_stream, d_p = rlca.rlca_rms_norm_backward(d_both @ p["into"], total, p["norm"], rstd, d_total=d_stream)
        grads.append(dict(norm=d_p, into=d_into, out=d_out))
    return d_stream.view(E, T, D), grads[::-1], d_norm


def act(embedded, layers, norm, states):
    """One token of E environments: the normalised rows [E, D]; the states are
    moved on in their own buffers."""
    E, D = embedded.shape
    stream, delta = embedded, None
    for p, state in zip(layers, states):
        y, stream, _, _, _ = rlca.rlca_rms_norm(stream if delta is None else delta, p["norm"],
                                                None if delta is None else stream)
        both = (y @ p["into"].t()).view(E, 1, 2 * D)
        h, _ = rlca.rlca_gated_scan(both[..., :D], both[..., D:], state=state, last=state)
        delta = h.view(E, D) @ p["out"].t()
    return rlca.rlca_rms_norm(delta, norm, stream)[0]


def update(embedded, layers, norm, head, terminated, states, tokens, advantages, *, keep_in_8_bits=True):
    """Gradients of the loss  -sum(A logp)  of ``tokens`` [E * T] int32 (-1: takes no part)."""
    x, lasts, saved = forward(embedded, layers, norm, terminated, states, keep_in_8_bits=keep_in_8_bits)
    logp, lse, _ = rlca.rlca_token_logprob(x, head, tokens, want_entropy=False)
    dx, d_head = rlca.rlca_token_logprob_backward(x, head, tokens, lse, -advantages)
    d_embedded, grads, d_norm = backward(dx, layers, norm, terminated, saved)
    return dict(logp=logp, states=lasts, embedded=d_embedded, layers=grads, norm=d_norm, head=d_head)


def synthetic(E, T, D, V, layers, seed=0, dtype=torch.bfloat16):
    """Inputs of :func:`update` on the current CUDA device."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    tokens = torch.randint(0, V, (E, T), generator=gen, device="cuda", dtype=torch.int32)
    tokens[:, :T // 4] = -1
    return dict(
        embedded=normal(E, T, D).to(dtype),
        layers=[dict(norm=(1 + 0.1 * normal(D)).to(dtype), into=(normal(2 * D, D) * D ** -0.5).to(dtype),
                     out=(normal(D, D) * D ** -0.5).to(dtype)) for _ in range(layers)],
        norm=(1 + 0.1 * normal(D)).to(dtype), head=(normal(V, D) * D ** -0.5).to(dtype),
        terminated=(torch.rand((E, T), generator=gen, device="cuda") < 0.02).to(torch.uint8),
        states=[0.5 * normal(E, D) for _ in range(layers)], tokens=tokens.view(-1), advantages=normal(E * T) / (E * T))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--envs", type=int, default=16)
    ap.add_argument("--steps", type=int, default=256)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--vocab", type=int, default=32768)
    a = ap.parse_args()
    batch = synthetic(a.envs, a.steps, a.dim, a.vocab, a.layers)
    for _ in range(3):
        update(**batch)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(10):
        update(**batch)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.envs} x {a.steps} tokens, {a.layers} layers of width {a.dim}, vocabulary {a.vocab}: "
          f"{begin.elapsed_time(end) / 10:.3f} ms an update")


if __name__ == "__main__":
    main()
