"""One update of a token policy, end to end through the library.

A policy over a vocabulary of tokens is a trunk (any model; here its output
rows are given), a final layer norm and a head.  One update on a batch of E
rollouts of T tokens runs

    layer norm -> log-probabilities and entropy -> V-Trace -> gradients -> clipping

and returns the trunk's gradient and the clipped gradients of the norm and
the head.  Rows whose token is -1 (prompts, padding) take no part.

    python examples/policy_update.py [--envs 64] [--steps 128] [--dim 1024] [--vocab 32768]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from first_order_linear_gb300 import rlca  # noqa: E402


def policy_update(trunk, norm_weight, norm_bias, head, tokens, behaviour_logp, rewards, values, terminated, *,
                  bootstrap=None, entropy_bonus=0.01, max_norm=1.0, temperature=1.0):
    """``trunk`` [E * T, D]: the trunk's output rows; ``tokens`` [E * T]
    int32; ``behaviour_logp``, ``rewards``, ``values`` [E, T] float32;
    ``terminated`` [E, T] uint8.  Returns a dict of the loss' gradients
    (clipped together by their global norm), the norm, the V-Trace targets
    and the log-probabilities.

    The loss per row that takes part is  -A logp - entropy_bonus * H,  A the
    V-Trace advantage, averaged over those rows."""
    E, T = rewards.shape
    x, mean, rstd = rlca.rlca_layer_norm(trunk, norm_weight, norm_bias)
    logp, lse, entropy = rlca.rlca_token_logprob(x, head, tokens, temperature=temperature)
    vs, advantages = rlca.rlca_vtrace(rewards, values, logp.view(E, T), behaviour_logp, terminated, bootstrap=bootstrap)

    part = (tokens >= 0) & (tokens < head.shape[0])
    scale = part.float() / part.sum().clamp(min=1)
    d_logp = -advantages.reshape(-1) * scale
    d_entropy = -entropy_bonus * scale
    d_x, d_head = rlca.rlca_token_logprob_backward(x, head, tokens, lse, d_logp, entropy=entropy, d_entropy=d_entropy,
                                                   temperature=temperature)
    d_trunk, d_weight, d_bias = rlca.rlca_layer_norm_backward(d_x, trunk, norm_weight, mean, rstd)
    grads = [d_trunk, d_weight, d_bias, d_head]
    _, norm = rlca.rlca_clip_grads(grads, max_norm, out=grads)
    return dict(trunk=d_trunk, norm_weight=d_weight, norm_bias=d_bias, head=d_head, norm=norm, targets=vs, logp=logp)


def synthetic(E, T, D, V, seed=0, dtype=torch.bfloat16, prompt=0.25):
    """Inputs of :func:`policy_update` on the current CUDA device."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    tokens = torch.randint(0, V, (E, T), generator=gen, device="cuda", dtype=torch.int32)
    tokens[:, :int(prompt * T)] = -1
    return dict(
        trunk=normal(E * T, D).to(dtype), norm_weight=(1 + 0.1 * normal(D)).to(dtype),
        norm_bias=(0.1 * normal(D)).to(dtype), head=(normal(V, D) * D ** -0.5).to(dtype), tokens=tokens.view(-1),
        behaviour_logp=-9.0 + 0.5 * normal(E, T), rewards=normal(E, T), values=normal(E, T),
        terminated=(torch.rand((E, T), generator=gen, device="cuda") < 0.01).to(torch.uint8), bootstrap=normal(E))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--envs", type=int, default=64)
    ap.add_argument("--steps", type=int, default=128)
    ap.add_argument("--dim", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32768)
    a = ap.parse_args()
    batch = synthetic(a.envs, a.steps, a.dim, a.vocab)
    for _ in range(3):
        out = policy_update(**batch)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(10):
        out = policy_update(**batch)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.envs} x {a.steps} tokens, width {a.dim}, vocabulary {a.vocab}: {begin.elapsed_time(end) / 10:.3f} ms an update, "
          f"gradient norm {out['norm'].item():.4g}")


if __name__ == "__main__":
    main()
