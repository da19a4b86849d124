"""A few training steps of a gated feed-forward block and the fused loss head.

Forward: the gated projection and the down projection that adds the residual
stream (two kernels), then the fused linear cross-entropy. Backward through all of
it, then the global gradient norm with clipping, and a plain SGD step.

    python examples/train_block.py --tokens 4096 --hidden 2048 --features 5632 --vocab 32000
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import linear_cross_entropy_gemm_gb300 as F  # noqa: E402


def train(tokens=512, hidden=256, features=704, vocab=2000, steps=8, lr=0.5, max_norm=1.0, seed=0):
    """Returns the loss before each step and the gradient norms."""
    torch.manual_seed(seed)
    block = F.GatedFeedForward(hidden, features, activation="silu", device="cuda")
    head = torch.nn.Parameter(torch.randn(vocab, hidden, device="cuda").mul_(hidden ** -0.5).bfloat16())
    loss_fn = F.FusedLinearCrossEntropyLoss()
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    y = torch.randint(0, vocab, (tokens,), device="cuda")
    params = [*block.parameters(), head]
    losses, norms = [], []
    for _ in range(steps):
        for p in params:
            p.grad = None
        loss = loss_fn(block(x), y, head)
        loss.backward()
        norms.append(F.clip_grad_norm_(params, max_norm))
        with torch.no_grad():
            for p in params:
                p.sub_(p.grad, alpha=lr)
        losses.append(loss.detach())
    return [float(v) for v in losses], [float(v) for v in norms]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 512), ("hidden", 256), ("features", 704), ("vocab", 2000),
                        ("steps", 8)):
        ap.add_argument("--" + name, type=int, default=value)
    losses, norms = train(**vars(ap.parse_args()))
    for i, (loss, norm) in enumerate(zip(losses, norms)):
        print(f"step {i}: loss {loss:.4f}, gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
