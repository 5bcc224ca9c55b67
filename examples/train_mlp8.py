"""Data-parallel training of two MLP blocks on one GPU with everything in few bits: activations kept
as unbiased 8-bit checkpoints, gradients of n workers compressed and averaged by Global-QSGD, and on request
products in 8-bit floating point and AdamW with states in 8 bits.

    python examples/train_mlp8.py [--workers 4] [--steps 30] [--width 256] [--tokens 512]
                                  [--products e4m3] [--optimizer adamw8]

Each step, every worker runs its own batch through the same model, and rounds its activations with random
words of its own (block.rank); the workers' gradients are the rows of one matrix, which gq_allreduce_mean
turns into the unbiased estimate of their mean.  The task is to
imitate a fixed teacher of the same shape.  Prints the loss and what the checkpoints take.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import allreduce_compatible_gradient_gb300 as gq  # noqa: E402
from allreduce_compatible_gradient_gb300.act8_layers import MlpBlock8  # noqa: E402
from allreduce_compatible_gradient_gb300.adamw import AdamW  # noqa: E402


def train(workers=4, steps=30, width=256, hidden=1024, tokens=512, lr=0.5, seed=0, products="bf16",
          optimizer="sgd"):
    """The losses of the steps, averaged over the workers."""
    torch.manual_seed(seed)
    teacher, model = (torch.nn.Sequential(*[MlpBlock8(width, hidden, device="cuda") for _ in range(2)])
                      for _ in range(2))
    for block in model:
        block.products = products
    params = list(model.parameters())
    adamw = AdamW(params, lr=3e-3, max_norm=1.0) if optimizer == "adamw8" else None
    d = sum(p.numel() for p in params)
    grads = torch.empty((workers, d), device="cuda")
    ws = gq.gq_workspace("cuda")
    losses = []
    for step in range(steps):
        total = 0.0
        for w in range(workers):
            for block in model:
                block.rank, block.step = w, step
            x = torch.randn((tokens, width), device="cuda").bfloat16()
            with torch.no_grad():
                want = teacher(x).float()
            loss = (model(x).float() - want).square().mean()
            total += loss.detach()
            row = torch.autograd.grad(loss, params)
            grads[w].copy_(torch.cat([g.reshape(-1) for g in row]))
        mean = gq.gq_allreduce_mean(grads, gq.NORM_INF, gq.NORM_INF, gq.LINEAR, 127, seed, step, ws=ws)
        parts = [g.view_as(p) for p, g in zip(params, mean.split([p.numel() for p in params]))]
        if adamw is not None:
            for p, g in zip(params, parts):
                p.grad = g
            adamw.step()
        else:
            with torch.no_grad():
                for p, g in zip(params, parts):
                    p -= lr * g
        losses.append(total / workers)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("workers", 4), ("steps", 30), ("width", 256), ("hidden", 1024), ("tokens", 512)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--products", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--optimizer", choices=("sgd", "adamw8"), default="sgd")
    a = ap.parse_args()
    losses = train(a.workers, a.steps, a.width, a.hidden, a.tokens, products=a.products, optimizer=a.optimizer)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %3d  loss %.5f" % (i, losses[i]))
    print("last      loss %.5f" % losses[-1])
    saved = a.tokens * (a.width + a.hidden)
    print("kept per block and worker: %.2f MB of 8-bit checkpoints instead of %.2f MB of bf16 activations"
          % (saved * (1 + 1 / 32) / 1e6, a.tokens * (2 * a.width + 2 * a.hidden) * 2 / 1e6))


if __name__ == "__main__":
    main()
