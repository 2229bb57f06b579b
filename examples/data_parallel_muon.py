"""A data-parallel training loop over virtual ranks, from the layers to the update.

Every rank holds the weights of a two-layer perceptron and its own batch:

    forward    h = gelu(x W1^T + b1),  y = h W2^T + b2 + x   (vc_linear_forward)
    backward   dW, db of both layers into the rank's tensors (vc_linear_backward)
    reduce     one bucket AllReduce (mean) over all ranks     (BucketPlan)
    update     a Muon step on the 32-bit weights of rank 0    (vc_muon_step)
    broadcast  the new weights to every rank                  (vc_broadcast)

The task is synthetic: the outputs of a fixed random perceptron.

    python examples/data_parallel_muon.py --ranks 4 --steps 40
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import allreduce_reducescatter_allgather_gb300 as vc  # noqa: E402

BF16 = torch.bfloat16


class Rank:
    """One virtual rank's weights, gradients and activations."""

    def __init__(self, weights, batch: int, dev):
        self.w = {k: v.to(BF16) for k, v in weights.items()}
        self.g = {k: torch.empty_like(v, dtype=torch.float32) for k, v in weights.items()}
        width, hidden = weights["w2"].shape
        new = lambda n: torch.empty(batch, n, dtype=BF16, device=dev)  # noqa: E731
        self.z, self.h, self.y = new(hidden), new(hidden), new(width)
        self.dy, self.dh = new(width), new(hidden)

    def forward(self, x):
        w = self.w
        vc.vc_linear_forward(x, w["w1"], self.h, bias=w["b1"], preact=self.z, activation="gelu")
        vc.vc_linear_forward(self.h, w["w2"], self.y, bias=w["b2"], residual=x)
        return self.y

    def backward(self, x):
        """dy holds the loss's gradient at y."""
        w, g = self.w, self.g
        vc.vc_linear_backward(self.dy, self.h, w["w2"], dx=self.dh, dweight=g["w2"],
                              dbias=g["b2"])
        vc.vc_linear_backward(self.dh, x, w["w1"], dweight=g["w1"], dbias=g["b1"],
                              preact=self.z, activation="gelu")


def train(ranks: int = 4, steps: int = 40, batch: int = 256, width: int = 256, hidden: int = 1024,
          lr: float = 0.02, seed: int = 0, device="cuda:0"):
    """The mean loss of each step, and the ranks."""
    dev = torch.device(device)
    rng = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=rng, device=dev)  # noqa: E731
    shapes = {"w1": (hidden, width), "b1": (hidden,), "w2": (width, hidden), "b2": (width,)}
    teacher = {k: rand(*s) * (s[-1] ** -0.5 if k[0] == "w" else 0.1) for k, s in shapes.items()}
    weights = {k: rand(*s) * (s[-1] ** -0.5 if k[0] == "w" else 0.0) for k, s in shapes.items()}
    momentum = {k: torch.zeros_like(v) for k, v in weights.items() if k[0] == "w"}

    group = [Rank(weights, batch, dev) for _ in range(ranks)]
    names = list(shapes)
    bucket = vc.BucketPlan([[r.g[k] for k in names] for r in group])
    muon = {k: vc.prepare_muon_step(weights[k], group[0].g[k], momentum[k]) for k in momentum}
    goal = Rank(teacher, batch, dev)

    losses = []
    for _ in range(steps):
        total = torch.zeros((), device=dev)
        for r in group:
            x = rand(batch, width).to(BF16)
            target = goal.forward(x).float()
            error = r.forward(x).float() - target
            total += error.square().mean() / ranks
            r.dy.copy_(error * (2.0 / error.numel()))
            r.backward(x)
        bucket.all_reduce(op="avg")
        for k in names:
            if k in muon:
                muon[k](lr)
            else:
                weights[k] -= 0.1 * lr * group[0].g[k].sign()
            group[0].w[k].copy_(weights[k])
            vc.vc_broadcast(group[0].w[k], [r.w[k] for r in group])
        losses.append(total)
    return torch.stack(losses).tolist(), group


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--batch", type=int, default=256)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    losses, _ = train(a.ranks, a.steps, a.batch, lr=a.lr)
    for i, loss in enumerate(losses):
        if i % 5 == 0 or i + 1 == len(losses):
            print(f"step {i:4d}  loss {loss:.5f}")


if __name__ == "__main__":
    main()
