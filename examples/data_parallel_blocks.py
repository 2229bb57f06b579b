"""A data-parallel training loop of a small token model over virtual ranks, from the
embedding to the clipped update.

Every rank holds the weights of L blocks of a two-layer perceptron, each between two norms
with a gate and the residual, and its own token sequences:

    embedding  x_0 = s E[ids],  n_0 = norm(x_0)                  (vc_embedding_forward,
    blocks     h = W2 gelu(W1 n_l),                               vc_linear_forward,
               x_{l+1} = x_l + gate_l * norm(h),                  vc_block_norm_forward)
               n_{l+1} = norm(x_{l+1})
    head       logits = n_L H^T
    backward   through all of it into the rank's tensors          (the same, _backward)
    reduce     one bucket AllReduce (mean) over all ranks         (BucketPlan)
    clip       the norm of all gradients, at most 1               (ClipPlan)
    update     Muon for the matrices of the blocks, signs for the rest
    broadcast  the new weights to every rank                      (vc_broadcast)

The task is synthetic: each token's successor is a fixed permutation's.

    python examples/data_parallel_blocks.py --ranks 4 --steps 40
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import allreduce_reducescatter_allgather_gb300 as vc  # noqa: E402

BF16 = torch.bfloat16


def make_weights(vocab: int, width: int, hidden: int, layers: int, rand):
    """Names and 32-bit values."""
    w = {"embed": rand(vocab, width) * width ** -0.5, "pre0": torch.ones_like(rand(width))}
    for i in range(layers):
        w[f"w1_{i}"] = rand(hidden, width) * width ** -0.5
        w[f"w2_{i}"] = rand(width, hidden) * hidden ** -0.5
        w[f"post{i}"] = torch.ones_like(w["pre0"])
        w[f"gate{i}"] = 0.5 * torch.ones_like(w["pre0"])
        w[f"pre{i + 1}"] = torch.ones_like(w["pre0"])
    w["head"] = rand(vocab, width) * width ** -0.5
    return w


class Rank:
    """One virtual rank's weights, gradients and activations."""

    def __init__(self, weights, tokens: int):
        self.w = {k: v.to(BF16) for k, v in weights.items()}
        self.g = {k: torch.empty_like(v) for k, v in weights.items()}
        self.layers = sum(k.startswith("w1_") for k in weights)
        vocab, width = weights["embed"].shape
        hidden = weights["w1_0"].shape[0]
        dev = weights["embed"].device
        new = lambda n: torch.empty(tokens, n, dtype=BF16, device=dev)  # noqa: E731
        many = lambda n, extra=0: [new(n) for _ in range(self.layers + extra)]  # noqa: E731
        self.x, self.n = many(width, 1), many(width, 1)
        self.z, self.a, self.h = many(hidden), many(hidden), many(width)
        self.logits, self.dlogits = new(vocab), new(vocab)
        self.dn, self.dx, self.dh, self.da = new(width), new(width), new(width), new(hidden)
        self.scale = width ** 0.5

    def forward(self, ids):
        w = self.w
        vc.vc_embedding_forward(ids, w["embed"], self.x[0], scale=self.scale)
        vc.vc_block_norm_forward(self.x[0], n=self.n[0], pre=w["pre0"])
        for i in range(self.layers):
            vc.vc_linear_forward(self.n[i], w[f"w1_{i}"], self.a[i], preact=self.z[i],
                                 activation="gelu")
            vc.vc_linear_forward(self.a[i], w[f"w2_{i}"], self.h[i])
            vc.vc_block_norm_forward(self.h[i], x=self.x[i], gate=w[f"gate{i}"], post=w[f"post{i}"],
                                     pre=w[f"pre{i + 1}"], r=self.x[i + 1], n=self.n[i + 1])
        vc.vc_linear_forward(self.n[-1], w["head"], self.logits)
        return self.logits

    def backward(self, ids):
        """dlogits holds the loss's gradient at the logits."""
        w, g = self.w, self.g
        vc.vc_linear_backward(self.dlogits, self.n[-1], w["head"], dx=self.dn, dweight=g["head"])
        dr = None
        for i in reversed(range(self.layers)):
            vc.vc_block_norm_backward(self.h[i], self.dh, dr=dr, dn=self.dn, r=self.x[i + 1],
                                      dx=self.dx, gate=w[f"gate{i}"], dgate=g[f"gate{i}"],
                                      post=w[f"post{i}"], dpost=g[f"post{i}"],
                                      pre=w[f"pre{i + 1}"], dpre=g[f"pre{i + 1}"])
            dr = self.dx  # read and written in place from here on
            vc.vc_linear_backward(self.dh, self.a[i], w[f"w2_{i}"], dx=self.da,
                                  dweight=g[f"w2_{i}"])
            vc.vc_linear_backward(self.da, self.n[i], w[f"w1_{i}"], dx=self.dn,
                                  dweight=g[f"w1_{i}"], preact=self.z[i], activation="gelu")
        vc.vc_block_norm_backward(dr=dr, dn=self.dn, r=self.x[0], dh=self.dh, pre=w["pre0"],
                                  dpre=g["pre0"])
        vc.vc_embedding_backward(self.dh, ids, g["embed"], scale=self.scale)

    def loss(self, targets):
        """The mean cross entropy, whose gradient goes to dlogits."""
        p = torch.log_softmax(self.logits.float(), -1)
        at = torch.arange(len(targets), device=targets.device)
        grad = p.exp()
        grad[at, targets] -= 1.0
        self.dlogits.copy_(grad / len(targets))
        return -p[at, targets].mean()


def train(ranks: int = 4, steps: int = 40, tokens: int = 512, vocab: int = 512, width: int = 256,
          hidden: int = 1024, layers: int = 2, lr: float = 0.02, max_norm: float = 1.0, seed: int = 0,
          device="cuda:0"):
    """The mean loss and the gradients' norm before clipping of each step, and the ranks."""
    dev = torch.device(device)
    rng = torch.Generator(device=dev).manual_seed(seed)
    weights = make_weights(vocab, width, hidden, layers,
                           lambda *s: torch.randn(*s, generator=rng, device=dev))
    follows = torch.randperm(vocab, generator=rng, device=dev)
    group = [Rank(weights, tokens) for _ in range(ranks)]
    names = list(weights)
    bucket = vc.BucketPlan([[r.g[k] for k in names] for r in group])
    clip = vc.ClipPlan([group[0].g[k] for k in names])
    momentum = {k: torch.zeros_like(v) for k, v in weights.items() if k[0] == "w"}
    muon = {k: vc.prepare_muon_step(weights[k], group[0].g[k], momentum[k]) for k in momentum}

    losses, norms = [], []
    for _ in range(steps):
        total, norm = torch.zeros((), device=dev), torch.empty((), device=dev)
        for r in group:
            ids = torch.randint(0, vocab, (tokens,), generator=rng, device=dev)
            r.forward(ids)
            total += r.loss(follows[ids]) / ranks
            r.backward(ids)
        bucket.all_reduce(op="avg")
        clip(max_norm, norm)
        for k in names:
            if k in muon:
                muon[k](lr)
            else:
                weights[k] -= 0.1 * lr * group[0].g[k].sign()
            group[0].w[k].copy_(weights[k])
            vc.vc_broadcast(group[0].w[k], [r.w[k] for r in group])
        losses.append(total)
        norms.append(norm)
    return torch.stack(losses).tolist(), torch.stack(norms).tolist(), group


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args()
    losses, norms, _ = train(a.ranks, a.steps, a.tokens, lr=a.lr)
    for i, (loss, norm) in enumerate(zip(losses, norms)):
        if i % 5 == 0 or i + 1 == len(losses):
            print(f"step {i:4d}  loss {loss:.5f}  gradient norm {norm:.4f}")


if __name__ == "__main__":
    main()
