"""examples/data_parallel_blocks.py: the embedding, the norms around the blocks, the
linear layers, the bucket AllReduce, clipping and the updates together.  It runs, every
rank holds the same weights, a second run gives the same bits, the gradients are those
of the formulas, and a captured step repeats them."""
from __future__ import annotations

import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, str(ROOT / "examples"))
    import data_parallel_blocks
    return torch, data_parallel_blocks


SMALL = dict(tokens=96, vocab=101, width=120, hidden=248, layers=2)


def test_runs_repeat_and_ranks_agree(example):
    torch, ex = example
    a, na, ga = ex.train(ranks=3, steps=3, **SMALL)
    b, nb, gb = ex.train(ranks=3, steps=3, **SMALL)
    assert a == b and na == nb and all(n > 0 and l == l for n, l in zip(na, a))
    for r in ga:
        for k in r.w:
            assert torch.equal(r.w[k], ga[0].w[k]) and torch.equal(r.w[k], gb[0].w[k])
    # what the optimiser saw had been clipped to 1, or left as it was
    norm = torch.stack([g.double().square().sum() for g in ga[0].g.values()]).sum().sqrt().item()
    assert abs(norm - min(1.0, na[-1])) < 1e-5


def reference(torch, ex, rank, ids, targets, width):
    """The loss and its gradients in 64 bits, from the rank's 16-bit weights."""
    w = {k: v.double().requires_grad_() for k, v in rank.w.items()}

    def norm(v, weight):
        return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight

    x = w["embed"][ids] * width ** 0.5
    n = norm(x, w["pre0"])
    for i in range(rank.layers):
        z = n @ w[f"w1_{i}"].t()
        h = (z * torch.special.ndtr(z)) @ w[f"w2_{i}"].t()
        x = x + w[f"gate{i}"] * norm(h, w[f"post{i}"])
        n = norm(x, w[f"pre{i + 1}"])
    p = torch.log_softmax(n @ w["head"].t(), -1)
    loss = -p[torch.arange(len(ids), device=ids.device), targets].mean()
    names = list(w)
    return loss, dict(zip(names, torch.autograd.grad(loss, [w[k] for k in names])))


@pytest.mark.parametrize("layers", [1, 2])
def test_gradients_are_those_of_the_formulas(example, layers):
    """Every activation and gradient between two operators is rounded to bfloat16: at
    most 2^-8 of a value, 2^-8 / sqrt(3) in the root mean square.  A gradient is behind at
    most seven such roundings a layer and six at the ends, forwards and backwards, which
    add up like independent errors, and the norms and the products' Jacobians of random
    weights raise them by less than two."""
    torch, ex = example
    dev = torch.device("cuda:0")
    shape = dict(SMALL, layers=layers)
    tokens = shape.pop("tokens")
    rng = torch.Generator(device=dev).manual_seed(3)
    weights = ex.make_weights(rand=lambda *s: torch.randn(*s, generator=rng, device=dev), **shape)
    for k in weights:  # weights of the norms that differ, so that their places matter
        if weights[k].dim() == 1:
            weights[k] += 0.2 * torch.randn(weights[k].shape, generator=rng, device=dev)
    rank = ex.Rank(weights, tokens)
    ids = torch.randint(0, shape["vocab"], (tokens,), generator=rng, device=dev)
    targets = torch.randint(0, shape["vocab"], (tokens,), generator=rng, device=dev)
    rank.forward(ids)
    loss = rank.loss(targets)
    rank.backward(ids)
    want, grads = reference(torch, ex, rank, ids, targets, shape["width"])
    roundings = 2 * (7 * layers + 6)
    bound = 2 * roundings ** 0.5 * 2.0 ** -8 / 3 ** 0.5
    assert abs(loss.item() - want.item()) < bound * abs(want.item())
    for k, g in grads.items():
        off = ((rank.g[k].double() - g).norm() / g.norm()).item()
        assert off < bound, (k, off, bound)


def test_a_captured_step(example):
    """Forward, loss, backward, clipping in one graph: the bits of the eager calls on
    other tokens, with the same graph."""
    torch, ex = example
    import allreduce_reducescatter_allgather_gb300 as vc
    dev = torch.device("cuda:0")
    shape = dict(SMALL)
    tokens = shape.pop("tokens")
    rng = torch.Generator(device=dev).manual_seed(4)
    weights = ex.make_weights(rand=lambda *s: torch.randn(*s, generator=rng, device=dev), **shape)
    rank = ex.Rank(weights, tokens)
    ids = torch.zeros(tokens, dtype=torch.int64, device=dev)
    norm = torch.empty((), device=dev)
    clip = vc.ClipPlan(list(rank.g.values()))

    def step():
        rank.forward(ids)
        loss = rank.loss(ids)
        rank.backward(ids)
        clip(0.25, norm)
        return loss

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step()
    for _ in range(2):
        ids.copy_(torch.randint(0, shape["vocab"], (tokens,), generator=rng, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        got = [loss.clone(), norm.clone(), *[g.clone() for g in rank.g.values()]]
        want = [step(), norm, *rank.g.values()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
