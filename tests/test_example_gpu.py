"""examples/data_parallel_muon.py: the layers, the bucket AllReduce, the Muon
step and the broadcast together.  The loss falls, every rank holds the same
weights, and a second run gives the same bits."""
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
    import data_parallel_muon
    return torch, data_parallel_muon


def test_loss_falls_and_ranks_agree(example):
    torch, ex = example
    losses, group = ex.train(ranks=3, steps=30, batch=96, width=120, hidden=250)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) < 0.35 * sum(losses[:5]), losses
    for r in group[1:]:
        for k in r.w:
            assert torch.equal(r.w[k], group[0].w[k])


def test_runs_repeat(example):
    torch, ex = example
    a, ga = ex.train(ranks=2, steps=4, batch=64, width=64, hidden=128)
    b, gb = ex.train(ranks=2, steps=4, batch=64, width=64, hidden=128)
    assert a == b
    assert all(torch.equal(ga[0].w[k], gb[0].w[k]) for k in ga[0].w)
