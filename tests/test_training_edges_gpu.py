"""The training-step operators where arguments are at the ends of their ranges.

The forms are those of test_training_gpu.py, in 64 bits; the bounds follow
from the same arithmetic (bf16 keeps 8 significant bits).
"""
from __future__ import annotations

import pytest

from test_training_gpu import env, rand

pytestmark = pytest.mark.gpu

assert env  # (the fixture; imported by name)


@pytest.mark.parametrize("m", [8, 100])
@pytest.mark.parametrize("name", ["none", "gelu", "silu"])
def test_infinite_gradients_stay_infinite(env, m, name):
    """An infinity in dy: its row of dx and its row of dW are infinite, with
    the signs of the other factors, and nothing else is touched."""
    torch, vc, dev = env
    n, k = 24, 40
    dy, z = rand(torch, dev, m, n, seed=1), rand(torch, dev, m, n, seed=2).abs() + 1
    x, w = rand(torch, dev, m, k, seed=3), rand(torch, dev, n, k, seed=4)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    dw, dw2 = torch.empty(n, k, device=dev), torch.empty(n, k, device=dev)
    vc.vc_linear_backward(dy, x, w, dx=dx, dweight=dw, preact=z, activation=name)
    dy[5, 3] = float("inf")
    vc.vc_linear_backward(dy, x, w, dx=dx2, dweight=dw2, preact=z, activation=name)
    inf = float("inf")
    assert torch.equal(dx2[5].float(), w[3].float().sign() * inf)
    assert torch.equal(dw2[3], x[5].float().sign() * inf)
    rows, features = torch.arange(m, device=dev) != 5, torch.arange(n, device=dev) != 3
    assert torch.equal(dx2[rows], dx[rows]) and torch.equal(dw2[features], dw[features])
