"""The training-step operators where arguments are at the ends of their ranges.

The forms are those of test_training_gpu.py, in 64 bits; the bounds follow
from the same arithmetic (bf16 keeps 8 significant bits).
"""
from __future__ import annotations

import subprocess
import sys

import pytest

from conftest import ROOT
from test_training_gpu import ACTS, BF16, COEF, ORTHO, act, env, ortho_exact, rand, relative

pytestmark = pytest.mark.gpu

assert env  # (the fixture; imported by name)

# beyond what an activation bends: from here on it is z or 0 (or z^2)
FAR = [2.0 ** 6, 1e4, 1e10, 1e13, 1e14, 1e18, 2e19, 1e25, 3e38]


def far_values(torch, dev):
    v = torch.tensor(FAR + [float("inf")], device=dev)
    return torch.cat([v, -v]).to(torch.bfloat16)


def limits(torch, z, name):
    """Value and derivative: the formulas' up to 64, their limits beyond,
    infinities included."""
    up = z > 0
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    if name == "none":
        return z, one
    if name == "relu2":
        return torch.where(up, z * z, zero), torch.where(up, 2 * z, zero)
    value, slope = act(torch, z.clamp(-64, 64), name)
    near = z.abs() <= 64
    return (torch.where(near, value, torch.where(up, z, zero)),
            torch.where(near, slope, torch.where(up, one, zero)))


def same(torch, got, want, what):
    """Equal after bf16's rounding, signs of zeros aside, infinities too."""
    off = (got.double() - want.to(torch.bfloat16).double()).abs()
    both_infinite = got.isinf() & want.to(torch.bfloat16).isinf() & (got.double().sign() == want.sign())
    ok = (off <= BF16 * want.abs()) | both_infinite
    assert ok.all(), (what, got[~ok].tolist(), want[~ok].tolist())


@pytest.mark.parametrize("repeat", [1, 20])  # up to 64 rows, and more
@pytest.mark.parametrize("name", ACTS)
def test_activations_far_out(env, name, repeat):
    torch, vc, dev = env
    z = far_values(torch, dev).repeat(repeat)
    x = torch.zeros(z.numel(), 16, dtype=torch.bfloat16, device=dev)
    x[:, 0] = z
    w = torch.zeros(40, 16, dtype=torch.bfloat16, device=dev)
    w[:, 0] = 1
    y = torch.empty(z.numel(), 40, dtype=torch.bfloat16, device=dev)
    vc.vc_linear_forward(x, w, y, activation=name)
    value, slope = limits(torch, z.double(), name)
    for column in (0, 31, 39):
        same(torch, y[:, column], value, name)
    x[:, 0] = float("nan")
    vc.vc_linear_forward(x, w, y, activation=name)
    assert y.isnan().all()
    # one output feature, so that dx's first column is dz itself
    one = torch.zeros(1, 16, dtype=torch.bfloat16, device=dev)
    one[0, 0] = 1
    dx = torch.empty_like(x)
    dy = torch.ones(z.numel(), 1, dtype=torch.bfloat16, device=dev)
    db = torch.empty(1, device=dev)
    vc.vc_linear_backward(dy, x, one, dx=dx, dbias=db, preact=z[:, None].contiguous(), activation=name)
    same(torch, dx[:, 0], slope, name + "'")


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


# ---------------------------------------------------------- orthogonalisation --

@pytest.mark.parametrize("shape", [(64, 100), (100, 64), (300, 257), (3, 130, 200), (2, 40, 600)])
def test_zero_matrices_without_eps(env, shape):
    """A zero matrix gives zeros, and leaves the weight, whatever eps is."""
    torch, vc, dev = env
    g = torch.zeros(*shape, device=dev)
    out = torch.full(shape, 5.0, dtype=torch.bfloat16, device=dev)
    vc.vc_orthogonalize(g, out, eps=0.0)
    assert (out == 0).all()
    w = rand(torch, dev, *shape, dtype=torch.float32)
    w0, m = w.clone(), torch.zeros_like(w)
    vc.vc_muon_step(w, g, m, 0.1, eps=0.0)
    assert torch.equal(w, w0) and (m == 0).all()


SMALL = [1.0, 1e-2, 1e-4, 1e-6, 1e-9, 1e-12]  # |G| / eps


@pytest.mark.parametrize("rows,cols", [(64, 100), (100, 64), (300, 257), (257, 300), (96, 1500)])
@pytest.mark.parametrize("eps", [1e-7, 1.0])
def test_norms_below_eps(env, rows, cols, eps):
    """Where eps is the larger part of the divisor, the result is as exact as
    anywhere else.  (norms from 1e-19: their squares are float32s)"""
    torch, vc, dev = env
    g0 = rand(torch, dev, rows, cols, seed=3, dtype=torch.float32)
    g0 /= g0.norm()
    for steps, coef in ((5, COEF), (1, COEF), (12, (1.5, -0.5, 0.0)), (30, (1.9, -1.2, 0.3)),
                        (2, (-3.0, 4.0, -1.5))):
        tol = max(ORTHO, ORTHO * (steps / 5) ** 0.5)
        for ratio in SMALL:
            g = g0 * (eps * ratio)
            out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
            vc.vc_orthogonalize(g, out, steps=steps, coefficients=coef, eps=eps)
            want = ortho_exact(torch, g, steps, coef, eps)
            assert relative(out, want) < tol, (steps, coef, ratio)


@pytest.mark.parametrize("rows,cols", [(64, 100), (300, 257)])
def test_scales_at_the_ends_of_float32(env, rows, cols):
    torch, vc, dev = env
    g = rand(torch, dev, rows, cols, seed=3, dtype=torch.float32)
    g /= g.norm()
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    for eps, scale in ((1e30, 1.0), (1e12, 1e-15), (1e12, 1e12), (0.0, 1e-18), (0.0, 1e18)):
        vc.vc_orthogonalize(g * scale, out, eps=eps)
        assert relative(out, ortho_exact(torch, g * scale, eps=eps)) < ORTHO, (eps, scale)
    # what falls out of float32 on the way becomes 0, not NaN
    for eps, coef, steps in ((3e38, COEF, 100), (1e-7, (0.01, 0.0, 0.0), 100), (1e30, (0.1, 0.0, 0.0), 9)):
        vc.vc_orthogonalize(g * 1e-10, out, eps=eps, coefficients=coef, steps=steps)
        want = ortho_exact(torch, g * 1e-10, steps, coef, eps)
        assert ((out.double() - want).abs() <= BF16 * want.abs().max() + 1e-37).all(), (eps, coef)
    # and what is not finite gives NaN everywhere
    for bad in (float("nan"), float("inf"), -float("inf")):
        for eps in (0.0, 1e-7, 1e9):
            h = g.clone()
            h[rows // 2, cols // 3] = bad
            vc.vc_orthogonalize(h, out, eps=eps)
            assert out.isnan().all(), (bad, eps)


def test_norms_below_eps_beside_others(env):
    """Matrices of a batch have their own scales; a Muon step too."""
    torch, vc, dev = env
    for rows, cols in ((60, 200), (260, 140)):
        g = rand(torch, dev, 4, rows, cols, seed=5, dtype=torch.float32)
        g /= g.norm(dim=(1, 2), keepdim=True)
        g *= torch.tensor([1.0, 1e-10, 1e-4, 1e-16], device=dev)[:, None, None]
        out = torch.empty(4, rows, cols, dtype=torch.bfloat16, device=dev)
        vc.vc_orthogonalize(g, out)
        want = ortho_exact(torch, g)
        for i in range(4):
            assert relative(out[i], want[i]) < ORTHO, i
        w = torch.zeros_like(g)
        vc.vc_muon_step(w, g, torch.zeros_like(g), 1.0, nesterov=False, scale=1.0)
        for i in range(4):
            assert relative(w[i], -want[i]) < ORTHO, i


# --------------------------------------------------------------------- slices --

def test_slices_of_one_tensor_that_interleave(env):
    """Inputs and outputs may be column slices of one wider tensor."""
    torch, vc, dev = env
    m, n, k = 70, 40, 48
    for at in (0, 3, 8):
        wide = rand(torch, dev, m, at + k + 2 * n + 9, seed=1)
        before = wide.clone()
        x, y, z = wide[:, at:at + k], wide[:, at + k:at + k + n], wide[:, at + k + n:at + k + 2 * n]
        w = rand(torch, dev, n, k, seed=2)
        y2, z2 = (torch.empty(m, n, dtype=torch.bfloat16, device=dev) for _ in range(2))
        vc.vc_linear_forward(x.contiguous(), w, y2, preact=z2, activation="silu")
        vc.vc_linear_forward(x, w, y, preact=z, activation="silu")
        assert torch.equal(y, y2) and torch.equal(z, z2)
        before[:, at + k:at + k + n] = y2
        before[:, at + k + n:at + k + 2 * n] = z2
        assert torch.equal(wide, before)
        both = rand(torch, dev, m, 2 * k + at, seed=4)
        x, dx = both[:, :k], both[:, k + at:]
        dx2, dy = torch.empty(m, k, dtype=torch.bfloat16, device=dev), rand(torch, dev, m, n, seed=5)
        vc.vc_linear_backward(dy, x.contiguous(), w, dx=dx2, preact=z2, activation="silu")
        vc.vc_linear_backward(dy, x, w, dx=dx, preact=z, activation="silu")
        assert torch.equal(dx, dx2)
    for rows, cols in ((30, 50), (200, 150)):
        wide = rand(torch, dev, 2, rows, 3 * cols, seed=6, dtype=torch.float32)
        parts = [wide[:, :, i * cols:(i + 1) * cols] for i in range(3)]
        alone = [p.contiguous() for p in parts]
        vc.vc_muon_step(*parts, 0.1)
        vc.vc_muon_step(*alone, 0.1)
        assert all(torch.equal(a, b) for a, b in zip(parts, alone))


def test_alignment_of_given_workspaces(env):
    """16 bytes for the linear layer, 256 for the rest, as the header says."""
    torch, vc, dev = env
    m, n, k = 70, 41, 51
    x, w, dy = (rand(torch, dev, *s, seed=i) for i, s in enumerate(((m, k), (n, k), (m, n))))
    y, y2, dx, dx2 = (torch.empty(m, c, dtype=torch.bfloat16, device=dev) for c in (n, n, k, k))
    g = rand(torch, dev, 140, 150, seed=4)
    out = torch.empty_like(g)
    need = max(vc.linear_forward_workspace(x, w), vc.linear_backward_workspace(dy, x, w, "relu"),
               vc.orthogonalize_workspace(g.shape))
    big = torch.empty(need + 512, dtype=torch.uint8, device=dev)
    vc.vc_linear_forward(x, w, y)
    vc.vc_linear_backward(dy, x, w, dx=dx, preact=y, activation="relu")
    for at in (16, 48, 256):
        y2.zero_(), dx2.zero_()
        vc.vc_linear_forward(x, w, y2, workspace=big[at:])
        vc.vc_linear_backward(dy, x, w, dx=dx2, preact=y, activation="relu", workspace=big[at:])
        assert torch.equal(y, y2) and torch.equal(dx, dx2)
    vc.vc_orthogonalize(g, out, workspace=big[256:])
    with pytest.raises(ValueError, match="aligned to 16 bytes"):
        vc.vc_linear_forward(x, w, y, workspace=big[8:])
    with pytest.raises(ValueError, match="aligned to 256 bytes"):
        vc.vc_orthogonalize(g, out, workspace=big[128:])


# -------------------------------------------------------------------- streams --

@pytest.mark.parametrize("how", ["argument", "current"])
def test_handle_dropped_while_another_stream_uses_its_workspace(env, how):
    """A handle prepared on one stream and called on another: its workspace is
    given to nobody else before that call has ended."""
    torch, vc, dev = env
    x, w = rand(torch, dev, 500, 301, seed=1), rand(torch, dev, 260, 301, seed=2)
    want, y = (torch.empty(500, 260, dtype=torch.bfloat16, device=dev) for _ in range(2))
    vc.vc_linear_forward(x, w, want)
    need = vc.linear_forward_workspace(x, w)
    assert need > 0
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    call = vc.prepare_linear_forward(x, w, y)
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        if how == "current":
            call()
    if how == "argument":
        call(stream=side)
    del call
    # whoever allocates next on the first stream writes at once
    for _ in range(4):
        torch.empty(need, dtype=torch.uint8, device=dev).fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_handle_waits_for_the_stream_that_prepared_it(env):
    """The workspace may hold a block that earlier work of the preparing
    stream still uses: a call on another stream starts behind it."""
    torch, vc, dev = env
    x, w = rand(torch, dev, 500, 301, seed=1), rand(torch, dev, 260, 301, seed=2)
    want, y = (torch.empty(500, 260, dtype=torch.bfloat16, device=dev) for _ in range(2))
    vc.vc_linear_forward(x, w, want)
    need = vc.linear_forward_workspace(x, w)
    side = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    block = torch.empty(need, dtype=torch.uint8, device=dev).fill_(255)
    del block  # free for this stream's next allocation, though its fill is still to come
    call = vc.prepare_linear_forward(x, w, y)
    call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_timeouts_wait_for_every_stream(env):
    torch, vc, dev = env
    side = torch.cuda.Stream(dev)
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    assert vc.train_timeouts() == 0
    assert side.query()  # its work has ended


# (in a process of its own: the count stays for as long as the library is loaded)
WAIT_OUT = """
import os, sys
sys.path.insert(0, sys.argv[1])
import torch
import allreduce_reducescatter_allgather_gb300 as vc
x = torch.randn(100, 64, device="cuda").bfloat16()
y, z = (torch.empty(100, 100, dtype=torch.bfloat16, device="cuda") for _ in range(2))
vc.vc_linear_forward(x, x, y)
assert vc.train_timeouts() == 0
os.environ["VC_TEST_WAIT_OUT"] = "1"
assert vc.train_timeouts() == 1
assert vc.train_timeouts() == 2
del os.environ["VC_TEST_WAIT_OUT"]
assert vc.train_timeouts() == 2
vc.vc_linear_forward(x, x, z)  # the context is as usable as before
assert torch.equal(y, z) and torch.isfinite(z.float()).all()
print("done")
"""


def test_a_wait_that_runs_out_is_counted(env):
    out = subprocess.run([sys.executable, "-c", WAIT_OUT, str(ROOT)], capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "done", out.stderr
