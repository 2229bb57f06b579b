"""The kernel of the large products (persistent pairs of blocks), whole outputs
against 64-bit forms: more tiles than pairs, ragged edges, two products in a
launch with uneven numbers of tiles, 32-bit sums in several segments,
symmetric products with mirrored tiles.  Which kernel ran is read from the
nodes of a captured graph.

The bounds are those of test_training_gpu.py.  A differences test that sees a
missing or a scaled gradient closes the file.
"""
from __future__ import annotations

import re
import warnings

import pytest

from test_training_gpu import (ACTS, BF16, ORTHO, accumulate_bound, act, check, env, forward_exact,
                               ortho_exact, rand, relative)

pytestmark = pytest.mark.gpu

assert env  # (the fixture; imported by name)


def kernels(torch, dev, call, tmp_path):
    """The names of the kernels that `call` launches, and how often."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    stream = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        call()
    path = tmp_path / "graph.dot"
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # (it says that it dumps)
        graph.debug_dump(str(path))
    names = re.findall(r"(pair_kernel|split_kernel|ns_small_kernel|dz_kernel|jobs_kernel|"
                       r"momentum_kernel|scale_kernel)", path.read_text(errors="replace"))
    return {n: names.count(n) for n in set(names)}


FORWARD = [(2100, 2600, 1000), (2304, 2560, 1024), (2050, 2309, 1501), (4099, 1288, 1280)]


@pytest.mark.parametrize("m,n,k", FORWARD)
@pytest.mark.parametrize("form", ["plain", "training", "residual", "in place"])
def test_forward(env, tmp_path, m, n, k, form):
    torch, vc, dev = env
    name = {"plain": "none", "training": "gelu", "residual": "silu", "in place": "relu2"}[form]
    x, w = rand(torch, dev, m, k, seed=1), rand(torch, dev, n, k, seed=2, std=k ** -0.5)
    b = rand(torch, dev, n, seed=3) if form != "plain" else None
    r = rand(torch, dev, m, n, seed=4) if form in ("residual", "in place") else None
    r0 = None if r is None else r.clone()
    y = r if form == "in place" else torch.full((m, n), 7.0, dtype=torch.bfloat16, device=dev)
    z = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=dev) if form == "training" else None
    call = vc.prepare_linear_forward(x, w, y, bias=b, residual=r, preact=z, activation=name)
    call()
    ez, dz, ey, dy = forward_exact(torch, x, w, b, r0, name)
    check(y, ey, dy + BF16 * (ey.abs() + dy), f"y {name}")
    if z is not None:
        check(z, ez, dz + BF16 * (ez.abs() + dz), "preact")
    ran = kernels(torch, dev, call, tmp_path)
    assert ran.get("pair_kernel") == 1 and "split_kernel" not in ran, ran


BACKWARD = [(4096, 2048, 1024), (4100, 1100, 1030), (2600, 1300, 1300), (3100, 2050, 1100)]


@pytest.mark.parametrize("m,n,k", BACKWARD)
@pytest.mark.parametrize("form", ["sums", "sums with dx", "sums with activation", "half", "half added"])
def test_backward(env, tmp_path, m, n, k, form):
    """dx and dW in one launch, or dW alone; 32-bit sums over several segments
    of 1024 rows, overwritten or added to."""
    torch, vc, dev = env
    name = "gelu" if form in ("sums with activation", "half") else "none"
    grad = torch.bfloat16 if form.startswith("half") else torch.float32
    add = form in ("sums with dx", "half added", "sums")
    dy, x = rand(torch, dev, m, n, seed=1), rand(torch, dev, m, k, seed=2)
    w, z = rand(torch, dev, n, k, seed=3, std=n ** -0.5), rand(torch, dev, m, n, seed=4)
    dx = None if form == "sums" else torch.full((m, k), 9.0, dtype=torch.bfloat16, device=dev)
    dw0 = rand(torch, dev, n, k, seed=5, dtype=grad)
    dw = dw0.clone()
    call = vc.prepare_linear_backward(dy, x, w, dx=dx, dweight=dw, preact=z, activation=name,
                                      accumulate=add)
    call()
    dz = dy.double()
    dzr = torch.zeros_like(dz)
    if name != "none":
        dz = dz * act(torch, z.double(), name)[1]
        dzr = dy.double().abs() * 2.0 ** -19 + dz.abs() * BF16
    X, W = x.double(), w.double()
    if dx is not None:
        want = dz @ W
        bound = dzr @ W.abs() + accumulate_bound(n, dz.abs() @ W.abs())
        check(dx, want, bound + BF16 * (want.abs() + bound), "dx")
    want = dz.t() @ X + (dw0.double() if add else 0)
    mag = dz.abs().t() @ X.abs() + dw0.double().abs()
    if grad == torch.float32:
        bound = (dzr.t() @ X.abs() + accumulate_bound(min(m, 1024), mag)
                 + (m / 1024 + 1) * 2.0 ** -24 * mag)
        check(dw, want, bound + 2.0 ** -24 * want.abs(), "dweight")
    else:
        bound = dzr.t() @ X.abs() + accumulate_bound(m, mag)
        check(dw, want, bound + BF16 * (want.abs() + bound), "dweight")
    if dx is not None or grad == torch.float32:
        ran = kernels(torch, dev, call, tmp_path)
        assert ran.get("pair_kernel") == 1 and "split_kernel" not in ran, ran


def test_one_launch_for_two_gradients_repeats(env):
    """The tiles of both products are shared out by a fixed rule: the same
    bits every time."""
    torch, vc, dev = env
    m, n, k = 4100, 1100, 1030
    dy, x = rand(torch, dev, m, n, seed=1), rand(torch, dev, m, k, seed=2)
    w = rand(torch, dev, n, k, seed=3)
    first = None
    for _ in range(4):
        dx, dw = torch.empty_like(x), torch.empty(n, k, device=dev)
        vc.vc_linear_backward(dy, x, w, dx=dx, dweight=dw)
        first = first or (dx, dw)
        assert torch.equal(first[0], dx) and torch.equal(first[1], dw)


SHAPES = [(2, 2048, 2100), (2, 2100, 2048), (3, 2000, 2300), (4, 1600, 1500)]


@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_orthogonalize(env, tmp_path, batch, rows, cols):
    torch, vc, dev = env
    g = rand(torch, dev, batch, rows, cols, seed=rows, std=1e-3)
    g[1] *= 1e-10  # eps outweighs its norm
    out = torch.full_like(g, 3.0)
    call = vc.prepare_orthogonalize(g, out)
    call()
    for i in range(batch):
        assert relative(out[i], ortho_exact(torch, g[i])) < ORTHO, i
    ran = kernels(torch, dev, call, tmp_path)
    assert ran.get("pair_kernel") == 15 and "split_kernel" not in ran, ran


@pytest.mark.parametrize("batch,rows,cols", SHAPES[:2])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_muon_step(env, batch, rows, cols, dtype):
    """Weights in slices of a wider tensor, whose other columns stay."""
    torch, vc, dev = env
    dtype = getattr(torch, dtype)
    for odd in (0, 3):
        wide = rand(torch, dev, batch, rows, cols + 8 + odd, seed=1, dtype=dtype)
        before, w = wide.clone(), wide[:, :, 8:8 + cols]
        g = rand(torch, dev, batch, rows, cols, seed=2, dtype=dtype)
        m = rand(torch, dev, batch, rows, cols, seed=3, dtype=torch.float32)
        m0 = m.double()
        vc.vc_muon_step(w, g, m, 0.02, beta=0.9, nesterov=True, weight_decay=0.1, scale=3.0)
        em = 0.9 * m0 + g.double()
        check(m, em, 2.0 ** -22 * (em.abs() + m0.abs() + g.double().abs()), "momentum")
        w0 = before[:, :, 8:8 + cols].double()
        half = BF16 if dtype == torch.bfloat16 else 2.0 ** -23
        for i in range(batch):
            o = ortho_exact(torch, g[i].double() + 0.9 * em[i])
            want = (1 - 0.02 * 0.1) * w0[i] - 0.06 * o
            off = (w[i].double() - want).norm().item()
            assert off <= ORTHO * 0.06 * o.norm().item() + half * want.norm().item()
        wide[:, :, 8:8 + cols] = before[:, :, 8:8 + cols]
        assert torch.equal(wide, before)


# ---------------------------------------------------------- against differences --

def norm_bound(torch, a):
    """At least the largest singular value: the 32nd root of the Frobenius norm
    of (a^T a)^16, the singular values' 32nd powers; at most n^(1/64) above it."""
    p = a.t() @ a if a.shape[0] >= a.shape[1] else a @ a.t()
    log = torch.zeros((), dtype=torch.float64, device=a.device)
    for power in (2, 4, 8, 16, 32):  # p is a's product to this power, over exp(log)
        size = p.norm()
        log, p = log + size.log(), p / size
        if power < 32:
            log, p = 2 * log, p @ p
    return (log / 32).exp().item()


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m", [40, 200, 3000])
def test_gradient_along_itself_against_differences(env, name, m):
    """Along the computed gradient's own direction the loss rises by its norm a
    unit.  The loss is that of the stored z, as the gradient is; what may
    differ is the rounding of dz, of bf16's 2^-8 a value (2^-16 for few rows),
    and of the result, together at most their norms.  A gradient that is zero,
    scaled or in the wrong place does not pass."""
    torch, vc, dev = env
    n, k = (1300, 1300) if m == 3000 else (96, 80)
    x, w, dy = (rand(torch, dev, *s, seed=i) for i, s in enumerate(((m, k), (n, k), (m, n))))
    w = (w.float() * k ** -0.5).to(torch.bfloat16)
    y, z = torch.empty_like(dy), torch.empty_like(dy)
    vc.vc_linear_forward(x, w, y, preact=z, activation=name)
    dx, dw = torch.empty_like(x), torch.empty(n, k, device=dev)
    db = torch.empty(n, device=dev)
    vc.vc_linear_backward(dy, x, w, dx=dx, dweight=dw, dbias=db, preact=z, activation=name)
    X, W, Z, G = x.double(), w.double(), z.double(), dy.double()
    dz = (G * act(torch, Z, name)[1]).norm().item()
    other = {"x": norm_bound(torch, W), "w": norm_bound(torch, X), "b": m ** 0.5}

    def compare(which, grad):
        """The gradient's norm, the loss's slope along it, and what they may differ by."""
        length = grad.double().norm().item()
        d = grad.double() / length
        step = d @ W.t() if which == "x" else X @ d.t() if which == "w" else d[None, :].expand_as(Z)
        h = 1e-3 / step.abs().max().item()  # no z moves by more than 1e-3
        up, down = (act(torch, Z + s * step, name)[0] for s in (h, -h))
        slope = ((up - down) * G).sum().item() / (2 * h)
        rounding = 0.0 if name == "none" or which == "b" else (2.0 ** -16 if m <= 64 else BF16)
        # dz, with its slopes' own error of 2^-19; the result (dx is bf16, the
        # rest 32-bit sums of up to 1024 products at a time)
        tol = ((rounding + 2.0 ** -19) * dz * other[which]
               + (BF16 if which == "x" else 0.0) * length + 2.0 ** -16 * dz * other[which])
        # differences: third derivatives of at most 4, and kinks within a step
        move = (G * step).abs()
        tol += 4e-6 / 6 * move.sum().item()
        if name.startswith("relu"):
            tol += move[Z.abs() <= h * step.abs()].sum().item()
        return length, slope, tol

    for which, grad in (("x", dx), ("w", dw), ("b", db)):
        length, slope, tol = compare(which, grad)
        assert abs(slope - length) <= tol, (which, length, slope, tol)
        assert tol < 0.08 * length, (which, length, tol)
        for wrong in (0.5 * grad, 0.9 * grad, 1.1 * grad, -grad, grad.roll(1, -1)):
            length, slope, tol = compare(which, wrong)
            assert abs(slope - length) > tol, which
