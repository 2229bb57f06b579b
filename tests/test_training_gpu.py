"""The training-step operators on the GPU against plain 64-bit forms.

Tolerances follow from the arithmetic that include/vc_train.h states:

  - bf16 keeps 8 significant bits: rounding is off by at most 2^-8 of a value.
  - A product of K terms in 32-bit accumulators that cut off: at most 2^-23 of
    the sum of magnitudes per group of 16 terms (and 16 more for the adds
    within a group and the epilogue): (K/16 + 16) 2^-23 sum |a b|.
  - 32-bit gradients add segments of 1024 terms rounded to nearest, so that K
    above is at most 1024 plus one rounding of 2^-24 a segment.
  - dz carries one more bf16 rounding into its products, or one of 2^-16 where
    its remainder is kept (batches of up to 64 rows).
  - Orthogonalisation: fp16 operands (11 significant bits) are off by 2^-11 at
    most and by 2^-11 / sqrt(3) in the root mean square; three roundings a pass
    count (X, A, B), whose effects the passes neither raise nor damp on
    matrices with a flat spectrum: 2^-11 / sqrt(3) sqrt(15) = 1.1e-3 of the
    norm, twice that as a bound, and bf16's own 2^-8 / sqrt(3) = 2.3e-3 at worst
    mantissas: 4.4e-3 together.
"""
from __future__ import annotations

import math

import pytest

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # unit roundoffs
FP16 = 2.0 ** -11
ORTHO = 2 * FP16 / 3 ** 0.5 * 15 ** 0.5 + BF16 / 3 ** 0.5

ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import allreduce_reducescatter_allgather_gb300 as vc
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    yield torch, vc, dev
    assert vc.train_timeouts() == 0


def rand(torch, dev, *shape, seed=0, std=1.0, dtype=None):
    g = torch.Generator(device=dev).manual_seed(1000 + seed)
    return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype or torch.bfloat16)


def act(torch, z, name):
    """Value and derivative in 64 bits."""
    one = torch.ones_like(z)
    if name == "none":
        return z, one
    if name == "relu":
        return z.clamp_min(0), (z > 0).double()
    if name == "relu2":
        return z.clamp_min(0) ** 2, 2 * z.clamp_min(0)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c
                                   * (1 + 3 * 0.044715 * z * z))
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s))


def accumulate_bound(K, magnitudes):
    return (K / 16 + 16) * 2.0 ** -23 * magnitudes


def check(got, want, bound, what):
    off = (got.double() - want).abs() - bound
    worst = off.max().item() if off.numel() else 0.0
    assert not worst > 0 and not math.isnan(worst), f"{what}: {worst:.3e} over its bound"


def forward_exact(torch, x, w, b, r, name):
    z = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    if b is not None:
        z = z + b.double()
        mag = mag + b.double().abs()
    y, slope = act(torch, z, name)
    # the largest slope within the error of z: these functions' second
    # derivatives are at most 2
    dz = accumulate_bound(x.shape[-1], mag) + 2.0 ** -24 * z.abs()
    dy = dz * (slope.abs() + 2 * dz) + 2.0 ** -20 * (y.abs() + z.abs() * 2.0 ** -3)
    if r is not None:
        y = y + r.double()
        dy = dy + 2.0 ** -23 * y.abs()
    return z, dz, y, dy


# one token to many, one feature, tile edges, odd rows, K of zero and one
SIZES = [(1, 1, 1), (1, 8, 16), (1, 4096, 1024), (3, 70, 65), (17, 129, 40), (32, 64, 2048),
         (64, 200, 72), (65, 64, 64), (127, 33, 257), (128, 64, 64), (129, 257, 129),
         (300, 1000, 24), (256, 256, 4096), (257, 513, 1000), (1003, 2049, 1021),
         (1024, 4096, 192), (2500, 1030, 96), (5, 7, 0), (200, 9, 0)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("i", range(3))
def test_forward(env, m, n, k, i):
    torch, vc, dev = env
    name = ACTS[(m + 2 * n + k + i) % 6] if i else "none"
    x = rand(torch, dev, m, k, seed=1)
    w = rand(torch, dev, n, k, seed=2, std=max(k, 1) ** -0.5)
    b = rand(torch, dev, n, seed=3) if i != 1 else None
    r = rand(torch, dev, m, n, seed=4) if i == 2 else None
    y = torch.full((m, n), 7.0, dtype=torch.bfloat16, device=dev)
    z = torch.full_like(y, 7.0) if i else None
    vc.vc_linear_forward(x, w, y, bias=b, residual=r, preact=z, activation=name)
    ez, dz, ey, dy = forward_exact(torch, x, w, b, r, name)
    check(y, ey, dy + BF16 * (ey.abs() + dy), f"y {name}")
    if z is not None:
        check(z, ez, dz + BF16 * (ez.abs() + dz), "preact")


def test_activations_over_their_range(env):
    """x W^T reproduces chosen pre-activations: every act over [-40, 40]."""
    torch, vc, dev = env
    z = torch.linspace(-40, 40, 4096, device=dev).to(torch.bfloat16)
    x = torch.zeros(4096, 16, dtype=torch.bfloat16, device=dev)
    x[:, 0] = z
    w = torch.zeros(64, 16, dtype=torch.bfloat16, device=dev)
    w[:, 0] = 1
    for name in ACTS:
        y = torch.empty(4096, 64, dtype=torch.bfloat16, device=dev)
        vc.vc_linear_forward(x, w, y, activation=name)
        want = act(torch, z.double(), name)[0][:, None].expand(4096, 64)
        # gelu's tail is good to 7.5e-8 |z|, absolutely
        check(y, want, BF16 * (1 + 2.0 ** -8) * want.abs() + 1e-7 * (1 + z.double().abs()[:, None]), name)
        dy = torch.ones_like(y)
        zz = z[:, None].expand(4096, 64).contiguous()
        dx = torch.empty(4096, 16, dtype=torch.bfloat16, device=dev)
        one = torch.zeros(64, 16, dtype=torch.bfloat16, device=dev)
        one[0, 0] = 1
        vc.vc_linear_backward(dy, x, one, dx=dx, preact=zz, activation=name)
        slope = act(torch, z.double(), name)[1]
        # (rounded as dz, and as dx)
        check(dx[:, 0], slope, 2.01 * BF16 * slope.abs() + 2e-6, name + "'")


def test_forward_of_rows_in_wider_tensors(env):
    """Strided rows, bases off 16 bytes, three dimensions, outputs between
    guard values."""
    torch, vc, dev = env
    m, n, k = 96, 80, 64
    wide = rand(torch, dev, m, 3 * k + 5, seed=1)
    w = rand(torch, dev, n, k, seed=2, std=0.1)
    for off in (0, 3, 8, k + 8):
        x = wide[:, off:off + k]
        big = torch.full((m, n + 40), 5.0, dtype=torch.bfloat16, device=dev)
        for at in (0, 1, 8):
            y = big[:, 16 + at:16 + at + n]
            vc.vc_linear_forward(x, w, y, activation="silu")
            _, _, ey, dy = forward_exact(torch, x, w, None, None, "silu")
            check(y, ey, dy + BF16 * (ey.abs() + dy), f"offset {off}, {at}")
            assert (big[:, :16 + at] == 5).all() and (big[:, 16 + at + n:] == 5).all()
            big.fill_(5.0)
    x3 = rand(torch, dev, 4, 24, k, seed=5)
    y3 = torch.empty(4, 24, n, dtype=torch.bfloat16, device=dev)
    vc.vc_linear_forward(x3, w, y3)
    flat = torch.empty(96, n, dtype=torch.bfloat16, device=dev)
    vc.vc_linear_forward(x3.view(96, k), w, flat)
    assert torch.equal(y3.view(96, n), flat)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_residual_in_place(env, m):
    torch, vc, dev = env
    x, w, r = (rand(torch, dev, *s, seed=i) for i, s in enumerate(((m, 64), (100, 64), (m, 100))))
    y = torch.empty_like(r)
    vc.vc_linear_forward(x, w, y, residual=r, activation="relu")
    vc.vc_linear_forward(x, w, r, residual=r, activation="relu")
    assert torch.equal(y, r)


@pytest.mark.parametrize("m", [3, 200])
def test_values_that_are_not_finite_stay_in_their_rows(env, m):
    torch, vc, dev = env
    x = rand(torch, dev, m, 72, seed=1)
    w = rand(torch, dev, 130, 72, seed=2)
    y, y2 = (torch.empty(m, 130, dtype=torch.bfloat16, device=dev) for _ in range(2))
    vc.vc_linear_forward(x, w, y, activation="gelu")
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[2, 7] = float("inf")
    vc.vc_linear_forward(x2, w, y2, activation="gelu")
    assert torch.isnan(y2[1]).all()
    assert not torch.isfinite(y2[2][w[:, 7] > 0]).any()
    keep = torch.ones(m, dtype=torch.bool, device=dev)
    keep[1:3] = False
    assert torch.equal(y[keep], y2[keep])


GRADS = [(1, 1, 1), (1, 64, 128), (2, 128, 401), (13, 64, 496), (64, 100, 33), (65, 100, 33),
         (129, 257, 65), (300, 520, 1000), (1003, 1000, 513), (4096, 256, 320), (2300, 1024, 260)]


@pytest.mark.parametrize("m,n,k", GRADS)
@pytest.mark.parametrize("i", range(4))
def test_backward(env, m, n, k, i):
    torch, vc, dev = env
    name = "none" if i < 2 else ACTS[1 + (m + n + k + i) % 5]
    grad = torch.float32 if i in (0, 3) else torch.bfloat16
    add = i in (0, 2)
    dy, x = rand(torch, dev, m, n, seed=1), rand(torch, dev, m, k, seed=2)
    w = rand(torch, dev, n, k, seed=3, std=n ** -0.5)
    z = rand(torch, dev, m, n, seed=4)
    dx = torch.empty_like(x)
    dw0, db0 = rand(torch, dev, n, k, seed=5, dtype=grad), rand(torch, dev, n, seed=6, dtype=grad)
    dw, db = dw0.clone(), db0.clone()
    vc.vc_linear_backward(dy, x, w, dx=dx, dweight=dw, dbias=db, preact=z, activation=name,
                          accumulate=add)
    dz = dy.double()
    dzr = 0.0 * dz
    if name != "none":
        slope = act(torch, z.double(), name)[1]
        dz = dz * slope
        # the slope's own error (functions good to 2^-20 of 1), and the rounding
        dzr = dy.double().abs() * 2.0 ** -19 + dz.abs() * 2.0 ** (-16 if m <= 64 else -8)
    X, W = x.double(), w.double()
    want = dz @ W
    bound = dzr @ W.abs() + accumulate_bound(2 * n, dz.abs() @ W.abs())
    check(dx, want, bound + BF16 * (want.abs() + bound), "dx")
    want = dz.t() @ X + (dw0.double() if add else 0)
    mag = dz.abs().t() @ X.abs() + dw0.double().abs()
    if grad == torch.float32:
        bound = dzr.t() @ X.abs() + accumulate_bound(min(m, 1024), mag) + (m / 1024 + 1) * 2.0 ** -24 * mag
        check(dw, want, bound + 2.0 ** -24 * want.abs(), "dweight")
    else:
        bound = dzr.t() @ X.abs() + accumulate_bound(2 * m, mag)
        check(dw, want, bound + BF16 * (want.abs() + bound), "dweight")
    want = dz.sum(0) + (db0.double() if add else 0)
    # column sums add at most m values one after the other, of 32-bit dz
    mag = dz.abs().sum(0) + db0.double().abs()
    bound = (m + 8) * 2.0 ** -24 * mag + (dy.double().abs() * 2.0 ** -19).sum(0)
    half = 2.0 ** -24 if grad == torch.float32 else BF16
    check(db, want, bound + half * (want.abs() + bound), "dbias")


@pytest.mark.parametrize("m", [1, 8, 33, 64])
@pytest.mark.parametrize("n,k", [(4096, 256), (2113, 1000), (64, 3000), (300, 65)])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_backward_of_few_rows(env, m, n, k, name):
    """dx by itself and with dW: the same values within the bounds, by
    whichever kernel."""
    torch, vc, dev = env
    dy, z = rand(torch, dev, m, n, seed=1), rand(torch, dev, m, n, seed=2)
    x, w = rand(torch, dev, m, k, seed=3), rand(torch, dev, n, k, seed=4, std=n ** -0.5)
    dz = dy.double() * act(torch, z.double(), name)[1]
    off = 0.0 if name == "none" else dy.double().abs() * 2.0 ** -19 + dz.abs() * 2.0 ** -16
    want = dz @ w.double()
    bound = accumulate_bound(2 * n, dz.abs() @ w.double().abs())
    bound = bound + (0.0 if name == "none" else off @ w.double().abs())
    for dw in (None, torch.empty(n, k, device=dev)):
        dx = torch.full((m, k + 3), 9.0, dtype=torch.bfloat16, device=dev)
        vc.vc_linear_backward(dy, x, w, dx=dx[:, :k], dweight=dw, preact=z, activation=name)
        check(dx[:, :k], want, bound + BF16 * (want.abs() + bound), "dx")
        assert (dx[:, k:] == 9).all()


def test_backward_parts_alone_and_strided(env):
    """Each output by itself gives the same bits as all together; gradients are
    written into the views of a bucket, whose other values stay."""
    torch, vc, dev = env
    m, n, k = 190, 96, 72
    dy, x, w, z = (rand(torch, dev, *s, seed=i)
                   for i, s in enumerate(((m, n), (m, k), (n, k), (m, n))))
    bucket = torch.full((n * k + n + 64,), 3.0, device=dev)
    dw, db = bucket[32:32 + n * k].view(n, k), bucket[32 + n * k:32 + n * k + n]
    dx = torch.empty_like(x)
    vc.vc_linear_backward(dy, x, w, dx=dx, dweight=dw, dbias=db, preact=z, activation="silu")
    assert (bucket[:32] == 3).all() and (bucket[32 + n * k + n:] == 3).all()
    one = torch.empty_like(dw)
    vc.vc_linear_backward(dy, x, w, dweight=one, preact=z, activation="silu")
    assert torch.equal(one, dw)
    one = torch.empty_like(db)
    vc.vc_linear_backward(dy, x, w, dbias=one, preact=z, activation="silu")
    assert torch.equal(one, db)
    one = torch.empty_like(dx)
    vc.vc_linear_backward(dy, x, w, dx=one, preact=z, activation="silu")
    assert torch.equal(one, dx)


def test_backward_of_no_rows(env):
    """No rows: dW and db are zero, or stay where they are added to."""
    torch, vc, dev = env
    dy, x = torch.empty(0, 40, dtype=torch.bfloat16, device=dev), torch.empty(
        0, 72, dtype=torch.bfloat16, device=dev)
    w = rand(torch, dev, 40, 72)
    for grad in (torch.float32, torch.bfloat16):
        dw, db = torch.ones(40, 72, dtype=grad, device=dev), torch.ones(40, dtype=grad, device=dev)
        vc.vc_linear_backward(dy, x, w, dweight=dw, dbias=db, accumulate=True)
        assert (dw == 1).all() and (db == 1).all()
        vc.vc_linear_backward(dy, x, w, dweight=dw, dbias=db)
        assert (dw == 0).all() and (db == 0).all()


def test_backward_of_no_features(env):
    """No outputs: dx is zero; no inputs: db alone is left."""
    torch, vc, dev = env
    none = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    dx = torch.ones(30, 70, dtype=torch.bfloat16, device=dev)
    vc.vc_linear_backward(none(30, 0), rand(torch, dev, 30, 70), none(0, 70), dx=dx,
                          dweight=none(0, 70))
    assert (dx == 0).all()
    dy, db = rand(torch, dev, 30, 20), torch.empty(20, device=dev)
    vc.vc_linear_backward(dy, none(30, 0), none(20, 0), dx=none(30, 0), dweight=none(20, 0),
                          dbias=db)
    check(db, dy.double().sum(0), 40 * 2.0 ** -24 * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("name", ACTS[1:])
def test_gradient_against_differences(env, name):
    """Along random directions the gradients agree with central differences of
    the 64-bit forward form."""
    torch, vc, dev = env
    m, n, k = 70, 64, 48
    x, w, b, dy = (rand(torch, dev, *s, seed=i)
                   for i, s in enumerate(((m, k), (n, k), (n,), (m, n))))
    w = (w.float() * k ** -0.5).to(torch.bfloat16)
    y, z = torch.empty_like(dy), torch.empty_like(dy)
    vc.vc_linear_forward(x, w, y, bias=b, preact=z, activation=name)
    dx = torch.empty_like(x)
    dw, db = torch.empty(n, k, device=dev), torch.empty(n, device=dev)
    vc.vc_linear_backward(dy, x, w, dx=dx, dweight=dw, dbias=db, preact=z, activation=name)

    def loss(X, W, B):
        return (act(torch, X @ W.t() + B, name)[0] * dy.double()).sum().item()

    h = 1e-5
    X, W, B = x.double(), w.double(), b.double()
    slope_change = 2.0 * BF16 * z.double().abs()  # act'' <= 2; z was rounded
    dz_off = dy.double().abs() * (slope_change + BF16)
    for which, grad, off in (("x", dx, dz_off @ W.abs()), ("w", dw, dz_off.t() @ X.abs()),
                             ("b", db, dz_off.sum(0))):
        d = rand(torch, dev, *grad.shape, seed=9, dtype=torch.float64)
        args = lambda s: (X + s * d if which == "x" else X, W + s * d if which == "w" else W,  # noqa: E731
                          B + s * d if which == "b" else B)
        slope = (loss(*args(h)) - loss(*args(-h))) / (2 * h)
        got = (grad.double() * d).sum().item()
        # errors of one sign at the worst; relu's kink within h counts as one slope
        tol = ((off + BF16 * grad.double().abs()) * d.abs()).sum().item() + 1e-4 * abs(slope)
        assert abs(got - slope) <= tol, (which, got, slope, tol)


# ---------------------------------------------------------- orthogonalisation --

COEF = (3.4445, -4.7750, 2.0315)


def ortho_exact(torch, g, steps=5, coef=COEF, eps=1e-7):
    a, b, c = coef
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1) if tall else x
    x = x / (x.norm(dim=(-2, -1), keepdim=True) + eps)
    for _ in range(steps):
        p = x @ x.transpose(-2, -1)
        x = a * x + (b * p + c * p @ p) @ x
    return x.transpose(-2, -1) if tall else x


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


SHAPES = [(1, 1), (1, 300), (300, 1), (2, 2), (7, 5), (16, 16), (33, 65), (64, 64), (100, 300),
          (300, 100), (128, 128), (128, 256), (129, 64), (128, 2048), (2050, 96), (120, 2100),
          (257, 129), (256, 256), (640, 200), (1000, 1003), (1024, 640)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_orthogonalize(env, rows, cols, dtype):
    torch, vc, dev = env
    g = rand(torch, dev, rows, cols, seed=rows, dtype=getattr(torch, dtype), std=1e-3)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    vc.vc_orthogonalize(g, out)
    assert relative(out, ortho_exact(torch, g)) < ORTHO


@pytest.mark.parametrize("rows,cols", [(48, 100), (300, 120), (512, 512), (400, 1300)])
def test_orthogonalize_falling_spectrum(env, rows, cols):
    torch, vc, dev = env
    r = min(rows, cols)
    u = rand(torch, dev, rows, r, seed=1, dtype=torch.float32)
    s = torch.exp(torch.linspace(0, -6, r, device=dev))
    g = (u * s) @ rand(torch, dev, r, cols, seed=2, dtype=torch.float32)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    vc.vc_orthogonalize(g, out)
    assert relative(out, ortho_exact(torch, g)) < 4e-3


@pytest.mark.parametrize("batch,rows,cols", [(3, 60, 100), (5, 100, 40), (2, 200, 333), (9, 128, 600)])
def test_orthogonalize_batches_with_strides(env, batch, rows, cols):
    """Matrices of a batch do not touch each other: each alone gives the same
    bits, strided rows and matrices too, and a NaN or a zero stays its own."""
    torch, vc, dev = env
    big = torch.full((batch, rows + 1, cols + 9), 3.0, device=dev)
    big[:, :rows, 3:3 + cols] = rand(torch, dev, batch, rows, cols, seed=4, dtype=torch.float32)
    g = big[:, :rows, 3:3 + cols]
    g[1].zero_()
    res = torch.full((batch, rows + 2, cols + 5), 4.0, dtype=torch.bfloat16, device=dev)
    out = res[:, :rows, 1:1 + cols]
    vc.vc_orthogonalize(g, out)
    assert (res[:, rows:] == 4).all() and (res[:, :, 0] == 4).all() and (res[:, :, 1 + cols:] == 4).all()
    assert (out[1] == 0).all()
    for i in range(batch):
        one = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
        vc.vc_orthogonalize(g[i].contiguous(), one)
        assert torch.equal(one, out[i])
    g[0, rows - 1, cols - 1] = float("nan")
    again = torch.empty(batch, rows, cols, dtype=torch.bfloat16, device=dev)
    vc.vc_orthogonalize(g, again)
    assert torch.isnan(again[0]).all()
    assert torch.equal(again[1:], out[1:])


def test_orthogonalize_in_place_steps_and_coefficients(env):
    torch, vc, dev = env
    g = rand(torch, dev, 96, 160, seed=1)
    for steps, coef in ((1, COEF), (3, COEF), (12, (1.5, -0.5, 0.0)), (8, (2.0, -1.5, 0.5))):
        want = ortho_exact(torch, g, steps, coef)
        out = g.clone()
        vc.vc_orthogonalize(out, out, steps=steps, coefficients=coef)
        # more passes, more roundings: sqrt(3 steps) of them
        tol = 2 * FP16 / 3 ** 0.5 * (3 * steps) ** 0.5 + BF16 / 3 ** 0.5
        assert relative(out, want) < tol, (steps, coef)


@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_orthogonalize_scale_of_the_input(env, scale):
    """The result does not depend on the input's scale while the squares' sum
    is a float32 (eps counts where the norm is near it)."""
    torch, vc, dev = env
    g = rand(torch, dev, 64, 100, seed=1, dtype=torch.float32) * scale
    out = torch.empty(64, 100, dtype=torch.bfloat16, device=dev)
    vc.vc_orthogonalize(g, out, eps=0.0)
    assert relative(out, ortho_exact(torch, g, eps=0.0)) < ORTHO


@pytest.mark.parametrize("shape", [(40, 100), (100, 40), (2, 300, 257), (1000, 200), (3, 128, 512)])
@pytest.mark.parametrize("i", range(4))
def test_muon_step(env, shape, i):
    torch, vc, dev = env
    wt, gt, mt = [(torch.float32, torch.float32, torch.float32),
                  (torch.bfloat16, torch.bfloat16, torch.float32),
                  (torch.float32, torch.bfloat16, torch.bfloat16),
                  (torch.bfloat16, torch.float32, torch.float32)][i]
    nesterov = i % 2 == 0
    w = rand(torch, dev, *shape, seed=1, dtype=wt)
    g = rand(torch, dev, *shape, seed=2, dtype=gt)
    m = rand(torch, dev, *shape, seed=3, dtype=mt)
    w0, m0, g0 = w.double(), m.double(), g.clone()
    lr, beta, wd, scale = 0.02, 0.9, 0.1, 3.0
    vc.vc_muon_step(w, g, m, lr, beta=beta, nesterov=nesterov, weight_decay=wd, scale=scale)
    assert torch.equal(g, g0)
    em = beta * m0 + g0.double()
    half = BF16 if mt == torch.bfloat16 else 2.0 ** -24
    check(m, em, (half + 2.0 ** -23) * (em.abs() + m0.abs() + g0.double().abs()), "momentum")
    used = m.double() if mt == torch.bfloat16 else em
    o = ortho_exact(torch, g0.double() + beta * used if nesterov else used)
    want = (1 - lr * wd) * w0 - lr * scale * o
    # the update without bf16's rounding, and the weight's one rounding
    off = (w.double() - want).norm().item()
    half = BF16 if wt == torch.bfloat16 else 2.0 ** -23
    assert off <= (ORTHO - BF16 / 3 ** 0.5) * lr * scale * o.norm().item() + half * want.norm().item()


def test_muon_default_scale(env):
    """scale None gives an update of 0.2 a value in the root mean square (the
    five passes bring singular values to between 0.68 and 1.13)."""
    torch, vc, dev = env
    for shape in ((64, 300), (300, 64), (256, 256)):
        w = torch.zeros(*shape, device=dev)
        vc.vc_muon_step(w, rand(torch, dev, *shape, seed=5), torch.zeros(*shape, device=dev), 1.0)
        rms = w.square().mean().sqrt().item() / 0.2
        lower = 0.68 if shape[0] != shape[1] else 0.5  # a square one has small ones too
        expect = math.sqrt(min(shape) * max(shape) / (shape[0] * shape[1]))
        assert lower * expect < rms < 1.14 * expect


# ------------------------------------------------------- calls, streams, sizes --

def test_calls_repeat_bit_for_bit_and_follow_their_stream(env):
    torch, vc, dev = env
    x, w = rand(torch, dev, 500, 300, seed=1), rand(torch, dev, 260, 300, seed=2)
    g = rand(torch, dev, 200, 500, seed=3)
    y, o = torch.empty(500, 260, dtype=torch.bfloat16, device=dev), torch.empty_like(g)
    vc.vc_linear_forward(x, w, y, activation="gelu")
    vc.vc_orthogonalize(g, o)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    x2, g2 = torch.zeros_like(x), torch.zeros_like(g)
    y2, o2 = torch.zeros_like(y), torch.zeros_like(o)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the inputs arrive late on this stream
        x2.copy_(x)
        g2.copy_(g)
    vc.vc_linear_forward(x2, w, y2, activation="gelu", stream=side)
    vc.vc_orthogonalize(g2, o2, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(o, o2)


def test_prepared_calls_and_given_workspaces(env):
    torch, vc, dev = env
    x, w = rand(torch, dev, 77, 65, seed=1), rand(torch, dev, 31, 65, seed=2)
    dy = rand(torch, dev, 77, 31, seed=3)
    z = rand(torch, dev, 77, 31, seed=4)
    y, y2 = (torch.empty(77, 31, dtype=torch.bfloat16, device=dev) for _ in range(2))
    ws = torch.empty(vc.linear_forward_workspace(x, w), dtype=torch.uint8, device=dev)
    vc.vc_linear_forward(x, w, y, workspace=ws)
    call = vc.prepare_linear_forward(x, w, y2)
    call()
    assert torch.equal(y, y2)
    need = vc.linear_backward_workspace(dy, x, w, "gelu", dbias=True)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    dx, dx2 = torch.empty_like(x), torch.empty_like(x)
    db, db2 = (torch.empty(31, device=dev) for _ in range(2))
    vc.vc_linear_backward(dy, x, w, dx=dx, dbias=db, preact=z, activation="gelu", workspace=ws)
    vc.prepare_linear_backward(dy, x, w, dx=dx2, dbias=db2, preact=z, activation="gelu")()
    assert torch.equal(dx, dx2) and torch.equal(db, db2)
    p = [rand(torch, dev, 40, 90, seed=i, dtype=torch.float32) for i in range(3)]
    q = [t.clone() for t in p]
    vc.vc_muon_step(*p, 0.1, workspace=torch.empty(vc.orthogonalize_workspace((40, 90)),
                                                   dtype=torch.uint8, device=dev))
    step = vc.prepare_muon_step(*q)
    step(0.1)
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    step(0.05)
    vc.vc_muon_step(*p, 0.05)
    assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_graph_capture(env):
    torch, vc, dev = env
    g = rand(torch, dev, 96, 700, seed=1)
    x, w = rand(torch, dev, 300, 64, seed=2), rand(torch, dev, 128, 64, seed=3)
    o, y = torch.empty_like(g), torch.empty(300, 128, dtype=torch.bfloat16, device=dev)
    a, b = vc.prepare_orthogonalize(g, o), vc.prepare_linear_forward(x, w, y)
    side = torch.cuda.Stream(dev)
    with torch.cuda.stream(side):
        a()
        b()
        side.synchronize()
        want = o.clone(), y.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            a()
            b()
    o.zero_()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(y, want[1])


def test_offsets_past_32_bits(env):
    torch, vc, dev = env
    # an operand of 2.3e9 values
    m, k, n = 70_000, 32_800, 8
    x = torch.empty(m, k, dtype=torch.bfloat16, device=dev).normal_(generator=torch.Generator(
        device=dev).manual_seed(1))
    w = rand(torch, dev, n, k, seed=2, std=k ** -0.5)
    y = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    vc.vc_linear_forward(x, w, y)
    rows = torch.tensor([0, 1, 65_472, 65_536, 69_998, 69_999], device=dev)
    _, _, ey, dy = forward_exact(torch, x[rows], w, None, None, "none")
    check(y[rows], ey, dy + BF16 * (ey.abs() + dy), "y")
    del x
    # an output of 2.3e9 values
    x, w = rand(torch, dev, m, 16, seed=3), rand(torch, dev, k, 16, seed=4)
    y = torch.empty(m, k, dtype=torch.bfloat16, device=dev)
    vc.vc_linear_forward(x, w, y)
    _, _, ey, dy = forward_exact(torch, x[rows], w, None, None, "none")
    check(y[rows], ey, dy + BF16 * (ey.abs() + dy), "y")


def test_refusals(env):
    torch, vc, dev = env
    t = rand(torch, dev, 8, 16)
    w = rand(torch, dev, 4, 16, seed=1)
    y = torch.empty(8, 4, dtype=torch.bfloat16, device=dev)
    cases = [
        (ValueError, "unknown activation", lambda: vc.vc_linear_forward(t, w, y, activation="tanh")),
        (TypeError, "dtype", lambda: vc.vc_linear_forward(t.float(), w, y)),
        (ValueError, "expected \\(N, 16\\)", lambda: vc.vc_linear_forward(t, w[:, :8], y)),
        (ValueError, "expected 8 x 4", lambda: vc.vc_linear_forward(t, w, y[:, :3])),
        (ValueError, "not contiguous", lambda: vc.vc_linear_forward(t, w, torch.empty(
            4, 8, dtype=torch.bfloat16, device=dev).t())),
        (ValueError, "bias has shape", lambda: vc.vc_linear_forward(t, w, y, bias=y[0, :3])),
        (ValueError, "needs preact", lambda: vc.vc_linear_backward(y, t, w, activation="gelu")),
        (ValueError, "overlap", lambda: vc.vc_linear_forward(t[:1].expand(8, 16), w, y)),
        (ValueError, "steps", lambda: vc.vc_orthogonalize(t, torch.empty_like(t), steps=0)),
        (ValueError, "out has shape", lambda: vc.vc_orthogonalize(t, y)),
        (ValueError, "workspace holds", lambda: vc.vc_orthogonalize(
            t, torch.empty_like(t), workspace=torch.empty(16, dtype=torch.uint8, device=dev))),
        (ValueError, "grad has shape", lambda: vc.vc_muon_step(t, w, t.clone(), 0.1)),
        (TypeError, "dtype", lambda: vc.vc_muon_step(t, t.half(), t.clone(), 0.1)),
        (vc.VcError, "ALIAS", lambda: vc.vc_muon_step(t, t, t.clone(), 0.1)),
        (vc.VcError, "ALIAS", lambda: vc.vc_linear_forward(t, w, t[:, :4])),
    ]
    for kind, text, call in cases:
        with pytest.raises(kind, match=text):
            call()
    before = t.clone()
    torch.cuda.synchronize()
    assert torch.equal(before, t)
