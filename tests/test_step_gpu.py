"""The embedding, the norms around a block and gradient clipping on the GPU against
plain 64-bit forms.

Tolerances follow from the arithmetic that include/vc_step.h states, with the unit
roundoffs u = 2^-24 of float32 and 2^-8 of bfloat16 (half a step):

  - A stored value is off by its type's roundoff, and by what the 32-bit arithmetic
    before it is off.
  - A lookup multiplies once in 32 bits: u.
  - A sum of n terms in 32 bits, in any order, is off by at most n u of the sum of
    magnitudes; scaling it and adding to what is there add 3 u.
  - The squares of gradients are added in 32 bits over at most 33 terms of a thread, then
    in 64: 33 u of the sum, half of that and one rounding for the root; c has three more.
  - A norm's statistics: sums of squares over D columns, of which a thread adds at most
    D / 512 + 16 in a row, and at most 32 partial sums follow; with the products and the root below
    128 u relative for D up to 20000.  Everything a row computes is then a few sums and products of
    terms whose magnitudes are added up beside it ("size"): 256 u of that.
  - Column sums over T rows: T + 256 u of the sum of magnitudes.
"""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}
ROWS = 256 * U


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


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def unit(t):
    return ROUND[str(t.dtype).split(".")[1]]


def rand(torch, dev, *shape, seed=0, std=1.0, mean=0.0, dtype=None):
    g = torch.Generator(device=dev).manual_seed(1000 + seed)
    return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dtype or torch.bfloat16)


def check(got, want, size, what):
    """|got - want| <= size + the rounding of what is stored."""
    off = (got.double() - want).abs()
    ok = off <= size + unit(got) * (want.abs() + size) + 1e-40
    assert ok.all(), (what, off[~ok][:4].tolist(), want[~ok][:4].tolist(), int((~ok).sum()))


def pitched(torch, dev, rows, cols, dtype, gap, offset=0, fill=7.0):
    """A tensor whose rows are `gap` values apart beyond their length, inside a
    larger one, and a call that checks that nothing around it was written."""
    flat = torch.full((offset + (rows + 1) * (cols + gap),), fill, dtype=dtype, device=dev)
    t = torch.as_strided(flat, (rows, cols), (cols + gap, 1), offset)
    mask = torch.ones_like(flat, dtype=torch.bool)
    torch.as_strided(mask, (rows, cols), (cols + gap, 1), offset).fill_(False)
    return t, lambda: bool((flat[mask] == fill).all())


# ---------------------------------------------------------------- embedding --

def lookup_want(torch, ids, weight, first, scale):
    row = ids.reshape(-1).long() - first
    live = (row >= 0) & (row < weight.shape[0])
    y = torch.zeros(row.numel(), weight.shape[1], dtype=torch.float64, device=ids.device)
    y[live] = weight.double()[row[live]] * scale
    return y


@pytest.mark.parametrize("ids_type", ["int32", "int64"])
@pytest.mark.parametrize("types", ["bf16-bf16", "f32-f32", "bf16-f32", "f32-bf16"])
@pytest.mark.parametrize("tokens,rows,cols", [(1, 1, 1), (1, 50, 1024), (7, 5, 3), (300, 40, 72),
                                              (1003, 501, 517), (5000, 300, 1030), (2100, 64, 2048)])
def test_lookup(env, tokens, rows, cols, types, ids_type):
    torch, vc, dev = env
    a, b = (dt(torch, k) for k in types.split("-"))
    g = torch.Generator(device=dev).manual_seed(tokens)
    for first in (0, 17):
        # ids below, inside and behind the table's rows
        ids = torch.randint(first - 3, first + rows + 3, (tokens,), generator=g, device=dev)
        ids = ids.to(getattr(torch, ids_type))
        w = rand(torch, dev, rows, cols, dtype=a)
        out = torch.full((tokens, cols), 9.0, dtype=b, device=dev)
        scale = float(cols) ** 0.5
        vc.vc_embedding_forward(ids, w, out, scale=scale, first=first)
        scale = torch.tensor(scale, dtype=torch.float32).item()
        want = lookup_want(torch, ids, w, first, scale)
        check(out, want, U * want.abs(), "y")


@pytest.mark.parametrize("gap,offset", [(0, 0), (8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
def test_lookup_strides(env, gap, offset):
    torch, vc, dev = env
    for cols in (64, 70, 129):
        w, _ = pitched(torch, dev, 33, cols, torch.bfloat16, gap, offset)
        w.copy_(rand(torch, dev, 33, cols))
        out, clean = pitched(torch, dev, 41, cols, torch.bfloat16, gap, offset)
        ids = torch.arange(41, device=dev) * 7 % 33
        vc.vc_embedding_forward(ids, w, out)
        assert torch.equal(out, w[ids]) and clean()
        three = torch.empty(2, 3, cols, dtype=torch.bfloat16, device=dev)
        vc.prepare_embedding_forward(ids[:6].view(2, 3), w, three)()
        assert torch.equal(three.view(6, cols), w[ids[:6]])


def test_ids_at_the_ends_of_their_range(env):
    torch, vc, dev = env
    low, high = -2 ** 63, 2 ** 63 - 1
    w = rand(torch, dev, 10, 16)
    for first in (0, 5, 2 ** 62):
        ids = torch.tensor([low, -1, high, first, first + 9, first + 10, low + first], device=dev)
        out = torch.empty(7, 16, dtype=torch.bfloat16, device=dev)
        vc.vc_embedding_forward(ids, w, out, first=first)
        want = torch.zeros_like(out)
        want[3], want[4] = w[0], w[9]
        assert torch.equal(out, want), first
        dw = torch.full((10, 16), 3.0, device=dev)
        vc.vc_embedding_backward(torch.ones(7, 16, device=dev), ids, dw, first=first)
        assert dw[0].eq(1).all() and dw[9].eq(1).all() and dw[1:9].eq(0).all()


def scatter_want(torch, dy, ids, rows, first, padding, scale):
    """The sums and the sums of magnitudes, and how many terms they have."""
    ids = ids.reshape(-1).long()
    dy = dy.reshape(ids.numel(), -1).double()
    row = ids - first
    live = (row >= 0) & (row < rows)
    if padding is not None:
        live &= ids != padding
    out = []
    for terms in (dy * scale, dy.abs() * abs(scale), torch.ones_like(dy)):
        s = torch.zeros(rows, dy.shape[1], dtype=torch.float64, device=dy.device)
        out.append(s.index_add_(0, row[live], terms[live]))
    return out


def check_scatter(torch, vc, dy, ids, dw, *, scale=0.75, first=0, padding=None, accumulate=False):
    before = dw.double().clone()
    vc.vc_embedding_backward(dy, ids, dw, scale=scale, first=first, padding=padding,
                             accumulate=accumulate)
    want, size, count = scatter_want(torch, dy, ids, dw.shape[0], first, padding, scale)
    tol = (count + 3) * U * size
    if accumulate:
        assert torch.equal(dw[count[:, 0] == 0].double(), before[count[:, 0] == 0])
        want, tol = want + before, tol + 3 * U * before.abs()
    check(dw, want, tol * (count > 0), "dweight")


@pytest.mark.parametrize("types", ["bf16-bf16", "bf16-f32", "f32-f32", "f32-bf16"])
@pytest.mark.parametrize("tokens,rows,cols", [
    (1, 1, 1), (1, 10, 8), (7, 5, 3), (64, 200, 64), (100, 50, 264), (1003, 5003, 517),
    (1000, 3, 256), (4097, 100, 40), (9000, 700, 300), (3000, 600, 1032)])
def test_scatter(env, tokens, rows, cols, types):
    torch, vc, dev = env
    a, b = (dt(torch, k) for k in types.split("-"))
    g = torch.Generator(device=dev).manual_seed(tokens + cols)
    u = torch.rand(tokens, generator=g, device=dev)
    ids = (u ** 3 * rows).long().clamp_max(rows - 1)  # some rows often, many never
    dy = rand(torch, dev, tokens, cols, dtype=a)
    dw = torch.full((rows, cols), 5.0, dtype=b, device=dev)
    check_scatter(torch, vc, dy, ids, dw)
    dw = rand(torch, dev, rows, cols, seed=1, dtype=b)
    check_scatter(torch, vc, dy, ids.int(), dw, accumulate=True, padding=0)
    shifted = ids - rows // 3 + 40  # some below and some behind the table
    check_scatter(torch, vc, dy, shifted, dw, first=40, padding=41)


@pytest.mark.parametrize("tokens,cols", [(9, 8), (64, 24), (65, 264), (5000, 264), (70001, 16)])
def test_scatter_of_one_id(env, tokens, cols):
    torch, vc, dev = env
    dy = rand(torch, dev, tokens, cols)
    for row in (0, 4, 11):
        ids = torch.full((tokens,), row, device=dev, dtype=torch.int32)
        dw = torch.full((12, cols), 5.0, device=dev)
        check_scatter(torch, vc, dy, ids, dw)
        # all of them padding, or outside of the table
        check_scatter(torch, vc, dy, ids, dw, padding=row)
        assert dw.eq(0).all()
        check_scatter(torch, vc, dy, ids, dw, first=12)
        assert dw.eq(0).all()


@pytest.mark.parametrize("tokens,rows,cols", [(70001, 700, 16), (131072, 5000, 8), (66000, 70000, 24)])
def test_scatter_of_many_tokens(env, tokens, rows, cols):
    """More tokens than the sorting blocks hold at a time."""
    torch, vc, dev = env
    g = torch.Generator(device=dev).manual_seed(tokens)
    ids = torch.randint(0, rows, (tokens,), generator=g, device=dev)
    check_scatter(torch, vc, rand(torch, dev, tokens, cols), ids,
                  torch.empty(rows, cols, device=dev))


@pytest.mark.parametrize("rows", [511, 512, 513, 262143, 262144, 600000])
def test_scatter_digits(env, rows):
    """Tables at the borders of the sort's passes; the last rows among the ids."""
    torch, vc, dev = env
    g = torch.Generator(device=dev).manual_seed(rows)
    ids = torch.randint(0, rows, (3000,), generator=g, device=dev)
    ids[:40] = rows - 1 - torch.arange(40, device=dev) % 20
    check_scatter(torch, vc, rand(torch, dev, 3000, 8), ids, torch.empty(rows, 8, device=dev))


def test_scatter_order_is_the_tokens(env):
    """A row's terms are added in an order that depends on the ids alone: the same
    bits in every run, with other tokens' values changed too."""
    torch, vc, dev = env
    g = torch.Generator(device=dev).manual_seed(3)
    ids = (torch.rand(20000, generator=g, device=dev) ** 4 * 3000).long()
    dy = rand(torch, dev, 20000, 136, dtype=torch.float32)
    a, b = (torch.empty(3000, 136, device=dev) for _ in range(2))
    vc.vc_embedding_backward(dy, ids, a)
    for _ in range(5):
        vc.vc_embedding_backward(dy, ids, b)
        assert torch.equal(a, b)
    dy[ids == 7] = float("nan")
    vc.vc_embedding_backward(dy, ids, b)
    assert b[7].isnan().all()
    b[7] = a[7]
    assert torch.equal(a, b)


@pytest.mark.parametrize("gap,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
def test_scatter_strides(env, gap, offset):
    torch, vc, dev = env
    for cols in (64, 70, 300):
        for b in (torch.bfloat16, torch.float32):
            dy, _ = pitched(torch, dev, 500, cols, torch.bfloat16, gap, offset)
            dy.copy_(rand(torch, dev, 500, cols))
            dw, clean = pitched(torch, dev, 90, cols, b, gap, offset)
            ids = torch.arange(500, device=dev) ** 2 % 83
            check_scatter(torch, vc, dy, ids, dw)
            check_scatter(torch, vc, dy, ids, dw, accumulate=True)
            assert clean()


def test_scatter_without_tokens(env):
    torch, vc, dev = env
    dw = torch.full((30, 20), 4.0, device=dev)
    none, ids = torch.empty(0, 20, device=dev), torch.empty(0, dtype=torch.int64, device=dev)
    vc.vc_embedding_backward(none, ids, dw, accumulate=True)
    assert dw.eq(4).all()
    vc.vc_embedding_backward(none, ids, dw)
    assert dw.eq(0).all()


def test_shards_of_a_vocabulary(env):
    """Ranks hold parts of the table: their lookups add up to the whole one's, and each
    has its part of the gradient."""
    torch, vc, dev = env
    rows, cols, tokens, ranks = 103, 48, 400, 4
    w, dy = rand(torch, dev, rows, cols), rand(torch, dev, tokens, cols, seed=1)
    ids = torch.arange(tokens, device=dev) * 31 % rows
    whole, dw = torch.empty_like(dy), torch.empty(rows, cols, device=dev)
    vc.vc_embedding_forward(ids, w, whole)
    vc.vc_embedding_backward(dy, ids, dw, padding=5)
    q = vc.vc_shard_count(rows, ranks)
    outs, grads = [], []
    for r in range(ranks):
        part = w[r * q:(r + 1) * q]
        outs.append(torch.empty_like(dy))
        vc.vc_embedding_forward(ids, part, outs[-1], first=r * q)
        grads.append(torch.empty(part.shape, device=dev))
        vc.vc_embedding_backward(dy, ids, grads[-1], first=r * q, padding=5)
    vc.vc_all_reduce(outs)
    assert all(torch.equal(o, whole) for o in outs)
    assert torch.equal(torch.cat(grads), dw)


# -------------------------------------------------------------- block norms --

def norm_parts(torch, v, kind, eps):
    """Hats, their magnitudes' bound and 1 / deviation."""
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    spread = v.abs().mean(-1, keepdim=True) if kind == "layer" else mean
    rstd = ((v - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    return (v - mean) * rstd, (v.abs() + spread) * rstd, rstd


class Block:
    """Inputs of a block's norms and the 64-bit forms of outputs and gradients, each
    with the sum of magnitudes that its terms have."""

    def __init__(self, torch, dev, rows, cols, norm="rms", stream="bf16", gates=None, post=True,
                 bias=False, act="none", gate_type="bf16", weight_type="bf16", residual=True,
                 scale=0.75, eps=1e-6, seed=0):
        s = dt(torch, stream)
        wt = dt(torch, weight_type)
        r = lambda *shape, **kw: rand(torch, dev, *shape, seed=seed + len(shape), **kw)  # noqa: E731
        self.torch, self.norm, self.act, self.scale, self.eps = torch, norm, act, scale, eps
        self.rows, self.cols, self.stream = rows, cols, s
        self.h = r(rows, cols, std=0.5, mean=0.1)
        self.x = rand(torch, dev, rows, cols, seed=seed + 3, std=2.0, dtype=s) if residual else None
        self.gate = None
        if gates is not None:
            self.gate = rand(torch, dev, gates, cols, seed=seed + 4, dtype=dt(torch, gate_type))
        vec = lambda k, **kw: rand(torch, dev, cols, seed=seed + k, dtype=wt, **kw)  # noqa: E731
        self.pre = vec(5, std=0.2, mean=1.0)
        self.post = vec(6, std=0.2, mean=1.0) if post else None
        self.pre_bias = vec(7) if bias else None
        self.post_bias = vec(8) if bias and post else None

    def keywords(self):
        return dict(gate=self.gate, post=self.post, post_bias=self.post_bias, pre=self.pre,
                    norm=self.norm, gate_act=self.act, residual_scale=self.scale, eps=self.eps)

    def wide(self, t):
        return None if t is None else t.double()

    def gate_values(self):
        if self.gate is None:
            one = self.torch.ones(1, 1, dtype=self.torch.float64, device=self.h.device)
            return one, one
        g = self.gate.double().repeat_interleave(self.rows // self.gate.shape[0], 0)
        if self.act == "none":
            return g, self.torch.ones_like(g)
        s = self.torch.sigmoid(g)
        return s, s * self.torch.sigmoid(-g)

    def post_values(self):
        """u, its size, hats, their size, 1 / deviation"""
        h = self.h.double()
        if self.post is None:
            return h, h.abs(), None, None, None
        hat, size, rstd = norm_parts(self.torch, h, self.norm, self.eps)
        w = self.post.double()
        u, us = hat * w, size * w.abs()
        if self.post_bias is not None:
            u, us = u + self.post_bias.double(), us + self.post_bias.double().abs()
        return u, us, hat, size, rstd

    def forward(self):
        """r, n and the sizes of what they are made of"""
        u, us, *_ = self.post_values()
        v, _ = self.gate_values()
        r, rs = v * u, v.abs() * us
        if self.x is not None:
            r, rs = r + self.scale * self.x.double(), rs + abs(self.scale) * self.x.double().abs()
        hat, size, rstd = norm_parts(self.torch, r, self.norm, self.eps)
        w = self.pre.double().abs()
        # what r is off moves the hats by as much, and through the statistics by as much again
        ns = w * (size + 2 * rs * rstd + size * (rs * rstd).square().mean(-1, keepdim=True).sqrt())
        n = hat * self.pre.double()
        if self.pre_bias is not None:
            n, ns = n + self.pre_bias.double(), ns + self.pre_bias.double().abs()
        return r, rs, n, ns

    def backward(self, dr, dn, r):
        """The gradients by their formulas, {name: (value, size)}."""
        out = {}
        t = self.torch
        layer = self.norm == "layer"

        def through(d, ds, hat, hs, rstd):
            m1 = d.mean(-1, keepdim=True) if layer else 0.0
            m1s = ds.mean(-1, keepdim=True) if layer else 0.0
            m2, m2s = (d * hat).mean(-1, keepdim=True), (ds * hs).mean(-1, keepdim=True)
            return rstd * (d - m1 - hat * m2), rstd * (ds + m1s + hs * m2s)

        all_, size = (dr.double(), dr.double().abs()) if dr is not None else (0.0, 0.0)
        if dn is not None:
            d = dn.double()
            hat, hs, rstd = norm_parts(t, r.double(), self.norm, self.eps)
            out["dpre"] = (d * hat).sum(0), (d.abs() * hs).sum(0)
            out["dpre_bias"] = d.sum(0), d.abs().sum(0)
            g, gs = through(d * self.pre.double(), (d * self.pre.double()).abs(), hat, hs, rstd)
            all_, size = all_ + g, size + gs
        out["dx"] = self.scale * all_, abs(self.scale) * size
        u, us, hat, hs, rstd = self.post_values()
        v, slope = self.gate_values()
        if self.gate is not None:
            groups = self.gate.shape[0]
            fold = lambda a: a.view(groups, -1, self.cols).sum(1)  # noqa: E731
            out["dgate"] = fold(all_ * u * slope), fold(size * us * slope)
        du, dus = all_ * v, size * v.abs()
        if self.post is None:
            out["dh"] = du, dus
            return out
        out["dpost"] = (du * hat).sum(0), (dus * hs).sum(0)
        out["dpost_bias"] = du.sum(0), dus.sum(0)
        w = self.post.double()
        out["dh"] = through(du * w, dus * w.abs(), hat, hs, rstd)
        return out


GATES = ["none", "shared", "full", "groups"]


def gates_of(kind, rows):
    groups = next(k for k in (5, 3, 2, 1) if rows % k == 0)
    return {"none": None, "shared": 1, "full": rows, "groups": groups}[kind]


def check_forward(env, b):
    torch, vc, dev = env
    r = torch.full((b.rows, b.cols), 9.0, dtype=b.stream, device=dev)
    n = torch.full((b.rows, b.cols), 9.0, dtype=torch.bfloat16, device=dev)
    vc.vc_block_norm_forward(b.h, r=r, n=n, x=b.x, pre_bias=b.pre_bias, **b.keywords())
    want, rs, wn, ns = b.forward()
    check(r, want, ROWS * rs, "r")
    check(n, wn, ROWS * ns, "n")
    return r, n


def check_backward(env, b, grad="f32", use=("dr", "dn"), accumulate=False):
    torch, vc, dev = env
    gt = dt(torch, grad)
    dr = rand(torch, dev, b.rows, b.cols, seed=21, dtype=b.stream) if "dr" in use else None
    dn = rand(torch, dev, b.rows, b.cols, seed=22) if "dn" in use else None
    r = rand(torch, dev, b.rows, b.cols, seed=23, std=2.0, mean=0.3, dtype=b.stream)
    want = b.backward(dr, dn, r)
    if b.norm == "rms":
        want = {k: v for k, v in want.items() if not k.endswith("_bias")}
    out = {}
    for i, (k, (v, _)) in enumerate(want.items()):
        kind = b.stream if k == "dx" else torch.bfloat16 if k == "dh" else gt
        out[k] = rand(torch, dev, *v.shape, seed=30 + i, dtype=kind)
    if "dgate" in out:
        out["dgate"] = out["dgate"].view(b.gate.shape)
    before = {k: v.double().clone() for k, v in out.items()}
    vc.vc_block_norm_backward(b.h, dr=dr, dn=dn, r=r if dn is not None else None,
                              accumulate=accumulate, **out, **b.keywords())
    for k, (v, size) in want.items():
        rows = b.rows if k in ("dpre", "dpre_bias", "dpost", "dpost_bias") else (
            b.rows // b.gate.shape[0] if k == "dgate" else 0)
        tol = (2 * ROWS + rows * U) * size
        if accumulate and k not in ("dx", "dh"):
            v, tol = v + before[k], tol + 2 * U * before[k].abs()
        check(out[k], v, tol, k)
    return out


COLS = [1, 3, 8, 100, 256, 257, 264, 512, 520, 1000, 1021, 1030, 2048, 2200, 4096, 4100, 5003, 8192,
        8200, 16384, 20000]


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_block_forward_widths(env, cols, stream, norm):
    torch, vc, dev = env
    for i, rows in enumerate((1, 30)):
        b = Block(torch, dev, rows, cols, norm, stream, gates=gates_of(GATES[(cols + i) % 4], rows),
                  bias=norm == "layer", act=("none", "sigmoid")[i])
        check_forward(env, b)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("cols", [32768, 33000, 40001, 65536, 70004])
def test_block_longest_rows(env, cols, norm):
    """Rows at the ends of what a cluster of blocks shares, and beyond."""
    for i, gate in enumerate(GATES):
        stream = ("bf16", "f32")[i % 2]
        b = Block(env[0], env[2], 6, cols, norm, stream, gates_of(gate, 6), True, norm == "layer",
                  ("none", "sigmoid")[i // 2])
        check_forward(env, b)
        check_backward(env, b)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("types", ["bf16-f32", "f32-bf16"])
def test_block_forward_options(env, norm, gate, post, types):
    torch, vc, dev = env
    gate_type, weight_type = types.split("-")
    for rows, cols in ((90, 136), (700, 1040), (2500, 72)):
        for residual in (True, False):
            b = Block(torch, dev, rows, cols, norm, "f32", gates_of(gate, rows), post, residual and
                      norm == "layer", "sigmoid" if rows == 90 else "none", gate_type, weight_type,
                      residual)
            check_forward(env, b)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_block_backward_widths(env, cols, stream, norm):
    torch, vc, dev = env
    for i, rows in enumerate((1, 30)):
        b = Block(torch, dev, rows, cols, norm, stream, gates=gates_of(GATES[(cols + i) % 4], rows),
                  bias=norm == "layer", act=("sigmoid", "none")[i])
        check_backward(env, b, ("bf16", "f32")[i])


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_block_backward_options(env, norm, gate, post, grad):
    torch, vc, dev = env
    for rows, cols in ((7, 40), (90, 136), (1500, 1040), (5000, 24), (640, 9000)):
        for i, use in enumerate((("dr", "dn"), ("dr",), ("dn",))):
            b = Block(torch, dev, rows, cols, norm, "f32" if i else "bf16", gates_of(gate, rows), post,
                      norm == "layer", "sigmoid" if rows == 90 else "none")
            check_backward(env, b, grad, use, accumulate=i == 1)


@pytest.mark.parametrize("rows,groups", [(10, 5), (3000, 1500), (3000, 2), (3000, 7 * 3), (4096, 64),
                                         (9999, 9)])
@pytest.mark.parametrize("cols", [40, 300, 1000, 3000, 8400])
def test_block_backward_groups(env, rows, groups, cols):
    """Gates shared by groups that span the rows of many teams, or lie inside of one's."""
    torch, vc, dev = env
    if rows % groups:
        groups = 3
    b = Block(torch, dev, rows, cols, gates=groups, act="sigmoid", gate_type="f32")
    check_backward(env, b)


@pytest.mark.parametrize("norm,stream", [("rms", "bf16"), ("layer", "f32")])
@pytest.mark.parametrize("gate_type", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1801, 2304, 2600, 4095, 5120, 8191, 8192])
def test_block_gates_of_wide_rows(env, cols, gate_type, norm, stream):
    """Gates for every element and for groups, where rows with them do and do not fit in
    shared memory."""
    torch, vc, dev = env
    for gates in (40, 4):
        b = Block(torch, dev, 40, cols, norm, stream, gates, bias=norm == "layer", act="sigmoid",
                  gate_type=gate_type)
        check_forward(env, b)
        check_backward(env, b, gate_type, accumulate=gates == 4)


@pytest.mark.parametrize("cols", [64, 130, 1040, 1801, 2301, 4099, 8300])
@pytest.mark.parametrize("gap,offset", [(8, 0), (8, 8), (3, 0), (0, 1), (0, 3)])
def test_block_strides(env, cols, gap, offset):
    """Rows of wider tensors, on and off 16 bytes; nothing beside them is written."""
    torch, vc, dev = env
    rows = 33
    b = Block(torch, dev, rows, cols, "layer", "f32", gates=11, bias=True)
    r0, n0 = check_forward(env, b)
    put = {}
    clean = []
    for name, kind in (("h", torch.bfloat16), ("x", torch.float32), ("r", torch.float32),
                       ("n", torch.bfloat16), ("dr", torch.float32), ("dn", torch.bfloat16),
                       ("dx", torch.float32), ("dh", torch.bfloat16)):
        put[name], c = pitched(torch, dev, rows, cols, kind, gap, offset)
        clean.append(c)
    for name, kind in (("gate", torch.bfloat16), ("dgate", torch.float32)):
        put[name], c = pitched(torch, dev, 11, cols, kind, gap, offset)
        clean.append(c)
    put["h"].copy_(b.h), put["x"].copy_(b.x), put["gate"].copy_(b.gate)
    kw = {**b.keywords(), "gate": put["gate"]}
    vc.vc_block_norm_forward(put["h"], r=put["r"], n=put["n"], x=put["x"], pre_bias=b.pre_bias, **kw)
    size = b.forward()
    check(put["r"], size[0], ROWS * size[1], "r")
    check(put["n"], size[2], ROWS * size[3], "n")
    put["dr"].copy_(rand(torch, dev, rows, cols, seed=1, dtype=torch.float32))
    put["dn"].copy_(rand(torch, dev, rows, cols, seed=2))
    want = b.backward(put["dr"], put["dn"], put["r"])
    vc.vc_block_norm_backward(put["h"], put["dh"], dr=put["dr"], dn=put["dn"], r=put["r"], dx=put["dx"],
                              dgate=put["dgate"], **kw)
    for k in ("dx", "dh", "dgate"):
        check(put[k], want[k][0], (2 * ROWS + rows * U) * want[k][1], k)
    assert all(c() for c in clean)


@pytest.mark.parametrize("cols", [40, 130, 1040, 3001, 8200, 17000])
def test_block_in_place(env, cols):
    torch, vc, dev = env
    b = Block(torch, dev, 50, cols, "layer", "f32", gates=50, bias=True)
    r, n = check_forward(env, b)
    x, h = b.x.clone(), b.h.clone()
    vc.vc_block_norm_forward(h, r=x, n=h, x=x, pre_bias=b.pre_bias, **b.keywords())
    assert torch.equal(x, r) and torch.equal(h, n)
    dr, dn = rand(torch, dev, 50, cols, seed=1, dtype=torch.float32), rand(torch, dev, 50, cols, seed=2)
    dx, dh, dg = torch.empty_like(dr), torch.empty_like(dn), torch.empty_like(b.gate)
    vc.vc_block_norm_backward(b.h, dh, dr=dr, dn=dn, r=r, dx=dx, dgate=dg, **b.keywords())
    dg2 = torch.empty_like(dg)
    vc.vc_block_norm_backward(b.h, dn, dr=dr, dn=dn, r=r, dx=dr, dgate=dg2, **b.keywords())
    assert torch.equal(dr, dx) and torch.equal(dn, dh) and torch.equal(dg, dg2)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("cols", [96, 1030, 9000])
def test_block_outputs_apart(env, norm, cols):
    """Each output asked for alone has the bits that it has among the others."""
    torch, vc, dev = env
    b = Block(torch, dev, 77, cols, norm, "bf16", gates=7, bias=norm == "layer", act="sigmoid")
    r, n = check_forward(env, b)
    r2, n2 = torch.empty_like(r), torch.empty_like(n)
    vc.vc_block_norm_forward(b.h, r=r2, x=b.x, pre_bias=b.pre_bias, **b.keywords())
    vc.vc_block_norm_forward(b.h, n=n2, x=b.x, pre_bias=b.pre_bias, **b.keywords())
    assert torch.equal(r, r2) and torch.equal(n, n2)
    dr, dn = rand(torch, dev, 77, cols, seed=1), rand(torch, dev, 77, cols, seed=2)
    new = {"dx": lambda: torch.empty_like(dr), "dh": lambda: torch.empty_like(dn),
           "dgate": lambda: torch.empty_like(b.gate)}
    for k in ("dpre", "dpost") + (("dpre_bias", "dpost_bias") if norm == "layer" else ()):
        new[k] = lambda: torch.empty(cols, device=dev)
    out = {k: f() for k, f in new.items()}
    vc.vc_block_norm_backward(b.h, dr=dr, dn=dn, r=r, **out, **b.keywords())
    for k, f in new.items():
        one = f()
        vc.vc_block_norm_backward(b.h, dr=dr, dn=dn, r=r, **{k: one}, **b.keywords())
        assert torch.equal(one, out[k]), k


def test_block_rows_at_the_ends(env):
    """Zero rows (0 / sqrt(eps)), rows with an infinity or a NaN (their own results are
    not numbers, their neighbours' are as before), and large and small values."""
    torch, vc, dev = env
    for cols in (72, 1040, 9000):
        for norm in ("rms", "layer"):
            b = Block(torch, dev, 8, cols, norm, "f32", post=True)
            r0, n0 = check_forward(env, b)
            b.h[2], b.x[2] = 0, 0
            b.h[4, 5], b.x[6, 7] = float("inf"), float("nan")
            r, n = torch.empty_like(r0), torch.empty_like(n0)
            vc.vc_block_norm_forward(b.h, r=r, n=n, x=b.x, **b.keywords())
            assert r[2].eq(0).all() and n[2].eq(0).all()
            assert n[4].isnan().all() and n[6].isnan().all()
            assert r[6].isnan().sum() == 1 and r[6, 7].isnan()
            for k in (0, 1, 3, 5, 7):
                assert torch.equal(r[k], r0[k]) and torch.equal(n[k], n0[k])
            # a row and the same row 2^40 times as large have one hat
            b = Block(torch, dev, 8, cols, norm, "f32", post=False, residual=False, eps=0.0)
            r, n = check_forward(env, b)
            big = torch.empty_like(n)
            b.h *= 2.0 ** 40
            vc.vc_block_norm_forward(b.h, n=big, **b.keywords())
            assert torch.equal(n, big)


def test_block_without_rows(env):
    torch, vc, dev = env
    none, w = torch.empty(0, 40, dtype=torch.bfloat16, device=dev), rand(torch, dev, 40)
    vc.vc_block_norm_forward(none, r=none.clone(), n=none.clone(), pre=w)
    dpre = torch.full((40,), 3.0, device=dev)
    kw = dict(dn=none, r=none.clone(), pre=w, dpre=dpre)
    vc.vc_block_norm_backward(accumulate=True, **kw)
    assert dpre.eq(3).all()
    vc.vc_block_norm_backward(**kw)
    assert dpre.eq(0).all()


@pytest.mark.parametrize("norm,act,gates", [("rms", "sigmoid", 6), ("layer", "none", 18), ("rms", "none", 1)])
def test_block_gradient_against_differences(env, norm, act, gates):
    """Along random directions: <gradient, v> against the central difference of the
    64-bit forward pass, whose error is of second order (1e-8 of its scale)."""
    torch, vc, dev = env
    rows, cols, step = 18, 136, 1e-4
    b = Block(torch, dev, rows, cols, norm, "f32", gates, True, norm == "layer", act, "f32", "f32")
    dr = rand(torch, dev, rows, cols, seed=1, dtype=torch.float32)
    dn = rand(torch, dev, rows, cols, seed=2)
    names = ["x", "h", "gate", "post", "pre"] + (["post_bias", "pre_bias"] if norm == "layer" else [])
    r = b.forward()[0].float()
    out = {"d" + k: torch.empty_like(getattr(b, k)) for k in names}
    vc.vc_block_norm_backward(b.h, dr=dr, dn=dn, r=r, **out, **b.keywords())
    size = {k: v[1] for k, v in b.backward(dr, dn, r).items()}

    def loss():
        want = b.forward()
        return ((want[0] * dr.double()).sum() + (want[2] * dn.double()).sum()).item()

    for k in names:
        at = getattr(b, k)
        v = rand(torch, dev, *at.shape, seed=40, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            setattr(b, k, at.double() + sign * step * v)
            ends.append(loss())
        setattr(b, k, at)
        got = (out["d" + k].double() * v).sum().item()
        scale = (size["d" + k].view(v.shape) * v.abs()).sum().item()
        tol = (2 * ROWS + rows * U) * scale + unit(out["d" + k]) * (
            out["d" + k].double() * v).abs().sum().item() + 1e-6 * scale
        assert abs(got - (ends[0] - ends[1]) / (2 * step)) <= tol, k


# ------------------------------------------------------------------ clipping --

NORM = 33 * U / 2 + 2 * U


def clip_want(torch, grads, max_norm, eps, kind):
    if kind == "max":
        norm = max(g.double().abs().max().item() for g in grads if g.numel())
    else:
        norm = sum(g.double().square().sum().item() for g in grads) ** 0.5
    return norm, min(1.0, max_norm / (norm + eps))


def check_clip(torch, vc, grads, out, max_norm, kind="l2", eps=1e-6):
    norm = torch.empty((), device=grads[0].device)
    before = [g.double().clone() for g in grads]
    want, c = clip_want(torch, grads, max_norm, eps, kind)
    plan = vc.ClipPlan(grads, out)
    plan.norm(norm, kind=kind)
    tol = NORM if kind == "l2" else U
    assert abs(norm.item() - want) <= tol * want, (norm.item(), want)
    assert all(torch.equal(g.double(), o) for g, o in zip(grads, before))
    norm.fill_(-1)
    plan.clip(max_norm, norm, kind=kind, eps=eps)
    assert abs(norm.item() - want) <= tol * want
    for o, g in zip(out if out is not None else grads, before):
        check(o, c * g, (tol + 4 * U) * c * g.abs(), "clipped")
    return c


SETS = [[1], [7], [8], [8192], [8193, 1], [3, 0, 5, 100000], [16385, 1, 2, 3, 4, 5, 6, 7, 9],
        [300] * 50, [1000003, 17], [4096 * 1024, 1024, 1024 * 1024]]


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("types", ["bf16", "f32", "both"])
@pytest.mark.parametrize("sizes", SETS)
def test_clip(env, sizes, types, kind):
    torch, vc, dev = env
    kinds = {"bf16": [torch.bfloat16], "f32": [torch.float32], "both": [torch.float32, torch.bfloat16]}[types]
    grads = [rand(torch, dev, n, seed=i, std=10.0 ** (-i % 4), dtype=kinds[i % len(kinds)])
             for i, n in enumerate(sizes)]
    out = [torch.empty_like(g) for g in grads]
    assert check_clip(torch, vc, grads, out, 0.5, kind) < 1
    assert check_clip(torch, vc, grads, out, 1e6, kind) == 1
    assert all(torch.equal(o, g) for o, g in zip(out, grads))
    copy = [g.clone() for g in grads]
    assert check_clip(torch, vc, grads, None, 1e6, kind) == 1
    assert all(torch.equal(o, g) for o, g in zip(copy, grads))
    check_clip(torch, vc, grads, None, 0.25, kind)
    check_clip(torch, vc, grads, None, 0.0, kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_unaligned_views(env, dtype):
    """Gradients packed without gaps, clipped into others that start elsewhere; what is
    around them stays."""
    torch, vc, dev = env
    kind = dt(torch, dtype)
    sizes = [1, 2, 3, 9, 30, 8191, 5, 20001]
    total = sum(sizes)
    src = rand(torch, dev, total + 16, dtype=kind)
    for shift in range(9):
        dst = torch.full((total + 32,), 7.0, dtype=kind, device=dev)
        at, grads, out = 1, [], []
        for n in sizes:
            grads.append(src[at:at + n])
            out.append(dst[at + shift:at + shift + n])
            at += n
        check_clip(torch, vc, grads, out, 0.5)
        assert dst[:1 + shift].eq(7).all() and dst[1 + shift + total:].eq(7).all()
    keep = src.clone()
    check_clip(torch, vc, grads, None, 0.5)
    assert torch.equal(src[:1], keep[:1]) and torch.equal(src[1 + total:], keep[1 + total:])


@pytest.mark.parametrize("scale", [1e-44, 1e-40, 1e-30, 1e-20, 1e-14, 1e10, 1e18, 1e25, 3e37])
def test_clip_scales(env, scale):
    """Squares that float32 does not hold, beside ones that it does."""
    torch, vc, dev = env
    for dtype in (torch.float32, torch.bfloat16):
        g = (rand(torch, dev, 30000, dtype=torch.float32).clamp(-3, 3) * scale).to(dtype)
        out = [torch.empty_like(g)]
        norm = torch.empty(1, device=dev)
        want, _ = clip_want(torch, [g], 1.0, 1e-6, "l2")
        plan = vc.ClipPlan([g], out)
        plan.clip(1.0, norm)
        if want < 3e38:
            assert abs(norm.item() - want) <= NORM * want + 2.0 ** -149
        else:
            assert norm.isinf().all()
        mixed = [g, rand(torch, dev, 9000, dtype=dtype), torch.zeros(5000, dtype=dtype, device=dev)]
        want, _ = clip_want(torch, mixed, 1.0, 1e-6, "l2")
        vc.ClipPlan(mixed, [torch.empty_like(t) for t in mixed]).norm(norm)
        if want < 3e38:
            assert abs(norm.item() - want) <= NORM * want


def test_clip_small_values_of_every_bit(env):
    """No value is taken for a zero: each bit of a subnormal alone."""
    torch, vc, dev = env
    norm = torch.empty(1, device=dev)
    for dtype, bits, unit_ in ((torch.float32, 23, 2.0 ** -149), (torch.bfloat16, 7, 2.0 ** -133)):
        raw = torch.int32 if dtype == torch.float32 else torch.int16
        for bit in range(bits):
            g = torch.zeros(40, dtype=raw, device=dev)
            g[bit] = 1 << bit
            vc.ClipPlan([g.view(dtype)]).norm(norm)
            assert norm.item() == unit_ * 2 ** bit


def test_clip_not_finite(env):
    torch, vc, dev = env
    norm = torch.empty(1, device=dev)
    for kind in ("l2", "max"):
        for dtype in (torch.float32, torch.bfloat16):
            for at in (0, 3, 20000, 39999):
                g = rand(torch, dev, 40000, dtype=dtype)
                out = [torch.empty_like(g)]
                plan = vc.ClipPlan([g], out)
                g[at] = float("nan")
                plan.clip(1.0, norm, kind=kind)
                assert norm.isnan().all() and out[0].isnan().all()
                g[at] = -float("inf")
                plan.clip(1.0, norm, kind=kind)
                assert norm.item() == float("inf")
                assert out[0][at].isnan() and out[0].nan_to_num(0).eq(0).all()
                plan.clip(float("inf"), norm, kind=kind)
                assert out[0].isnan().all()


def test_clip_of_nothing(env):
    torch, vc, dev = env
    norm = torch.full((), 5.0, device=dev)
    plan = vc.ClipPlan([torch.empty(0, device=dev)])
    plan.norm(norm)
    assert norm.item() == 0
    norm.fill_(5)
    plan(1.0, norm)
    assert norm.item() == 0
    zero = torch.zeros(100, device=dev)
    vc.ClipPlan([zero]).clip(0.0, norm, eps=0.0)  # 0 / 0
    assert norm.item() == 0 and zero.isnan().all()


def test_clip_repeats_and_streams(env):
    """The same bits in every run and on every stream, and a plan dropped while its call
    is under way."""
    torch, vc, dev = env
    grads = [rand(torch, dev, n, seed=i, dtype=torch.float32) for i, n in enumerate((3000001, 5, 70000))]
    norm, out = torch.empty(1, device=dev), [torch.empty_like(g) for g in grads]
    vc.ClipPlan(grads, out).clip(1.0, norm)
    side = torch.cuda.Stream()
    for _ in range(4):
        n2, o2 = torch.empty(1, device=dev), [torch.empty_like(g) for g in grads]
        torch.cuda.synchronize()
        plan = vc.ClipPlan(grads, o2)
        plan.clip(1.0, n2, stream=side)
        del plan
        trash = [torch.full((1 << 18,), 3.0, device=dev) for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(out, o2))
        del trash


def test_refusals(env):
    torch, vc, dev = env
    w, ids = rand(torch, dev, 10, 8), torch.zeros(4, dtype=torch.int64, device=dev)
    y, norm = rand(torch, dev, 4, 8), torch.empty(1, device=dev)
    for call, error in (
            (lambda: vc.vc_embedding_forward(ids.float(), w, y), TypeError),
            (lambda: vc.vc_embedding_forward(ids[::2], w, y[:2]), ValueError),
            (lambda: vc.vc_embedding_forward(ids, w, y[:3]), ValueError),
            (lambda: vc.vc_embedding_forward(ids, w.half(), y), TypeError),
            (lambda: vc.vc_embedding_forward(ids, w[None], y), ValueError),
            (lambda: vc.vc_embedding_forward(ids, w, y, first=-1), ValueError),
            (lambda: vc.vc_embedding_forward(ids, w, w[:4]), vc.VcError),
            (lambda: vc.vc_embedding_backward(y, ids, w, padding=-3), ValueError),
            (lambda: vc.vc_embedding_backward(y, ids, w, workspace=norm), TypeError),
            (lambda: vc.vc_embedding_backward(y[:, :7], ids, w), ValueError),
            (lambda: vc.vc_block_norm_forward(y, n=y.clone()), ValueError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), post_bias=w[0]), ValueError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), post=w[0], post_bias=w[1]), ValueError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), x=y.float()), TypeError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), gate=w[:3]), ValueError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), norm="batch"), ValueError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), gate_act="gelu"), ValueError),
            (lambda: vc.vc_block_norm_forward(y, r=y.clone(), eps=-1.0), ValueError),
            (lambda: vc.vc_block_norm_backward(y, dh=y.clone()), ValueError),
            (lambda: vc.vc_block_norm_backward(y, dn=y, dh=y.clone()), ValueError),
            (lambda: vc.vc_block_norm_backward(y, dr=y, dgate=w[0].clone()), ValueError),
            (lambda: vc.vc_block_norm_backward(None, dr=y, dh=y.clone(), post=w[0]), ValueError),
            (lambda: vc.vc_block_norm_backward(y, dr=y, dpre=w[0].clone(), pre=w[1]), ValueError),
            (lambda: vc.vc_block_norm_backward(y, dr=y, dpost=w[0].clone()), ValueError),
            (lambda: vc.ClipPlan([w, w]), vc.VcError),
            (lambda: vc.ClipPlan([w], [w.float()]), TypeError),
            (lambda: vc.ClipPlan([w], [w[:9]]), ValueError),
            (lambda: vc.ClipPlan([w[:, :4]]), ValueError),
            (lambda: vc.ClipPlan([w], []), ValueError),
            (lambda: vc.ClipPlan([ids]), TypeError),
            (lambda: vc.ClipPlan([w]).clip(-1.0, norm), ValueError),
            (lambda: vc.ClipPlan([w]).clip(float("nan"), norm), ValueError),
            (lambda: vc.ClipPlan([w]).clip(1.0, norm.double()), TypeError),
            (lambda: vc.ClipPlan([w]).clip(1.0, y), TypeError),
            (lambda: vc.ClipPlan([w]).norm(norm.expand(2).contiguous()), ValueError),
            (lambda: vc.ClipPlan([w]).norm(norm, kind="l1"), ValueError)):
        with pytest.raises(error):
            call()


# ------------------------------------------------------------------- far rows --

def test_tables_beyond_32_bit_offsets(env):
    """A table of 2^31 and more elements: its last rows are looked up, and their
    gradients land there and nowhere else."""
    torch, vc, dev = env
    cols = 4096
    rows = 2 ** 31 // cols + 300
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device=dev)
    last = rand(torch, dev, 64, cols)
    w[-64:] = last
    ids = torch.arange(rows - 64, rows, device=dev).flip(0)
    out = torch.empty(64, cols, dtype=torch.bfloat16, device=dev)
    vc.vc_embedding_forward(ids, w, out)
    assert torch.equal(out, last.flip(0))
    w.fill_(3)
    vc.vc_embedding_backward(last, ids, w)
    assert torch.equal(w[-64:], last.flip(0))
    assert not w[:-64].any()
    vc.vc_embedding_backward(last, ids, w, accumulate=True)
    assert torch.equal(w[-64:], last.flip(0) * 2) and not w[:-64].any()


def test_rows_beyond_32_bit_offsets(env):
    torch, vc, dev = env
    cols = 4096
    rows = 2 ** 31 // cols + 40
    h = torch.zeros(rows, cols, dtype=torch.bfloat16, device=dev)
    h[-40:] = rand(torch, dev, 40, cols)
    w = rand(torch, dev, cols, mean=1.0)
    n, few = torch.empty_like(h), torch.empty(40, cols, dtype=torch.bfloat16, device=dev)
    vc.vc_block_norm_forward(h, n=n, pre=w)
    vc.vc_block_norm_forward(h[-40:], n=few, pre=w)
    assert torch.equal(n[-40:], few) and not n[:-40].any()
    dx, dpre = torch.empty_like(h), torch.empty(cols, device=dev)
    fx, fpre = torch.empty_like(few), torch.empty(cols, device=dev)
    vc.vc_block_norm_backward(dr=h, dn=h, r=h, dx=dx, pre=w, dpre=dpre)
    vc.vc_block_norm_backward(dr=h[-40:], dn=h[-40:], r=h[-40:], dx=fx, pre=w, dpre=fpre)
    assert torch.equal(dx[-40:], fx) and not dx[:-40].any()
    assert ((dpre - fpre).abs() <= 80 * U * (h[-40:].double().square().sum(0) * 40)).all()


def test_gradients_beyond_32_bit_offsets(env):
    torch, vc, dev = env
    g = torch.zeros(2 ** 31 + 100, dtype=torch.bfloat16, device=dev)
    g[-100:] = 4
    norm = torch.empty((), device=dev)
    plan = vc.ClipPlan([g])
    plan.clip(10.0, norm, eps=0.0)
    assert norm.item() == 40 and g[-100:].eq(1).all() and not g[:-100].any()


# ------------------------------------------------------- streams and graphs --

def test_replays_of_a_graph_see_new_inputs(env):
    """All operators captured as a run of them is used, replayed on other inputs."""
    torch, vc, dev = env
    rows, cols, vocab = 96, 136, 500
    b = Block(torch, dev, rows, cols, "rms", "bf16", gates=4)
    ids = torch.zeros(rows, dtype=torch.int64, device=dev)
    w, dw = rand(torch, dev, vocab, cols), torch.empty(vocab, cols, device=dev)
    emb, r, n, dx, dh = (torch.empty(rows, cols, dtype=torch.bfloat16, device=dev) for _ in range(5))
    dn, dr = rand(torch, dev, rows, cols, seed=1), rand(torch, dev, rows, cols, seed=2)
    dpre, norm = torch.empty(cols, device=dev), torch.empty(1, device=dev)
    plan = vc.ClipPlan([dw, dpre])
    calls = [vc.prepare_embedding_forward(ids, w, emb),
             vc.prepare_block_norm_forward(b.h, r=r, n=n, x=emb, **b.keywords()),
             vc.prepare_block_norm_backward(b.h, dh, dr=dr, dn=dn, r=r, dx=dx, dpre=dpre, **b.keywords()),
             vc.prepare_embedding_backward(dx, ids, dw)]

    def run():
        for c in calls:
            c()
        plan.clip(0.5, norm)

    outs = [emb, r, n, dx, dh, dpre, dw, norm]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    g = torch.Generator(device=dev).manual_seed(0)
    for _ in range(3):
        ids.copy_(torch.randint(0, vocab, (rows,), generator=g, device=dev))
        b.h.copy_(torch.randn(rows, cols, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.fill_(3)
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(got, outs))


def test_calls_on_other_streams(env):
    """Unprepared calls with workspaces of their own on two streams at a time."""
    torch, vc, dev = env
    rows, cols, vocab = 3000, 520, 900
    dy = rand(torch, dev, rows, cols)
    ids = torch.arange(rows, device=dev) * 17 % vocab
    b = Block(torch, dev, rows, cols, gates=30, act="sigmoid")
    want_dw, want_dg = torch.empty(vocab, cols, device=dev), torch.empty_like(b.gate)
    vc.vc_embedding_backward(dy, ids, want_dw)
    vc.vc_block_norm_backward(b.h, dr=dy, dgate=want_dg, **b.keywords())
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        dw, dg = torch.empty_like(want_dw), torch.empty_like(want_dg)
        outs.append((dw, dg))
        streams[0].wait_stream(torch.cuda.current_stream())
        streams[1].wait_stream(torch.cuda.current_stream())
        vc.vc_embedding_backward(dy, ids, dw, stream=streams[i % 2])
        vc.vc_block_norm_backward(b.h, dr=dy, dgate=dg, stream=streams[1 - i % 2], **b.keywords())
    torch.cuda.synchronize()
    for dw, dg in outs:
        assert torch.equal(dw, want_dw) and torch.equal(dg, want_dg)
