"""The operators of a training step between the linear layers and around the
buckets, as measurable cases.

  clip      N = the norm of many gradients taken as one vector (2-norm or the
            largest magnitude);  c = min(1, max_norm / (N + 1e-6));  out = c g
  lookup    y_t = s W[id_t - first], zero where the table has no such row (a
            vocabulary shard)
  scatter   the lookup's gradient: dW_v (+)= s * the sum of dy_t over the tokens t
            of row v, the padding token left out
  block     u = post-norm(h);  r = a x + act(gate) u;  n = pre-norm(r)
  block_grad  its gradient: from dr and dn to dx, dh, dgate and the gradients of
            the norms' weights and biases

`own` false computes them from elementary torch operations in 32 bits, `own`
true through the framework's entry points.
"""
import math
import random

import torch

own = False

CLIP_EPS = 1e-6
NORM_EPS = 1e-6
MAX_CLIP_BYTES = 8 * 4 * 67_000_003
MAX_ROWS_VALUES = 65536 * 4096
MAX_BLOCK_VALUES = 32768 * 4096


def _package():
    import allreduce_reducescatter_allgather_gb300 as vc
    return vc


def listed():
    return [
        # the example's perceptron (256 wide, 1024 hidden), 32-bit gradients:
        # two matrices, two biases; bound by latency
        {"name": "clip_perceptron", "op": "clip", "layout": "perceptron", "tensors": 4,
         "values": 525_568, "dtype": "fp32", "kind": "l2", "clipped": True},
        # the synthetic transformer's 145 16-bit gradients, clipped into the
        # buffers that the optimiser reads
        {"name": "clip_transformer", "op": "clip", "layout": "transformer", "tensors": 145,
         "values": 183_922_688, "dtype": "bf16", "kind": "l2", "clipped": True},
        # eight ranks' 32-bit shards of an odd length, in place, whose norm is
        # below the bound as it mostly is late in training
        {"name": "clip_shards", "op": "clip", "layout": "shards", "tensors": 8,
         "values": 8 * 67_000_003, "dtype": "fp32", "kind": "l2", "clipped": False},
        # eight sequences decoded together through the synthetic transformer's table
        {"name": "lookup_decode", "op": "lookup", "tokens": 8, "rows": 32000, "cols": 1024,
         "first": 0, "weight": "bf16", "out": "bf16", "ids": "int64"},
        # a large micro-batch from a large vocabulary
        {"name": "lookup_large", "op": "lookup", "tokens": 65536, "rows": 131072, "cols": 4096,
         "first": 0, "weight": "bf16", "out": "bf16", "ids": "int32"},
        # one rank's part of a vocabulary, a padded batch, odd widths
        {"name": "scatter_ragged", "op": "scatter", "tokens": 1003, "rows": 5003, "cols": 517,
         "first": 1201, "padded": 0.25, "dy": "bf16", "grad": "fp32", "ids": "int64",
         "accumulate": False},
        # the synthetic transformer's table on a micro-batch, into a bucket view
        {"name": "scatter_transformer", "op": "scatter", "tokens": 16384, "rows": 32000,
         "cols": 1024, "first": 0, "padded": 0.0, "dy": "bf16", "grad": "bf16", "ids": "int64",
         "accumulate": False},
        # a large micro-batch and vocabulary
        {"name": "scatter_large", "op": "scatter", "tokens": 65536, "rows": 131072, "cols": 4096,
         "first": 0, "padded": 0.1, "dy": "bf16", "grad": "bf16", "ids": "int32",
         "accumulate": False},
        # one token between two blocks: latency
        {"name": "block_token", "op": "block", "tokens": 1, "cols": 4096, "norm": "rms",
         "stream": "bf16", "post": True, "bias": False, "gates": 0, "act": "none",
         "scale": 1.0},
        # a large micro-batch, a gate value for every element
        {"name": "block_large", "op": "block", "tokens": 32768, "cols": 4096, "norm": "rms",
         "stream": "bf16", "post": True, "bias": False, "gates": 32768, "act": "sigmoid",
         "scale": 1.0},
        # layer norms with biases, odd widths, one gate vector for each of 17 sequences
        {"name": "block_grad_ragged", "op": "block_grad", "tokens": 1003, "cols": 1021,
         "norm": "layer", "stream": "fp32", "post": True, "bias": True, "gates": 17,
         "act": "none", "scale": 0.75, "grad": "fp32"},
        # a large micro-batch, one gate vector for all of it
        {"name": "block_grad_large", "op": "block_grad", "tokens": 16384, "cols": 8192,
         "norm": "rms", "stream": "bf16", "post": True, "bias": False, "gates": 1, "act": "none",
         "scale": 1.0, "grad": "fp32"},
    ]


def _size(rng, low, high):
    """Log-uniform; half of them whole multiples of 64 where that is possible."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 64 and rng.random() < 0.5:
        v -= v % 64
    return max(low, min(high, v))


def draw(rng):
    while True:
        op = rng.choice(("clip", "lookup", "scatter", "block", "block_grad"))
        if op == "clip":
            layout = rng.choice(("mixed", "shards"))
            tensors = _size(rng, 1, 200 if layout == "mixed" else 16)
            case = {"op": op, "layout": layout, "tensors": tensors,
                    "values": _size(rng, max(1000, 4 * tensors), 8 * 67_000_003),
                    "dtype": rng.choice(("fp32", "bf16", "both")),
                    "kind": "max" if rng.random() < 0.25 else "l2",
                    "clipped": rng.random() < 0.6}
            return case
        if op in ("lookup", "scatter"):
            case = {"op": op, "tokens": _size(rng, 1, 65536), "rows": _size(rng, 1000, 262144),
                    "cols": _size(rng, 64, 8192), "first": 0,
                    "ids": rng.choice(("int32", "int64"))}
            if rng.random() < 0.3:
                case["first"] = rng.randrange(1, 4) * case["rows"]
            if op == "lookup":
                case["weight"] = rng.choice(("fp32", "bf16"))
                case["out"] = rng.choice(("fp32", "bf16"))
            else:
                case["padded"] = rng.choice((0.0, 0.1, 0.5))
                case["dy"] = rng.choice(("bf16", "bf16", "fp32"))
                case["grad"] = rng.choice(("fp32", "bf16"))
                # 16-bit sums over micro-batches would lose what the later ones add
                case["accumulate"] = case["grad"] == "fp32" and rng.random() < 0.4
            if (case["tokens"] * case["cols"] > MAX_ROWS_VALUES
                    or case["rows"] * case["cols"] > 131072 * 4096
                    or work(case)["bytes"] > 1.5 * MAX_ROWS_VALUES * 4):
                continue
            return case
        case = {"op": op, "tokens": _size(rng, 1, 32768), "cols": _size(rng, 64, 16384),
                "norm": rng.choice(("rms", "layer")), "stream": rng.choice(("bf16", "fp32")),
                "post": rng.random() < 0.7, "act": rng.choice(("none", "sigmoid")),
                "scale": rng.choice((1.0, 0.75))}
        case["bias"] = case["norm"] == "layer" and rng.random() < 0.5
        groups = _size(rng, 1, case["tokens"])
        while case["tokens"] % groups:
            groups -= 1
        case["gates"] = rng.choice((0, 1, groups, case["tokens"]))
        if op == "block_grad":
            case["grad"] = rng.choice(("fp32", "bf16"))
        if case["tokens"] * case["cols"] > MAX_BLOCK_VALUES:
            continue
        return case


_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"fp32": 4, "bf16": 2}


# ------------------------------------------------------------------- sizes --

def _gradient_sizes(case):
    """The sizes and types of the gradients, from the case alone."""
    layout, n, total = case["layout"], case["tensors"], case["values"]
    if layout == "perceptron":
        sizes = [1024 * 256, 1024, 256 * 1024, 256]
    elif layout == "transformer":
        h, vocab = 1024, 32000
        sizes = [vocab * h]
        for _ in range(12):
            sizes += [h, h, 3 * h * h, 3 * h, h * h, h, h, h, 4 * h * h, 4 * h, 4 * h * h, h]
    elif layout == "shards":
        sizes = [max(1, total // n)] * n
    else:  # matrices and their biases, of sizes from a few values to most of the sum
        rng = random.Random(f"{n} {total}")
        shares = [math.exp(rng.gauss(0.0, 2.5)) for _ in range(n)]
        scale = total / sum(shares)
        sizes = [max(1, int(s * scale)) for s in shares]
    types = {"fp32": ["fp32"], "bf16": ["bf16"], "both": ["bf16", "fp32"]}[case["dtype"]]
    return [(s, types[i % len(types)]) for i, s in enumerate(sizes)]


def _buffers(case, sizes):
    """How the gradients lie: shards are tensors of their own, others views into one
    buffer for each type, packed as they come or (as in a bucket) each on a
    16-byte boundary.  (buffers' sizes and types, [buffer, offset] of each gradient)"""
    if case["layout"] == "shards":
        return sizes, [(i, 0) for i in range(len(sizes))]
    align = 1 if case["layout"] == "mixed" else 8
    types = sorted({t for _, t in sizes})
    ends, places = [0] * len(types), []
    for n, t in sizes:
        b = types.index(t)
        ends[b] = -(-ends[b] // align) * align
        places.append((b, ends[b]))
        ends[b] += n
    return list(zip(ends, types)), places


def _zipf(case):
    """Cumulative frequencies of the vocabulary's tokens: the k-th most
    frequent one's falls like 1 / (k + 2.7)."""
    n = case["first"] + case["rows"] + (case["rows"] if case["first"] else 0)
    f = 1.0 / (torch.arange(n, dtype=torch.float64) + 2.7)
    return torch.cumsum(f / f.sum(), 0)


def _distinct(case):
    """The expected number of rows that some token has."""
    cdf = _zipf(case)
    p = torch.diff(cdf, prepend=torch.zeros(1, dtype=torch.float64))
    p = p[case["first"]:case["first"] + case["rows"]]
    live = case["tokens"] * (1.0 - case.get("padded", 0.0))
    return int(-torch.expm1(live * torch.log1p(-p)).sum().item()) + 1


def work(case):
    """Inputs read once, outputs written once."""
    op = case["op"]
    if op == "clip":
        each = sum(s * _BYTES[t] for s, t in _gradient_sizes(case))
        n = sum(s for s, _ in _gradient_sizes(case))
        return {"bytes": each * (2 if case["clipped"] else 1),
                "flops": n * (3 if case["clipped"] else 2)}
    if op in ("lookup", "scatter"):
        t, d = case["tokens"], case["cols"]
        ids = t * (8 if case["ids"] == "int64" else 4)
        rows = _distinct(case)
        if op == "lookup":
            return {"bytes": ids + d * (rows * _BYTES[case["weight"]] + t * _BYTES[case["out"]]),
                    "flops": t * d}
        live = int(t * (1.0 - case["padded"]))
        written = 2 * rows if case["accumulate"] else case["rows"]
        return {"bytes": ids + d * (live * _BYTES[case["dy"]] + written * _BYTES[case["grad"]]),
                "flops": live * d}
    t, d, g, s = case["tokens"], case["cols"], case["gates"], _BYTES[case["stream"]]
    weights = (1 + case["post"]) * (1 + case["bias"]) * d
    if op == "block":
        return {"bytes": t * d * (2 + 2 * s + 2) + 2 * g * d + 2 * weights, "flops": 12 * t * d}
    recompute = 2 if case["post"] or g else 0  # h
    grads = (weights + (d if g == 1 else 0)) * _BYTES[case["grad"]] + (2 * g * d if g > 1 else 0)
    return {"bytes": t * d * (3 * s + 2 + recompute + 2) + 2 * g * d + 2 * weights + grads,
            "flops": 30 * t * d}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _tokens(g, case):
    cdf = _zipf(case).to("cuda")
    u = torch.rand(case["tokens"], generator=g, device="cuda", dtype=torch.float64)
    ids = torch.searchsorted(cdf, u).clamp_max(cdf.numel() - 1)
    padding = case["first"]  # the table's first row is the padding token's
    padded = case.get("padded", 0.0)
    if padded:
        drop = torch.rand(case["tokens"], generator=g, device="cuda") < padded
        ids = torch.where(drop, torch.full_like(ids, padding), ids)
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "clip":
        sizes = _gradient_sizes(case)
        buffers, places = _buffers(case, sizes)
        s["buffers"] = [torch.zeros(n, dtype=_DTYPES[t], device="cuda") for n, t in buffers]
        s["out_buffers"] = ([torch.zeros_like(x) for x in s["buffers"]] if case["clipped"]
                            else s["buffers"])
        views = lambda bufs: [bufs[b][at:at + n]  # noqa: E731
                              for (b, at), (n, _) in zip(places, sizes)]
        s["grads"], s["out"] = views(s["buffers"]), views(s["out_buffers"])
        # layers' gradients differ in size by orders of magnitude
        for i, x in enumerate(s["grads"]):
            x.copy_(_normal(g, x.numel(), std=1e-3 * 10.0 ** (-(i % 5) / 2), dtype=x.dtype))
        s["norm"] = torch.empty((), device="cuda")
        total = sum(n for n, _ in sizes)
        size = 1e-3 * (1.0 if case["kind"] == "max" else math.sqrt(total))
        s["max_norm"] = 0.05 * size if case["clipped"] else 100.0 * size
    elif op in ("lookup", "scatter"):
        s["ids"] = _tokens(g, case)
        s["scale"] = math.sqrt(case["cols"])
        t, v, d = case["tokens"], case["rows"], case["cols"]
        if op == "lookup":
            s["weight"] = _normal(g, v, d, std=d ** -0.5, dtype=_DTYPES[case["weight"]])
            s["out"] = torch.empty(t, d, dtype=_DTYPES[case["out"]], device="cuda")
        else:
            s["padding"] = case["first"] if case["padded"] else None
            s["dy"] = _normal(g, t, d, std=1e-2, dtype=_DTYPES[case["dy"]])
            s["dweight"] = _normal(g, v, d, std=1e-2, dtype=_DTYPES[case["grad"]])
    else:
        t, d, stream = case["tokens"], case["cols"], _DTYPES[case["stream"]]
        s["h"] = _normal(g, t, d, std=0.5)
        s["gate"] = _normal(g, case["gates"], d, std=0.5, mean=0.5) if case["gates"] else None
        s["pre"] = _normal(g, d, std=0.1, mean=1.0)
        s["post"] = _normal(g, d, std=0.1, mean=1.0) if case["post"] else None
        s["pre_bias"] = _normal(g, d, std=0.1) if case["bias"] else None
        s["post_bias"] = _normal(g, d, std=0.1) if case["bias"] and case["post"] else None
        # a residual stream of several layers, a few of whose features are large
        column = 1.0 + 20.0 * (torch.rand(d, generator=g, device="cuda") < 0.003)
        x = (torch.randn(t, d, generator=g, device="cuda") * 2.0 * column).to(stream)
        if op == "block":
            s["x"] = x
            s["r"], s["n"] = torch.empty_like(x), torch.empty_like(s["h"])
        else:
            grad = _DTYPES[case["grad"]]
            s["r"] = x
            s["dr"] = _normal(g, t, d, std=1e-2, dtype=stream)
            s["dn"] = _normal(g, t, d, std=1e-2)
            s["dx"], s["dh"] = torch.empty_like(x), torch.empty_like(s["h"])
            for name in ("post", "post_bias", "pre", "pre_bias"):
                s["d" + name] = None if s[name] is None else torch.empty(d, dtype=grad, device="cuda")
            s["dgate"] = None
            if case["gates"]:
                s["dgate"] = torch.empty(case["gates"], d, device="cuda",
                                         dtype=grad if case["gates"] == 1 else torch.bfloat16)
    if own:  # the handle of fixed buffers that a program keeps beside them
        s["call"] = _handle(s)
    return s


def _handle(s):
    vc, case = _package(), s["case"]
    op = case["op"]
    if op == "clip":
        return vc.ClipPlan(s["grads"], s["out"])
    if op == "lookup":
        return vc.prepare_embedding_forward(s["ids"], s["weight"], s["out"], scale=s["scale"],
                                            first=case["first"])
    if op == "scatter":
        return vc.prepare_embedding_backward(s["dy"], s["ids"], s["dweight"], scale=s["scale"],
                                             first=case["first"], padding=s["padding"],
                                             accumulate=case["accumulate"])
    common = {"gate": s["gate"], "post": s["post"], "post_bias": s["post_bias"], "pre": s["pre"],
              "norm": case["norm"], "gate_act": case["act"], "residual_scale": case["scale"],
              "eps": NORM_EPS}
    if op == "block":
        return vc.prepare_block_norm_forward(s["h"], x=s["x"], r=s["r"], n=s["n"],
                                             pre_bias=s["pre_bias"], **common)
    return vc.prepare_block_norm_backward(s["h"], s["dh"], dr=s["dr"], dn=s["dn"], r=s["r"],
                                          dx=s["dx"], dgate=s["dgate"], dpost=s["dpost"],
                                          dpost_bias=s["dpost_bias"], dpre=s["dpre"],
                                          dpre_bias=s["dpre_bias"], **common)


# ---------------------------------------------------------------- plain form --

def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _normalise(v, kind):
    """The normalised rows and what they were divided by, inverted."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = 1.0 / (v.square().mean(-1, keepdim=True) + NORM_EPS).sqrt()
    return v * rstd, rstd


def _normalise_grad(d, hat, rstd, kind):
    d = d - hat * (d * hat).mean(-1, keepdim=True) if kind == "rms" else (
        d - d.mean(-1, keepdim=True) - hat * (d * hat).mean(-1, keepdim=True))
    return d * rstd


def _by_group(v, groups):
    return v.view(groups, -1, v.shape[-1])


def _outputs(s):
    op = s["case"]["op"]
    if op == "clip":
        return {"norm": s["norm"], "grads": s["out_buffers"]}
    if op == "lookup":
        return {"y": s["out"]}
    if op == "scatter":
        return {"dweight": s["dweight"]}
    if op == "block":
        return {"r": s["r"], "n": s["n"]}
    return {k: s[k] for k in ("dx", "dh", "dgate", "dpost", "dpost_bias", "dpre", "dpre_bias")}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "clip":
            s["call"].clip(s["max_norm"], s["norm"], kind=case["kind"], eps=CLIP_EPS)
        else:
            s["call"]()
        return _outputs(s)
    if op == "clip":
        if case["kind"] == "max":
            norm = torch.stack([x.float().abs().max() for x in s["grads"]]).max()
        else:
            norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
        s["norm"].copy_(norm)
        c = (s["max_norm"] / (norm + CLIP_EPS)).clamp_max(1.0)
        for x, y in zip(s["grads"], s["out"]):
            y.copy_(x.float() * c)
    elif op == "lookup":
        row = s["ids"].long() - case["first"]
        inside = (row >= 0) & (row < case["rows"])
        y = s["weight"][row.clamp(0, case["rows"] - 1)].float() * s["scale"]
        s["out"].copy_(y * inside[:, None])
    elif op == "scatter":
        ids = s["ids"].long()
        row = ids - case["first"]
        live = (row >= 0) & (row < case["rows"])
        if s["padding"] is not None:
            live &= ids != s["padding"]
        dw = torch.zeros(case["rows"], case["cols"], device="cuda")
        dw.index_add_(0, row.clamp(0, case["rows"] - 1),
                      s["dy"].float() * (live[:, None] * s["scale"]))
        s["dweight"].copy_(s["dweight"] + dw if case["accumulate"] else dw)
    else:
        _block(s) if op == "block" else _block_grad(s)
    return _outputs(s)


def _block(s):
    case = s["case"]
    u = s["h"].float()
    if s["post"] is not None:
        u = _normalise(u, case["norm"])[0] * s["post"].float()
        if s["post_bias"] is not None:
            u = u + s["post_bias"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        gate = _sigmoid(gate) if case["act"] == "sigmoid" else gate
        u = (_by_group(u, case["gates"]) * gate[:, None]).view_as(u)
    r = case["scale"] * s["x"].float() + u
    s["r"].copy_(r)
    n = _normalise(r, case["norm"])[0] * s["pre"].float()
    if s["pre_bias"] is not None:
        n = n + s["pre_bias"].float()
    s["n"].copy_(n)


def _block_grad(s):
    case = s["case"]
    kind, groups = case["norm"], case["gates"]
    dn = s["dn"].float()
    hat, rstd = _normalise(s["r"].float(), kind)
    s["dpre"].copy_((dn * hat).sum(0))
    if s["dpre_bias"] is not None:
        s["dpre_bias"].copy_(dn.sum(0))
    dr = s["dr"].float() + _normalise_grad(dn * s["pre"].float(), hat, rstd, kind)
    s["dx"].copy_(case["scale"] * dr)
    u = s["h"].float()
    if s["post"] is not None:
        hat, rstd = _normalise(u, kind)
        u = hat * s["post"].float()
        if s["post_bias"] is not None:
            u = u + s["post_bias"].float()
    du = dr
    if s["gate"] is not None:
        gate = s["gate"].float()
        value, slope = gate, torch.ones_like(gate)
        if case["act"] == "sigmoid":
            value = _sigmoid(gate)
            slope = value * (1.0 - value)
        s["dgate"].copy_(_by_group(dr * u, groups).sum(1) * slope)
        du = (_by_group(dr, groups) * value[:, None]).view_as(dr)
    if s["post"] is None:
        s["dh"].copy_(du)
        return
    s["dpost"].copy_((du * hat).sum(0))
    if s["dpost_bias"] is not None:
        s["dpost_bias"].copy_(du.sum(0))
    s["dh"].copy_(_normalise_grad(du * s["post"].float(), hat, rstd, kind))


# --------------------------------------------------- the definitions, 64 bits --

def _exact_norm(v, kind, weight, bias):
    """The norm of rows as a function that torch differentiates."""
    if kind == "layer":
        v = v - v.sum(-1, keepdim=True) / v.shape[-1]
    y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + NORM_EPS) * weight
    return y if bias is None else y + bias


def _exact_block(h, x, gate, post, post_bias, case):
    u = h if post is None else _exact_norm(h, case["norm"], post, post_bias)
    if gate is not None:
        gate = torch.sigmoid(gate) if case["act"] == "sigmoid" else gate
        u = u * gate.repeat_interleave(case["tokens"] // case["gates"], 0)
    return u if x is None else case["scale"] * x + u


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    wide = lambda k: None if s.get(k) is None else s[k].double()  # noqa: E731
    if op == "clip":
        if case["kind"] == "max":
            norm = max(torch.linalg.vector_norm(x.double(), math.inf).item() for x in s["grads"])
        else:
            norm = math.sqrt(math.fsum(torch.linalg.vector_norm(x.double()).item() ** 2
                                       for x in s["grads"]))
        c = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                "grads": [x.double() * c for x in s["buffers"]]}
    if op == "lookup":
        y = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        at = torch.nonzero((s["ids"] >= case["first"])
                           & (s["ids"] < case["first"] + case["rows"]))[:, 0]
        y[at] = s["weight"].double()[s["ids"][at].long() - case["first"]] * s["scale"]
        return {"y": y}
    if op == "scatter":
        keep = (s["ids"] >= case["first"]) & (s["ids"] < case["first"] + case["rows"])
        if s["padding"] is not None:
            keep &= s["ids"] != s["padding"]
        at = torch.nonzero(keep)[:, 0]
        rows, order = torch.sort(s["ids"][at].long() - case["first"], stable=True)
        dw = torch.zeros(case["rows"], case["cols"], dtype=torch.float64, device="cuda")
        dw.index_put_((rows,), s["dy"][at[order]].double() * s["scale"], accumulate=True)
        return {"dweight": dw + s["dweight"].double() if case["accumulate"] else dw}
    if op == "block":
        r = _exact_block(wide("h"), wide("x"), wide("gate"), wide("post"), wide("post_bias"), case)
        return {"r": r, "n": _exact_norm(r, case["norm"], wide("pre"), wide("pre_bias"))}
    # the gradient by differentiating the formulas, rows in pieces: r as stored is
    # where the second norm is differentiated, h where the first one is
    sums = {k: wide(k) for k in ("post", "post_bias", "pre", "pre_bias")}
    total = {k: None if v is None else torch.zeros_like(v) for k, v in sums.items()}
    gates, tokens = case["gates"], case["tokens"]
    dx, dh = [], []
    dgate = None if not gates else torch.zeros(gates, case["cols"], dtype=torch.float64,
                                               device="cuda")
    for lo in range(0, tokens, 4096):
        hi = min(tokens, lo + 4096)
        leaf = {k: None if v is None else v.clone().requires_grad_() for k, v in sums.items()}
        h = s["h"][lo:hi].double().requires_grad_()
        r = s["r"][lo:hi].double().requires_grad_()
        which = None
        gate = None
        if gates:
            which = torch.arange(lo, hi, device="cuda") // (tokens // gates)
            gate = s["gate"][which].double().requires_grad_()
        n = _exact_norm(r, case["norm"], leaf["pre"], leaf["pre_bias"])
        pre = [v for k, v in leaf.items() if k[:3] == "pre" and v is not None]
        first = torch.autograd.grad(n, [r, *pre], s["dn"][lo:hi].double())
        dr = s["dr"][lo:hi].double() + first[0]
        each = dict(case, tokens=hi - lo, gates=hi - lo if gates else 0)
        out = _exact_block(h, None, gate, leaf["post"], leaf["post_bias"], each)
        names = [k for k in ("post", "post_bias") if leaf[k] is not None]
        inputs = [h, *([gate] if gates else []), *[leaf[k] for k in names]]
        second = list(torch.autograd.grad(out, inputs, dr)) if out is not h else [dr]
        dx.append(case["scale"] * dr)
        dh.append(second.pop(0))
        if gates:
            dgate.index_add_(0, which, second.pop(0))
        for k, v in zip(names, second):
            total[k] += v
        for k, v in zip([k for k in ("pre", "pre_bias") if leaf[k] is not None], first[1:]):
            total[k] += v
    return {"dx": torch.cat(dx), "dh": torch.cat(dh), "dgate": dgate, "dpost": total["post"],
            "dpost_bias": total["post_bias"], "dpre": total["pre"],
            "dpre_bias": total["pre_bias"]}
