"""The training-step operators beside the collectives, as measurable cases.

A data-parallel step computes a linear layer's gradients on every rank,
reduces them in buckets, and turns each reduced matrix into an orthogonalised
update.  Four operators:

  linear    y = act(x W^T + b) + r, keeping the pre-activation z for training
  backward  dz = dy * act'(z);  dx = dz W,  dW (+)= dz^T x,  db (+)= sum dz
  ortho     Newton-Schulz: X_0 = G / (|G|_F + eps),
            X <- a X + (b A + c A^2) X with A = X X^T, five times
  muon      M <- mu M + G;  O = ortho(G + mu M);
            W <- (1 - lr wd) W - lr scale O

`own` false computes them from elementary torch operations in 32 bits, `own`
true through the framework's entry points.
"""
import math

import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
BETA = 0.95
LR = 1e-4
WEIGHT_DECAY = 0.1
ACTIVATIONS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")
MAX_LINEAR_FLOPS = 2 * 8192 * 16384 * 4096
MAX_ORTHO_FLOPS = 5 * (3 * 4096 * 4096 * 16384 + 4096 ** 3)


def _package():
    import allreduce_reducescatter_allgather_gb300 as vc
    return vc


def listed():
    return [
        # one token through the synthetic transformer's MLP (hidden 1024): latency
        {"name": "linear_token", "op": "linear", "m": 1, "n": 4096, "k": 1024,
         "act": "gelu", "bias": True, "residual": False, "preact": False},
        # a small serving batch: bound by reading the weight
        {"name": "linear_batch", "op": "linear", "m": 32, "n": 4096, "k": 4096,
         "act": "silu", "bias": True, "residual": True, "preact": False},
        # a ragged batch through odd widths: rows that no 16-byte vector divides
        {"name": "linear_ragged", "op": "linear", "m": 1003, "n": 2049, "k": 1021,
         "act": "relu2", "bias": True, "residual": True, "preact": True},
        # a large layer in training: the pre-activation is kept
        {"name": "linear_large", "op": "linear", "m": 8192, "n": 16384, "k": 4096,
         "act": "gelu", "bias": True, "residual": False, "preact": True},
        # its gradient on a ragged batch
        {"name": "backward_ragged", "op": "backward", "m": 1003, "n": 1000, "k": 513,
         "act": "silu", "bias": True, "grad": "bf16", "accumulate": False},
        # a projection with no activation whose gradient adds to 32-bit sums
        # over micro-batches
        {"name": "backward_accumulate", "op": "backward", "m": 16384, "n": 1024, "k": 4096,
         "act": "none", "bias": True, "grad": "fp32", "accumulate": True},
        # a large layer's gradient
        {"name": "backward_large", "op": "backward", "m": 16384, "n": 4096, "k": 4096,
         "act": "gelu", "bias": True, "grad": "bf16", "accumulate": False},
        # one small matrix: latency of fifteen dependent products
        {"name": "ortho_small", "op": "ortho", "batch": 1, "rows": 128, "cols": 256,
         "grad": "bf16"},
        # the largest single matrix
        {"name": "ortho_large", "op": "ortho", "batch": 1, "rows": 4096, "cols": 16384,
         "grad": "bf16"},
        # the synthetic transformer's MLP matrix with 32-bit weights, taller than wide
        {"name": "muon_mlp", "op": "muon", "batch": 1, "rows": 4096, "cols": 1024,
         "weight": "fp32", "grad": "fp32", "nesterov": True},
        # odd sizes, several matrices in one call
        {"name": "muon_ragged", "op": "muon", "batch": 3, "rows": 1003, "cols": 517,
         "weight": "bf16", "grad": "bf16", "nesterov": False},
        # eight experts' matrices in one call
        {"name": "muon_experts", "op": "muon", "batch": 8, "rows": 2048, "cols": 8192,
         "weight": "bf16", "grad": "bf16", "nesterov": True},
    ]


def _size(rng, low, high):
    """Log-uniform; half of them whole multiples of 64 where that is possible."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if v >= 64 and rng.random() < 0.5:
        v -= v % 64
    return max(low, min(high, v))


def draw(rng):
    while True:
        op = rng.choice(("linear", "backward", "ortho", "muon"))
        if op in ("linear", "backward"):
            case = {"op": op, "m": _size(rng, 1, 16384), "n": _size(rng, 64, 16384),
                    "k": _size(rng, 64, 16384), "act": rng.choice(ACTIVATIONS),
                    "bias": rng.random() < 0.7}
            if op == "linear":
                case["residual"] = rng.random() < 0.5
                case["preact"] = rng.random() < 0.5
            else:
                # sums in 32 bits go with layers that have no activation: its
                # derivative is rounded to 16 bits before the products
                case["grad"] = rng.choice(("fp32", "bf16")) if case["act"] == "none" else "bf16"
                case["accumulate"] = case["grad"] == "fp32" and rng.random() < 0.5
            if work(case)["flops"] > MAX_LINEAR_FLOPS:
                continue
        else:
            case = {"op": op, "batch": _size(rng, 1, 8), "rows": _size(rng, 16, 8192),
                    "cols": _size(rng, 16, 8192), "grad": rng.choice(("fp32", "bf16"))}
            if op == "muon":
                case["weight"] = rng.choice(("fp32", "bf16"))
                case["nesterov"] = rng.random() < 0.5
            if work(case)["flops"] > MAX_ORTHO_FLOPS:
                continue
        return case


_DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"fp32": 4, "bf16": 2}


def work(case):
    """Inputs read once, outputs written once; a symmetric product has half of
    a full one's multiplications."""
    op = case["op"]
    if op in ("linear", "backward"):
        m, n, k = case["m"], case["n"], case["k"]
        if op == "linear":
            return {"bytes": 2 * (m * k + n * k + m * n * (1 + case["residual"] + case["preact"])
                                  + n * case["bias"]),
                    "flops": 2 * m * n * k}
        g = _BYTES[case["grad"]] * (2 if case["accumulate"] else 1)
        return {"bytes": 2 * (m * n * (1 if case["act"] == "none" else 2) + 2 * m * k + n * k)
                + g * (n * k + n * case["bias"]),
                "flops": 4 * m * n * k}
    r, c = sorted((case["rows"], case["cols"]))
    flops = case["batch"] * STEPS * (3 * r * r * c + r * r * r)
    each = _BYTES[case["grad"]] + (2 if op == "ortho" else 8 + 2 * _BYTES[case["weight"]])
    return {"bytes": case["batch"] * r * c * each, "flops": flops}


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _gradient(g, batch, rows, cols, dtype):
    """A matrix gradient: a sum of fewer outer products than rows or columns,
    of falling weight, and noise."""
    rank = max(1, min(rows, cols) // 4)
    fall = torch.exp(torch.linspace(0.0, -3.0, rank, device="cuda")) / rank ** 0.5
    u = torch.randn(batch, rows, rank, generator=g, device="cuda") * fall
    v = torch.randn(batch, rank, cols, generator=g, device="cuda")
    noise = torch.randn(batch, rows, cols, generator=g, device="cuda")
    return ((u @ v + 0.1 * noise) * 1e-3).to(dtype)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    if op in ("linear", "backward"):
        m, n, k = case["m"], case["n"], case["k"]
        s = {"x": _normal(g, m, k), "weight": _normal(g, n, k, std=k ** -0.5)}
        if op == "linear":
            s["bias"] = _normal(g, n, std=0.1) if case["bias"] else None
            s["residual"] = _normal(g, m, n) if case["residual"] else None
            s["preact"] = torch.empty_like(_normal(g, m, n)) if case["preact"] else None
            s["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        else:
            grad = _DTYPES[case["grad"]]
            s["dy"] = _normal(g, m, n, std=0.01)
            s["preact"] = None if case["act"] == "none" else _normal(g, m, n)
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = _normal(g, n, k, std=0.1, dtype=grad)
            s["dbias"] = _normal(g, n, std=0.1, dtype=grad) if case["bias"] else None
    else:
        shape = (case["batch"], case["rows"], case["cols"])
        s = {"grad": _gradient(g, *shape, _DTYPES[case["grad"]])}
        if op == "ortho":
            s["out"] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        else:
            s["weight"] = _normal(g, *shape, std=0.02, dtype=_DTYPES[case["weight"]])
            s["momentum"] = _gradient(g, *shape, torch.float32) * 4
    s["case"] = case
    if own:  # the handle of fixed buffers that a program keeps beside them
        s["call"] = _handle(s)
    return s


def _handle(s):
    vc, case = _package(), s["case"]
    if case["op"] == "linear":
        return vc.prepare_linear_forward(s["x"], s["weight"], s["out"], bias=s["bias"],
                                         residual=s["residual"], preact=s["preact"],
                                         activation=case["act"])
    if case["op"] == "backward":
        return vc.prepare_linear_backward(s["dy"], s["x"], s["weight"], dx=s["dx"],
                                          dweight=s["dweight"], dbias=s["dbias"],
                                          preact=s["preact"], activation=case["act"],
                                          accumulate=case["accumulate"])
    if case["op"] == "ortho":
        return vc.prepare_orthogonalize(s["grad"], s["out"], steps=STEPS,
                                        coefficients=COEFFICIENTS, eps=EPS)
    return vc.prepare_muon_step(s["weight"], s["grad"], s["momentum"], beta=BETA,
                                nesterov=case["nesterov"], weight_decay=WEIGHT_DECAY,
                                steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)


# ---------------------------------------------------------------- plain form --

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "relu2":
        return z.clamp_min(0.0).square()
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1.0 + torch.exp(-z))


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2.0 * z.clamp_min(0.0)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return (0.5 * (1.0 + t)
                + 0.5 * z * (1.0 - t * t) * math.sqrt(2 / math.pi) * (1.0 + 3 * 0.044715 * z * z))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _orthogonal(g):
    a, b, c = COEFFICIENTS
    tall = g.shape[-2] > g.shape[-1]
    x = g.transpose(-2, -1) if tall else g
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = x @ x.transpose(-2, -1)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(-2, -1) if tall else x


def _scale(rows, cols):
    """The step that has the size of an elementwise optimiser's: 0.2 a value."""
    return 0.2 * math.sqrt(max(rows, cols))


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "muon":
            s["call"](lr=LR)
            return {"weight": s["weight"], "momentum": s["momentum"]}
        s["call"]()
        if op == "linear":
            return {"y": s["out"], "preact": s["preact"]}
        if op == "backward":
            return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
        return {"out": s["out"]}
    if op == "linear":
        z = s["x"].float() @ s["weight"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        s["out"].copy_(y)
        if s["preact"] is not None:
            s["preact"].copy_(z)
        return {"y": s["out"], "preact": s["preact"]}
    if op == "backward":
        dz = s["dy"].float()
        if s["preact"] is not None:
            dz = dz * _act_grad(s["preact"].float(), case["act"])
        s["dx"].copy_(dz @ s["weight"].float())
        dw = dz.t() @ s["x"].float()
        s["dweight"].copy_(s["dweight"] + dw if case["accumulate"] else dw)
        if s["dbias"] is not None:
            db = dz.sum(0)
            s["dbias"].copy_(s["dbias"] + db if case["accumulate"] else db)
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "ortho":
        s["out"].copy_(_orthogonal(s["grad"].float()))
        return {"out": s["out"]}
    grad = s["grad"].float()
    s["momentum"].mul_(BETA).add_(grad)
    update = _orthogonal(grad + BETA * s["momentum"] if case["nesterov"] else s["momentum"])
    step = LR * _scale(case["rows"], case["cols"])
    s["weight"].copy_((1.0 - LR * WEIGHT_DECAY) * s["weight"].float() - step * update)
    return {"weight": s["weight"], "momentum": s["momentum"]}


# --------------------------------------------------- the definitions, 64 bits --

def _exact_orthogonal(g):
    """One matrix: the same polynomial, as a product with the smaller Gram
    matrix on whichever side it is."""
    a, b, c = COEFFICIENTS
    x = g.double()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        if x.shape[0] <= x.shape[1]:
            p = x @ x.t()
            x = (a * eye + p @ (b * eye + c * p)) @ x
        else:
            p = x.t() @ x
            x = x @ (a * eye + p @ (b * eye + c * p))
    return x


def _exact_act(z, act):
    """The value and the derivative."""
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return torch.where(z > 0, z, zero), torch.where(z > 0, one, zero)
    if act == "relu2":
        return torch.where(z > 0, z * z, zero), torch.where(z > 0, 2 * z, zero)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        k = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(k * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * (1 - s) * k * (1 + 0.134145 * z * z)
    s = torch.sigmoid(z)
    return z * s, s + z * s * (1 - s)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "linear":
        z = torch.einsum("mk,nk->mn", s["x"].double(), s["weight"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "preact": z if case["preact"] else None}
    if op == "backward":
        dz = s["dy"].double()
        if s["preact"] is not None:
            dz = dz * _exact_act(s["preact"].double(), case["act"])[1]
        dx = torch.einsum("mn,nk->mk", dz, s["weight"].double())
        dw = torch.einsum("mn,mk->nk", dz, s["x"].double())
        db = torch.einsum("mn->n", dz) if case["bias"] else None
        if case["accumulate"]:
            dw = dw + s["dweight"].double()
            db = None if db is None else db + s["dbias"].double()
        return {"dx": dx, "dweight": dw, "dbias": db}
    if op == "ortho":
        return {"out": torch.stack([_exact_orthogonal(g) for g in s["grad"]])}
    moment = BETA * s["momentum"].double() + s["grad"].double()
    update = BETA * moment + s["grad"].double() if case["nesterov"] else moment
    update = torch.stack([_exact_orthogonal(u) for u in update])
    step = LR * 0.2 * max(case["rows"], case["cols"]) ** 0.5
    weight = s["weight"].double() * (1.0 - LR * WEIGHT_DECAY) - step * update
    return {"weight": weight, "momentum": moment}
