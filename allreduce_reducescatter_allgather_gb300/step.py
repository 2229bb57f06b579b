"""The operators of include/vc_step.h on torch tensors: the embedding lookup
and its gradient, the norms before and after a block with its gate and residual,
and the norm of all gradients with clipping.

The conventions are those of training.py: outputs are the caller's tensors, rows
may be further apart than they are long, a `workspace` (a CUDA uint8 tensor on 256
bytes) may be passed in, and the prepare_* functions check fixed buffers once.
"""
from __future__ import annotations

import bisect
import ctypes
import math

from ._binding import _torch, check_status, pointer_table
from .training import (
    Matrix, PreparedOperator, _code, _lib as _train_lib, _matrix, _once, _ref, _shape, _tensor,
    _vector, _workspace)

NORMS = {"rms": 0, "layer": 1}
GATE_ACTS = {"none": 0, "sigmoid": 1}
GRAD_NORMS = {"l2": 0, "max": 1}

# Every function include/vc_step.h declares.
STEP_EXPORTS = ("vc_embedding_forward", "vc_embedding_backward_workspace", "vc_embedding_backward",
                "vc_block_norm_forward", "vc_block_norm_backward_workspace",
                "vc_block_norm_backward", "vc_clip_plan", "vc_clip_workspace", "vc_grad_norm",
                "vc_clip_grad_norm")


class Affine(ctypes.Structure):
    """vc_affine_t."""
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("dtype", ctypes.c_int)]


class BlockNorm(ctypes.Structure):
    """vc_block_norm_t."""
    _fields_ = [("norm", ctypes.c_int), ("gate_act", ctypes.c_int),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class BlockNormIn(ctypes.Structure):
    """vc_block_norm_in_t."""
    _fields_ = [(k, ctypes.POINTER(Matrix)) for k in ("dr", "dn", "r", "h", "gate")]


class BlockNormOut(ctypes.Structure):
    """vc_block_norm_out_t."""
    _fields_ = [(k, ctypes.POINTER(Matrix)) for k in ("dx", "dh", "dgate")] + [
        ("dpost", Affine), ("dpre", Affine)]


class ClipTile(ctypes.Structure):
    """vc_clip_tile_t."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("count", ctypes.c_int),
                ("flags", ctypes.c_int), ("index", ctypes.c_longlong)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = _train_lib()
        mp, ap, vp = ctypes.POINTER(Matrix), ctypes.POINTER(Affine), ctypes.c_void_p
        sz, i32, i64, f32 = ctypes.c_size_t, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        vpp, np_ = ctypes.POINTER(vp), ctypes.POINTER(BlockNorm)
        L.vc_embedding_forward.argtypes = [vp, i32, i64, mp, i64, f32, mp, vp]
        L.vc_embedding_backward_workspace.argtypes = [i64] * 3
        L.vc_embedding_backward.argtypes = [mp, vp, i32, i64, i64, f32, mp, i32, vp, sz, vp]
        L.vc_block_norm_forward.argtypes = [mp, mp, mp, ap, ap, np_, mp, mp, vp]
        L.vc_block_norm_backward_workspace.argtypes = [i64] * 3
        L.vc_block_norm_backward.argtypes = [ctypes.POINTER(BlockNormIn), ap, ap, np_,
                                             ctypes.POINTER(BlockNormOut), i32, vp, sz, vp]
        L.vc_clip_plan.argtypes = [vpp, vpp, ctypes.POINTER(sz), ctypes.POINTER(i32), i32,
                                   ctypes.POINTER(ClipTile), i32, ctypes.POINTER(i32)]
        L.vc_clip_workspace.argtypes = [i32]
        L.vc_grad_norm.argtypes = [vp, i32, i32, vp, vp, sz, vp]
        L.vc_clip_grad_norm.argtypes = [vp, i32, i32, f32, f32, vp, vp, sz, vp]
        for name in STEP_EXPORTS:
            getattr(L, name).restype = sz if name.endswith("_workspace") else i32
        _ready = L
    return _ready


def _float_types():
    torch = _torch()
    return torch.bfloat16, torch.float32


def _choice(what, name, table):
    code = table.get(name)
    if code is None:
        raise ValueError(f"unknown {what} {name!r}; use one of {', '.join(table)}")
    return code


# --------------------------------------------------------------- embedding --

def _ids(ids, device):
    """Pointer, type code and number of token ids."""
    torch = _torch()
    _tensor("ids", ids, (torch.int32, torch.int64), device)
    if not ids.is_contiguous():
        raise ValueError("ids is not contiguous")
    return ctypes.c_void_p(ids.data_ptr()), 0 if ids.dtype == torch.int32 else 1, ids.numel()


def _table(name, weight, device):
    _tensor(name, weight, _float_types(), device)
    if weight.dim() != 2:
        raise ValueError(f"{name} has {weight.dim()} dimensions, expected 2")
    return _matrix(name, weight, _float_types(), device)


def _first(first):
    if not 0 <= int(first) <= 1 << 62:
        raise ValueError(f"first is {first}, expected 0 to 2^62")
    return int(first)


def _embedding_forward(ids, weight, out, scale, first):
    wm = _table("weight", weight, None)
    dev = weight.device
    ptr, code, tokens = _ids(ids, dev)
    om = _matrix("out", out, _float_types(), dev)
    _shape("out", om, tokens, wm.cols)
    args = (ptr, code, tokens, _ref(wm), _first(first), float(scale), _ref(om))
    return _lib().vc_embedding_forward, args, dev, (ids, weight, out, wm, om), None


def vc_embedding_forward(ids, weight, out, scale: float = 1.0, first: int = 0, stream=None):
    """out[t] <- scale * weight[ids[t] - first] for every token, and zeros where
    weight [V, D] has no such row: it may hold the rows from `first` on of a
    vocabulary that ranks share, whose outputs an AllReduce adds up.  ids
    (int32 or int64, contiguous) of any shape, out [..., D]; weight and out float32
    or bfloat16."""
    _once(stream, *_embedding_forward(ids, weight, out, scale, first))


def prepare_embedding_forward(ids, weight, out, scale: float = 1.0, first: int = 0):
    """vc_embedding_forward on these buffers."""
    return PreparedOperator(*_embedding_forward(ids, weight, out, scale, first))


def embedding_backward_workspace(tokens: int, rows: int, cols: int) -> int:
    """Bytes of workspace vc_embedding_backward needs for this many tokens and a
    table of [rows, cols]."""
    return int(_lib().vc_embedding_backward_workspace(tokens, rows, cols))


def _embedding_backward(dy, ids, dweight, scale, first, padding, accumulate, workspace, stream):
    wm = _table("dweight", dweight, None)
    dev = dweight.device
    ptr, code, tokens = _ids(ids, dev)
    ym = _matrix("dy", dy, _float_types(), dev)
    _shape("dy", ym, tokens, wm.cols)
    if padding is not None and not 0 <= int(padding) < 1 << 63:  # (what an id can be)
        raise ValueError(f"padding is {padding}, expected an id")
    need = embedding_backward_workspace(tokens, wm.rows, wm.cols)
    ws, size, held, made = _workspace(workspace, need, dev, stream, 256)
    args = (_ref(ym), ptr, code, _first(first), -1 if padding is None else int(padding),
            float(scale), _ref(wm), int(bool(accumulate)), ws, size)
    return _lib().vc_embedding_backward, args, dev, (dy, ids, dweight, held, ym, wm), made


def vc_embedding_backward(dy, ids, dweight, scale: float = 1.0, first: int = 0, padding=None,
                          accumulate: bool = False, workspace=None, stream=None):
    """The gradient of vc_embedding_forward: dweight[v] (+)= scale * the sum of dy[t]
    over the tokens with ids[t] - first = v, in 32 bits.  Tokens whose id is
    `padding` are left out.  dweight may be a view into a gradient bucket; rows without a
    token become zero, or with accumulate stay as they are.  dy [..., D] and
    dweight [V, D] float32 or bfloat16."""
    _once(stream, *_embedding_backward(dy, ids, dweight, scale, first, padding, accumulate,
                                       workspace, stream))


def prepare_embedding_backward(dy, ids, dweight, scale: float = 1.0, first: int = 0, padding=None,
                               accumulate: bool = False, workspace=None):
    """vc_embedding_backward on these buffers."""
    return PreparedOperator(*_embedding_backward(dy, ids, dweight, scale, first, padding,
                                                 accumulate, workspace, None))


# -------------------------------------------------------------- block norms --

def _affine(name, weight, bias, cols, device):
    """vc_affine_t of a norm's weight and bias, or of their gradients."""
    there = weight if weight is not None else bias
    if there is None:
        return Affine(None, None, 3)
    for what, t in ((name, weight), (name + "_bias", bias)):
        if t is not None:
            _vector(what, t, cols, _float_types(), device)
            if t.dtype != there.dtype:
                raise TypeError(f"{what} has dtype {t.dtype}, expected {there.dtype}")
    return Affine(weight.data_ptr() if weight is not None else None,
                  bias.data_ptr() if bias is not None else None, _code(there))


def _norm_args(norm, gate_act, residual_scale, eps, biases):
    if not eps >= 0:
        raise ValueError(f"eps is {eps}, expected 0 or more")
    code = _choice("norm", norm, NORMS)
    if code == 0 and any(b is not None for b in biases):
        raise ValueError("rms norms have no bias")
    return BlockNorm(code, _choice("gate_act", gate_act, GATE_ACTS), float(residual_scale),
                     float(eps))


def _gate(name, gate, rows, cols, device):
    if gate is None:
        return None
    gm = _matrix(name, gate, _float_types(), device)
    if gm.cols != cols or gm.rows < 1 or rows % gm.rows:
        raise ValueError(f"{name} holds {gm.rows} x {gm.cols} values, expected {cols} columns and "
                         f"a number of rows that divides {rows}")
    return gm


def _stream_matrix(name, t, like, rows, cols, device):
    """A matrix of the residual stream, whose type all of its matrices share."""
    if t is None:
        return None
    m = _matrix(name, t, _float_types(), device)
    _shape(name, m, rows, cols)
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
    return m


def _half_matrix(name, t, rows, cols, device):
    if t is None:
        return None
    m = _matrix(name, t, (_torch().bfloat16,), device)
    _shape(name, m, rows, cols)
    return m


def _block_forward(h, r, n, x, gate, post, post_bias, pre, pre_bias, norm, gate_act,
                   residual_scale, eps):
    hm = _matrix("h", h, (_torch().bfloat16,))
    dev, rows, cols = h.device, hm.rows, hm.cols
    xm = _stream_matrix("x", x, None, rows, cols, dev)
    rm = _stream_matrix("r", r, x, rows, cols, dev)
    nm = _half_matrix("n", n, rows, cols, dev)
    gm = _gate("gate", gate, rows, cols, dev)
    if n is not None and pre is None:
        raise ValueError("n needs pre, the weight of its norm")
    for name, w, b in (("post", post, post_bias), ("pre", pre, pre_bias)):
        if b is not None and w is None:
            raise ValueError(f"{name}_bias needs {name}")
    pa, qa = _affine("post", post, post_bias, cols, dev), _affine("pre", pre, pre_bias, cols, dev)
    na = _norm_args(norm, gate_act, residual_scale, eps, (post_bias, pre_bias))
    args = (_ref(hm), _ref(xm), _ref(gm), _ref(pa), _ref(qa), _ref(na), _ref(rm), _ref(nm))
    keep = (h, r, n, x, gate, post, post_bias, pre, pre_bias, hm, xm, gm, rm, nm, pa, qa, na)
    return _lib().vc_block_norm_forward, args, dev, keep, None


def vc_block_norm_forward(h, r=None, n=None, x=None, gate=None, post=None, post_bias=None,
                          pre=None, pre_bias=None, norm: str = "rms", gate_act: str = "none",
                          residual_scale: float = 1.0, eps: float = 1e-6, stream=None):
    """The end of one block and the start of the next:

        u = post-norm(h)                               (h itself without post)
        r <- residual_scale * x + gate_act(gate) * u   (u alone without x and gate)
        n <- pre-norm(r)

    h [..., D] is a block's output and n the next one's input (bfloat16), x and r the
    residual stream (float32 or bfloat16).  post and pre are the norms' weights ([D], float32 or
    bfloat16), with biases for norm "layer".  gate [D], [G, D] (one row for each of G
    equal groups of rows, such as sequences) or of h's shape.  r or n may be left out; r
    may be x itself and n may be h itself."""
    _once(stream, *_block_forward(h, r, n, x, gate, post, post_bias, pre, pre_bias, norm, gate_act,
                                  residual_scale, eps))


def prepare_block_norm_forward(h, r=None, n=None, x=None, gate=None, post=None, post_bias=None,
                               pre=None, pre_bias=None, norm: str = "rms", gate_act: str = "none",
                               residual_scale: float = 1.0, eps: float = 1e-6):
    """vc_block_norm_forward on these buffers."""
    return PreparedOperator(*_block_forward(h, r, n, x, gate, post, post_bias, pre, pre_bias, norm,
                                            gate_act, residual_scale, eps))


def block_norm_backward_workspace(rows: int, cols: int, gates: int = 0) -> int:
    """Bytes of workspace vc_block_norm_backward needs for [rows, cols] and a gate of
    `gates` rows (0: none)."""
    return int(_lib().vc_block_norm_backward_workspace(rows, cols, gates))


def _block_backward(h, dh, dr, dn, r, dx, gate, dgate, post, post_bias, dpost, dpost_bias, pre,
                    dpre, dpre_bias, norm, gate_act, residual_scale, eps, accumulate, workspace,
                    stream):
    like = dr if dr is not None else dn
    if like is None:
        raise ValueError("dr or dn is needed")
    shape = _matrix("dr" if dr is not None else "dn", like, _float_types())
    dev, rows, cols = like.device, shape.rows, shape.cols
    if dn is not None and (r is None or pre is None):
        raise ValueError("dn needs r and pre")
    first = dr if dr is not None else r
    drm = _stream_matrix("dr", dr, None, rows, cols, dev)
    rm = _stream_matrix("r", r, first, rows, cols, dev)
    dxm = _stream_matrix("dx", dx, first, rows, cols, dev)
    dnm, hm, dhm = (_half_matrix(k, t, rows, cols, dev)
                    for k, t in (("dn", dn), ("h", h), ("dh", dh)))
    gm = _gate("gate", gate, rows, cols, dev)
    dgm = None
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate needs gate")
        dgm = _matrix("dgate", dgate, _float_types(), dev)
        _shape("dgate", dgm, gm.rows, cols)
    sums = [("post", post, dpost), ("post", post, dpost_bias), ("pre", pre, dpre),
            ("pre", pre, dpre_bias)]
    for name, w, d in sums:
        if d is not None and (w is None or (name == "pre" and dn is None)):
            raise ValueError(f"the gradient of {name} needs {name}" + (" and dn" if name == "pre" else ""))
    if post_bias is not None and post is None:
        raise ValueError("post_bias needs post")
    needs_h = dgate is not None or (post is not None
                                    and any(t is not None for t in (dh, dpost, dpost_bias)))
    if needs_h and h is None:
        raise ValueError("h is needed for the gradients of post and gate")
    pa, qa = _affine("post", post, post_bias, cols, dev), _affine("pre", pre, None, cols, dev)
    na = _norm_args(norm, gate_act, residual_scale, eps, (post_bias, dpost_bias, dpre_bias))

    def pointer(m):
        return ctypes.pointer(m) if m is not None else None

    ins = BlockNormIn(*(pointer(m) for m in (drm, dnm, rm, hm, gm)))
    outs = BlockNormOut(pointer(dxm), pointer(dhm), pointer(dgm),
                        _affine("dpost", dpost, dpost_bias, cols, dev),
                        _affine("dpre", dpre, dpre_bias, cols, dev))
    need = block_norm_backward_workspace(rows, cols, gm.rows if gm is not None else 0)
    ws, size, held, made = _workspace(workspace, need, dev, stream, 256)
    args = (_ref(ins), _ref(pa), _ref(qa), _ref(na), _ref(outs), int(bool(accumulate)), ws, size)
    keep = (h, dh, dr, dn, r, dx, gate, dgate, post, post_bias, dpost, dpost_bias, pre, dpre,
            dpre_bias, held, ins, outs, pa, qa, na, drm, dnm, rm, hm, gm, dxm, dhm, dgm)
    return _lib().vc_block_norm_backward, args, dev, keep, made


def vc_block_norm_backward(h=None, dh=None, dr=None, dn=None, r=None, dx=None, gate=None,
                           dgate=None, post=None, post_bias=None, dpost=None, dpost_bias=None,
                           pre=None, dpre=None, dpre_bias=None, norm: str = "rms",
                           gate_act: str = "none", residual_scale: float = 1.0, eps: float = 1e-6,
                           accumulate: bool = False, workspace=None, stream=None):
    """The gradient of vc_block_norm_forward, from dr (at r, where later blocks added
    to the residual stream; None: 0) and dn (at n; None where there was no n) and what the
    forward pass read (h, gate) and stored (r).  Writes those of dx, dh, dgate, dpost,
    dpost_bias, dpre and dpre_bias that are given.  dgate has gate's shape; where rows share
    a gate row it is the sum over them.  The weights' and biases' gradients and dgate are
    float32 or bfloat16, may be views into a gradient bucket, and accumulate adds to
    them.  dx may be dr itself, and dh may be dn itself."""
    _once(stream, *_block_backward(h, dh, dr, dn, r, dx, gate, dgate, post, post_bias, dpost,
                                   dpost_bias, pre, dpre, dpre_bias, norm, gate_act,
                                   residual_scale, eps, accumulate, workspace, stream))


def prepare_block_norm_backward(h=None, dh=None, dr=None, dn=None, r=None, dx=None, gate=None,
                                dgate=None, post=None, post_bias=None, dpost=None,
                                dpost_bias=None, pre=None, dpre=None, dpre_bias=None,
                                norm: str = "rms", gate_act: str = "none",
                                residual_scale: float = 1.0, eps: float = 1e-6,
                                accumulate: bool = False, workspace=None):
    """vc_block_norm_backward on these buffers."""
    return PreparedOperator(*_block_backward(h, dh, dr, dn, r, dx, gate, dgate, post, post_bias,
                                             dpost, dpost_bias, pre, dpre, dpre_bias, norm,
                                             gate_act, residual_scale, eps, accumulate, workspace,
                                             None))


# ----------------------------------------------------------------- clipping --

class ClipPlan(PreparedOperator):
    """The norm of many gradients taken as one vector, and clipping to it: `grads`
    are contiguous float32 or bfloat16 tensors of one device (matrices and biases, views
    into buckets, the ranks' shards of a ReduceScatter), `out` where the clipped ones
    go (None: in place).  No two gradients share memory where `out` is None, and no two
    outputs do: a weight that is tied is given once.  A call is two launches.  The plan keeps
    the tensors' addresses: make a new one if they change.  Planning (checks, aliasing, a table
    of the tensors' parts of 16 KiB, its copy to the GPU) takes longer than a call: 0.1 ms
    for 2 MB in 4 tensors, 1.4 ms for 368 MB in 145, 5 ms for 2.1 GB, 13 ms where the
    tensors do not follow one another in memory.  So gradients that keep their places from step
    to step (views into buckets) are planned once.
    Calls of one plan that may overlap on the GPU share its workspace and must be
    ordered by the caller.

        plan = ClipPlan(grads)
        plan.clip(1.0, norm)      # norm: a float32 CUDA tensor of one value
        plan.norm(norm)           # the norm alone

    norm lies outside of the gradients and outputs.
    """

    def __init__(self, grads, out=None):
        torch = _torch()
        grads = list(grads)
        if not grads:
            raise ValueError("a plan needs at least one gradient")
        outs = grads if out is None else list(out)
        if len(outs) != len(grads):
            raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
        _tensor("grads[0]", grads[0], _float_types(), None)
        dev = grads[0].device
        for k, (g, o) in enumerate(zip(grads, outs)):
            _tensor(f"grads[{k}]", g, _float_types(), dev)
            _tensor(f"out[{k}]", o, (g.dtype,), dev)
            if not g.is_contiguous() or not o.is_contiguous():
                raise ValueError(f"grads[{k}] or out[{k}] is not contiguous")
            if o.numel() != g.numel():
                raise ValueError(f"out[{k}] holds {o.numel()} elements, expected {g.numel()}")
        n, L = len(grads), _lib()
        counts = (ctypes.c_size_t * n)(*(g.numel() for g in grads))
        types = (ctypes.c_int * n)(*(_code(g) for g in grads))
        ntiles = ctypes.c_int(0)
        tables = (pointer_table([g.data_ptr() for g in grads]),
                  pointer_table([o.data_ptr() for o in outs]), counts, types, n)
        check_status(L.vc_clip_plan(*tables, None, 0, ctypes.byref(ntiles)))
        tiles = (ClipTile * max(1, ntiles.value))()
        check_status(L.vc_clip_plan(*tables, tiles, ntiles.value, ctypes.byref(ntiles)))
        self.ntiles = ntiles.value
        # the table and the workspace are one allocation, which follows the calls' streams
        table = torch.frombuffer(tiles, dtype=torch.uint8)
        at = -(-table.numel() // 256) * 256
        size = int(L.vc_clip_workspace(self.ntiles))
        ws, _, held, made = _workspace(None, at + size, dev, None, 256)
        held[:table.numel()].copy_(table)
        self._table = (ws, self.ntiles)
        self._space = (ctypes.c_void_p(ws.value + at), size)
        # the memory that a call reads and writes, as runs in order that do not overlap
        self._starts, self._ends = [], []
        for lo, hi in sorted({(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                              for t in (*grads, *outs) if t.numel()}):
            if self._ends and lo <= self._ends[-1]:
                self._ends[-1] = max(self._ends[-1], hi)
            else:
                self._starts.append(lo)
                self._ends.append(hi)
        super().__init__(None, (), dev, (grads, outs, held), made)

    def _norm_pointer(self, norm):
        # (before every call: with as few objects as it can do with)
        _tensor("norm", norm, (_torch().float32,), self._device)
        if norm.numel() != 1:
            raise ValueError(f"norm holds {norm.numel()} elements, expected 1")
        at = norm.data_ptr()
        run = bisect.bisect_left(self._starts, at + 4) - 1
        if run >= 0 and self._ends[run] > at:
            raise ValueError("norm lies in a gradient or an output")
        return at

    def norm(self, norm, kind: str = "l2", stream=None):
        """norm <- the 2-norm ("l2") of the gradients, or their largest magnitude
        ("max"); 0 where they are empty."""
        args = (*self._table, _choice("kind", kind, GRAD_NORMS), self._norm_pointer(norm),
                *self._space)
        self._launch(_lib().vc_grad_norm, args, stream)

    def clip(self, max_norm: float, norm, kind: str = "l2", eps: float = 1e-6, stream=None):
        """norm <- the gradients' norm, and every output <- min(1, max_norm /
        (norm + eps)) times its gradient.  Gradients in place are left as they are
        where that is 1.  A norm that is NaN makes all outputs NaN."""
        if not (max_norm >= 0 and eps >= 0) or math.isinf(eps):
            raise ValueError(f"max_norm is {max_norm} and eps {eps}, expected 0 or more")
        args = (*self._table, _choice("kind", kind, GRAD_NORMS), float(max_norm), float(eps),
                self._norm_pointer(norm), *self._space)
        self._launch(_lib().vc_clip_grad_norm, args, stream)

    def __call__(self, max_norm: float, norm, kind: str = "l2", eps: float = 1e-6, stream=None):
        self.clip(max_norm, norm, kind, eps, stream)
