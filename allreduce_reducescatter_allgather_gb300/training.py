"""The training-step operators of include/vc_train.h on torch tensors: the
linear layer and its gradient, Newton-Schulz orthogonalisation, and the Muon
step.

Argument marshalling only, as for the collectives: tensors in, device
pointers and a CUDA stream out to libvc.so.  Outputs are the caller's tensors;
nothing is returned.  A `workspace` (a CUDA uint8 tensor of the size the
*_workspace functions give, on 16 bytes for the linear layer and on 256 for
the others) may be passed in; without one it comes from
torch's allocator, on the stream of the call.

Matrices are tensors of two dimensions (three for a batch of them) whose last
dimension is contiguous; rows may be further apart than they are long, as in
a slice of a wider tensor.  The linear layer also takes leading dimensions
that can be viewed as one.

The prepare_* functions check fixed buffers once and keep a workspace; every
call of the handle is then one C call.
"""
from __future__ import annotations

import ctypes
import math

from ._binding import _OnDevice, _torch, check_status, lib

ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "gelu": 3, "gelu_tanh": 4, "silu": 5}
# Quintic whose repeated application takes singular values in (0, 1] to about 1.
COEFFICIENTS = (3.4445, -4.7750, 2.0315)

# Every function include/vc_train.h declares.
TRAIN_EXPORTS = ("vc_linear_forward_workspace", "vc_linear_forward",
                 "vc_linear_backward_workspace", "vc_linear_backward",
                 "vc_orthogonalize_workspace", "vc_orthogonalize", "vc_muon_step",
                 "vc_train_timeouts")


class Matrix(ctypes.Structure):
    """vc_matrix_t."""
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_longlong),
                ("rows", ctypes.c_longlong), ("cols", ctypes.c_longlong),
                ("ld", ctypes.c_longlong), ("batch_stride", ctypes.c_longlong),
                ("dtype", ctypes.c_int)]


class NewtonSchulz(ctypes.Structure):
    """vc_newton_schulz_t."""
    _fields_ = [("steps", ctypes.c_int), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("eps", ctypes.c_float)]


class Muon(ctypes.Structure):
    """vc_muon_t."""
    _fields_ = [("lr", ctypes.c_float), ("beta", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("scale", ctypes.c_float),
                ("nesterov", ctypes.c_int), ("ns", NewtonSchulz)]


_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = lib()
        mp, vp, sz, i32 = ctypes.POINTER(Matrix), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.vc_linear_forward_workspace.argtypes = [mp, mp]
        L.vc_linear_forward.argtypes = [mp, mp, vp, mp, mp, mp, i32, vp, sz, vp]
        L.vc_linear_backward_workspace.argtypes = [mp, mp, mp, i32, i32]
        L.vc_linear_backward.argtypes = [mp, mp, mp, mp, i32, mp, mp, vp, i32, i32, vp, sz, vp]
        L.vc_orthogonalize_workspace.argtypes = [ctypes.c_longlong] * 3
        L.vc_orthogonalize.argtypes = [mp, mp, ctypes.POINTER(NewtonSchulz), vp, sz, vp]
        L.vc_muon_step.argtypes = [mp, mp, mp, ctypes.POINTER(Muon), vp, sz, vp]
        L.vc_train_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        for name in TRAIN_EXPORTS:
            getattr(L, name).restype = sz if name.endswith("_workspace") else i32
        _ready = L
    return _ready


# ----------------------------------------------------------------- arguments --

def _tensor(name, t, dtypes, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} is not a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} is not a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected "
                        + " or ".join(str(d) for d in dtypes))


def _code(t):
    return 2 if t.dtype == _torch().float32 else 3


def _matrix(name, t, dtypes, device=None, batched=False):
    """vc_matrix_t of a tensor.  Leading dimensions: one batch dimension
    (batched), or dimensions that can be viewed as rows."""
    _tensor(name, t, dtypes, device)
    if batched:
        if t.dim() not in (2, 3):
            raise ValueError(f"{name} has {t.dim()} dimensions, expected 2 or 3")
        rows, cols = t.shape[-2], t.shape[-1]
        batch = t.shape[0] if t.dim() == 3 else 1
        ld = t.stride(-2)
        skip = t.stride(0) if t.dim() == 3 else 0
    else:
        if t.dim() < 1:
            raise ValueError(f"{name} has no dimensions")
        if t.dim() != 2:
            try:
                t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(
                    math.prod(t.shape[:-1]), t.shape[-1])
            except RuntimeError:
                raise ValueError(f"{name}: leading dimensions cannot be viewed as rows; "
                                 f"make it contiguous first") from None
        batch, skip = 1, 0
        rows, cols = t.shape
        ld = t.stride(0)
    if cols > 1 and t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension is not contiguous")
    if rows > 1 and t.numel() and ld < cols:
        raise ValueError(f"{name}: rows overlap (stride {ld}, {cols} columns)")
    if batch > 1 and t.numel() and skip < (rows - 1) * ld + cols:
        raise ValueError(f"{name}: matrices of the batch overlap or are not in order")
    return Matrix(t.data_ptr(), batch, rows, cols, ld, skip, _code(t))


def _vector(name, t, size, dtypes, device):
    _tensor(name, t, dtypes, device)
    if t.dim() != 1 or t.numel() != size:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({size},)")
    if t.numel() > 1 and not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous")


def _shape(name, m, rows, cols):
    if (m.rows, m.cols) != (rows, cols):
        raise ValueError(f"{name} holds {m.rows} x {m.cols} values, expected {rows} x {cols}")


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"unknown activation {name!r}; use one of {', '.join(ACTIVATIONS)}")
    return code


def _ref(m):
    return ctypes.byref(m) if m is not None else None


def _workspace(workspace, need, device, stream, align):
    """The pointer and size to pass, the tensor to keep until the call has
    been enqueued, and it again where it is new.  A new one is allocated on the
    call's stream, so that torch's allocator gives it out again only behind the
    call."""
    torch = _torch()
    new = workspace is None
    if new:
        if need == 0:
            return ctypes.c_void_p(0), 0, None, None
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _tensor("workspace", workspace, (torch.uint8,), device)
        if not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace holds {workspace.numel()} bytes, {need} are needed")
        if workspace.data_ptr() % align != 0:
            raise ValueError(f"workspace is not aligned to {align} bytes")
    return (ctypes.c_void_p(workspace.data_ptr()), workspace.numel(), workspace,
            workspace if new else None)


class PreparedOperator:
    """A training-step operator on fixed buffers, checked once.  Holds its
    tensors and its workspace; calls of one handle that may overlap on the
    GPU (on different streams) share the workspace and must be ordered by the
    caller.

        forward = prepare_linear_forward(x, weight, out, bias=b, activation="gelu")
        forward()                # on the current stream
        forward(stream=s)        # on another torch stream

    A workspace that the handle has made itself follows it from stream to
    stream: a call on another stream than the preparing one starts behind what
    that one had to do when the workspace was allocated, and the allocator
    gives the workspace to nobody else before the call has ended, even where
    the handle is dropped meanwhile.  (The operands are the caller's to keep.)
    A handle whose call was captured in a graph is kept as long as the graph.
    """

    def __init__(self, fn, args, device, keep, made=None):
        """made: the workspace, where it was allocated for this handle on the
        current stream."""
        self._fn, self._args, self._device, self._keep = fn, args, device, keep
        self._index = device.index if device.index is not None else _torch().cuda.current_device()
        self._made, self._stream, self._allocated = made, None, None
        if made is not None:
            torch = _torch()
            self._stream = torch._C._cuda_getCurrentRawStream(self._index)
            with _OnDevice(self._device):
                if not torch.cuda.is_current_stream_capturing():
                    self._allocated = torch.cuda.Event()
                    self._allocated.record()

    def _move(self, stream, raw):
        """The workspace goes to another stream than that of the last call."""
        torch = _torch()
        with _OnDevice(self._device):
            if stream is None:
                stream = torch.cuda.current_stream()
            with torch.cuda.stream(stream):
                # (a stream under capture cannot wait for work outside of it;
                # torch.cuda.graph waits for all work before it captures)
                capturing = torch.cuda.is_current_stream_capturing()
            if not capturing:
                self._stream = raw
                if self._allocated is not None:
                    stream.wait_event(self._allocated)
            self._made.record_stream(stream)

    def __call__(self, stream=None):
        self._launch(self._fn, self._args, stream)

    def _launch(self, fn, args, stream):
        torch = _torch()
        # (short calls are bound by the host: the common case makes no objects)
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(self._index)
        else:
            raw = stream.cuda_stream
        if self._made is not None and raw != self._stream:
            self._move(stream, raw)
        if torch.cuda.current_device() == self._index:
            status = fn(*args, raw)
        else:
            with _OnDevice(self._device):
                status = fn(*args, raw)
        if status != 0:
            check_status(status)


def _once(stream, fn, args, device, keep, made):
    """One call, whose new workspace was allocated on its own stream."""
    PreparedOperator(fn, args, device, keep)(stream)


# ------------------------------------------------------------- linear layer --

def linear_forward_workspace(x, weight) -> int:
    """Bytes of workspace vc_linear_forward needs (0 where x and weight lie on
    16 bytes)."""
    bf16 = (_torch().bfloat16,)
    return int(_lib().vc_linear_forward_workspace(
        _ref(_matrix("x", x, bf16)), _ref(_matrix("weight", weight, bf16))))


def _forward(x, weight, out, bias, residual, preact, activation, workspace, stream):
    bf16 = (_torch().bfloat16,)
    xm = _matrix("x", x, bf16)
    dev = x.device
    wm = _matrix("weight", weight, bf16, dev)
    if weight.dim() != 2 or wm.cols != xm.cols:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected (N, {xm.cols})")
    om = _matrix("out", out, bf16, dev)
    _shape("out", om, xm.rows, wm.rows)
    rm = pm = None
    if residual is not None:
        rm = _matrix("residual", residual, bf16, dev)
        _shape("residual", rm, xm.rows, wm.rows)
    if preact is not None:
        pm = _matrix("preact", preact, bf16, dev)
        _shape("preact", pm, xm.rows, wm.rows)
    if bias is not None:
        _vector("bias", bias, wm.rows, bf16, dev)
    act = _activation(activation)
    L = _lib()
    need = int(L.vc_linear_forward_workspace(_ref(xm), _ref(wm)))
    ws, size, held, made = _workspace(workspace, need, dev, stream, 16)
    args = (_ref(xm), _ref(wm), ctypes.c_void_p(bias.data_ptr() if bias is not None else 0),
            _ref(rm), _ref(om), _ref(pm), act, ws, size)
    return L.vc_linear_forward, args, dev, (x, weight, out, bias, residual, preact, held,
                                            xm, wm, om, rm, pm), made


def vc_linear_forward(x, weight, out, bias=None, residual=None, preact=None,
                      activation: str = "none", workspace=None, stream=None):
    """out <- act(x W^T + bias) + residual, x [..., K], weight [N, K], out
    [..., N], all bfloat16.  preact receives x W^T + bias (for the backward
    pass).  residual may be out itself."""
    _once(stream, *_forward(x, weight, out, bias, residual, preact, activation, workspace, stream))


def prepare_linear_forward(x, weight, out, bias=None, residual=None, preact=None,
                           activation: str = "none", workspace=None):
    """vc_linear_forward on these buffers."""
    return PreparedOperator(*_forward(x, weight, out, bias, residual, preact, activation,
                                      workspace, None))


def linear_backward_workspace(dy, x, weight, activation: str = "none", dbias: bool = False) -> int:
    """Bytes of workspace vc_linear_backward needs."""
    bf16 = (_torch().bfloat16,)
    return int(_lib().vc_linear_backward_workspace(
        _ref(_matrix("dy", dy, bf16)), _ref(_matrix("x", x, bf16)),
        _ref(_matrix("weight", weight, bf16)), _activation(activation), int(dbias)))


def _backward(dy, x, weight, dx, dweight, dbias, preact, activation, accumulate, workspace,
              stream):
    torch = _torch()
    bf16, grads = (torch.bfloat16,), (torch.bfloat16, torch.float32)
    xm = _matrix("x", x, bf16)
    dev = x.device
    wm = _matrix("weight", weight, bf16, dev)
    if weight.dim() != 2 or wm.cols != xm.cols:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected (N, {xm.cols})")
    ym = _matrix("dy", dy, bf16, dev)
    _shape("dy", ym, xm.rows, wm.rows)
    act = _activation(activation)
    pm = dxm = dwm = None
    if act != 0:
        if preact is None:
            raise ValueError(f"the gradient of {activation} needs preact")
        pm = _matrix("preact", preact, bf16, dev)
        _shape("preact", pm, xm.rows, wm.rows)
    if dx is not None:
        dxm = _matrix("dx", dx, bf16, dev)
        _shape("dx", dxm, xm.rows, xm.cols)
    if dweight is not None:
        dwm = _matrix("dweight", dweight, grads, dev)
        _shape("dweight", dwm, wm.rows, wm.cols)
    if dbias is not None:
        _vector("dbias", dbias, wm.rows, grads, dev)
    L = _lib()
    need = int(L.vc_linear_backward_workspace(_ref(ym), _ref(xm), _ref(wm), act,
                                              int(dbias is not None)))
    ws, size, held, made = _workspace(workspace, need, dev, stream, 16)
    args = (_ref(ym), _ref(xm), _ref(wm), _ref(pm), act, _ref(dxm), _ref(dwm),
            ctypes.c_void_p(dbias.data_ptr() if dbias is not None else 0),
            _code(dbias) if dbias is not None else 3, int(bool(accumulate)), ws, size)
    return L.vc_linear_backward, args, dev, (dy, x, weight, dx, dweight, dbias, preact, held,
                                             ym, xm, wm, pm, dxm, dwm), made


def vc_linear_backward(dy, x, weight, dx=None, dweight=None, dbias=None, preact=None,
                       activation: str = "none", accumulate: bool = False, workspace=None,
                       stream=None):
    """The gradient of vc_linear_forward: dz = dy * act'(preact);
    dx <- dz W, dweight (+)= dz^T x, dbias (+)= column sums of dz.  dweight and
    dbias are bfloat16 or float32 and may be views into a gradient bucket;
    accumulate adds to them.  The residual's gradient is dy itself.  dz is
    rounded to bfloat16 before the products."""
    _once(stream, *_backward(dy, x, weight, dx, dweight, dbias, preact, activation, accumulate,
                             workspace, stream))


def prepare_linear_backward(dy, x, weight, dx=None, dweight=None, dbias=None, preact=None,
                            activation: str = "none", accumulate: bool = False, workspace=None):
    """vc_linear_backward on these buffers."""
    return PreparedOperator(*_backward(dy, x, weight, dx, dweight, dbias, preact, activation,
                                       accumulate, workspace, None))


# ------------------------------------------------------- orthogonalisation --

def orthogonalize_workspace(shape) -> int:
    """Bytes of workspace for tensors of this shape (two or three dimensions),
    for vc_orthogonalize and vc_muon_step."""
    batch = int(shape[0]) if len(shape) == 3 else 1
    return int(_lib().vc_orthogonalize_workspace(batch, int(shape[-2]), int(shape[-1])))


def _newton_schulz(steps, coefficients, eps):
    a, b, c = coefficients
    if not 1 <= int(steps) <= 100:
        raise ValueError(f"steps is {steps}, expected 1 to 100")
    return NewtonSchulz(int(steps), a, b, c, eps)


def _same_shape(name, t, like):
    if t.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")


def _orthogonalize(g, out, steps, coefficients, eps, workspace, stream):
    torch = _torch()
    gm = _matrix("g", g, (torch.bfloat16, torch.float32), batched=True)
    om = _matrix("out", out, (torch.bfloat16,), g.device, batched=True)
    _same_shape("out", out, g)
    ns = _newton_schulz(steps, coefficients, eps)
    need = orthogonalize_workspace(g.shape)
    ws, size, held, made = _workspace(workspace, need, g.device, stream, 256)
    return _lib().vc_orthogonalize, (_ref(gm), _ref(om), _ref(ns), ws, size), g.device, (
        g, out, held, gm, om, ns), made


def vc_orthogonalize(g, out, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7,
                     workspace=None, stream=None):
    """out <- g / (|g|_F + eps) after `steps` passes of
    X <- a X + (b A + c A^2) X, A = X X^T: each matrix of g [rows, cols] or
    [batch, rows, cols] (float32 or bfloat16) brought near the closest matrix
    with orthonormal rows (or columns).  out is bfloat16 and may be g."""
    _once(stream, *_orthogonalize(g, out, steps, coefficients, eps, workspace, stream))


def prepare_orthogonalize(g, out, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7,
                          workspace=None):
    """vc_orthogonalize on these buffers."""
    return PreparedOperator(*_orthogonalize(g, out, steps, coefficients, eps, workspace, None))


class PreparedMuon(PreparedOperator):
    """vc_muon_step on fixed buffers; the learning rate goes with each call."""

    def __init__(self, fn, args, device, keep, made, muon):
        super().__init__(fn, args, device, keep, made)
        self._muon = muon

    def __call__(self, lr: float, stream=None):
        self._muon.lr = lr
        super().__call__(stream)


def _muon(weight, grad, momentum, beta, nesterov, weight_decay, scale, steps, coefficients, eps,
          workspace, stream):
    torch = _torch()
    types = (torch.bfloat16, torch.float32)
    wm = _matrix("weight", weight, types, batched=True)
    gm = _matrix("grad", grad, types, weight.device, batched=True)
    mm = _matrix("momentum", momentum, types, weight.device, batched=True)
    _same_shape("grad", grad, weight)
    _same_shape("momentum", momentum, weight)
    if scale is None:
        scale = 0.2 * math.sqrt(max(weight.shape[-2], weight.shape[-1]))
    args = Muon(0.0, beta, weight_decay, scale, int(bool(nesterov)),
                _newton_schulz(steps, coefficients, eps))
    need = orthogonalize_workspace(weight.shape)
    ws, size, held, made = _workspace(workspace, need, weight.device, stream, 256)
    return (_lib().vc_muon_step, (_ref(wm), _ref(gm), _ref(mm), _ref(args), ws, size),
            weight.device, (weight, grad, momentum, held, wm, gm, mm), made, args)


def vc_muon_step(weight, grad, momentum, lr: float, beta: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, scale: float | None = None, steps: int = 5,
                 coefficients=COEFFICIENTS, eps: float = 1e-7, workspace=None, stream=None):
    """One Muon step in place: momentum <- beta momentum + grad;
    O = orthogonalize(grad + beta momentum, or momentum without nesterov);
    weight <- (1 - lr weight_decay) weight - lr scale O.  weight, grad and
    momentum are float32 or bfloat16, of one shape, [rows, cols] or
    [batch, rows, cols].  scale None: 0.2 sqrt(max(rows, cols)), which gives
    the update 0.2 a value in the root mean square."""
    *call, args = _muon(weight, grad, momentum, beta, nesterov, weight_decay, scale, steps,
                        coefficients, eps, workspace, stream)
    args.lr = lr
    _once(stream, *call)


def prepare_muon_step(weight, grad, momentum, beta: float = 0.95, nesterov: bool = True,
                      weight_decay: float = 0.0, scale: float | None = None, steps: int = 5,
                      coefficients=COEFFICIENTS, eps: float = 1e-7, workspace=None):
    """vc_muon_step on these buffers: handle(lr) does one step."""
    return PreparedMuon(*_muon(weight, grad, momentum, beta, nesterov, weight_decay, scale, steps,
                               coefficients, eps, workspace, None))


def train_timeouts() -> int:
    """Blocks on the current device, of product kernels and of clusters that
    share a row of a block norm, whose bounded waits ran out since the library
    was loaded: 0 unless something is broken.
    Waits for the device."""
    n = ctypes.c_uint(0)
    check_status(_lib().vc_train_timeouts(ctypes.byref(n)))
    return int(n.value)
