"""Calls of the embedding, block norms and clipping at the ends of what they allow, and beside
each other."""
from __future__ import annotations

import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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


def rand(torch, dev, *shape, seed=0, dtype=None):
    g = torch.Generator(device=dev).manual_seed(2000 + seed)
    return torch.randn(*shape, generator=g, device=dev).to(dtype or torch.bfloat16)


# ---------------------------------------------------------------- embedding --

def test_padding_beyond_64_bits(env):
    """Not taken for the id that its low 64 bits are."""
    torch, vc, dev = env
    ids, dy = torch.tensor([5, 2 ** 63 - 1], device=dev), torch.ones(2, 8, device=dev)
    for padding in (2 ** 63, 2 ** 64, 2 ** 64 + 5):
        dw = torch.full((10, 8), 3.0, device=dev)
        with pytest.raises(ValueError, match="expected an id"):
            vc.vc_embedding_backward(dy, ids, dw, padding=padding)
        assert dw.eq(3).all()
    vc.vc_embedding_backward(dy, ids, dw, padding=2 ** 63 - 1)
    assert dw[5].eq(1).all() and dw.sum().item() == 8


# ------------------------------------------------------------------ clipping --

@pytest.mark.parametrize("values", [500_002_816, 2 ** 31])
@pytest.mark.parametrize("eleven_bits", [1543, 1913])
def test_long_sums_of_equal_squares(env, values, eleven_bits):
    """Equal values round every addition of a plain sum the same way.  A value of 11 bits
    has a square of 22, of which four and sixteen add up exactly in 32 bits; tiles of
    4096 such values are all full.  From there on sums are pairs, each addition of which
    is off by less than 2^-44, and fewer than 2^12 follow one another.  That leaves the rounding
    to 32 bits (u of the sum, half of it in the root) and the root's: 2 u."""
    torch, vc, dev = env
    assert values % 4096 == 0
    value = eleven_bits / 2048
    g = torch.full((values,), value, device=dev)
    norm, want = torch.empty(1, device=dev), value * values ** 0.5
    plan = vc.ClipPlan([g])
    plan.norm(norm)
    assert abs(norm.item() - want) <= 2 * U * want, norm.item() / want - 1
    norm.fill_(0)
    plan.clip(2 * want, norm)
    assert abs(norm.item() - want) <= 2 * U * want
    del plan, g
    torch.cuda.empty_cache()


def test_norm_inside_of_what_is_read_or_written(env):
    """Refused before anything is launched; neighbours are not."""
    torch, vc, dev = env
    flat, other = torch.ones(3000, device=dev), torch.ones(3000, device=dev)
    grads, out = [flat[8:1000], flat[1000:1000], flat[1004:2000]], [other[0:992], other[992:992], other[992:1988]]
    half = torch.ones(100, dtype=torch.bfloat16, device=dev)
    elsewhere, in_place = vc.ClipPlan(grads, out), vc.ClipPlan(grads + [half])
    bad = [flat[k:k + 1] for k in (8, 500, 999, 1004, 1999)]
    for plan, inside in ((elsewhere, bad + [other[k:k + 1] for k in (0, 991, 992, 1987)]),
                         (in_place, bad + [half[98:].view(torch.float32)])):
        for norm in inside:
            for call in (plan.norm, lambda n: plan.clip(1.0, n), lambda n: plan(1.0, n)):
                with pytest.raises(ValueError, match="norm lies in"):
                    call(norm)
    torch.cuda.synchronize()
    assert flat.eq(1).all() and other.eq(1).all() and half.eq(1).all()
    want = (992 + 996) ** 0.5  # (the sum is exact)
    for norm in [flat[k:k + 1] for k in (7, 1000, 1003, 2000)] + [other[1988:1989]]:
        elsewhere.norm(norm)
        assert abs(norm.item() - want) <= 2 * U * want
        norm.fill_(1)
    for norm in (flat[7:8], flat[1000], other[0:1]):
        in_place.norm(norm)
        assert abs(norm.item() - 2088 ** 0.5) <= 2 * U * 2088 ** 0.5
        norm.fill_(1)


# --------------------------------------------------------------- block norms --

@pytest.mark.parametrize("gates", [1, 3, 40])
@pytest.mark.parametrize("act", ["none", "sigmoid"])
@pytest.mark.parametrize("grad", ["bfloat16", "float32"])
@pytest.mark.parametrize("cols", [5, 130, 4100])
def test_gates_without_rows(env, cols, grad, act, gates):
    """A sum over no rows is zero, whatever the gate is, and adds nothing."""
    torch, vc, dev = env
    none, w = torch.empty(0, cols, dtype=torch.bfloat16, device=dev), rand(torch, dev, cols)
    gate = rand(torch, dev, gates, cols)
    gate[0, 0] = float("nan")
    whole = torch.full((gates + 2, cols + 3), 3.0, dtype=getattr(torch, grad), device=dev)
    dgate, dpre = whole[1:-1, :cols], torch.full((cols,), 3.0, device=dev)
    plain = dict(h=none, dr=none, gate=gate, dgate=dgate, gate_act=act)
    both = dict(dn=none, r=none, pre=w, dpre=dpre, **plain)
    for kw in (plain, both):
        vc.vc_block_norm_backward(accumulate=True, **kw)
        assert whole.eq(3).all() and dpre.eq(3).all()
    for kw in (plain, both):
        whole.fill_(3)
        vc.vc_block_norm_backward(**kw)
        assert dgate.eq(0).all()
        assert whole[0].eq(3).all() and whole[-1].eq(3).all() and whole[:, cols:].eq(3).all()
        assert dpre.eq(0 if kw is both else 3).all()


def test_threads_with_other_operands(env):
    """Host threads that call one kernel with more and fewer operands, which need more and
    less shared memory, do not take it from each other."""
    torch, vc, dev = env
    rows, cols = 4, 4096
    f = lambda i: rand(torch, dev, rows, cols, seed=i, dtype=torch.float32)  # noqa: E731
    h, dn, w = rand(torch, dev, rows, cols), rand(torch, dev, rows, cols, seed=1), rand(torch, dev, cols)
    x, gate, r, dr = f(2), f(3), f(4), f(5)

    def calls():
        """Forward and backward with few operands and with many, of one kernel each."""
        o = [torch.empty_like(x) for _ in range(4)]
        b = [torch.empty_like(h) for _ in range(2)]
        few = (vc.prepare_block_norm_forward(h, r=o[0], x=x),
               vc.prepare_block_norm_backward(dr=dr, dn=dn, r=r, dx=o[1], pre=w))
        many = (vc.prepare_block_norm_forward(h, r=o[2], x=x, gate=gate, post=w, pre=w, n=b[0]),
                vc.prepare_block_norm_backward(h, b[1], dr=dr, dn=dn, r=r, dx=o[3], gate=gate, post=w,
                                               pre=w))
        return few, many, o, b

    few, many, want, want_b = calls()
    for c in (*few, *many):
        c()
    torch.cuda.synchronize()
    errors, outs = [], []
    start = threading.Barrier(4)

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                f_, m_, o, b = calls()
                outs.append((o, b))
                mine = m_ if k % 2 else f_
                start.wait(60)
                for _ in range(4000):
                    for c in mine:
                        c()
                for c in (*f_, *m_):
                    c()
            stream.synchronize()
        except Exception as e:  # reported below, on the main thread
            errors.append((k, e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for o, b in outs:
        assert all(torch.equal(p, q) for p, q in zip(o + b, want + want_b))


# ----------------------------------------------------------- failed launches --

def test_a_failed_launch_leaves_no_error_behind(env):
    """A launch that the runtime refuses (here on a stream whose capture has been
    invalidated) is reported by its own call alone, and not again by the next one that asks
    the runtime for its last error.  An error that the program has left itself is not taken
    for a launch's."""
    torch, vc, dev = env
    rt = ctypes.CDLL("libcudart.so.13")
    x, w = rand(torch, dev, 4, 4096), rand(torch, dev, 16, 4096)
    out, y = torch.empty_like(x), torch.empty(4, 16, dtype=torch.bfloat16, device=dev)
    wide = [t.float() for t in (x, x)]
    ids = torch.zeros(4, dtype=torch.int64, device=dev)
    torch.cuda.synchronize()
    raw = ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(raw), 1) == 0
    stream = torch.cuda.ExternalStream(raw.value, device=dev)
    calls = {
        "embedding": vc.prepare_embedding_forward(ids, w, out),
        "block": vc.prepare_block_norm_forward(x, r=wide[0], x=wide[1], pre=w[0], n=out),
        "linear": vc.prepare_linear_forward(x, w, y),
        "all_reduce": lambda stream: vc.vc_all_reduce([x, out], stream=stream),
    }
    torch.cuda.synchronize()
    left = {}
    for name, call in calls.items():
        assert rt.cudaStreamBeginCapture(raw, 2) == 0  # relaxed
        assert rt.cudaStreamSynchronize(raw) != 0      # not allowed: ends the capture's validity
        rt.cudaGetLastError()
        with pytest.raises(vc.VcError):
            call(stream=stream)
        left[name] = rt.cudaPeekAtLastError()
        rt.cudaGetLastError()
        graph = ctypes.c_void_p()
        assert rt.cudaStreamEndCapture(raw, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
    assert rt.cudaStreamDestroy(raw) == 0
    assert not any(left.values()), left
    assert rt.cudaSetDevice(1 << 20) != 0  # leaves its error
    try:
        for name, call in calls.items():
            call(stream=torch.cuda.current_stream())
            left[name] = rt.cudaPeekAtLastError()
    finally:
        rt.cudaGetLastError()
    assert all(left.values()), left
    torch.cuda.synchronize()
