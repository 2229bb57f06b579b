"""The ABI of include/vc_step.h without a GPU: the library exports what the header
declares and rejects bad arguments before it launches anything.

No call reaches a launch: validation fails first, or the launch hook
(VC_TEST_FAIL_LAUNCH) turns the launch into VC_ERR_CUDA.  The fake device pointers are
never dereferenced.
"""
from __future__ import annotations

import ctypes
import re
import subprocess

import pytest

from conftest import ROOT

SUCCESS, INVALID, UNSUPPORTED, ALIAS, CUDA = 0, 1, 2, 3, 4
I32, I64, F32, BF16 = 0, 1, 2, 3
GiB = 1 << 30


@pytest.fixture(scope="module")
def st():
    import __graft_entry__
    __graft_entry__.build()
    from allreduce_reducescatter_allgather_gb300 import step
    step._lib()
    return step


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setenv("VC_TEST_FAIL_LAUNCH", "1")


def mat(st, at, rows, cols, ld=None, dtype=BF16, batch=1):
    ld = cols if ld is None else ld
    return st.Matrix(at, batch, rows, cols, ld, rows * ld, dtype)


def ref(m):
    return ctypes.byref(m) if m is not None else None


def test_library_exports_what_the_header_declares(st):
    text = (ROOT / "include" / "vc_step.h").read_text()
    declared = sorted(set(re.findall(r"^\S.*?\b(vc_\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(st.STEP_EXPORTS)
    from allreduce_reducescatter_allgather_gb300._binding import LIB_PATH
    out = subprocess.run(["nm", "-D", "--defined-only", str(LIB_PATH)], capture_output=True,
                         text=True, check=True).stdout
    assert set(declared) <= set(re.findall(r"\bT (vc_\w+)$", out, flags=re.M))


def test_entry_points_do_not_throw(st):
    """Nothing in the host code allocates or throws."""
    from allreduce_reducescatter_allgather_gb300 import _build
    for stem in ("vc_step_embed", "vc_step_norm", "vc_step_norm_grad", "vc_step_clip"):
        out = subprocess.run(["nm", "-u", "-C", str(_build.BUILD / f"{stem}.o")],
                             capture_output=True, text=True, check=True).stdout
        assert "cudaLaunchKernel" in out
        bad = [line for line in out.splitlines()
               if re.search(r"operator new|throw|__once|_Rb_tree", line)]
        assert not bad, (stem, bad)


# ---------------------------------------------------------------- embedding --

def lookup(st, w, out, ids=5 * GiB, code=I64, tokens=10, first=0):
    return st._lib().vc_embedding_forward(ids, code, tokens, ref(w), first, 1.0, ref(out), None)


def test_embedding_forward_arguments(st):
    w, y = mat(st, GiB, 100, 64), mat(st, 2 * GiB, 10, 64)
    assert lookup(st, w, y) == CUDA  # valid: the hook fires
    assert lookup(st, mat(st, GiB, 100, 64, dtype=F32), y, code=I32) == CUDA
    assert lookup(st, w, mat(st, 2 * GiB, 10, 64, dtype=F32)) == CUDA
    assert lookup(st, None, y) == INVALID
    assert lookup(st, w, None) == INVALID
    assert lookup(st, w, mat(st, 2 * GiB, 11, 64)) == INVALID  # another number of tokens
    assert lookup(st, w, mat(st, 2 * GiB, 10, 63)) == INVALID
    assert lookup(st, w, y, code=F32) == INVALID
    assert lookup(st, w, y, ids=0) == INVALID
    assert lookup(st, w, y, ids=5 * GiB + 4) == INVALID  # int64 on 4 bytes
    assert lookup(st, w, y, ids=5 * GiB + 4, code=I32) == CUDA
    assert lookup(st, w, y, tokens=-1) == INVALID
    assert lookup(st, w, y, first=-1) == INVALID
    assert lookup(st, w, y, first=1 << 63 - 1) in (INVALID, CUDA)
    assert lookup(st, w, y, first=(1 << 62) + 1) == INVALID
    assert lookup(st, mat(st, GiB, 100, 64, batch=2), y) == INVALID
    assert lookup(st, w, mat(st, GiB + 64, 10, 64)) == ALIAS
    assert lookup(st, w, y, ids=2 * GiB) == ALIAS
    assert lookup(st, w, mat(st, 0, 0, 64), ids=0, tokens=0) == SUCCESS
    assert lookup(st, mat(st, 0, 100, 0), mat(st, 0, 10, 0)) == SUCCESS
    assert lookup(st, mat(st, 0, 0, 64), y) == CUDA  # a table without rows: zeros


def scatter(st, dy, dw, ids=5 * GiB, code=I64, first=0, padding=-1, acc=0, ws=8 * GiB, size=GiB):
    return st._lib().vc_embedding_backward(ref(dy), ids, code, first, padding, 1.0, ref(dw), acc,
                                           ws, size, None)


def test_embedding_backward_arguments(st):
    L = st._lib()
    dy, dw = mat(st, GiB, 10, 64), mat(st, 2 * GiB, 100, 64, dtype=F32)
    assert scatter(st, dy, dw) == CUDA
    assert scatter(st, dy, dw, padding=3, acc=1) == CUDA
    assert scatter(st, None, dw) == INVALID
    assert scatter(st, dy, None) == INVALID
    assert scatter(st, dy, mat(st, 2 * GiB, 100, 65)) == INVALID
    assert scatter(st, dy, dw, code=BF16) == INVALID
    assert scatter(st, dy, dw, ids=0) == INVALID
    assert scatter(st, dy, dw, ids=5 * GiB + 2, code=I32) == INVALID
    assert scatter(st, dy, dw, first=-5) == INVALID
    need = L.vc_embedding_backward_workspace(10, 100, 64)
    assert need > 0 and need % 256 == 0
    assert scatter(st, dy, dw, size=need) == CUDA
    assert scatter(st, dy, dw, size=need - 1) == INVALID
    assert scatter(st, dy, dw, ws=8 * GiB + 16) == INVALID
    assert scatter(st, dy, dw, ws=0) == INVALID
    assert scatter(st, dy, dw, ws=2 * GiB) == ALIAS
    assert scatter(st, dy, dw, ws=GiB, size=GiB // 2) == ALIAS
    assert scatter(st, dy, mat(st, GiB, 100, 64)) == ALIAS
    assert scatter(st, dy, dw, ids=2 * GiB + 128) == ALIAS
    assert scatter(st, dy, dw, ids=8 * GiB) == ALIAS
    empty = mat(st, 0, 0, 64)
    assert scatter(st, empty, dw, ids=0, ws=0, size=0) == CUDA  # zeros
    assert scatter(st, empty, dw, ids=0, acc=1, ws=0, size=0) == SUCCESS
    assert scatter(st, dy, mat(st, 0, 0, 64), ws=0, size=0) == SUCCESS
    assert L.vc_embedding_backward_workspace(-1, 100, 64) == 0
    assert L.vc_embedding_backward_workspace(10, 1 << 31, 64) == 0
    assert L.vc_embedding_backward_workspace((1 << 30) + 1, 100, 64) == 0
    assert L.vc_embedding_backward_workspace(1 << 30, 1 << 30, 1 << 22) > 0
    # more columns than a grid covers
    assert L.vc_embedding_backward_workspace(10, 100, (1 << 22) + 1) == 0
    wide = mat(st, 40 * GiB, 1, (1 << 22) + 8)
    assert scatter(st, mat(st, GiB, 1, (1 << 22) + 8), wide) == INVALID


# -------------------------------------------------------------- block norms --

def affine(st, weight=None, bias=None, dtype=BF16):
    return st.Affine(weight, bias, dtype)


def block(st, h, x=None, gate=None, post=None, pre=None, r=None, n=None, norm=0, act=0, eps=1e-6):
    args = st.BlockNorm(norm, act, 1.0, eps)
    return st._lib().vc_block_norm_forward(ref(h), ref(x), ref(gate), ref(post), ref(pre),
                                           ref(args), ref(r), ref(n), None)


def test_block_forward_arguments(st):
    h, x = mat(st, GiB, 12, 64), mat(st, 2 * GiB, 12, 64, dtype=F32)
    r, n = mat(st, 3 * GiB, 12, 64, dtype=F32), mat(st, 4 * GiB, 12, 64)
    post, pre = affine(st, 5 * GiB), affine(st, 6 * GiB, dtype=F32)
    gate = mat(st, 7 * GiB, 4, 64, dtype=F32)
    full = dict(h=h, x=x, gate=gate, post=post, pre=pre, r=r, n=n)
    assert block(st, **full) == CUDA
    assert block(st, **{**full, "norm": 1, "act": 1}) == CUDA
    assert block(st, h, r=r) == CUDA
    assert block(st, h, pre=pre, n=n) == CUDA
    assert block(st, h, x, pre=pre, post=post) == SUCCESS  # nothing asked for
    for change in ({"h": None}, {"h": mat(st, GiB, 12, 64, dtype=F32)},
                   {"n": mat(st, 4 * GiB, 12, 64, dtype=F32)}, {"x": mat(st, 2 * GiB, 12, 64)},
                   {"r": mat(st, 3 * GiB, 12, 64)}, {"x": mat(st, 2 * GiB, 11, 64, dtype=F32)},
                   {"r": mat(st, 3 * GiB, 12, 63, dtype=F32)}, {"n": mat(st, 4 * GiB, 13, 64)},
                   {"pre": None}, {"pre": affine(st)}, {"pre": affine(st, None, 6 * GiB)},
                   {"post": affine(st, None, 5 * GiB)}, {"post": affine(st, 5 * GiB + 1)},
                   {"pre": affine(st, 6 * GiB + 2, dtype=F32)}, {"pre": affine(st, 6 * GiB, dtype=I32)},
                   {"gate": mat(st, 7 * GiB, 5, 64)}, {"gate": mat(st, 7 * GiB, 24, 64)},
                   {"gate": mat(st, 7 * GiB, 4, 32)}, {"gate": mat(st, 0, 0, 64)},
                   {"norm": 2}, {"norm": -1}, {"act": 2}, {"eps": -1.0}, {"eps": float("nan")}):
        assert block(st, **{**full, **change}) == INVALID, change
    # r may be x and n may be h, exactly
    assert block(st, **{**full, "r": x}) == CUDA
    assert block(st, **{**full, "n": h}) == CUDA
    for change in ({"r": mat(st, 2 * GiB + 4, 12, 64, dtype=F32)}, {"n": mat(st, GiB + 2, 12, 64)},
                   {"r": mat(st, 4 * GiB, 12, 64, dtype=F32)}, {"r": mat(st, GiB, 12, 64, dtype=F32)},
                   {"n": mat(st, 2 * GiB, 12, 64)}, {"n": mat(st, 5 * GiB, 12, 64)},
                   {"r": mat(st, 6 * GiB, 12, 64, dtype=F32)}, {"n": mat(st, 7 * GiB, 12, 64)}):
        assert block(st, **{**full, **change}) == ALIAS, change
    assert block(st, mat(st, 0, 0, 64), r=mat(st, 0, 0, 64)) == SUCCESS
    assert block(st, mat(st, 0, 12, 0), r=mat(st, 0, 12, 0)) == SUCCESS


def block_grad(st, post=None, pre=None, dr=None, dn=None, r=None, h=None, gate=None, dx=None,
               dh=None, dgate=None, dpost=None, dpre=None, norm=0, acc=0, ws=20 * GiB, size=GiB):
    args = st.BlockNorm(norm, 0, 1.0, 1e-6)

    def ptr(m):
        return ctypes.pointer(m) if m is not None else None

    ins = st.BlockNormIn(ptr(dr), ptr(dn), ptr(r), ptr(h), ptr(gate))
    outs = st.BlockNormOut(ptr(dx), ptr(dh), ptr(dgate), dpost or affine(st), dpre or affine(st))
    return st._lib().vc_block_norm_backward(ref(ins), ref(post), ref(pre), ref(args), ref(outs),
                                            acc, ws, size, None)


def test_block_backward_arguments(st):
    L = st._lib()
    at = lambda i, **kw: mat(st, i * GiB, 12, 64, **kw)  # noqa: E731
    full = dict(dr=at(1, dtype=F32), dn=at(2), r=at(3, dtype=F32), h=at(4),
                gate=mat(st, 5 * GiB, 4, 64), post=affine(st, 6 * GiB), pre=affine(st, 7 * GiB),
                dx=at(8, dtype=F32), dh=at(9), dgate=mat(st, 10 * GiB, 4, 64, dtype=F32),
                dpost=affine(st, 11 * GiB, dtype=F32), dpre=affine(st, 12 * GiB, dtype=F32))
    assert block_grad(st, **full) == CUDA
    biases = dict(post=affine(st, 6 * GiB, 13 * GiB), dpost=affine(st, 11 * GiB, 14 * GiB),
                  dpre=affine(st, 12 * GiB, 15 * GiB))
    assert block_grad(st, **{**full, **biases, "norm": 1}) == CUDA
    assert block_grad(st, dr=full["dr"], dh=at(9)) == CUDA  # the residual's gradient, narrowed
    assert block_grad(st, dn=at(2), r=at(3), pre=full["pre"], dx=at(8)) == CUDA
    assert block_grad(st, dr=at(1)) == SUCCESS  # nothing asked for
    for change in ({"dr": None, "dn": None}, {"r": None}, {"h": None}, {"pre": None},
                   {"gate": None}, {"dx": at(8)}, {"r": at(3)}, {"dn": at(2, dtype=F32)},
                   {"h": at(4, dtype=F32)}, {"dh": at(9, dtype=F32)},
                   {"dgate": mat(st, 10 * GiB, 5, 64)}, {"gate": mat(st, 5 * GiB, 5, 64)},
                   {"dh": mat(st, 9 * GiB, 13, 64)}, {"dpost": affine(st, 11 * GiB + 2, dtype=F32)},
                   {"dpre": affine(st, 12 * GiB, dtype=I64)}, {"post": None},
                   {"dpost": affine(st, 11 * GiB, 13 * GiB)},  # rms norms have no bias
                   {"post": affine(st, 6 * GiB, 13 * GiB)}, {"norm": 3},
                   {"ws": 20 * GiB + 8}, {"ws": 0}, {"size": 100}):
        assert block_grad(st, **{**full, **change}) == INVALID, change
    # dx may be dr and dh may be dn, exactly
    assert block_grad(st, **{**full, "dx": full["dr"]}) == CUDA
    assert block_grad(st, **{**full, "dh": full["dn"]}) == CUDA
    for change in ({"dx": at(3, dtype=F32)}, {"dh": at(4)}, {"dh": at(3)}, {"dgate": mat(st, 5 * GiB, 4, 64)},
                   {"dpost": affine(st, 6 * GiB)}, {"dpre": affine(st, 11 * GiB + 8, dtype=F32)},
                   {"dx": mat(st, GiB + 4, 12, 64, dtype=F32)}, {"dh": at(8)}, {"ws": 9 * GiB},
                   {"ws": 4 * GiB}):
        assert block_grad(st, **{**full, **change}) == ALIAS, change
    need = L.vc_block_norm_backward_workspace(12, 64, 4)
    assert block_grad(st, **full, size=need) == CUDA
    assert block_grad(st, **full, size=need - 1) == INVALID
    assert L.vc_block_norm_backward_workspace(0, 64, 0) == 0
    assert L.vc_block_norm_backward_workspace(12, -1, 0) == 0
    assert L.vc_block_norm_backward_workspace(12, 64, 13) == 0
    # no rows: the sums are zeros, or stay as they are
    none = dict(dr=mat(st, 0, 0, 64), dn=mat(st, 0, 0, 64), r=mat(st, 0, 0, 64), pre=full["pre"],
                dpre=full["dpre"], ws=0, size=0)
    assert block_grad(st, **none) == CUDA
    assert block_grad(st, **none, acc=1) == SUCCESS


# ------------------------------------------------------------------ clipping --

def plan(st, grads, outs, counts, types=None, room=1000):
    from allreduce_reducescatter_allgather_gb300._binding import pointer_table
    n = len(grads)
    types = [BF16] * n if types is None else types
    count = ctypes.c_int(-1)
    tiles = (st.ClipTile * max(1, room))()
    args = (pointer_table(grads), pointer_table(outs) if outs is not None else None,
            (ctypes.c_size_t * n)(*counts), (ctypes.c_int * n)(*types), n)
    asked = st._lib().vc_clip_plan(*args, None, 0, ctypes.byref(count))
    status = st._lib().vc_clip_plan(*args, tiles, room, ctypes.byref(count))
    return asked, status, count.value, tiles


def test_clip_plan_covers_every_element_once(st):
    per = (1 << 14) // 2
    counts = [1, 0, per, per + 1, 5 * per - 3]
    grads = [GiB + 2, 0, 2 * GiB, 3 * GiB + 6, 4 * GiB]
    outs = [9 * GiB, 0, 7 * GiB, 6 * GiB, 5 * GiB]  # in another order
    asked, status, n, tiles = plan(st, grads, outs, counts)
    assert (asked, status, n) == (SUCCESS, SUCCESS, 1 + 1 + 2 + 5)
    want = [(g + 2 * a, o + 2 * a, min(per, c - a))
            for g, o, c in zip(grads, outs, counts) for a in range(0, c, per)]
    assert [(t.src, t.dst, t.count) for t in tiles[:n]] == want
    assert [t.index for t in tiles[:n]] == list(range(n))
    assert all(t.flags & 1 == 0 for t in tiles[:n])
    _, status, n, tiles = plan(st, [GiB, 2 * GiB], None, [10, 10], [F32, BF16])
    assert status == SUCCESS and [t.flags & 1 for t in tiles[:n]] == [1, 0]
    assert [t.dst for t in tiles[:n]] == [None, None]


def test_clip_plan_refusals(st):
    for args in ((([0], None, [5])), ([GiB + 1], None, [5]), ([GiB], [0], [5]),
                 ([GiB], [2 * GiB + 1], [5]), ([GiB], None, [1 << 47])):
        assert plan(st, *args)[:2] == (INVALID, INVALID), args
    assert plan(st, [GiB], None, [5], [I32])[1] == INVALID
    assert plan(st, [GiB + 2], None, [5], [F32])[1] == INVALID
    asked, status, n, _ = plan(st, [GiB], None, [20000], room=2)
    assert (asked, status, n) == (SUCCESS, INVALID, 3)
    # in place is allowed, any other overlap is not
    assert plan(st, [GiB, 2 * GiB], [GiB, 2 * GiB], [9000, 9000])[1] == SUCCESS
    assert plan(st, [GiB, 2 * GiB], [GiB, 3 * GiB], [9000, 9000])[1] == SUCCESS
    assert plan(st, [GiB, 2 * GiB], [2 * GiB, GiB], [9000, 9000])[1] == ALIAS
    assert plan(st, [GiB], [GiB + 2], [9000])[1] == ALIAS
    assert plan(st, [GiB, 2 * GiB], [3 * GiB, 3 * GiB + 17998], [9000, 9000])[1] == ALIAS
    assert plan(st, [GiB, 2 * GiB], [3 * GiB, 3 * GiB + 18000], [9000, 9000])[1] == SUCCESS
    assert plan(st, [GiB, GiB + 40000], [GiB + 30000, 5 * GiB], [9000, 9000])[1] == ALIAS
    assert plan(st, [GiB, GiB], [GiB, GiB], [9000, 9000])[1] == ALIAS
    assert plan(st, [GiB, GiB], [2 * GiB, 3 * GiB], [9000, 9000])[1] == SUCCESS  # read twice
    assert plan(st, [GiB, GiB], None, [9000, 9000])[1] == SUCCESS


def test_clip_arguments(st):
    L = st._lib()
    need = L.vc_clip_workspace(100)
    assert need % 256 == 0 and L.vc_clip_workspace(-1) == 0

    def clip(tiles=GiB, n=100, kind=0, max_norm=1.0, eps=1e-6, norm=2 * GiB, ws=3 * GiB, size=need):
        a = L.vc_clip_grad_norm(tiles, n, kind, max_norm, eps, norm, ws, size, None)
        b = L.vc_grad_norm(tiles, n, kind, norm, ws, size, None)
        return a, b

    ok, bad, alias = (CUDA, CUDA), (INVALID, INVALID), (ALIAS, ALIAS)
    assert clip() == ok and clip(kind=1) == ok and clip(max_norm=float("inf")) == ok
    assert clip(tiles=0, n=0) == ok  # the norm of nothing
    for change in ({"tiles": 0}, {"n": -1}, {"tiles": GiB + 8}, {"kind": 2}, {"kind": -1}, {"norm": 0},
                   {"norm": 2 * GiB + 2}, {"ws": 0}, {"ws": 3 * GiB + 128}, {"size": need - 1}):
        assert clip(**change) == bad, change
    for change in ({"max_norm": -1.0}, {"max_norm": float("nan")}, {"eps": -1e-6},
                   {"eps": float("nan")}):
        assert clip(**change)[0] == INVALID, change
    assert clip(norm=GiB + 32) == alias
    assert clip(norm=3 * GiB) == alias
    assert clip(ws=GiB) == alias


# ------------------------------------------------------------ tensor checks --

def test_tensors_are_checked(st):
    """The binding names what is wrong before anything reaches the library."""
    import torch
    import allreduce_reducescatter_allgather_gb300 as vc
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        vc.vc_embedding_forward(torch.zeros(4, dtype=torch.int64), t, t)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        vc.vc_embedding_backward(t, torch.zeros(4, dtype=torch.int64), t)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        vc.vc_block_norm_forward(t, r=t)
    with pytest.raises(ValueError, match="dr or dn"):
        vc.vc_block_norm_backward(t)
    with pytest.raises(ValueError, match="at least one"):
        vc.ClipPlan([])
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        vc.ClipPlan([t])
    with pytest.raises(TypeError, match="not a tensor"):
        vc.ClipPlan([3.0])
