"""The training-step ABI (include/vc_train.h) without a GPU: the library exports
what the header declares, and rejects bad arguments before launching anything.

As in test_abi_cpu.py, no call reaches a launch: validation fails first, or the
launch hook (VC_TEST_FAIL_LAUNCH) turns the launch into VC_ERR_CUDA.  The fake
device pointers are never dereferenced.
"""
from __future__ import annotations

import ctypes
import re
import subprocess
import sys

import pytest

from conftest import ROOT

SUCCESS, INVALID, UNSUPPORTED, ALIAS, CUDA = 0, 1, 2, 3, 4
F32, BF16, I32 = 2, 3, 0
GiB = 1 << 30
NONE, RELU, GELU = 0, 1, 3


@pytest.fixture(scope="module")
def tr():
    import __graft_entry__
    __graft_entry__.build()
    from allreduce_reducescatter_allgather_gb300 import training
    training._lib()
    return training


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    monkeypatch.setenv("VC_TEST_FAIL_LAUNCH", "1")


def mat(tr, at, rows, cols, ld=None, dtype=BF16, batch=1, stride=None):
    ld = cols if ld is None else ld
    return tr.Matrix(at, batch, rows, cols, ld, rows * ld if stride is None else stride, dtype)


def ref(m):
    return ctypes.byref(m) if m is not None else None


def header_functions():
    text = (ROOT / "include" / "vc_train.h").read_text()
    return sorted(set(re.findall(r"^\S.*?\b(vc_\w+)\s*\(", text, flags=re.M)))


def test_library_exports_what_the_header_declares(tr):
    assert header_functions() == sorted(tr.TRAIN_EXPORTS)
    from allreduce_reducescatter_allgather_gb300._binding import LIB_PATH
    out = subprocess.run(["nm", "-D", "--defined-only", str(LIB_PATH)], capture_output=True,
                         text=True, check=True).stdout
    exported = set(re.findall(r"\bT (vc_\w+)$", out, flags=re.M))
    assert set(header_functions()) <= exported


def test_an_edit_of_any_source_is_noticed(tr, monkeypatch, tmp_path):
    """The library counts as old when any file that one of its sources
    includes is newer."""
    import os
    from allreduce_reducescatter_allgather_gb300 import _build
    included = set()
    for f in _build.CSRC.iterdir():
        assert f in _build.dependencies(), f.name
        included |= set(re.findall(r'#include "(.*?)"', f.read_text()))
    assert {"vc_ns_small.cuh", "vc_train.h"} <= included
    assert included <= {f.name for f in _build.dependencies()}
    lib = tmp_path / "lib.so"
    lib.touch()
    monkeypatch.setattr(_build, "LIB", lib)
    newest = max(f.stat().st_mtime for f in _build.dependencies())
    os.utime(lib, (newest, newest))
    assert not _build._stale()
    os.utime(lib, (newest - 1, newest - 1))
    assert _build._stale()


def test_entry_points_do_not_throw(tr):
    """What the training operators are compiled to neither allocates host
    memory nor throws: no exception can leave a C entry point."""
    from allreduce_reducescatter_allgather_gb300 import _build
    for stem in ("vc_gemm", "vc_train_linear", "vc_train_muon"):
        out = subprocess.run(["nm", "-u", "-C", str(_build.BUILD / f"{stem}.o")],
                             capture_output=True, text=True, check=True).stdout
        assert "cudaLaunchKernel" in out or "cudaFuncSetAttribute" in out
        bad = [line.split(" U ")[-1] for line in out.splitlines()
               if re.search(r"operator new|throw|__once|_Rb_tree", line)]
        assert not bad, (stem, bad)


def forward(tr, x, w, y, bias=0, res=None, z=None, act=NONE, ws=0, size=0):
    return tr._lib().vc_linear_forward(ref(x), ref(w), bias, ref(res), ref(y), ref(z), act, ws,
                                       size, None)


def test_forward_shapes_types_and_pointers(tr):
    x, w, y = mat(tr, GiB, 10, 64), mat(tr, 2 * GiB, 24, 64), mat(tr, 3 * GiB, 10, 24)
    assert forward(tr, x, w, y) == CUDA  # valid: the hook fires
    assert forward(tr, None, w, y) == INVALID
    assert forward(tr, x, None, y) == INVALID
    assert forward(tr, x, w, None) == INVALID
    assert forward(tr, mat(tr, 0, 10, 64), w, y) == INVALID          # null
    assert forward(tr, mat(tr, GiB + 1, 10, 64), w, y) == INVALID    # not on an element
    assert forward(tr, mat(tr, GiB, 10, 63), w, y) == INVALID        # K differs
    assert forward(tr, x, w, mat(tr, 3 * GiB, 11, 24)) == INVALID    # M differs
    assert forward(tr, x, w, mat(tr, 3 * GiB, 10, 23)) == INVALID    # N differs
    assert forward(tr, x, w, mat(tr, 3 * GiB, 10, 24, dtype=F32)) == INVALID
    assert forward(tr, mat(tr, GiB, 10, 64, dtype=I32), w, y) == INVALID
    assert forward(tr, mat(tr, GiB, 10, 64, ld=63), w, y) == INVALID  # rows overlap
    assert forward(tr, mat(tr, GiB, 10, 64, batch=2), w, y) == INVALID
    assert forward(tr, mat(tr, GiB, -1, 64), w, y) == INVALID
    assert forward(tr, x, w, y, act=6) == INVALID
    assert forward(tr, x, w, y, act=-1) == INVALID
    assert forward(tr, x, w, y, bias=4 * GiB + 1) == INVALID
    assert forward(tr, x, w, y, res=mat(tr, 5 * GiB, 10, 25)) == INVALID
    assert forward(tr, x, w, y, z=mat(tr, 5 * GiB, 9, 24)) == INVALID
    # sizes beyond the kernels' coordinates, strides whose bytes would wrap
    assert forward(tr, mat(tr, GiB, 1 << 31, 64), w, mat(tr, 3 * GiB, 1 << 31, 24)) == INVALID
    assert forward(tr, mat(tr, GiB, 10, 64, ld=1 << 61), w, y) == INVALID


def test_forward_aliases(tr):
    x, w, y = mat(tr, GiB, 10, 64), mat(tr, 2 * GiB, 24, 64), mat(tr, 3 * GiB, 10, 24)
    assert forward(tr, x, w, mat(tr, GiB, 10, 24)) == ALIAS
    assert forward(tr, x, w, mat(tr, 2 * GiB + 100, 10, 24)) == ALIAS
    assert forward(tr, x, w, y, bias=3 * GiB) == ALIAS
    assert forward(tr, x, w, y, res=y) == CUDA  # in place
    assert forward(tr, x, w, y, res=mat(tr, 3 * GiB + 2, 10, 24)) == ALIAS
    assert forward(tr, x, w, mat(tr, 3 * GiB, 10, 24, ld=32), res=y) == ALIAS  # other rows
    assert forward(tr, x, w, y, z=y) == ALIAS
    assert forward(tr, x, w, y, z=mat(tr, GiB, 10, 24)) == ALIAS


def test_forward_workspace(tr):
    L = tr._lib()
    y = mat(tr, 3 * GiB, 10, 24)
    assert L.vc_linear_forward_workspace(ref(mat(tr, GiB, 10, 64)), ref(mat(tr, 2 * GiB, 24, 64))) == 0
    assert L.vc_linear_forward_workspace(None, ref(mat(tr, 2 * GiB, 24, 64))) == 0
    x, w = mat(tr, GiB, 10, 65), mat(tr, 2 * GiB, 24, 65)  # rows off 16 bytes
    need = L.vc_linear_forward_workspace(ref(x), ref(w))
    assert need >= (10 + 24) * 65 * 2
    assert forward(tr, x, w, y, ws=6 * GiB, size=need) == CUDA
    assert forward(tr, x, w, y, ws=6 * GiB, size=need - 1) == INVALID
    assert forward(tr, x, w, y) == INVALID
    assert forward(tr, x, w, y, ws=6 * GiB + 8, size=need) == INVALID
    assert forward(tr, x, w, y, ws=3 * GiB, size=need) == ALIAS
    # one row's length does not matter, a base off 16 bytes does
    one = mat(tr, GiB, 1, 65)
    assert L.vc_linear_forward_workspace(ref(one), ref(mat(tr, 2 * GiB, 24, 65))) < need
    assert L.vc_linear_forward_workspace(ref(mat(tr, GiB + 2, 10, 64)),
                                         ref(mat(tr, 2 * GiB, 24, 64))) > 0


def test_forward_empty(tr):
    w, y = mat(tr, 2 * GiB, 24, 64), mat(tr, 3 * GiB, 10, 24)
    assert forward(tr, mat(tr, 0, 0, 64), w, mat(tr, 0, 0, 24)) == SUCCESS
    assert forward(tr, mat(tr, GiB, 10, 64), mat(tr, 0, 0, 64), mat(tr, 0, 10, 0)) == SUCCESS
    assert forward(tr, mat(tr, 0, 10, 0), mat(tr, 0, 24, 0), y) == CUDA  # K = 0: y = act(b) + r


def backward(tr, dy, x, w, dx=None, dw=None, db=0, db_type=F32, z=None, act=NONE, acc=0,
             ws=8 * GiB, size=GiB):
    return tr._lib().vc_linear_backward(ref(dy), ref(x), ref(w), ref(z), act, ref(dx), ref(dw), db,
                                        db_type, acc, ws, size, None)


def test_backward_arguments(tr):
    dy, x, w = mat(tr, GiB, 100, 24), mat(tr, 2 * GiB, 100, 64), mat(tr, 3 * GiB, 24, 64)
    dx, dw = mat(tr, 4 * GiB, 100, 64), mat(tr, 5 * GiB, 24, 64, dtype=F32)
    z = mat(tr, 6 * GiB, 100, 24)
    assert backward(tr, dy, x, w, dx, dw, 7 * GiB) == CUDA
    assert backward(tr, dy, x, w, dx) == CUDA
    assert backward(tr, dy, x, w, dw=mat(tr, 5 * GiB, 24, 64)) == CUDA
    assert backward(tr, dy, x, w) == SUCCESS  # nothing asked for
    assert backward(tr, dy, x, w, dx, act=GELU) == INVALID  # needs preact
    assert backward(tr, dy, x, w, dx, act=GELU, z=z) == CUDA
    assert backward(tr, dy, x, w, dx, act=GELU, z=mat(tr, 6 * GiB, 100, 24, dtype=F32)) == INVALID
    assert backward(tr, dy, x, w, mat(tr, 4 * GiB, 100, 64, dtype=F32)) == INVALID
    assert backward(tr, dy, x, w, mat(tr, 4 * GiB, 100, 63)) == INVALID
    assert backward(tr, dy, x, w, dw=mat(tr, 5 * GiB, 64, 24)) == INVALID
    assert backward(tr, mat(tr, GiB, 99, 24), x, w, dx) == INVALID
    assert backward(tr, dy, x, w, dx, db=7 * GiB, db_type=I32) == INVALID
    assert backward(tr, dy, x, w, dx, db=7 * GiB + 2) == INVALID
    assert backward(tr, dy, x, w, dx, db=7 * GiB + 2, db_type=BF16) == CUDA
    assert backward(tr, dy, x, w, dx, act=9) == INVALID


def test_backward_aliases_and_workspace(tr):
    dy, x, w = mat(tr, GiB, 100, 24), mat(tr, 2 * GiB, 100, 64), mat(tr, 3 * GiB, 24, 64)
    z = mat(tr, 6 * GiB, 100, 24)
    assert backward(tr, dy, x, w, mat(tr, 2 * GiB, 100, 64)) == ALIAS  # dx over x
    assert backward(tr, dy, x, w, mat(tr, GiB, 100, 64)) == ALIAS
    assert backward(tr, dy, x, w, dw=mat(tr, 3 * GiB, 24, 64)) == ALIAS
    assert backward(tr, dy, x, w, mat(tr, 4 * GiB, 100, 64),
                    mat(tr, 4 * GiB + 16, 24, 64)) == ALIAS
    assert backward(tr, dy, x, w, db=6 * GiB, act=GELU, z=z) == ALIAS
    L = tr._lib()
    need = L.vc_linear_backward_workspace(ref(dy), ref(x), ref(w), GELU, 1)
    assert need >= 100 * 24 * 2 + 24 * 4
    dx = mat(tr, 4 * GiB, 100, 64)
    assert backward(tr, dy, x, w, dx, db=7 * GiB, act=GELU, z=z, size=need) == CUDA
    assert backward(tr, dy, x, w, dx, db=7 * GiB, act=GELU, z=z, size=need - 1) == INVALID
    assert backward(tr, dy, x, w, dx, db=7 * GiB, act=GELU, z=z, ws=2 * GiB, size=need) == ALIAS
    # without an activation, a bias or odd rows nothing is needed
    assert L.vc_linear_backward_workspace(ref(dy), ref(x), ref(w), NONE, 0) == 0
    assert backward(tr, dy, x, w, dx, ws=0, size=0) == CUDA
    # small batches keep dz's rounding remainder: a second plane
    few = [mat(tr, GiB, 64, 24), mat(tr, 2 * GiB, 64, 64)]
    more = [mat(tr, GiB, 65, 24), mat(tr, 2 * GiB, 65, 64)]
    assert (L.vc_linear_backward_workspace(ref(few[0]), ref(few[1]), ref(w), GELU, 0)
            > L.vc_linear_backward_workspace(ref(more[0]), ref(more[1]), ref(w), GELU, 0))


# Every side may be 0, with every output.  (In a process of its own: a division
# by zero ends it.)
EMPTY_SIDES = """
import ctypes, itertools, sys
sys.path.insert(0, sys.argv[1])
from allreduce_reducescatter_allgather_gb300 import training as tr
L, GiB = tr._lib(), 1 << 30
mat = lambda at, r, c, t=3: ctypes.byref(tr.Matrix(at * GiB, 1, r, c, c, 0, t))
for m, n, k, act, db in itertools.product((0, 10), (0, 24), (0, 64), (0, 3), (0, 1)):
    dy, x, w, z = mat(1, m, n), mat(2, m, k), mat(3, n, k), mat(4, m, n)
    need = L.vc_linear_backward_workspace(dy, x, w, act, db)
    assert need < GiB, need
    status = L.vc_linear_backward(dy, x, w, z, act, mat(5, m, k), mat(6, n, k, 2), 7 * GiB * db, 2,
                                  0, 8 * GiB, GiB, None)
    assert status == (0 if n == 0 and m * k == 0 else 4), (m, n, k, act, db, status)
print("done")
"""


def test_backward_of_empty_sides(tr):
    out = subprocess.run([sys.executable, "-c", EMPTY_SIDES, str(ROOT)], capture_output=True,
                         text=True)
    assert out.returncode == 0 and out.stdout.strip() == "done", (out.returncode, out.stderr)


def ns(tr, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7):
    return tr.NewtonSchulz(steps, a, b, c, eps)


def ortho(tr, g, out, n=None, ws=8 * GiB, size=4 * GiB):
    return tr._lib().vc_orthogonalize(ref(g), ref(out), ref(n or ns(tr)), ws, size, None)


def test_orthogonalize_arguments(tr):
    g, out = mat(tr, GiB, 100, 64, dtype=F32), mat(tr, 2 * GiB, 100, 64)
    assert ortho(tr, g, out) == CUDA
    assert ortho(tr, mat(tr, GiB, 100, 64), out) == CUDA
    assert ortho(tr, out, out) == CUDA  # in place
    assert ortho(tr, mat(tr, 2 * GiB + 2, 100, 64), out) == ALIAS
    assert ortho(tr, mat(tr, GiB, 100, 64, dtype=I32), out) == INVALID
    assert ortho(tr, g, mat(tr, 2 * GiB, 100, 64, dtype=F32)) == INVALID
    assert ortho(tr, g, mat(tr, 2 * GiB, 64, 100)) == INVALID
    assert ortho(tr, g, out, ns(tr, steps=0)) == INVALID
    assert ortho(tr, g, out, ns(tr, steps=101)) == INVALID
    assert ortho(tr, g, out, ns(tr, a=float("nan"))) == INVALID
    assert ortho(tr, g, out, ns(tr, eps=-1.0)) == INVALID
    assert ortho(tr, g, out, ws=0) == INVALID
    assert ortho(tr, g, out, ws=8 * GiB + 16) == INVALID
    assert ortho(tr, g, out, ws=GiB) == ALIAS
    need = tr._lib().vc_orthogonalize_workspace(1, 100, 64)
    assert need > 0
    assert ortho(tr, g, out, size=need) == CUDA
    assert ortho(tr, g, out, size=need - 1) == INVALID
    assert ortho(tr, mat(tr, GiB, 100, 64, batch=3, stride=100 * 64 - 1),
                 mat(tr, 2 * GiB, 100, 64, batch=3)) == INVALID  # matrices overlap
    for shape in ((0, 100, 64), (1, 0, 64), (1, 100, 0)):
        assert tr._lib().vc_orthogonalize_workspace(*shape) == 0
        assert ortho(tr, mat(tr, 0, shape[1], shape[2], batch=shape[0]),
                     mat(tr, 0, shape[1], shape[2], batch=shape[0]), ws=0, size=0) == SUCCESS
    assert tr._lib().vc_orthogonalize_workspace(-1, 4, 4) == 0
    assert tr._lib().vc_orthogonalize_workspace(1, 1 << 25, 4) == 0


def muon(tr, w, g, m, ws=8 * GiB, size=4 * GiB, **kw):
    args = tr.Muon(kw.get("lr", 0.1), kw.get("beta", 0.9), kw.get("wd", 0.0), kw.get("scale", 1.0),
                   1, kw.get("ns", ns(tr)))
    return tr._lib().vc_muon_step(ref(w), ref(g), ref(m), ctypes.byref(args), ws, size, None)


def test_muon_arguments(tr):
    w, g, m = (mat(tr, (1 + i) * GiB, 100, 64, dtype=F32) for i in range(3))
    assert muon(tr, w, g, m) == CUDA
    assert muon(tr, mat(tr, GiB, 100, 64), mat(tr, 2 * GiB, 100, 64), m) == CUDA
    assert muon(tr, w, w, m) == ALIAS
    assert muon(tr, w, g, g) == ALIAS
    assert muon(tr, w, g, m, ws=2 * GiB) == ALIAS
    assert muon(tr, w, mat(tr, 2 * GiB, 64, 100, dtype=F32), m) == INVALID
    assert muon(tr, w, g, mat(tr, 3 * GiB, 100, 64, dtype=I32)) == INVALID
    assert muon(tr, w, g, None) == INVALID
    for bad in ({"lr": float("inf")}, {"beta": float("nan")}, {"wd": float("nan")},
                {"scale": float("inf")}, {"ns": ns(tr, steps=0)}):
        assert muon(tr, w, g, m, **bad) == INVALID
    assert tr._lib().vc_muon_step(ref(w), ref(g), ref(m), None, 8 * GiB, GiB, None) == INVALID


def test_timeouts_reports_errors(tr):
    assert tr._lib().vc_train_timeouts(None) == INVALID
    n = ctypes.c_uint(7)
    assert tr._lib().vc_train_timeouts(ctypes.byref(n)) == CUDA


def test_binding_refuses_host_tensors(tr):
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tr.vc_linear_forward(t, t, t)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tr.vc_orthogonalize(t, t)
    with pytest.raises(TypeError, match="not a tensor"):
        tr.vc_muon_step([1.0], t, t, lr=0.1)


def test_slices_that_interleave_are_no_aliases(tr):
    """Columns 0..63 and 64..87 of rows of 100 values share no element; one
    column more, from either side, does."""
    def x(first, n, ld=100, rows=10):
        return mat(tr, GiB + 2 * first, rows, n, ld=ld)
    def fwd(*a, ws=8 * GiB, size=GiB, **kw):
        return forward(tr, *a, ws=ws, size=size, **kw)
    w = mat(tr, 2 * GiB, 24, 64)
    assert fwd(x(0, 64), w, x(64, 24)) == CUDA
    assert fwd(x(36, 64), w, x(12, 24)) == CUDA
    assert fwd(x(36, 64), w, x(100, 24)) == CUDA       # from the next row on
    assert fwd(x(0, 64), w, x(63, 24)) == ALIAS
    assert fwd(x(36, 64), w, x(13, 24)) == ALIAS
    assert fwd(x(36, 64), w, x(77, 24)) == ALIAS       # reaches into the next row
    assert fwd(x(0, 64), w, x(64, 24, ld=101)) == ALIAS  # rows drift over each other
    assert fwd(x(0, 64), w, x(64, 24, ld=200)) == ALIAS
    # one row, or a vector, between the rows of a matrix
    one = mat(tr, GiB + 2 * 164, 1, 24, ld=0)
    assert fwd(mat(tr, 3 * GiB, 1, 64), w, one, res=one) == CUDA
    assert fwd(x(0, 64), w, mat(tr, 4 * GiB, 10, 24), bias=GiB + 2 * 164) == CUDA
    assert fwd(mat(tr, 3 * GiB, 10, 64), w, x(0, 24), bias=GiB + 2 * 164) == CUDA
    assert fwd(mat(tr, 3 * GiB, 10, 64), w, x(0, 24), bias=GiB + 2 * 176) == CUDA
    assert fwd(mat(tr, 3 * GiB, 10, 64), w, x(0, 24), bias=GiB + 2 * 177) == ALIAS
    assert fwd(mat(tr, 3 * GiB, 10, 64), w, x(0, 24), bias=GiB + 2 * 123) == ALIAS
    # a workspace may not reach into a matrix's rows
    odd, wo = mat(tr, 3 * GiB, 10, 65), mat(tr, 2 * GiB, 24, 65)
    need = tr._lib().vc_linear_forward_workspace(ref(odd), ref(wo))
    assert fwd(odd, wo, x(0, 24), ws=GiB + 128, size=need) == ALIAS

    def three(first, stride=100 * 100, cols=30):
        return mat(tr, GiB + 4 * first, 100, cols, ld=100, dtype=F32, batch=3, stride=stride)
    assert muon(tr, three(0), three(30), three(60)) == CUDA
    assert muon(tr, three(0), three(30), three(59)) == ALIAS
    assert muon(tr, three(0), three(30, stride=100 * 101), three(60)) == CUDA
    assert muon(tr, three(0), three(30, stride=100 * 101 + 1), three(60)) == ALIAS


def test_sizes_that_no_launch_could_take(tr):
    """Refused before anything is launched: more tiles than ints count, rows
    further apart than a tensor map can say."""
    big, far = 1 << 20, (1 << 39) - 8
    w = mat(tr, 2 * GiB, big, 8)
    assert forward(tr, mat(tr, GiB, big, 8), w, mat(tr, 1 << 45, big, big)) == INVALID
    assert forward(tr, mat(tr, GiB, big // 4, 8), w, mat(tr, 1 << 45, big // 4, big)) == CUDA
    one = mat(tr, 3 * GiB, 10, 24)
    assert forward(tr, mat(tr, 1 << 45, 10, 64, ld=far), mat(tr, 2 * GiB, 24, 64), one) == CUDA
    assert forward(tr, mat(tr, 1 << 45, 10, 64, ld=far + 8), mat(tr, 2 * GiB, 24, 64), one) == INVALID
    assert ortho(tr, mat(tr, GiB, 1 << 19, 1 << 19, batch=2), mat(tr, 1 << 45, 1 << 19, 1 << 19, batch=2)) == INVALID


class PlainMuon:
    """vc_muon_step on the host; the ways in which it can be wrong."""

    def __init__(self, fault=None):
        self.fault = fault

    def vc_muon_step(self, w, grad, m, lr, scale):
        if self.fault == "nothing written":
            return
        m.copy_(0.95 * m + grad)
        if self.fault == "momentum alone":
            return
        o = (m if self.fault == "no nesterov" else grad + 0.95 * m).double()
        o = o / o.norm()
        for _ in range(4 if self.fault == "a pass short" else 5):
            a = o @ o.t()
            o = 3.4445 * o + (-4.7750 * a + 2.0315 * (a @ a)) @ o
        w.sub_((lr * scale * o * (1.01 if self.fault == "scale" else 1)).float())
        if self.fault == "momentum":
            m.mul_(1.001)


@pytest.mark.parametrize("fault", [None, "nothing written", "momentum alone", "momentum",
                                   "no nesterov", "a pass short", "scale"])
def test_smoke_rejects_wrong_muon_steps(fault):
    torch = pytest.importorskip("torch")
    import __graft_entry__ as entry
    if fault is None:
        entry._check_muon(torch, PlainMuon(), torch.device("cpu"))
        return
    with pytest.raises(AssertionError):
        entry._check_muon(torch, PlainMuon(fault), torch.device("cpu"))


class FakeCuda:
    """What PreparedOperator asks of torch: streams by number, events, and a
    log of what is done with them."""

    def __init__(self):
        self.log, self.now, self.capturing, self.device = [], 0, False, 0
        fake = self

        class Stream:
            def __init__(self, raw):
                self.cuda_stream = raw

            def wait_event(self, event):
                fake.log.append(("wait", self.cuda_stream, event.at))

            def __enter__(self):
                self.before, fake.now = fake.now, self.cuda_stream

            def __exit__(self, *exc):
                fake.now = self.before

        class Event:
            def record(self):
                assert not fake.capturing
                self.at = fake.now

        class Cuda:
            current_device = staticmethod(lambda: fake.device)
            current_stream = staticmethod(lambda: Stream(fake.now))
            is_current_stream_capturing = staticmethod(lambda: fake.capturing)
            stream = staticmethod(lambda s: s)

        class C:
            _cuda_getCurrentRawStream = staticmethod(lambda index: fake.now)

        self.Stream, Cuda.Event, self.cuda, self._C = Stream, Event, Cuda, C

    def workspace(self):
        fake = self

        class Tensor:
            def record_stream(self, stream):
                fake.log.append(("record", stream.cuda_stream))
        return Tensor()


@pytest.fixture
def fake_cuda(tr, monkeypatch):
    import contextlib
    fake = FakeCuda()
    monkeypatch.setattr(tr, "_torch", lambda: fake)
    monkeypatch.setattr(tr, "_OnDevice", lambda device: contextlib.nullcontext())
    return fake


def handle(tr, fake, made):
    class Device:
        index = 0
    return tr.PreparedOperator(lambda stream: fake.log.append(("call", stream)) or 0, (), Device,
                               (made,), made)


def test_a_handles_workspace_follows_its_calls(tr, fake_cuda):
    """On another stream than the preparing one, by argument or by a change of
    the current stream, a call waits for what preceded the allocation and the
    allocator learns of the stream, before the launch."""
    fake = fake_cuda
    fake.now = 7
    call = handle(tr, fake, fake.workspace())
    call()
    call(stream=fake.Stream(7))
    assert fake.log == [("call", 7), ("call", 7)]
    fake.log.clear()
    call(stream=fake.Stream(8))
    call(stream=fake.Stream(8))
    assert fake.log == [("wait", 8, 7), ("record", 8), ("call", 8), ("call", 8)]
    fake.log.clear()
    fake.now = 9
    call()
    assert fake.log == [("wait", 9, 7), ("record", 9), ("call", 9)]
    assert fake.now == 9
    # nothing to follow where the caller brought the workspace
    fake.log.clear()
    handle(tr, fake, None)(stream=fake.Stream(8))
    assert fake.log == [("call", 8)]


def test_a_handles_workspace_under_capture(tr, fake_cuda):
    """A stream under capture waits for nothing outside of it, and no event is
    recorded there."""
    fake = fake_cuda
    call = handle(tr, fake, fake.workspace())
    fake.capturing = True
    call(stream=fake.Stream(3))
    assert fake.log == [("record", 3), ("call", 3)]
    fake.log.clear()
    fake.capturing = False
    call(stream=fake.Stream(3))  # the same stream, after its capture
    assert fake.log == [("wait", 3, 0), ("record", 3), ("call", 3)]
    fake.log.clear()
    fake.capturing = True
    call = handle(tr, fake, fake.workspace())
    fake.capturing = False
    call(stream=fake.Stream(4))
    assert fake.log == [("record", 4), ("call", 4)]
