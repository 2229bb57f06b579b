"""Arguments of include/vc_step.h's entry points without a GPU: calls that are refused, or
that have to reach a launch (the launch hook turns it into VC_ERR_CUDA).  The fake
device pointers are never dereferenced."""
from __future__ import annotations

import ctypes

import pytest

SUCCESS, INVALID, ALIAS, CUDA = 0, 1, 3, 4
F32, BF16 = 2, 3
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


def mat(st, at, rows, cols, dtype=BF16):
    return st.Matrix(at, 1, rows, cols, cols, rows * cols, dtype)


@pytest.mark.parametrize("cols", [64, 70000])
def test_rms_norms_have_no_bias(st, cols):
    """Of any width, before or behind a block, in both directions; layer norms have."""
    L = st._lib()
    h, r, n = (mat(st, (k + 1) * GiB, 12, cols) for k in range(3))
    weight, biased = st.Affine(8 * GiB, None, BF16), st.Affine(9 * GiB, 10 * GiB, BF16)
    by = ctypes.byref
    for post, pre in ((biased, weight), (weight, biased), (biased, biased), (weight, weight)):
        args = st.BlockNorm(0, 0, 1.0, 1e-6)
        want = CUDA if post is weight and pre is weight else INVALID
        call = (by(h), None, None, by(post), by(pre), by(args), by(r), by(n), None)
        assert L.vc_block_norm_forward(*call) == want
        args.norm = 1
        assert L.vc_block_norm_forward(*call) == CUDA


@pytest.mark.parametrize("gates", [1, 3])
def test_gates_without_rows_reach_a_launch(st, gates):
    """The gradient of a gate that no row has is zeros, and has to be written."""
    L = st._lib()
    none, gate, dgate = mat(st, 0, 0, 64), mat(st, GiB, gates, 64), mat(st, 2 * GiB, gates, 64, F32)
    at = ctypes.pointer
    ins = st.BlockNormIn(at(none), None, None, at(none), at(gate))
    empty = st.Affine(None, None, BF16)
    outs = st.BlockNormOut(None, None, at(dgate), empty, empty)
    args = st.BlockNorm(0, 0, 1.0, 1e-6)
    call = lambda acc: L.vc_block_norm_backward(  # noqa: E731
        ctypes.byref(ins), None, None, ctypes.byref(args), ctypes.byref(outs), acc, None, 0, None)
    assert call(0) == CUDA
    assert call(1) == SUCCESS
