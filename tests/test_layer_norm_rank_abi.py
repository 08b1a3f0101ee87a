"""Host-side checks of layer norm on one rank's shard, without a GPU."""
import ctypes

import pytest

import video_dit_sequence_b200 as sp

A = 0x1000000  # a 16-byte aligned address that no call gets to use


@pytest.fixture(scope="module")
def lib():
    from video_dit_sequence_b200 import build
    build.build()
    return sp.load()


def _forward(lib, rank, shape, ptrs=(A,) * 6, hidden=64):
    s = ctypes.byref(shape.c()) if shape else None
    return lib.sp_layer_norm_rank(*ptrs, hidden, 1e-6, 0, 0, rank, s, None)


def _backward(lib, rank, shape, ptrs=(A,) * 9, hidden=64):
    s = ctypes.byref(shape.c()) if shape else None
    return lib.sp_layer_norm_backward_rank(*ptrs, hidden, 0, 0, rank, s, None)


@pytest.mark.parametrize("call,n", [(_forward, 6), (_backward, 9)])
def test_refusals(lib, call, n):
    shape = sp.Shape(2, 10, 1, 128, 4)
    for rank in (-1, -2, 4, 2 ** 31 - 1, -2 ** 31):
        assert call(lib, rank, shape) == sp.SP_ERR_SHAPE
    assert call(lib, 0, None) == sp.SP_ERR_NULL
    assert call(lib, 3, shape, hidden=60) == sp.SP_ERR_SHAPE
    assert call(lib, 3, sp.Shape(2, 0, 1, 128, 4)) == sp.SP_ERR_SHAPE
    for i in range(n):
        bad = [A] * n
        bad[i] = A + 2
        assert call(lib, 3, shape, bad) == sp.SP_ERR_ALIGN
    bad = [A] * n
    bad[0] = None
    assert call(lib, 3, shape, bad) == sp.SP_ERR_NULL


def test_workspace_is_that_of_a_shard(lib):
    for B, N, P, C in ((1, 9, 8, 64), (3, 1001, 4, 1160), (2, 300, 2, 5120)):
        shape = sp.Shape(B, N, 1, 128, P)
        want = sp.layer_norm_backward_workspace(sp.Shape(B, shape.Nl, 1, 128, 1), C)
        assert all(sp.layer_norm_backward_workspace(shape, C, r) == want for r in range(P))
