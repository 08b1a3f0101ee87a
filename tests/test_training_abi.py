"""Host-side checks of the training calls (layer norm, attention backward) on
a machine without a GPU: bad arguments come back before anything is
enqueued."""
import ctypes

import pytest

import video_dit_sequence_b200 as sp

A = 0x1000000  # a 16-byte aligned address that no call gets to use


@pytest.fixture(scope="module")
def lib():
    from video_dit_sequence_b200 import build
    build.build()
    return sp.load()


def _p(v):
    return ctypes.c_void_p(v) if v else None


def _norm(lib, x=A, w=A, b=A, y=A, mean=A, rstd=A, hidden=64, eps=1e-6, layout=0, ptype=0,
          shape=sp.Shape(1, 10, 1, 128, 2)):
    s = shape.c() if shape is not None else None
    return lib.sp_layer_norm(_p(x), _p(w), _p(b), _p(y), _p(mean), _p(rstd), hidden, eps, layout,
                             ptype, ctypes.byref(s) if s is not None else None, None)


def _norm_back(lib, dy=A, x=A, w=A, mean=A, rstd=A, dx=A, dw=A, db=A, ws=A, hidden=64, layout=0,
               ptype=0, shape=sp.Shape(1, 10, 1, 128, 2)):
    s = shape.c()
    return lib.sp_layer_norm_backward(_p(dy), _p(x), _p(w), _p(mean), _p(rstd), _p(dx), _p(dw),
                                      _p(db), _p(ws), hidden, layout, ptype, ctypes.byref(s), None)


def test_layer_norm_refusals(lib):
    assert _norm(lib, shape=None) == sp.SP_ERR_NULL
    for name in ("x", "y"):
        assert _norm(lib, **{name: 0}) == sp.SP_ERR_NULL
    for name in ("x", "y", "w", "b"):
        assert _norm(lib, **{name: A + 8}) == sp.SP_ERR_ALIGN
    for name in ("mean", "rstd"):
        assert _norm(lib, **{name: A + 2}) == sp.SP_ERR_ALIGN
    for hidden in (0, -8, 4, 12, sp.NORM_MAX_HIDDEN + 8):
        assert _norm(lib, hidden=hidden) == sp.SP_ERR_SHAPE
    for kw in ({"layout": 2}, {"layout": -1}, {"ptype": 2}, {"ptype": -1}):
        assert _norm(lib, **kw) == sp.SP_ERR_SHAPE
    for s in (sp.Shape(0, 10, 1, 128, 1), sp.Shape(1, 0, 1, 128, 1), sp.Shape(1, 10, 1, 128, 0),
              sp.Shape(65536, 10, 1, 128, 1), sp.Shape(1, 10, 1, 128, 65536),
              sp.Shape(2, 2 ** 30, 1, 128, 1), sp.Shape(1, 2 ** 31 - 1, 1, 128, 65535)):
        assert _norm(lib, shape=s) == sp.SP_ERR_SHAPE


def test_layer_norm_backward_refusals(lib):
    for name in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert _norm_back(lib, **{name: 0}) == sp.SP_ERR_NULL
    assert _norm_back(lib, dw=0) == sp.SP_ERR_NULL and _norm_back(lib, db=0) == sp.SP_ERR_NULL
    for name in ("dy", "x", "w", "dx", "dw", "db", "ws"):
        assert _norm_back(lib, **{name: A + 4}) == sp.SP_ERR_ALIGN
    assert _norm_back(lib, hidden=60) == sp.SP_ERR_SHAPE
    assert _norm_back(lib, layout=7) == sp.SP_ERR_SHAPE


def test_layer_norm_workspace(lib):
    for B, N, C in ((1, 1, 8), (2, 77, 1536), (1, 75600, 5120), (3, 1001, 1160), (500, 10, 64)):
        n = sp.layer_norm_backward_workspace(sp.Shape(B, N, 1, 128, 1), C)
        assert n % (2 * C * 4) == 0
        # at least one partial row of both gradients per sample
        assert n >= B * 2 * C * 4
        assert n == sp.layer_norm_backward_workspace(sp.Shape(B, N, 1, 128, 4), C)
    with pytest.raises(sp.SpError):
        sp.layer_norm_backward_workspace(sp.Shape(1, 10, 1, 128, 1), 60)


def _attn_back(lib, seq=True, shape=sp.Shape(1, 10, 2, 128, 2), **kw):
    a = {n: A for n in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv", "ws")}
    a.update(kw)
    s = shape.c() if shape is not None else None
    fn = lib.sp_attention_backward_seqsharded if seq else lib.sp_attention_backward
    return fn(*[_p(v) for v in a.values()], ctypes.byref(s) if s is not None else None, None)


@pytest.mark.parametrize("seq", [True, False])
def test_attention_backward_refusals(lib, seq):
    names = ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv", "ws")
    for n in names:
        assert _attn_back(lib, seq, **{n: 0}) == sp.SP_ERR_NULL
        assert _attn_back(lib, seq, **{n: A + 2}) == sp.SP_ERR_ALIGN
        if n != "lse":
            assert _attn_back(lib, seq, **{n: A + 8}) == sp.SP_ERR_ALIGN
    assert _attn_back(lib, seq, shape=None) == sp.SP_ERR_NULL
    assert _attn_back(lib, seq, shape=sp.Shape(1, 10, 2, 96, 2)) == sp.SP_ERR_UNSUPPORTED_D
    for s in (sp.Shape(0, 10, 2, 128, 2), sp.Shape(1, 0, 2, 128, 2), sp.Shape(1, 10, 0, 128, 2),
              sp.Shape(1, 10, 2, 128, 0), sp.Shape(1, 2 ** 30, 16, 128, 2)):
        assert _attn_back(lib, seq, shape=s) == sp.SP_ERR_SHAPE
    if not seq:
        assert _attn_back(lib, seq, shape=sp.Shape(1, 10, 3, 128, 2)) == sp.SP_ERR_HEADS_NOT_DIVISIBLE


def test_attention_backward_workspace(lib):
    for B, N, H, D in ((1, 1, 1, 64), (2, 777, 6, 128), (1, 4096, 40, 128), (1, 75600, 40, 128)):
        n = sp.attention_backward_workspace(sp.Shape(B, N, H, D, 1))
        tiles = -(-N // 128)
        # two statistics a row at least
        assert n >= B * H * tiles * 128 * 8
        assert n == sp.attention_backward_workspace(sp.Shape(B, N, H, D, 5))
    with pytest.raises(sp.SpError):
        sp.attention_backward_workspace(sp.Shape(1, 10, 1, 32, 1))


def test_backward_step_needs_a_step():
    torch = pytest.importorskip("torch")
    rank = sp.UlyssesRank(sp.Shape(1, 10, 2, 64, 2))
    with pytest.raises(RuntimeError, match="there was none"):
        rank.backward_step(torch.zeros(1), None, lambda send, recv: None)
