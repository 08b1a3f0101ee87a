"""Host logic of UlyssesRank without a GPU: the library calls are replaced by
plain torch on CPU tensors, streams by recording fakes."""
import contextlib
import types

import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")

SHAPE = sp.Shape(1, 10, 4, 64, 2)


class Streams:
    """Fakes of the streams and of the allocator: which stream was current
    when a tensor was allocated, and which streams it was recorded on."""

    def __init__(self, monkeypatch):
        self.current, self.allocated, self.recorded = 0, {}, []
        empty = torch.empty

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, self.current if stream is None else stream.cuda_stream
            yield
            self.current = before

        def allocate(*args, **kw):
            t = empty(*args, **kw)
            self.allocated[t.data_ptr()] = self.current
            return t

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stream(self.current))
        monkeypatch.setattr(torch, "empty", allocate)
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: self.recorded.append((t.data_ptr(), s.cuda_stream)))
        monkeypatch.setattr(sp, "_stream",
                            lambda s, device: self.current if s is None else s.cuda_stream)

    @staticmethod
    def stream(handle):
        return types.SimpleNamespace(cuda_stream=handle, device=torch.device("cpu"))


def _phases(monkeypatch):
    """The local phases without arithmetic."""
    for name in ("exchange_pack", "exchange_unpack", "attention_seqsharded",
                 "attention_backward_seqsharded"):
        monkeypatch.setattr(sp, name, lambda *a, **kw: None)
    monkeypatch.setattr(sp, "attention_backward_workspace", lambda shape: 64)


def test_buffers_belong_to_the_stream_of_their_phase(monkeypatch):
    """A phase on a stream other than the current one must not take memory of
    the current one, whose earlier work may still use it."""
    fake = Streams(monkeypatch)
    _phases(monkeypatch)
    x = torch.zeros(SHAPE.rank_shard, dtype=torch.bfloat16)
    chunks = torch.zeros(SHAPE.send_chunks, dtype=torch.bfloat16)
    lse = torch.zeros(SHAPE.head_group().lse_shape)
    workspaces = []
    monkeypatch.setattr(sp, "attention_backward_seqsharded",
                        lambda *a, workspace=None, **kw: workspaces.append(workspace))
    rank, side = sp.UlyssesRank(SHAPE), fake.stream(7)
    bufs = (rank.send_qkv(x, x, x, stream=side) + [rank.attend(chunks, chunks, chunks, lse, side)] +
            [rank.finish(chunks, side), rank.send_grad(x, side)] +
            rank.attend_backward(chunks, chunks, chunks, chunks, lse, chunks, side) +
            rank.finish_grads([chunks] * 3, side) + workspaces)
    assert len(bufs) == 13
    assert all(fake.allocated[b.data_ptr()] == 7 for b in bufs), fake.allocated
    assert not fake.recorded
    # the next step on the same stream, then one on another: the same memory,
    # recorded for the second
    again = rank.send_qkv(x, x, x, stream=side)
    assert [t.data_ptr() for t in again] == [t.data_ptr() for t in bufs[:3]] and not fake.recorded
    rank.send_qkv(x, x, x, stream=fake.stream(9))
    assert fake.recorded == [(t.data_ptr(), 9) for t in bufs[:3]]
    fake.recorded.clear()
    rank.send_grad(x)                       # (the current stream)
    assert fake.recorded == [(bufs[5].data_ptr(), 0)]


def _plain_ptr(t, shape, name, dtype=None):
    """The binding's checks of an operand, without a device."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != (dtype or torch.bfloat16):
        raise TypeError(f"{name} must be {dtype or torch.bfloat16}, got {t.dtype}")
    if not t.is_contiguous() or t.numel() != torch.Size(shape).numel():
        raise ValueError(f"{name} has shape {tuple(t.shape)}")
    return t.data_ptr()


def _pack(x, send, shape, stream=None):
    """[B][Nl][H][D] -> [P][B][Nl][Hl][D]"""
    B, Nl, H, D = shape.rank_shard
    send.copy_(x.reshape(B, Nl, shape.P, H // shape.P, D).permute(2, 0, 1, 3, 4))


def _unpack(recv, out, shape, stream=None):
    out.copy_(recv.permute(1, 2, 0, 3, 4).reshape(out.shape))


def _heads(x, shape):
    """[P][B][Nl][H][D] -> [B][H][N][D] in 64 bits."""
    full = x.double().transpose(0, 1).reshape(shape.B, shape.Np, shape.H, shape.D)
    return full[:, :shape.N].transpose(1, 2)


def _back(x, shape):
    full = x.new_zeros(shape.B, shape.Np, shape.H, shape.D)
    full[:, :shape.N] = x.transpose(1, 2)
    return full.view(shape.B, shape.P, shape.Nl, shape.H, shape.D).transpose(0, 1)


def _attend(q, k, v, o, shape, lse=None, stream=None):
    qd, kd, vd = (_heads(t, shape) for t in (q, k, v))
    s = qd @ kd.transpose(2, 3) / shape.D ** 0.5
    o.copy_(_back(torch.softmax(s, -1) @ vd, shape))
    if lse is not None:
        lse.fill_(float("-inf"))
        lse[..., :shape.N] = torch.logsumexp(s, -1)


def _attend_backward(q, k, v, o, lse, do, dq, dk, dv, shape, workspace=None, stream=None):
    qd, kd, vd, od, dod = (_heads(t, shape) for t in (q, k, v, o, do))
    f = shape.D ** -0.5
    p = torch.exp(f * qd @ kd.transpose(2, 3) - lse[..., :shape.N, None].double())
    ds = p * (dod @ vd.transpose(2, 3) - (dod * od).sum(-1, keepdim=True))
    for out, g in ((dq, f * ds @ kd), (dk, f * ds.transpose(2, 3) @ qd), (dv, p.transpose(2, 3) @ dod)):
        out.copy_(_back(g, shape))


def _play(patch):
    """The local phases in plain torch, on the current (only) stream."""
    for name, f in (("exchange_pack", _pack), ("exchange_unpack", _unpack),
                    ("attention_seqsharded", _attend), ("_stream", lambda s, device: 0),
                    ("attention_backward_seqsharded", _attend_backward), ("_ptr", _plain_ptr),
                    ("attention_backward_workspace", lambda shape: 64)):
        patch(sp, name, f)


def _inputs(shape, seed, n=4):
    """n tensors [P][B][Nl][H][D] with zero padding."""
    g = torch.Generator().manual_seed(seed)
    rows = (torch.randn(shape.B, shape.H, shape.N, shape.D, generator=g) for _ in range(n))
    return [_back(x, shape).to(torch.bfloat16).contiguous() for x in rows]


def _copy(send, recv):
    recv.copy_(send)


def test_backward_step_goes_back_over_what_attend_took(monkeypatch):
    """attend as a phase, on the caller's own tensors: backward_step uses
    those, and no buffer that nothing was written to."""
    _play(monkeypatch.setattr)
    shape = sp.Shape(2, 9, 2, 64, 1)
    q, k, v, do = _inputs(shape, 1)
    rank, lse = sp.UlyssesRank(shape), torch.empty(shape.lse_shape)
    o = rank.attend(q, k, v, lse=lse)
    got = rank.backward_step(do[0], lse, _copy)
    want = [torch.empty_like(q) for _ in range(3)]
    _attend_backward(q, k, v, o, lse, do, *want, shape)
    assert all(torch.equal(g, w[0]) for g, w in zip(got, want))


def test_backward_step_refuses_and_keeps_the_step(monkeypatch):
    _play(monkeypatch.setattr)
    shape = sp.Shape(2, 9, 2, 64, 1)
    q, k, v, do = (t[0] for t in _inputs(shape, 2))
    lse, other = torch.empty(shape.lse_shape), torch.empty(shape.lse_shape)
    rank = sp.UlyssesRank(shape)
    rank.step(q, k, v, _copy, lse=lse)
    want = [g.clone() for g in rank.backward_step(do, lse, _copy)]
    exchanges = []
    for bad in (do.float(), do[:1], do.transpose(0, 1), None):
        with pytest.raises((TypeError, ValueError)):
            rank.backward_step(bad, lse, lambda *a: exchanges.append(a))
    for bad in (None, other):
        with pytest.raises(ValueError, match="lse"):
            rank.backward_step(do, bad, lambda *a: exchanges.append(a))
    assert not exchanges
    # a correct call after a refused one
    assert all(torch.equal(g, w) for g, w in zip(rank.backward_step(do, lse, _copy), want))
    # a later step that kept no lse, or another one
    rank.step(k, q, v, _copy)
    with pytest.raises(RuntimeError, match="kept none"):
        rank.backward_step(do, lse, _copy)
    rank.step(k, q, v, _copy, lse=other)
    with pytest.raises(ValueError, match="lse"):
        rank.backward_step(do, lse, _copy)
    # a step that broke off, one that has only begun
    def broken(send, recv):
        raise OSError("peer left")
    with pytest.raises(OSError):
        rank.step(q, k, v, broken, lse=lse)
    with pytest.raises(RuntimeError, match="there was none"):
        rank.backward_step(do, other, _copy)
    rank.step(q, k, v, _copy, lse=lse)
    rank.recv_buffers(q)
    with pytest.raises(RuntimeError, match="there was none"):
        rank.backward_step(do, lse, _copy)


def test_step_refuses_an_lse_before_any_exchange(monkeypatch):
    """(The other ranks would wait in an exchange that this one never joins.)"""
    _play(monkeypatch.setattr)
    shape = sp.Shape(2, 9, 2, 64, 1)
    q, k, v, _ = (t[0] for t in _inputs(shape, 2))
    exchanges = []
    for bad in (torch.empty(shape.lse_shape).double(), torch.empty(shape.lse_shape)[..., 1:],
                torch.empty(2, 2, 10)[..., :9], torch.empty(shape.lse_shape, device="meta")):
        with pytest.raises((TypeError, ValueError)):
            sp.UlyssesRank(shape).step(q, k, v, lambda *a: exchanges.append(a), lse=bad)
    assert not exchanges


def test_distributed_call_keeps_an_lse(monkeypatch):
    _play(monkeypatch.setattr)
    shape = sp.Shape(1, 9, 2, 64, 1)
    q, k, v, do = (t[0] for t in _inputs(shape, 3))
    rank, lse = sp.UlyssesRank(shape), torch.empty(shape.lse_shape)
    out = sp.ulysses_attention_distributed(q, k, v, shape, all_to_all=_copy, rank=rank, lse=lse)
    got = [out.clone()] + [g.clone() for g in rank.backward_step(do, lse, _copy)]
    want = [rank.step(q, k, v, _copy, lse=lse)] + rank.backward_step(do, lse, _copy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
