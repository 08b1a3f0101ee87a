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
