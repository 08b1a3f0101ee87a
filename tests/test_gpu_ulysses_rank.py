"""UlyssesRank on the GPU: its buffers and its way back."""
import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _shards(shape, n, seed):
    """n tensors [P][B][Nl][H][D], padding slots zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(n):
        x = torch.randn(shape.seq_sharded, generator=g, device="cuda")
        slot = torch.arange(shape.Np, device="cuda").view(shape.P, 1, shape.Nl, 1, 1)
        out.append((x * (slot < shape.N)).to(torch.bfloat16))
    return out


def _stream_of(t):
    """Handle of the stream whose memory t lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def test_phases_on_a_stream_of_their_own():
    """Every buffer lies in the memory of the stream that its phase was given,
    and the results are those of the current stream."""
    shape = sp.Shape(2, 301, 2, 64, 1)
    q, k, v, do = (t[0] for t in _shards(shape, 4, seed=3))
    lse = torch.empty(shape.head_group().lse_shape, device="cuda")

    def there_and_back(rank, stream=None):
        send = rank.send_qkv(q, k, v, stream=stream)
        o = rank.attend(*send, lse=lse, stream=stream)
        out = rank.finish(o, stream=stream)
        grads = rank.attend_backward(*send, o, lse, rank.send_grad(do, stream=stream), stream=stream)
        return send + [o, out] + grads + rank.finish_grads(grads, stream=stream)

    want = [t.clone() for t in there_and_back(sp.UlyssesRank(shape))]
    side = torch.cuda.Stream()
    rank = sp.UlyssesRank(shape)
    torch.cuda.synchronize()
    for _ in range(2):
        got = there_and_back(rank, side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert side.cuda_stream != torch.cuda.current_stream().cuda_stream
    assert all(_stream_of(t) == side.cuda_stream for t in got)
    assert sp.device_status() == sp.SP_OK


@pytest.mark.parametrize("B,N,H,D,P", [(1, 700, 4, 128, 4), (2, 333, 6, 64, 3), (2, 9, 8, 64, 8)])
def test_there_and_back_on_virtual_ranks(B, N, H, D, P):
    """step and backward_step of P ranks, a thread each, whose exchanges meet
    at a host barrier and copy chunks on the one stream they share (no kernel
    waits for another): bit-equal to the calls on all shards, twice in a row
    with the same objects."""
    import threading
    shape = sp.Shape(B, N, H, D, P)
    ranks = [sp.UlyssesRank(shape) for _ in range(P)]
    lses = [torch.empty(shape.head_group().lse_shape, device="cuda") for _ in ranks]
    for seed in (5, 6):
        q, k, v, do = _shards(shape, 4, seed)
        o, lse = torch.empty_like(q), torch.empty(shape.lse_shape, device="cuda")
        sp.attention_seqsharded(q, k, v, o, shape, lse=lse)
        want = [torch.empty_like(q) for _ in range(3)]
        sp.attention_backward_seqsharded(q, k, v, o, lse, do, *want, shape)
        barrier, sent, got, errors = threading.Barrier(P), [None] * P, [None] * P, []

        def main(r):
            def exchange(send, recv):
                sent[r] = send
                barrier.wait(60)           # every rank's pack is enqueued
                for i in range(P):
                    recv[i].copy_(sent[i][r])
                barrier.wait(60)           # every copy is, before a buffer is packed again
            try:
                out = ranks[r].step(q[r], k[r], v[r], exchange, lse=lses[r])
                got[r] = [out] + ranks[r].backward_step(do[r], lses[r], exchange)
            except BaseException as e:
                errors.append(e)
                barrier.abort()

        threads = [threading.Thread(target=main, args=(r,)) for r in range(P)]
        for t in threads:
            t.start()
        for t in threads:
            t.join(120)
        assert not errors, errors
        torch.cuda.synchronize()
        for r in range(P):
            assert all(torch.equal(g, w[r]) for g, w in zip(got[r], [o] + want)), (seed, r)
        assert torch.equal(torch.cat(lses, 1)[..., :N], lse[..., :N])
    assert sp.device_status() == sp.SP_OK


def test_refused_way_back():
    """A dO or lse that does not fit is refused before any exchange, and the
    call with the right ones gives the step's gradients all the same."""
    shape = sp.Shape(1, 200, 2, 64, 1)
    q, k, v, do = (t[0] for t in _shards(shape, 4, seed=8))
    rank, lse = sp.UlyssesRank(shape), torch.empty(shape.lse_shape, device="cuda")
    copy = lambda send, recv: recv.copy_(send)
    rank.step(q, k, v, copy, lse=lse)
    want = [g.clone() for g in rank.backward_step(do, lse, copy)]
    calls = []
    refuse = lambda send, recv: calls.append(send)
    for bad in (do.float(), do.cpu(), do[:, :-1], do.transpose(1, 2)):
        with pytest.raises((TypeError, ValueError)):
            rank.backward_step(bad, lse, refuse)
    for bad in (None, lse.clone()):
        with pytest.raises(ValueError):
            rank.backward_step(do, bad, refuse)
    assert not calls
    assert all(torch.equal(g, w) for g, w in zip(rank.backward_step(do, lse, copy), want))
    assert sp.device_status() == sp.SP_OK


@pytest.mark.parametrize("eager_first", [True, False])
def test_step_and_way_back_in_a_graph(eager_first):
    """Captured with buffers of an earlier eager step, or its own; replayed on
    new data, with eager steps of the same object between the replays."""
    shape = sp.Shape(2, 150, 2, 64, 1)
    data = [[t[0] for t in _shards(shape, 4, seed=s)] for s in (11, 12)]
    copy = lambda send, recv: recv.copy_(send)
    want = []
    for q, k, v, do in data:
        rank, lse = sp.UlyssesRank(shape), torch.empty(shape.lse_shape, device="cuda")
        out = rank.step(q, k, v, copy, lse=lse)
        want.append([t.clone() for t in [out] + rank.backward_step(do, lse, copy)])
    rank, lse = sp.UlyssesRank(shape), torch.empty(shape.lse_shape, device="cuda")
    static = [t.clone() for t in data[0]]

    def there_and_back():
        out = rank.step(*static[:3], copy, lse=lse)
        return [out] + rank.backward_step(static[3], lse, copy)

    if eager_first:
        assert all(torch.equal(a, b) for a, b in zip(there_and_back(), want[0]))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = there_and_back()
    for i in (0, 1, 0):
        for s, t in zip(static, data[i]):
            s.copy_(t)
        for t in captured:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want[i]))
        assert all(torch.equal(a, b) for a, b in zip(there_and_back(), want[i]))
    assert sp.device_status() == sp.SP_OK
