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
