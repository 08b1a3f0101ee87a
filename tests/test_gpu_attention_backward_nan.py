"""A NaN among the row statistics reaches every gradient that it enters, as
NaN, and no other."""
import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [0, 1, 2, 3, 7, 9, 40, 97, 127, 129, 199])
def test_nan_in_one_row_s_lse(D, at):
    """P of that query is NaN for every key, whichever unit computes its
    exponentials: dV, dK and the query's dQ are NaN, not infinite or finite;
    the other queries' dQ and the other head are as without it."""
    B, N, H = 1, 200, 2
    shape = sp.Shape(B, N, H, D, 1)
    g = torch.Generator(device="cuda").manual_seed(at)
    q, k, v, do = (torch.randn(shape.seq_sharded, generator=g, device="cuda").to(torch.bfloat16)
                   for _ in range(4))
    o, lse = torch.empty_like(q), torch.empty(shape.lse_shape, device="cuda")
    sp.attention_seqsharded(q, k, v, o, shape, lse=lse)

    def backward():
        d = [torch.empty_like(q) for _ in range(3)]
        sp.attention_backward_seqsharded(q, k, v, o, lse, do, *d, shape)
        return [t[0, 0].transpose(0, 1) for t in d]     # [H][N][D]

    clean = backward()
    lse[0, 0, at] = float("nan")
    dq, dk, dv = backward()
    assert torch.isnan(dv[0]).all() and torch.isnan(dk[0]).all() and torch.isnan(dq[0, at]).all()
    rest = torch.arange(N, device="cuda") != at
    assert torch.equal(dq[0, rest], clean[0][0, rest])
    for got, want in zip((dq, dk, dv), clean):
        assert torch.equal(got[1], want[1])
    assert sp.device_status() == sp.SP_OK
