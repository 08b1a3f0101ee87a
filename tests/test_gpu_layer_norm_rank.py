"""Layer norm of one rank's shard, as every rank of the multi-GPU form has it,
against the call on all shards: rows bit for bit, sums over the ranks."""
import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CASES = [
    # (B, N, P, C, parameters): ranks that are full, ragged and without a token
    (1, 100, 4, 64, "shared"), (2, 101, 4, 1160, "sample"), (3, 9, 8, 264, "shared"),
    (3, 9, 8, 8, "sample"), (2, 5, 4, 1536, "none"), (2, 1, 3, 128, "shared"),
    (2, 1999, 3, 2816, "sample"), (1, 4000, 7, 5120, "shared"), (40, 33, 4, 72, "sample"),
]


@pytest.mark.parametrize("B,N,P,C,params", CASES)
def test_ranks_against_all_shards(B, N, P, C, params):
    shape = sp.Shape(B, N, 1, 128, P)
    Nl = shape.Nl
    g = torch.Generator(device="cuda").manual_seed(N + C)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    tokens = torch.arange(P * Nl, device="cuda").view(P, 1, Nl)
    pad = (tokens >= N).expand(P, B, Nl)
    x, dy = ((r(P, B, Nl, C) + 0.5).to(torch.bfloat16) for _ in range(2))
    for t in (x, dy):
        t[pad] = float("nan")            # padding slots are not read
    w = b = None
    if params != "none":
        ps = (C,) if params == "shared" else (B, C)
        w, b = 1 + 0.3 * r(*ps), r(*ps)
    empty = lambda *s: torch.full(s, float("nan"), device="cuda")

    def run(x, dy, rows, rank=None):
        y, dx, mean, rstd = empty(*x.shape).to(torch.bfloat16), empty(*x.shape).to(torch.bfloat16), \
            empty(*rows), empty(*rows)
        sp.layer_norm(x, w, b, y, shape, mean=mean, rstd=rstd, rank=rank)
        dw, db = (empty(*w.shape), empty(*w.shape)) if w is not None else (None, None)
        sp.layer_norm_backward(dy, x, w, mean, rstd, dx, shape, dweight=dw, dbias=db, rank=rank)
        return y, mean, rstd, dx, dw, db

    whole = run(x, dy, (P, B, Nl))
    xd, d = x.double(), dy.double()
    xh = (xd - whole[1].double()[..., None]) * whole[2].double()[..., None]
    live = (~pad)[..., None]
    terms = torch.where(live, d * xh, 0.0), torch.where(live, d, 0.0)
    for k in range(P):
        got = run(x[k].contiguous(), dy[k].contiguous(), (B, Nl), rank=k)
        for a, c in zip(got[:4], whole[:4]):
            assert torch.equal(a, c[k])
            assert (a[pad[k]].float() == 0).all() and not torch.signbit(a[pad[k]].float()).any()
        if w is not None:
            for a, t in zip(got[4:], terms):
                sums = t[k].sum((0, 1)) if params == "shared" else t[k].sum(1)
                size = t[k].abs().sum((0, 1)) if params == "shared" else t[k].abs().sum(1)
                # at most 3 roundings of a term and 300 additions on a path
                assert ((a.double() - sums).abs() <= 303 * U * size).all()
                if k * Nl >= N:
                    assert (a == 0).all() and not torch.signbit(a).any()
    assert sp.device_status() == sp.SP_OK


def test_refusals_of_the_binding():
    shape = sp.Shape(2, 10, 1, 128, 4)
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    sp.layer_norm(x, None, None, y, shape, rank=3)
    for rank in (-1, 4):
        with pytest.raises(sp.SpError):
            sp.layer_norm(x, None, None, y, shape, rank=rank)
    with pytest.raises(ValueError):        # all shards, given one
        sp.layer_norm(x, None, None, y, shape)
    with pytest.raises(ValueError):        # one shard, given all
        sp.layer_norm(torch.zeros(4, 2, 3, 64, dtype=torch.bfloat16, device="cuda"), None, None, y,
                      shape, rank=0)


def test_ranks_in_a_graph_and_on_a_stream():
    B, N, P, C = 2, 301, 2, 768
    shape = sp.Shape(B, N, 1, 128, P)
    rank = 1
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(B, shape.Nl, C, generator=g, device="cuda").to(torch.bfloat16)
             for _ in range(2))
    w = torch.randn(C, generator=g, device="cuda")
    mean = torch.empty(B, shape.Nl, device="cuda")
    ws = torch.empty(sp.layer_norm_backward_workspace(shape, C, rank), dtype=torch.uint8, device="cuda")

    def buffers():
        return (torch.empty_like(x), torch.empty_like(mean), torch.empty_like(mean),
                torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))

    def run(out, **kw):
        y, m, r, dx, dw, db = out
        sp.layer_norm(x, w, w, y, shape, mean=m, rstd=r, rank=rank, **kw)
        sp.layer_norm_backward(dy, x, w, m, r, dx, shape, dweight=dw, dbias=db, workspace=ws,
                               rank=rank, **kw)

    want, got, replayed = buffers(), buffers(), buffers()
    run(want)
    torch.cuda.synchronize()
    run(got, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(replayed)
    graph.replay()
    torch.cuda.synchronize()
    for a, c, e in zip(want, got, replayed):
        assert torch.equal(a, c) and torch.equal(a, e)
