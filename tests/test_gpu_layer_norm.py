"""Layer norm, forward and backward, against the formulas in 64 bits.

Tolerances: a result rounded to bf16 may be off by half a step (2^-8
relative), one held in fp32 by 2^-24; the arithmetic before it is fp32, whose
sums of a row or over rows carry at most DEPTH roundings of 2^-24 of their
absolute values on any path (lane sums of at most 256 terms, 5 to 9 tree
steps, and for the parameters' gradients the rows of one block plus the
blocks' partial sums)."""
import numpy as np
import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEPTH = 300
HALF = {"bf16": 2.0 ** -8, "fp32": U}


def _shape(B, N, P):
    return sp.Shape(B, N, 1, 128, P)


def _shard(x, P):
    """[B][N][...] -> [P][B][Nl][...], padding slots NaN: the calls must not
    read them."""
    B, N = x.shape[:2]
    Nl = -(-N // P)
    full = torch.full((B, P * Nl) + tuple(x.shape[2:]), float("nan"), dtype=x.dtype, device=x.device)
    full[:, :N] = x
    return full.view((B, P, Nl) + tuple(x.shape[2:])).transpose(0, 1).contiguous()


def _unshard(xs, N):
    P, B, Nl = xs.shape[:3]
    full = xs.transpose(0, 1).reshape((B, P * Nl) + tuple(xs.shape[3:]))
    return full[:, :N], full[:, N:]


def _inputs(B, N, C, params, seed, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = (r(B, N, C) * torch.exp(0.5 * r(C)) + offset).to(torch.bfloat16)
    dy = r(B, N, C).to(torch.bfloat16)
    if params == "none":
        return x, dy, None, None
    dt = torch.bfloat16 if params.endswith("bf16") else torch.float32
    ps = (C,) if params.startswith("shared") else (B, C)
    return x, dy, (1 + 0.3 * r(*ps)).to(dt), (0.3 * r(*ps)).to(dt)


def _p64(t, B):
    return None if t is None else t.double().view(-1, 1, t.shape[-1])


def _oracle(x, dy, w, b, eps=1e-6):
    """Everything in 64 bits on the logical tensors, with the error bounds."""
    B, N, C = x.shape
    xd, d = x.double(), dy.double()
    mean = xd.mean(-1, keepdim=True)
    var = ((xd - mean) ** 2).mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    xh = (xd - mean) * rstd
    W = _p64(w, B) if w is not None else torch.ones(1, 1, 1, dtype=torch.float64, device=x.device)
    Bb = _p64(b, B) if b is not None else torch.zeros(1, 1, 1, dtype=torch.float64, device=x.device)
    y = xh * W + Bb
    exh = DEPTH * U * (xd.abs().mean(-1, keepdim=True) * rstd + xh.abs())  # error of xh
    ey = W.abs() * exh + 4 * U * (xh.abs() * W.abs() + Bb.abs())
    g = d * W
    c1, c2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    ec2 = (g.abs() * exh).mean(-1, keepdim=True) + DEPTH * U * (g * xh).abs().mean(-1, keepdim=True)
    edx = rstd * (DEPTH * U * (g.abs() + g.abs().mean(-1, keepdim=True) + (xh * c2).abs())
                  + exh * c2.abs() + xh.abs() * ec2)
    dims = (0, 1) if w is None or w.dim() == 1 else (1,)
    dw, db = (d * xh).sum(dims), d.sum(dims)
    edw = (d.abs() * exh).sum(dims) + DEPTH * U * (d * xh).abs().sum(dims)
    edb = DEPTH * U * d.abs().sum(dims)
    return dict(mean=mean[..., 0], rstd=rstd[..., 0], y=y, ey=ey, dx=dx, edx=edx, dw=dw, edw=edw,
                db=db, edb=edb, emean=DEPTH * U * xd.abs().mean(-1),
                erstd=rstd[..., 0] * DEPTH * U * (1 + (xd.abs().mean(-1) * rstd[..., 0]) ** 2))


def _close(got, ref, err, kind, where):
    got = got.double()
    assert torch.isfinite(got).all(), where
    bad = (got - ref).abs() > HALF[kind] * ref.abs() + err * (1 + HALF[kind]) + 1e-30
    assert not bad.any(), (where, (got - ref).abs().max().item(), int(bad.sum()))


def _forward(x, w, b, P, stats=True):
    B, N, C = x.shape
    xs = _shard(x, P)
    y = torch.full_like(xs, float("nan"))
    mean = torch.full(xs.shape[:3], float("nan"), device="cuda") if stats else None
    rstd = mean.clone() if stats else None
    sp.layer_norm(xs, w, b, y, _shape(B, N, P), mean=mean, rstd=rstd)
    return xs, y, mean, rstd


def _backward(xs, dy, w, mean, rstd, N, P, grads=True, dtype=None, pshape=None, ws=None):
    B, C = xs.shape[1], xs.shape[-1]
    dx = torch.full_like(xs, float("nan"))
    dw = db = None
    if grads:
        like = w if w is not None else torch.empty(pshape or (C,), dtype=dtype or torch.float32,
                                                   device="cuda")
        dw, db = torch.full_like(like, float("nan")), torch.full_like(like, float("nan"))
    sp.layer_norm_backward(_shard(dy, P), xs, w, mean, rstd, dx, _shape(B, N, P), dweight=dw,
                           dbias=db, workspace=ws)
    return dx, dw, db


CASES = [
    # (B, N, P, C, params)
    (1, 1, 1, 8, "shared_fp32"), (1, 1, 1, 1536, "shared_bf16"), (1, 2, 4, 64, "sample_fp32"),
    (2, 77, 1, 1536, "none"), (3, 101, 4, 1160, "sample_fp32"), (2, 45, 2, 264, "sample_bf16"),
    (2, 33, 3, 1024, "shared_bf16"), (1, 50, 7, 1032, "shared_fp32"), (1, 40, 2, 2048, "sample_bf16"),
    (1, 31, 1, 3968, "shared_bf16"), (2, 19, 2, 5120, "sample_fp32"), (1, 9, 1, 8192, "shared_fp32"),
    (2, 13, 2, 8184, "sample_bf16"), (2, 700, 2, 6400, "shared_fp32"), (1, 900, 3, 7160, "shared_bf16"),
    (3, 411, 2, 2816, "sample_fp32"), (2, 1500, 4, 5120, "shared_fp32"), (1, 2000, 1, 4096, "shared_bf16"),
    (2, 1333, 2, 1536, "shared_bf16"), (300, 5, 2, 72, "sample_fp32"),
    (1, 5001, 2, 8, "shared_fp32"), (2, 9001, 4, 32, "shared_bf16"), (3, 7, 2, 56, "sample_fp32"),
    (1, 40001, 1, 128, "shared_fp32"), (2, 20000, 3, 248, "sample_bf16"), (1, 3000, 2, 256, "shared_fp32"), (1, 2500, 1, 32, "none"),
]


@pytest.mark.parametrize("B,N,P,C,params", CASES)
def test_forward_and_backward(B, N, P, C, params):
    x, dy, w, b = _inputs(B, N, C, params, seed=N * 7 + C)
    ref = _oracle(x, dy, w, b)
    xs, y, mean, rstd = _forward(x, w, b, P)
    for got, name, kind in ((y, "y", "bf16"), (mean, "mean", "fp32"), (rstd, "rstd", "fp32")):
        rows, pad = _unshard(got, N)
        _close(rows, ref[name], ref["e" + name], kind, name)
        assert (pad.float() == 0).all() and not torch.signbit(pad.float()).any(), name
    dx, dw, db = _backward(xs, dy, w, mean, rstd, N, P, grads=w is not None)
    rows, pad = _unshard(dx, N)
    _close(rows, ref["dx"], ref["edx"], "bf16", "dx")
    assert (pad.float() == 0).all() and not torch.signbit(pad.float()).any()
    if w is not None:
        kind = "bf16" if w.dtype == torch.bfloat16 else "fp32"
        _close(dw, ref["dw"], ref["edw"], kind, "dweight")
        _close(db, ref["db"], ref["edb"], kind, "dbias")
    assert sp.device_status() == sp.SP_OK


def test_results_do_not_depend_on_the_degree_and_repeat():
    B, N, C = 2, 1000, 640
    x, dy, w, b = _inputs(B, N, C, "sample_fp32", seed=5)
    first = None
    for P in (1, 3, 8, 1):
        xs, y, mean, rstd = _forward(x, w, b, P)
        dx, dw, db = _backward(xs, dy, w, mean, rstd, N, P)
        out = [_unshard(t, N)[0] for t in (y, mean, rstd, dx)] + [dw, db]
        first = first or out
        assert all(torch.equal(a, c) for a, c in zip(out, first)), P


def test_large_mean_and_constant_rows():
    """A mean of 1,000 standard deviations costs no digits of the variance;
    a constant row has xh = 0 and rstd = 1 / sqrt(eps)."""
    x, dy, w, b = _inputs(1, 40, 512, "shared_fp32", seed=9)
    x = (1024 + 8 * torch.randn(1, 40, 512, device="cuda")).to(torch.bfloat16)
    x[0, 7] = 3.0
    ref = _oracle(x, dy, w, b)
    xs, y, mean, rstd = _forward(x, w, b, 1)
    _close(_unshard(y, 40)[0], ref["y"], ref["ey"], "bf16", "y")
    assert torch.equal(y[0, 0, 7].float(), b.to(torch.bfloat16).float())
    assert abs(rstd[0, 0, 7].item() - 1e3) < 1e-3
    dx, dw, db = _backward(xs, dy, w, mean, rstd, 40, 1)
    _close(_unshard(dx, 40)[0], ref["dx"], ref["edx"], "bf16", "dx")


def test_frozen_parameters_and_bias_or_weight_alone():
    x, dy, w, b = _inputs(2, 30, 320, "sample_bf16", seed=3)
    ref = _oracle(x, dy, w, None)
    xs, y, mean, rstd = _forward(x, w, None, 2)
    _close(_unshard(y, 30)[0], ref["y"], ref["ey"], "bf16", "weight alone")
    dx, _, _ = _backward(xs, dy, w, mean, rstd, 30, 2, grads=False)
    _close(_unshard(dx, 30)[0], ref["dx"], ref["edx"], "bf16", "dx, frozen")
    ref = _oracle(x, dy, None, b)
    _, y, _, _ = _forward(x, None, b, 2, stats=False)
    _close(_unshard(y, 30)[0], ref["y"], ref["ey"], "bf16", "bias alone")
    # gradients of parameters that are not given (weight 1): shape and type of dweight
    dx, dw, db = _backward(xs, dy, None, mean, rstd, 30, 2, dtype=torch.float32, pshape=(2, 320))
    d, xd = dy.double(), x.double()
    xh = (xd - xd.mean(-1, keepdim=True)) * (xd.var(-1, keepdim=True, correction=0) + 1e-6) ** -0.5
    assert torch.allclose(dw.double(), (d * xh).sum(1), rtol=0, atol=DEPTH * U * 30 * 30)
    assert torch.allclose(db.double(), d.sum(1), rtol=0, atol=DEPTH * U * 30 * 6)


def test_gradients_against_differences():
    """(L(x + h v) - L(x - h v)) / 2h of L = sum(dy * y), with L in 64 bits by
    the formula, against <dx, v>: the difference's own error is O(h^2)."""
    x, dy, w, b = _inputs(2, 12, 256, "sample_fp32", seed=21)
    xs, _, mean, rstd = _forward(x, w, b, 1)
    dx, dw, db = _backward(xs, dy, w, mean, rstd, 12, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = 1e-4

    def loss(xd, wd, bd):
        m = xd.mean(-1, keepdim=True)
        r = (((xd - m) ** 2).mean(-1, keepdim=True) + 1e-6) ** -0.5
        return (dy.double() * ((xd - m) * r * wd[:, None] + bd[:, None])).sum()

    vx = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    vw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
    X, W, Bb = x.double(), w.double(), b.double()
    # x, and the parameters with w's direction for both
    num = (loss(X + h * vx, W, Bb) - loss(X - h * vx, W, Bb)) / (2 * h)
    got = (_unshard(dx, 12)[0].double() * vx).sum()
    bound = 2.0 ** -8 * (_unshard(dx, 12)[0].double().abs() * vx.abs()).sum()
    assert abs(num - got) <= bound
    num = (loss(X, W + h * vw, Bb + h * vw) - loss(X, W - h * vw, Bb - h * vw)) / (2 * h)
    got = ((dw + db).double() * vw).sum()
    assert abs(num - got) <= DEPTH * U * 12 * 256 * 2 * 30 + 1e-6 * abs(num)


def test_streams_workspaces_and_graphs():
    """Two streams with a workspace each, a call on a stream that is not the
    current one, and a captured forward + backward replayed on new data."""
    B, N, C, P = 2, 300, 768, 2
    shape = _shape(B, N, P)
    data = [_inputs(B, N, C, "sample_fp32", seed=s) for s in (1, 2)]
    want = []
    for x, dy, w, b in data:
        xs, y, mean, rstd = _forward(x, w, b, P)
        want.append((y,) + _backward(xs, dy, w, mean, rstd, N, P))
    streams = [torch.cuda.Stream() for _ in data]
    ws = [torch.empty(sp.layer_norm_backward_workspace(shape, C), dtype=torch.uint8, device="cuda")
          for _ in data]
    got = []
    torch.cuda.synchronize()
    for (x, dy, w, b), st, k in zip(data, streams, ws):
        xs, dys = _shard(x, P), _shard(dy, P)
        y, dx = torch.empty_like(xs), torch.empty_like(xs)
        mean = torch.empty(xs.shape[:3], device="cuda")
        rstd, dw, db = torch.empty_like(mean), torch.empty_like(w), torch.empty_like(w)
        torch.cuda.synchronize()
        for it in range(3):
            sp.layer_norm(xs, w, b, y, shape, mean=mean, rstd=rstd, stream=st)
            sp.layer_norm_backward(dys, xs, w, mean, rstd, dx, shape, dweight=dw, dbias=db,
                                   workspace=k if it else None, stream=st)
        got.append((y, dx, dw, db))
    torch.cuda.synchronize()
    for a, c in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(a, c))
    # graph
    x, dy, w, b = data[0]
    xs, dys = _shard(x, P), _shard(dy, P)
    y, dx = torch.empty_like(xs), torch.empty_like(xs)
    mean = torch.empty(xs.shape[:3], device="cuda")
    rstd, dw, db = torch.empty_like(mean), torch.empty_like(w), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sp.layer_norm(xs, w, b, y, shape, mean=mean, rstd=rstd)
        sp.layer_norm_backward(dys, xs, w, mean, rstd, dx, shape, dweight=dw, dbias=db)
    for (x, dy, w1, b1), ref in zip(data, want):
        xs.copy_(_shard(x, P))
        dys.copy_(_shard(dy, P))
        w.copy_(w1)
        b.copy_(b1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip((y, dx, dw, db), ref))


def test_outputs_stay_inside_their_buffers():
    B, N, C, P = 2, 37, 136, 3
    x, dy, w, b = _inputs(B, N, C, "sample_bf16", seed=4)
    shape = _shape(B, N, P)
    xs, dys = _shard(x, P), _shard(dy, P)
    guard = 1024

    def guarded(like):
        n = like.numel() * like.element_size()
        buf = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf[guard:guard + n].view(like.dtype).view(like.shape)

    stat = torch.empty(xs.shape[:3], device="cuda")
    need = sp.layer_norm_backward_workspace(shape, C)
    bufs = {n: guarded(t) for n, t in dict(
        y=xs, mean=stat, rstd=stat, dx=xs, dw=w, db=w,
        ws=torch.empty(need, dtype=torch.uint8, device="cuda")).items()}
    v = {n: t for n, (_, t) in bufs.items()}
    sp.layer_norm(xs, w, b, v["y"], shape, mean=v["mean"], rstd=v["rstd"])
    sp.layer_norm_backward(dys, xs, w, v["mean"], v["rstd"], v["dx"], shape, dweight=v["dw"],
                           dbias=v["db"], workspace=v["ws"])
    torch.cuda.synchronize()
    for n, (buf, _) in bufs.items():
        assert (buf[:guard] == 0xA5).all() and (buf[-guard:] == 0xA5).all(), n
    ref = _oracle(x, dy, w, b)
    _close(_unshard(v["dx"], N)[0], ref["dx"], ref["edx"], "bf16", "dx")


def test_every_hidden_size():
    """Every hidden size (the teams' warps, vectors and shared memory follow
    from it) with enough rows for full blocks: y, the statistics and dx of a
    few rows, and dweight, in 64 bits."""
    N = 2500
    g = torch.Generator(device="cuda").manual_seed(7)
    big = torch.randn(N * 8192, generator=g, device="cuda").to(torch.bfloat16)
    bigd = torch.randn(N * 8192, generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([0, 1, 147, 1201, N - 2, N - 1], device="cuda")
    for C in range(8, sp.NORM_MAX_HIDDEN + 1, 8):
        x, dy = (t[:N * C].view(1, 1, N, C) for t in (big, bigd))
        w = (1 + 0.3 * torch.randn(C, generator=g, device="cuda"))
        b = 0.3 * torch.randn(C, generator=g, device="cuda")
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean = torch.empty(1, 1, N, device="cuda")
        rstd, dw, db = torch.empty_like(mean), torch.empty_like(w), torch.empty_like(w)
        shape = _shape(1, N, 1)
        sp.layer_norm(x, w, b, y, shape, mean=mean, rstd=rstd)
        sp.layer_norm_backward(dy, x, w, mean, rstd, dx, shape, dweight=dw, dbias=db)
        ref = _oracle(x[0, :, rows], dy[0, :, rows], w, b)
        for got, name, kind in ((y, "y", "bf16"), (mean, "mean", "fp32"), (rstd, "rstd", "fp32"),
                                (dx, "dx", "bf16")):
            _close(got[0, :, rows], ref[name], ref["e" + name], kind, (C, name))
        xd, d = x[0, 0].float(), dy[0, 0].float()   # (fp32 products, summed in 64 bits)
        xh = (xd - mean[0, 0, :, None]) * rstd[0, 0, :, None]
        terms = d * xh
        assert ((dw - terms.sum(0, dtype=torch.float64)).abs()
                <= DEPTH * U * (terms.abs().sum(0, dtype=torch.float64) + d.abs().sum(0))).all(), C
        assert ((db - d.sum(0, dtype=torch.float64)).abs() <= DEPTH * U * d.abs().sum(0)).all(), C


def test_rows_that_are_not_finite_stay_alone():
    x, dy, w, b = _inputs(1, 50, 1160, "shared_fp32", seed=13)
    xs, y0, _, _ = _forward(x, w, b, 1)
    x[0, 20, 3] = float("nan")
    x[0, 31, 7] = float("inf")
    xs, y, mean, rstd = _forward(x, w, b, 1)
    dx, dw, db = _backward(xs, dy, w, mean, rstd, 50, 1)
    bad = torch.zeros(50, dtype=torch.bool, device="cuda")
    bad[[20, 31]] = True
    assert torch.isnan(y[0, 0][bad]).any(1).all() and torch.equal(y[0, 0][~bad], y0[0, 0][~bad])
    assert torch.isnan(dx[0, 0][bad]).any(1).all() and torch.isfinite(dx[0, 0][~bad]).all()
    assert torch.isnan(dw).any() and torch.isfinite(db).all()


def test_offsets_past_32_bits():
    """More than 2^31 elements: the first and the last rows against the call on
    them alone."""
    B, N, C, P = 2, 140000, 8192, 1
    assert B * N * C > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.empty(P, B, N, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
             for _ in range(2))
    w = 1 + 0.3 * torch.randn(B, C, generator=g, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean = torch.empty(P, B, N, device="cuda")
    rstd, dw, db = torch.empty_like(mean), torch.empty_like(w), torch.empty_like(w)
    shape = _shape(B, N, P)
    sp.layer_norm(x, w, w, y, shape, mean=mean, rstd=rstd)
    sp.layer_norm_backward(dy, x, w, mean, rstd, dx, shape, dweight=dw, dbias=db)
    for b, n in ((0, 0), (1, N - 40), (0, N - 40)):
        part = x[:, b:b + 1, n:n + 40].contiguous()
        pd = dy[:, b:b + 1, n:n + 40].contiguous()
        yp, dxp = torch.empty_like(part), torch.empty_like(part)
        m = torch.empty(1, 1, 40, device="cuda")
        r = torch.empty_like(m)
        sp.layer_norm(part, w[b], w[b], yp, _shape(1, 40, 1), mean=m, rstd=r)
        sp.layer_norm_backward(pd, part, w[b], m, r, dxp, _shape(1, 40, 1))
        assert torch.equal(y[:, b:b + 1, n:n + 40], yp) and torch.equal(rstd[:, b:b + 1, n:n + 40], r)
        assert torch.equal(dx[:, b:b + 1, n:n + 40], dxp)
    # the sums over all rows, in 64 bits by blocks of rows
    ref_w, ref_b = torch.zeros(B, C, dtype=torch.float64, device="cuda"), torch.zeros(B, C, dtype=torch.float64, device="cuda")
    abs_w = torch.zeros_like(ref_w)
    for n in range(0, N, 4000):
        d = dy[0, :, n:n + 4000].double()
        xh = (x[0, :, n:n + 4000].double() - mean[0, :, n:n + 4000, None]) * rstd[0, :, n:n + 4000, None]
        ref_w += (d * xh).sum(1)
        ref_b += d.sum(1)
        abs_w += (d * xh).abs().sum(1)
    # a block's rows (up to N / 148 of a team) and the blocks' sums in fp32
    depth = N / 148 + 200
    assert ((dw - ref_w).abs() <= depth * U * abs_w).all()
    assert ((db - ref_b).abs() <= depth * U * N * 6).all()


def test_binding_refusals():
    B, N, C, P = 1, 10, 64, 1
    x, dy, w, b = _inputs(B, N, C, "shared_fp32", seed=1)
    shape = _shape(B, N, P)
    xs, y, mean, rstd = _forward(x, w, b, P)
    dys, dx = _shard(dy, P), torch.empty_like(xs)
    bad = [
        lambda: sp.layer_norm(xs, w, b.to(torch.bfloat16), y, shape),        # mixed types
        lambda: sp.layer_norm(xs, w[:32], b, y, shape),                      # short weight
        lambda: sp.layer_norm(xs, w.half(), None, y, shape),                 # fp16
        lambda: sp.layer_norm(xs.float(), w, b, y, shape),                   # fp32 x
        lambda: sp.layer_norm(xs.cpu(), w, b, y, shape),                     # host x
        lambda: sp.layer_norm(xs, w, b, y[..., ::2], shape),                 # not contiguous
        lambda: sp.layer_norm_backward(dys, xs, w, mean, rstd, dx, shape, dweight=w.clone()),
        lambda: sp.layer_norm_backward(dys, xs, w, mean, rstd, dx, shape, dweight=w.clone(),
                                       dbias=w.clone(), workspace=torch.empty(8, device="cuda")),
        lambda: sp.layer_norm_backward(dys, xs, w, mean, None, dx, shape),
    ]
    for f in bad:
        with pytest.raises((TypeError, ValueError, sp.SpError)):
            f()
