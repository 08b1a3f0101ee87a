"""Attention's backward pass against its formula in 64 bits.

Two bars.  (a) Element by element, the worst case of the arithmetic: P and dS
are rounded to bf16 once (half a step, 2^-8 relative), every gradient is
rounded to bf16 once, and everything else is fp32: products of D terms or sums
over the tokens whose roundings (2^-23 a step, the tensor core may truncate)
are counted on the sum of absolute terms.  (b) Per head in the 2-norm, for
random inputs from 16 tokens on: the roundings to bf16 are independent with a
root mean square of at most 2^-8 / sqrt(3) of the term (two of them, the
operand's and the result's: 0.82 * 2^-8), so the error stays below 2^-8 of the
gradient's norm."""
import math

import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
U = 2.0 ** -23


def _to_layout(x, layout, P, fill=float("nan")):
    """Logical [B][N][H][D] -> the layout, padding slots `fill`: the calls
    must not use them."""
    B, N, H, D = x.shape
    Nl = -(-N // P)
    full = torch.full((B, P * Nl, H, D), fill, dtype=x.dtype, device=x.device)
    full[:, :N] = x
    if layout == "seq":
        return full.view(B, P, Nl, H, D).transpose(0, 1).contiguous()
    return full.view(B, P * Nl, P, H // P, D).permute(2, 0, 1, 3, 4).contiguous()


def _from_layout(x, layout, B, N, H, D, P):
    Nl = -(-N // P)
    if layout == "seq":
        full = x.transpose(0, 1).reshape(B, P * Nl, H, D)
    else:
        full = x.permute(1, 2, 0, 3, 4).reshape(B, P * Nl, H, D)
    return full[:, :N], full[:, N:]


def _inputs(B, N, H, D, seed, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, do = (torch.randn(B, N, H, D, generator=g, device="cuda") for _ in range(4))
    return [t.to(torch.bfloat16) for t in (q * amp, k, v, do)]


def _forward64(q, k, v, scale):
    """o (bf16) and lse (fp32) as a forward pass leaves them."""
    qd, kd, vd = (t.double().transpose(1, 2) for t in (q, k, v))
    s = scale * qd @ kd.transpose(2, 3)
    lse = torch.logsumexp(s, -1)
    o = torch.exp(s - lse[..., None]) @ vd
    return o.transpose(1, 2).to(torch.bfloat16), lse.float()


def _oracle(q, k, v, o, lse, do, scale):
    """Gradients [B][H][N][D] in 64 bits and bounds on the kernel's error."""
    D, N = q.shape[-1], q.shape[1]
    q, k, v, o, do = (t.double().transpose(1, 2) for t in (q, k, v, o, do))
    lse = lse.double()[..., None]
    s = scale * q @ k.transpose(2, 3)
    p = torch.where(lse > -math.inf, torch.exp(s - lse), torch.zeros_like(s))
    delta = (do * o).sum(-1, keepdim=True)
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - delta)
    out = (scale * ds @ k, scale * ds.transpose(2, 3) @ q, p.transpose(2, 3) @ do)
    # relative error of a probability, absolute error of dP - delta
    ep = D * U * scale * (q.abs() @ k.abs().transpose(2, 3)) + 4 * U * (s.abs() + lse.abs()) + 4 * U
    if D == 64:   # the polynomial for 2^r is off by at most 2.9e-6 < 2^-18
        ep = ep + 2.0 ** -18
    ep = torch.where(lse > -math.inf, ep, torch.zeros_like(ep))
    ed = D * U * (do.abs() @ v.abs().transpose(2, 3) + (do.abs() * o.abs()).sum(-1, keepdim=True))
    eds = ds.abs() * (HALF + ep) + (1 + HALF) * p * ed
    acc = (N + 130) * U
    eq = scale * (eds + acc * ds.abs()) @ k.abs()
    ek = scale * (eds + acc * ds.abs()).transpose(2, 3) @ q.abs()
    ev = (p * (HALF + ep + acc)).transpose(2, 3) @ do.abs()
    return out, (eq, ek, ev)


def _call(layout, shape, q, k, v, o, lse, do, workspace=None, stream=None, fill=float("nan")):
    P, N = shape.P, shape.N
    t = [_to_layout(x, layout, P, fill) for x in (q, k, v, o, do)]
    lp = torch.full(shape.lse_shape, float("nan"), device="cuda")
    lp[..., :N] = lse
    d = [torch.full_like(t[0], float("nan")) for _ in range(3)]
    fn = sp.attention_backward_seqsharded if layout == "seq" else sp.attention_backward
    fn(t[0], t[1], t[2], t[3], lp, t[4], *d, shape, workspace=workspace, stream=stream)
    return d


def _check(d, ref, err, layout, shape, norms=True):
    B, N, H, D, P = shape.B, shape.N, shape.H, shape.D, shape.P
    assert sp.device_status() == sp.SP_OK
    for got, r, e, name in zip(d, ref, err, ("dq", "dk", "dv")):
        rows, pad = _from_layout(got, layout, B, N, H, D, P)
        assert (pad.float() == 0).all() and not torch.signbit(pad.float()).any(), name
        g = rows.double().transpose(1, 2)
        assert torch.isfinite(g).all(), name
        diff = (g - r).abs()
        bad = diff > e + HALF * (r.abs() + e) + 1e-37
        assert not bad.any(), (name, int(bad.sum()), (diff / (e + HALF * r.abs() + 1e-37)).max().item())
        if norms and N >= 16:
            rel = diff.square().sum((2, 3)).sqrt() / r.square().sum((2, 3)).sqrt()
            assert rel.max() < HALF, (name, rel.max().item())


CASES = [
    # (layout, B, N, H, D, P)
    ("seq", 1, 128, 1, 128, 1), ("seq", 1, 256, 2, 128, 1), ("seq", 1, 256, 1, 64, 1),
    ("seq", 1, 1, 1, 128, 1), ("seq", 2, 2, 2, 64, 2), ("seq", 1, 3, 1, 128, 8),
    ("seq", 1, 33, 3, 64, 2), ("head", 1, 127, 2, 128, 2), ("head", 2, 129, 2, 64, 1),
    ("seq", 2, 200, 3, 128, 3), ("seq", 2, 255, 2, 64, 2), ("head", 2, 257, 4, 128, 4),
    ("seq", 3, 640, 2, 128, 2), ("seq", 2, 777, 6, 128, 3), ("seq", 2, 1000, 1, 64, 4),
    ("head", 3, 511, 6, 64, 3), ("seq", 2, 1537, 4, 64, 3),
    # shards of 5, 8, 13, 29, 32, 37 and 98 tokens, some of them empty
    ("seq", 2, 33, 2, 128, 8), ("seq", 2, 300, 2, 64, 60), ("seq", 3, 200, 1, 128, 25),
    ("seq", 2, 300, 2, 128, 24), ("seq", 2, 260, 2, 64, 9), ("seq", 2, 500, 2, 128, 16),
    ("seq", 2, 361, 1, 128, 10), ("seq", 2, 777, 3, 64, 8),
    # more than 16 key tiles, and more tiles than the GPU runs at once
    ("seq", 1, 2177, 1, 128, 2), ("head", 1, 2100, 8, 128, 8), ("seq", 3, 1300, 5, 128, 4),
    ("seq", 2, 2500, 3, 64, 3), ("seq", 70, 150, 3, 128, 1), ("seq", 1, 4099, 3, 128, 1),
]


@pytest.mark.parametrize("layout,B,N,H,D,P", CASES)
def test_gradients(layout, B, N, H, D, P):
    shape = sp.Shape(B, N, H, D, P)
    scale = 1 / math.sqrt(D)
    q, k, v, do = _inputs(B, N, H, D, seed=N + D)
    o, lse = _forward64(q, k, v, scale)
    d = _call(layout, shape, q, k, v, o, lse, do)
    ref, err = _oracle(q, k, v, o, lse, do, scale)
    _check(d, ref, err, layout, shape)


@pytest.mark.parametrize("amp,scale", [(1.0, 0.02), (8.0, 0.0), (1e-3, 1.0)])
def test_scales_and_peaked_rows(amp, scale):
    """A scale of the user's, rows whose softmax is nearly one-hot (most
    probabilities underflow), and nearly uniform rows."""
    B, N, H, D, P = 1, 300, 2, 128, 2
    q, k, v, do = _inputs(B, N, H, D, seed=11, amp=amp)
    s = scale or 1 / math.sqrt(D)
    o, lse = _forward64(q, k, v, s)
    shape = sp.Shape(B, N, H, D, P, scale)
    d = _call("seq", shape, q, k, v, o, lse, do)
    ref, err = _oracle(q, k, v, o, lse, do, s)
    _check(d, ref, err, "seq", shape, norms=False)


def test_rows_without_a_key_and_negative_statistics():
    """lse = -inf: no probability, no gradient, nothing added to dK and dV.
    A strongly negative lse: the zero rows past N would overflow exp(0 - lse)
    if they were not left out."""
    B, N, H, D, P = 1, 300, 2, 64, 1
    scale = 1 / math.sqrt(D)
    q, k, v, do = _inputs(B, N, H, D, seed=12)
    k = (k.abs() + 4).to(torch.bfloat16)
    q = (-q.abs() - 4).to(torch.bfloat16)
    o, lse = _forward64(q, k, v, scale)
    assert lse.max() < -120
    lse[:, :, 7] = -math.inf
    lse[:, 1, 290:] = -math.inf
    shape = sp.Shape(B, N, H, D, P)
    d = _call("seq", shape, q, k, v, o, lse, do)
    ref, err = _oracle(q, k, v, o, lse, do, scale)
    _check(d, ref, err, "seq", shape, norms=False)
    dq = _from_layout(d[0], "seq", B, N, H, D, P)[0]
    assert (dq[:, 7] == 0).all() and (dq[:, 290:, 1] == 0).all()


@pytest.mark.parametrize("layout,D,P", [("seq", 128, 3), ("seq", 64, 1), ("head", 64, 2), ("head", 128, 2)])
def test_values_that_are_not_finite_stay_in_their_head(layout, D, P):
    """A NaN in one query reaches that query's gradient and, through its row of
    probabilities, every dK and dV of the head, and nothing else; one in a row of
    dO likewise.  The other heads repeat bit for bit."""
    B, N, H = 2, 333, 2
    scale = 1 / math.sqrt(D)
    shape = sp.Shape(B, N, H, D, P)
    clean = _inputs(B, N, H, D, seed=21)
    o, lse = _forward64(*clean[:3], scale)
    base = _call(layout, shape, *clean[:3], o, lse, clean[3])
    base = [_from_layout(t, layout, B, N, H, D, P)[0] for t in base]
    for which in (0, 3):    # q, dO
        for row in (5, 18, 200):
            t = [x.clone() for x in clean]
            t[which][1, row, 1, :] = float("nan")
            o, lse = _forward64(*t[:3], scale)
            d = _call(layout, shape, *t[:3], o, lse, t[3])
            dq, dk, dv = (_from_layout(x, layout, B, N, H, D, P)[0] for x in d)
            assert not torch.isfinite(dq[1, row, 1]).any()
            rest = torch.ones(B, N, H, dtype=torch.bool, device="cuda")
            rest[1, row, 1] = False
            assert torch.equal(dq[rest], base[0][rest])
            assert not torch.isfinite(dk[1, :, 1]).any() and not torch.isfinite(dv[1, :, 1]).any()
            for got, want in ((dk, base[1]), (dv, base[2])):
                assert torch.equal(got[0], want[0]) and torch.equal(got[1, :, 0], want[1, :, 0])
    assert sp.device_status() == sp.SP_OK


@pytest.mark.parametrize("B,N,H", [(1, 1025, 4), (2, 2200, 12)])
def test_results_repeat_and_depend_on_neither_degree_nor_layout(B, N, H):
    D = 128
    q, k, v, do = _inputs(B, N, H, D, seed=3)
    o, lse = _forward64(q, k, v, 1 / math.sqrt(D))
    first = None
    for layout, P in (("seq", 1), ("seq", 3), ("head", 2), ("head", 4), ("seq", 8), ("seq", 1)):
        d = _call(layout, sp.Shape(B, N, H, D, P), q, k, v, o, lse, do)
        out = [_from_layout(t, layout, B, N, H, D, P)[0] for t in d]
        first = first or out
        assert all(torch.equal(a, c) for a, c in zip(out, first)), (layout, P)
    assert sp.device_status() == sp.SP_OK


def test_gradients_against_differences():
    """(L(x + h u) - L(x - h u)) / 2h with L = sum(dO * O) in 64 bits, along a
    direction in q, k and v, against the products with the gradients, whose
    worst-case error the oracle's bounds give; the difference's own error is
    O(h^2)."""
    B, N, H, D = 1, 150, 2, 64
    scale = 1 / math.sqrt(D)
    q, k, v, do = _inputs(B, N, H, D, seed=5)
    o, lse = _forward64(q, k, v, scale)
    shape = sp.Shape(B, N, H, D, 1)
    d = _call("seq", shape, q, k, v, o, lse, do)
    _, err = _oracle(q, k, v, o, lse, do, scale)
    g = torch.Generator(device="cuda").manual_seed(1)

    def loss(a, b, c):
        a, b, c = (t.transpose(1, 2) for t in (a, b, c))
        return ((torch.softmax(scale * a @ b.transpose(2, 3), -1) @ c).transpose(1, 2) * do.double()).sum()

    x = [t.double() for t in (q, k, v)]
    for i in range(3):
        u = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + h * u, x[i] - h * u
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        got = _from_layout(d[i], "seq", B, N, H, D, 1)[0].double()
        # o was rounded to bf16 before delta: delta_i off by 2^-8 sum |dO o|
        ed = HALF * (do.double().abs() * o.double().abs()).sum(-1, keepdim=True)
        extra = scale * ((ed * q.double().abs().amax(1, keepdim=True) * u.abs()).sum()
                         if i == 1 else (ed * k.double().abs().amax(1, keepdim=True) * u.abs()).sum())
        bound = ((err[i].transpose(1, 2) + HALF * got.abs()) * u.abs()).sum() + extra
        assert abs(num - (got * u).sum()) <= bound + 1e-6 * abs(num), i
        # (the worst case is loose: independent roundings give a sharper bar)
        noise = HALF * ((got * u).square().sum().sqrt() + (ed * u).square().sum().sqrt())
        assert abs(num - (got * u).sum()) <= 8 * noise, i


def test_streams_workspaces_and_graphs():
    """Two streams at once with a workspace each, fresh workspaces, and a
    captured call replayed on new data."""
    B, N, H, D, P = 2, 1400, 8, 128, 2
    shape = sp.Shape(B, N, H, D, P)
    data, want = [], []
    for seed in (1, 2):
        q, k, v, do = _inputs(B, N, H, D, seed=seed)
        o, lse = _forward64(q, k, v, 1 / math.sqrt(D))
        data.append((q, k, v, o, lse, do))
        want.append(_call("seq", shape, *data[-1]))
    need = sp.attention_backward_workspace(shape)
    streams = [torch.cuda.Stream() for _ in data]
    ws = [torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") for _ in data]
    args = []
    for q, k, v, o, lse, do in data:
        t = [_to_layout(x, "seq", P) for x in (q, k, v, o, do)]
        lp = torch.full(shape.lse_shape, float("nan"), device="cuda")
        lp[..., :N] = lse
        args.append(t[:4] + [lp, t[4]] + [torch.empty_like(t[0]) for _ in range(3)])
    torch.cuda.synchronize()
    for it in range(3):
        for a, st, w in zip(args, streams, ws):
            sp.attention_backward_seqsharded(*a, shape, workspace=w if it else None, stream=st)
    torch.cuda.synchronize()
    for a, c in zip(args, want):
        assert all(torch.equal(s, t) for s, t in zip(a[6:], c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.attention_backward_seqsharded(*args[0], shape)
    for i in (1, 0, 1):
        for dst, src in zip(args[0][:6], args[i][:6] if i else None or _saved(data[0], shape)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(args[0][6:], want[i]))
    assert sp.device_status() == sp.SP_OK


def test_beside_other_kernels():
    """The forward pass and the norm on other streams at the same time (D = 64:
    a CTA of each fits an SM's shared memory, and one waits for the other's
    tensor memory), and one workspace in two graphs replayed in turn."""
    B, N, H, D, P = 1, 3000, 16, 64, 1
    shape = sp.Shape(B, N, H, D, P)
    q, k, v, do = (_to_layout(t, "seq", P, 0.0) for t in _inputs(B, N, H, D, seed=9))
    o, lse = torch.empty_like(q), torch.empty(shape.lse_shape, device="cuda")
    sp.attention_seqsharded(q, k, v, o, shape, lse=lse)
    want = [torch.empty_like(q) for _ in range(3)]
    sp.attention_backward_seqsharded(q, k, v, o, lse, do, *want, shape)
    x = q.view(P, B, N, H * D)
    norm = torch.empty_like(x)
    sp.layer_norm(x, None, None, norm, shape)
    s = [torch.cuda.Stream() for _ in range(3)]
    d = [torch.empty_like(q) for _ in range(3)]
    o2, n2 = torch.empty_like(o), torch.empty_like(norm)
    torch.cuda.synchronize()
    for _ in range(8):
        sp.attention_backward_seqsharded(q, k, v, o, lse, do, *d, shape, stream=s[0])
        sp.attention_seqsharded(q, k, v, o2, shape, stream=s[1])
        sp.layer_norm(x, None, None, n2, shape, stream=s[2])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(d + [o2, n2], want + [o, norm]))
    ws = torch.empty(sp.attention_backward_workspace(shape), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for t in ((q, k, v, o, lse, do), (q, k, v, o, lse, 2 * do)):
        outs.append([torch.empty_like(q) for _ in range(3)])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sp.attention_backward_seqsharded(*t, *outs[-1], shape, workspace=ws)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], want))
    # twice dO: every gradient doubles exactly
    assert all(torch.equal(a, 2 * b) for a, b in zip(outs[1], want))
    assert sp.device_status() == sp.SP_OK


def _saved(d, shape):
    q, k, v, o, lse, do = d
    t = [_to_layout(x, "seq", shape.P) for x in (q, k, v, o, do)]
    lp = torch.full(shape.lse_shape, float("nan"), device="cuda")
    lp[..., :shape.N] = lse
    return t[:4] + [lp, t[4]]


@pytest.mark.parametrize("B,N,H,D,P", [(2, 333, 2, 128, 3), (1, 2433, 9, 64, 2)])
def test_outputs_stay_inside_their_buffers(B, N, H, D, P):
    shape = sp.Shape(B, N, H, D, P)
    q, k, v, do = _inputs(B, N, H, D, seed=4)
    o, lse = _forward64(q, k, v, 1 / math.sqrt(D))
    a = _saved((q, k, v, o, lse, do), shape)
    before = [t.clone() for t in a]
    guard = 4096

    def guarded(nbytes):
        return torch.full((nbytes + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")

    nb = a[0].numel() * 2
    bufs = [guarded(nb) for _ in range(3)] + [guarded(sp.attention_backward_workspace(shape))]
    d = [b[guard:guard + nb].view(torch.bfloat16).view(a[0].shape) for b in bufs[:3]]
    sp.attention_backward_seqsharded(*a, *d, shape, workspace=bufs[3][guard:-guard])
    torch.cuda.synchronize()
    for b in bufs:
        assert (b[:guard] == 0xA5).all() and (b[-guard:] == 0xA5).all()
    for x, y in zip(a, before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    ref, err = _oracle(q, k, v, o, lse, do, 1 / math.sqrt(D))
    _check(d, ref, err, "seq", shape)


def test_forward_then_backward():
    """On what the framework's own forward pass leaves (its O and lse)."""
    B, N, H, D, P = 2, 900, 4, 128, 2
    shape = sp.Shape(B, N, H, D, P)
    scale = 1 / math.sqrt(D)
    q, k, v, do = _inputs(B, N, H, D, seed=8)
    for layout, fwd, bwd in (("seq", sp.attention_seqsharded, sp.attention_backward_seqsharded),
                             ("head", sp.attention, sp.attention_backward)):
        t = [_to_layout(x, layout, P, 0.0) for x in (q, k, v, do)]
        o = torch.empty_like(t[0])
        lse = torch.empty(shape.lse_shape, device="cuda")
        fwd(t[0], t[1], t[2], o, shape, lse=lse)
        d = [torch.empty_like(t[0]) for _ in range(3)]
        bwd(t[0], t[1], t[2], o, lse, t[3], *d, shape)
        ol = _from_layout(o, layout, B, N, H, D, P)[0]
        ref, err = _oracle(q, k, v, ol, lse[..., :N], do, scale)
        _check(d, ref, err, layout, shape)


def test_block_of_norm_projection_attention_and_back():
    """Layer norm -> q, k, v projection -> attention -> O projection and the
    way back through attention and the norm (the projections' own gradients
    are plain matrix products of torch), against autograd in 64 bits."""
    B, N, H, D, P, C = 2, 300, 2, 64, 2, 192
    shape = sp.Shape(B, N, H, D, P)
    g = torch.Generator(device="cuda").manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    Nl = -(-N // P)
    rows = (P, B, Nl)
    x = (r(*rows, C) + 0.3).to(torch.bfloat16)
    w_ln, b_ln = 1 + 0.2 * r(B, C), 0.2 * r(B, C)
    wqkv = (r(3 * H * D, C) / C ** 0.5).to(torch.bfloat16)
    wo = (r(C, H * D) / (H * D) ** 0.5).to(torch.bfloat16)
    dy = r(*rows, C).to(torch.bfloat16)
    e = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    h, y = e(*rows, C), e(*rows, C)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    q, k, v, o = (e(*rows, H, D) for _ in range(4))
    lse = torch.empty(shape.lse_shape, device="cuda")
    sp.layer_norm(x, w_ln, b_ln, h, shape, mean=mean, rstd=rstd)
    sp.qkv_projection(h, wqkv, None, q, k, v, shape)
    sp.attention_seqsharded(q, k, v, o, shape, lse=lse)
    sp.out_projection(o, wo, None, y, shape)
    do = (dy.float().reshape(-1, C) @ wo.float()).to(torch.bfloat16).view(*rows, H, D)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    sp.attention_backward_seqsharded(q, k, v, o, lse, do, dq, dk, dv, shape)
    dqkv = torch.cat([t.reshape(-1, H * D) for t in (dq, dk, dv)], 1)
    dh = (dqkv.float() @ wqkv.float()).to(torch.bfloat16).view(*rows, C)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w_ln), torch.empty_like(b_ln)
    sp.layer_norm_backward(dh, x, w_ln, mean, rstd, dx, shape, dweight=dw, dbias=db)

    xd = x.double().requires_grad_()
    W, Bb = w_ln.double().requires_grad_(), b_ln.double().requires_grad_()
    m = xd.mean(-1, keepdim=True)
    xh = (xd - m) * ((xd - m).square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    hd = xh * W[None, :, None] + Bb[None, :, None]
    qkv = (hd @ wqkv.double().t()).view(P, B, Nl, 3, H, D).permute(3, 1, 4, 0, 2, 5).reshape(3, B, H, N, D)
    att = torch.softmax(qkv[0] @ qkv[1].transpose(2, 3) / D ** 0.5, -1) @ qkv[2]
    od = att.view(B, H, P, Nl, D).permute(2, 0, 3, 1, 4).reshape(P, B, Nl, H * D)
    yd = od @ wo.double().t()
    (yd * dy.double()).sum().backward()
    # h, q, k, v, o, dO, P, dS, dq, dk, dv, dh, dx: 13 roundings to bf16 in a
    # row at 2^-8 / sqrt(3) each, independent, and at most doubled by the
    # softmax's differences and the norm's projection
    bar = 2 * math.sqrt(13 / 3) * HALF
    for got, ref in ((y, yd), (dx, xd.grad), (dw, W.grad), (db, Bb.grad)):
        assert (got.double() - ref).norm() <= bar * ref.norm()
    assert sp.device_status() == sp.SP_OK


@pytest.mark.parametrize("B,N,H,D,P", [(1, 700, 4, 128, 4), (2, 333, 6, 64, 3)])
def test_ranks_of_the_multi_gpu_form(B, N, H, D, P):
    """UlyssesRank's phases for P virtual ranks, the all-to-alls as copies:
    bit-equal to the call on all shards (a row's arithmetic depends neither on
    the layout nor on which heads a call holds); and one rank's whole step."""
    shape = sp.Shape(B, N, H, D, P)
    q, k, v, do = (_to_layout(t, "seq", P, 0.0) for t in _inputs(B, N, H, D, seed=6))
    o, lse = torch.empty_like(q), torch.empty(shape.lse_shape, device="cuda")
    sp.attention_seqsharded(q, k, v, o, shape, lse=lse)
    want = [torch.empty_like(q) for _ in range(3)]
    sp.attention_backward_seqsharded(q, k, v, o, lse, do, *want, shape)
    ranks = [sp.UlyssesRank(shape) for _ in range(P)]

    def exchange(sends):  # recv[r] = chunk r of every rank, in rank order
        return [torch.stack([s[r] for s in sends]) for r in range(P)]

    qkv = [exchange(list(s)) for s in zip(*[r.send_qkv(q[i], k[i], v[i]) for i, r in enumerate(ranks)])]
    lses = [torch.empty(shape.head_group().lse_shape, device="cuda") for _ in ranks]
    outs = [r.attend(*(t[i] for t in qkv), lse=lses[i]) for i, r in enumerate(ranks)]
    dos = exchange([r.send_grad(do[i]) for i, r in enumerate(ranks)])
    grads = [r.attend_backward(*(t[i] for t in qkv), outs[i], lses[i], dos[i])
             for i, r in enumerate(ranks)]
    backs = [exchange(list(g)) for g in zip(*grads)]
    for i, r in enumerate(ranks):
        got = r.finish_grads([b[i] for b in backs])
        assert all(torch.equal(g, w[i]) for g, w in zip(got, want)), i
    one = sp.Shape(B, N, H, D, 1)
    x = [_to_layout(t, "seq", 1, 0.0)[0] for t in _inputs(B, N, H, D, seed=6)]
    rank, lse = sp.UlyssesRank(one), torch.empty(one.lse_shape, device="cuda")
    copy = lambda send, recv: recv.copy_(send)
    rank.step(*x[:3], copy, lse=lse)
    for g, w in zip(rank.backward_step(x[3], lse, copy), want):
        assert torch.equal(g, _from_layout(w, "seq", B, N, H, D, P)[0])
    assert sp.device_status() == sp.SP_OK


@pytest.mark.parametrize("B,N,H,D,P", [(2049, 128, 64, 128, 1), (1025, 256, 64, 128, 2)])
def test_offsets_past_32_bits(B, N, H, D, P):
    """Tensors of more than 2^31 elements: the first and the last heads, by
    the formula and against a call on them alone."""
    shape = sp.Shape(B, N, H, D, P)
    assert B * N * H * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v, do = (torch.empty(shape.seq_sharded, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
                   for _ in range(4))
    o, lse = torch.empty_like(q), torch.empty(shape.lse_shape, device="cuda")
    sp.attention_seqsharded(q, k, v, o, shape, lse=lse)
    d = [torch.empty_like(q) for _ in range(3)]
    sp.attention_backward_seqsharded(q, k, v, o, lse, do, *d, shape)
    assert sp.device_status() == sp.SP_OK
    small = sp.Shape(1, N, 2, D, P)
    for b, h in ((0, 0), (B // 2, 30), (B - 1, H - 2)):
        part = [t[:, b:b + 1, :, h:h + 2].contiguous() for t in (q, k, v, o, do)]
        l = lse[b:b + 1, h:h + 2].contiguous()
        w = [torch.empty_like(part[0]) for _ in range(3)]
        sp.attention_backward_seqsharded(*part[:4], l, part[4], *w, small)
        assert all(torch.equal(x[:, b:b + 1, :, h:h + 2], y) for x, y in zip(d, w))
        logical = [_from_layout(t, "seq", 1, N, 2, D, P)[0] for t in part]
        ref, err = _oracle(*logical[:4], l[..., :N], logical[4], 1 / math.sqrt(D))
        _check(w, ref, err, "seq", small)


def test_binding_refusals():
    B, N, H, D, P = 1, 100, 2, 128, 2
    shape = sp.Shape(B, N, H, D, P)
    q, k, v, do = _inputs(B, N, H, D, seed=1)
    o, lse = _forward64(q, k, v, 1 / math.sqrt(D))
    a = _saved((q, k, v, o, lse, do), shape)
    d = [torch.empty_like(a[0]) for _ in range(3)]
    f = sp.attention_backward_seqsharded
    f(*a, *d, shape)
    for i in range(9):
        args = a + d
        for bad in (None, args[i].cpu(), args[i].double(), args[i][..., :1].expand_as(args[i]),
                    args[i].flatten()[1:]):
            args = a + d
            args[i] = bad
            with pytest.raises((TypeError, ValueError, sp.SpError)):
                f(*args, shape)
    need = sp.attention_backward_workspace(shape)
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need, dtype=torch.uint8),
               torch.empty(need + 1, dtype=torch.uint8, device="cuda")[1:], "workspace"):
        with pytest.raises((TypeError, ValueError, sp.SpError)):
            f(*a, *d, shape, workspace=ws)
    with pytest.raises(sp.SpError):
        f(*a, *d, sp.Shape(B, N, 1, 256, P))
    with pytest.raises((ValueError, sp.SpError)):  # three heads in two groups
        t = [torch.empty(P, B, 50, 3, D, dtype=torch.bfloat16, device="cuda") for _ in range(8)]
        sp.attention_backward(*t[:4], torch.empty(B, 3, 100, device="cuda"), *t[4:],
                              sp.Shape(B, N, 3, D, P))
