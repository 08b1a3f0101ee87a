"""Layer norm of rows whose mean is far larger than their spread, in both
directions.  Where the mean is a number of fp32, x - mean is exact, and the
errors do not grow with |mean| * rstd."""
import pytest

import video_dit_sequence_b200 as sp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LEVELS = (3.0, -100.0, 1000.0, 9984.0, -59904.0)   # numbers of bf16
# hidden sizes whose reciprocal fp32 does not hold, or does; every team shape
SIZES = (24, 104, 328, 512, 840, 1160, 2048, 5120, 7160, 8192)


def _forward(x, w, b):
    N, C = x.shape
    shape = sp.Shape(1, N, 1, 128, 1)
    y = torch.empty_like(x)
    mean = torch.empty(N, device="cuda")
    rstd = torch.empty_like(mean)
    sp.layer_norm(x, w, b, y, shape, mean=mean, rstd=rstd)
    return shape, y, mean, rstd


def _params(C, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.3 * torch.randn(C, generator=g, device="cuda"), torch.randn(C, generator=g, device="cuda")


def _levels(N, C):
    v = torch.tensor(LEVELS, device="cuda").repeat(-(-N // len(LEVELS)))[:N]
    return v, v[:, None].expand(N, C).to(torch.bfloat16).contiguous()


@pytest.mark.parametrize("C", SIZES)
def test_constant_rows_forward(C):
    """The mean is the row's value, xh is 0 and y the bias, whatever 1 / C
    rounds to (a row's sum is a number of fp32)."""
    v, x = _levels(60, C)
    w, b = _params(C, C)
    _, y, mean, rstd = _forward(x, w, b)
    assert torch.equal(mean, v)
    assert torch.equal(y, b.to(torch.bfloat16).expand_as(y))
    # var = 0: eps itself (rounded to fp32), its root and the quotient rounded
    assert ((rstd.double() - 1e3).abs() <= 1e3 * 3 * U).all()


def _backward(x, dy, w, shape, mean, rstd):
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    sp.layer_norm_backward(dy, x, w, mean, rstd, dx, shape, dweight=dw, dbias=db)
    assert sp.device_status() == sp.SP_OK
    return dx, dw, db


@pytest.mark.parametrize("C", SIZES)
def test_constant_rows_backward(C):
    """xh = 0: such rows add nothing to dweight, and dx = rstd (g - mean(g))."""
    v, x = _levels(300, C)
    w, b = _params(C, C)
    g = torch.Generator(device="cuda").manual_seed(C + 1)
    dy = (torch.randn(x.shape, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    shape, _, mean, rstd = _forward(x, w, b)
    dx, dw, db = _backward(x, dy, w, shape, mean, rstd)
    assert (dw == 0).all()
    gd = dy.double() * w.double()
    # half a bf16 step; fp32: g, the sum's tree (9 lane terms of at most 4 vectors
    # and 9 steps: below 40 roundings), the quotient and four products
    ref = 1e3 * (gd - gd.mean(1, keepdim=True))
    err = 1e3 * 48 * U * (gd.abs() + gd.abs().mean(1, keepdim=True))
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + err) + err).all()
    # (the frozen form computes the same dx)
    alone = torch.empty_like(dx)
    sp.layer_norm_backward(dy, x, w, mean, rstd, alone, shape)
    assert torch.equal(alone, dx)


@pytest.mark.parametrize("C", [64, 512, 2048, 8192])
def test_one_value_stands_out(C):
    """Rows of 9,984 with one value 64 above: the mean and x - mean are numbers
    of fp32 (C a power of two), so xh carries the roundings of rstd and one
    product, at a mean of up to 14,000 deviations."""
    N = 100
    x = torch.full((N, C), 9984.0, device="cuda")
    at = torch.arange(N, device="cuda") * 7 % C
    x[torch.arange(N, device="cuda"), at] += 64
    x = x.to(torch.bfloat16)
    w, b = _params(C, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    dy = torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16)
    shape, y, mean, rstd = _forward(x, w, b)
    dx, dw, db = _backward(x, dy, w, shape, mean, rstd)
    xd, d, wd = x.double(), dy.double(), w.double()
    xc = xd - xd.mean(1, keepdim=True)
    r = (xc.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    xh = xc * r
    assert torch.equal(mean.double(), xd.mean(1))
    # the sum of squares, whose large term meets at most 12 terms of its lane, 5
    # of its warp and 4 of its team (halved by the root), eps, root, quotient
    assert ((rstd.double() - r[:, 0]).abs() <= 16 * U * r[:, 0]).all()
    yd = xh * wd + b.double()
    ey = 20 * U * (xh * wd).abs() + 2 * U * b.abs()
    assert ((y.double() - yd).abs() <= 2.0 ** -8 * (yd.abs() + ey) + ey).all()
    # xh's 20 roundings, the product, the rows of a team and the sums of teams
    # and blocks: at most N + 20 additions
    edw = (N + 42) * U * (d * xh).abs().sum(0)
    assert ((dw.double() - (d * xh).sum(0)).abs() <= edw).all()
    assert ((db.double() - d.sum(0)).abs() <= (N + 20) * U * d.abs().sum(0)).all()
    gd = d * wd
    c2 = (gd * xh).mean(1, keepdim=True)
    ref = r * (gd - gd.mean(1, keepdim=True) - xh * c2)
    # rstd three times over, the sum of 16 terms a lane and 10 steps, 5 products
    err = 100 * U * r * (gd.abs() + gd.abs().mean(1, keepdim=True)
                        + xh.abs() * (gd * xh).abs().mean(1, keepdim=True))
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + err) + err).all()


@pytest.mark.parametrize("C", [24, 40, 104, 200, 264, 328])
def test_rows_whose_mean_over_their_deviation_is_past_fp32(C):
    """Constant rows of 1e36: mean * rstd is infinite, and lanes of a team that
    have no columns must not bring that into the row's sums."""
    x = torch.full((70, C), 1e36, device="cuda").to(torch.bfloat16)
    w, b = _params(C, 5)
    dy = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(6),
                     device="cuda").to(torch.bfloat16)
    shape, y, mean, rstd = _forward(x, w, b)
    assert torch.equal(mean, x[:, 0].float()) and torch.equal(y, b.to(torch.bfloat16).expand_as(y))
    dx, dw, db = _backward(x, dy, w, shape, mean, rstd)
    assert (dw == 0).all()
    gd = dy.double() * w.double()
    ref = 1e3 * (gd - gd.mean(1, keepdim=True))
    err = 1e3 * 48 * U * (gd.abs() + gd.abs().mean(1, keepdim=True))   # (as above)
    assert ((dx.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + err) + err).all()
