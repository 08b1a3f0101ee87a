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
