"""Layer norm of rows that are far from zero and nearly, or quite, constant."""
import math

import pytest

from test_gpu_training import DT, HALF_STEP, LEAST, TINY, U, chain, f32, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


def reference(s, gamma, beta, eps, dtype):
    """y, mean, rstd in binary64 with tolerances, for a mean that is taken twice:
    the second time of the deviations from the first.

    The first mean is off by h <= (k + 2) u mean|s|.  A deviation from it is
    rounded once (u).  Their mean, and so the corrected mean and deviations, is
    off by (k + 2) u of their mean magnitude, at most that of the true ones plus
    h; the corrected mean is rounded once more.  The variance is the mean square
    less the squared correction: each is off by (k + 4) u of the mean square, at
    most twice the variance plus h^2."""
    dim = s.shape[1]
    k = chain(dim)
    mean = s.mean(1, keepdim=True)
    d = s - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    h = (k + 2) * U * s.abs().mean(1, keepdim=True)
    size = d.abs().mean(1, keepdim=True) + h
    off = (k + 2) * U * size
    tol_mean = U * mean.abs() + 2 * off + TINY
    tol_d = off + U * (d.abs() + h) + U * d.abs()
    tol_var = 2 * (k + 4) * U * 2 * (var + h * h) + off * off
    low = (var + eps - tol_var).clamp_min(eps * (1 - 2 * U))
    tol_rstd = (low ** -0.5 - rstd) + 5 * U * rstd
    y = d * rstd * gamma + beta
    tol_y = gamma.abs() * (tol_d * (rstd + tol_rstd) + d.abs() * tol_rstd + 2 * U * (d * rstd).abs()) + U * y.abs()
    tol_y = tol_y * 1.01 + HALF_STEP[dtype] * (y.abs() + tol_y) + LEAST[dtype]
    return (y, tol_y), (mean[:, 0], tol_mean[:, 0]), (rstd[:, 0], tol_rstd[:, 0])


DIMS = [64, 100, 257, 1001, 2500, 5120, 8193, 16384, 20001]


def check(ga, x, res=None):
    rows, dim = x.shape
    gen = torch.Generator().manual_seed(dim)
    gamma, beta = (1 + 0.2 * torch.randn(dim, generator=gen)).cuda(), torch.randn(dim, generator=gen).cuda()
    s = x if res is None else (x.float() + res.float()).to(x.dtype)
    want = reference(s.double(), gamma.double(), beta.double(), f32(1e-5), x.dtype)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ga.LayerNorm(dim, x.dtype, torch.float32, backward=False).forward(x, gamma, beta, y, mean, rstd, residual=res, eps=1e-5)
    for name, got, (ref, tol) in zip(("mean", "rstd", "y"), (mean, rstd, y), (want[1], want[2], want[0])):
        within(got, ref, tol, name)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype", list(DT))
def test_constant_rows(ga, dim, dtype):
    values = torch.tensor([0.1, -3.7, 1000.1, -1000.3, 9999.7, 12345.6, 60000.0], dtype=torch.float64)
    x = values.to(DT[dtype]).cuda()[:, None].expand(-1, dim).contiguous()
    check(ga, x)
    check(ga, x, res=(x * 0.0625).contiguous())            # 63750 at most: below fp16's largest


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("offset", [1e3, -1e4, 1e6])
def test_little_spread(ga, dim, offset):
    """A spread of a few units in the last place of the offset, and one of 1e-3
    of it."""
    gen = torch.Generator().manual_seed(dim)
    for size in (4 * U * abs(offset), 1e-3 * abs(offset)):
        x = (offset + size * torch.randn(6, dim, generator=gen, dtype=torch.float64)).float().cuda()
        check(ga, x)
        check(ga, x, res=(0.5 * x).contiguous())


@pytest.mark.parametrize("dim,rows", [(61, 70000), (509, 19000), (2047, 4800), (4093, 4800), (8189, 2400), (12289, 1200),
                                      (16390, 2400)])
def test_far_and_near_rows_in_turn(ga, dim, rows):
    """A workgroup's rows, two or three of them, need the correction or not."""
    gen = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    far = torch.rand(rows, 1, generator=gen, device="cuda") < 0.5
    check(ga, x + torch.where(far, 1e4, 0.0))


def test_one_far_element(ga):
    """An outlier at the row's start or end."""
    for at in (0, -1):
        x = torch.randn(5, 3001, generator=torch.Generator().manual_seed(1)).cuda()
        x[:, at] = 1e5
        check(ga, x)
    assert math.isfinite(float(x.sum()))
