"""How near group norm's statistics and outputs come to their definitions, with bounds
that hold for what the kernels claim and for little more: an outlier among a thread's
first values, groups beside ones of another size, in every way that groups lie on vectors,
held in registers and in two kernels.

U = 2^-24.  A mean is off by at most some roundings of the deviations that it is a mean
of: the sums of thousands of roundings of either sign, divided by the count, stay below
8 U of the deviation (a model in binary32 of the threads' sums gives up to 1.5, and 30 to
500000 where the rounding of the first mean is not made good).  The variance: of a thread
whose sums of squares are taken up before they hold eight rows, each step is off by U of
what the thread's values have about their own mean: 16 U of 1/deviation together where no
value stands out (the model: up to 6), 40 where one does (up to 14; 40 to 400 without)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_groupnorm import DT, U, grouped, half_step, spread  # noqa: E402

TINY_EPS = 1e-30


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


def check(ga, x, G, rel=16, samples=None, eps=TINY_EPS):
    """All of x through the kernels; the `samples` (all, if None) against binary64."""
    N, S, C = x.shape
    gn = ga.GroupNorm(C, G, x.dtype, backward=False)
    y = torch.empty(x.shape, dtype=x.dtype, device="cuda")
    mean, rstd = torch.empty(2, N, G, device="cuda")
    gn.forward(x, None, None, y, mean, rstd, eps=eps)
    for n in range(N) if samples is None else samples:
        xd = x[n:n + 1].double()
        m = grouped(xd, G)
        d = xd - spread(m, C)
        sigma = grouped(d.square(), G).sqrt()
        r = (sigma.square() + eps) ** -0.5
        mean_err = 8 * U * (sigma + U * m.abs())
        assert bool(((mean[n:n + 1].double() - m).abs() <= mean_err + U * m.abs()).all())
        assert bool(((rstd[n:n + 1].double() / r - 1).abs() <= rel * U).all())
        want = d * spread(r, C)
        err = spread(mean_err * r, C) + (rel + 4) * U * want.abs()
        tol = err + half_step(x.dtype) * (want.abs() + err) + torch.finfo(x.dtype).tiny
        assert bool(((y[n:n + 1].double() - want).abs() <= tol).all())


def normal(N, S, C, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 7 * C + S)
    return torch.randn(N, S, C, generator=gen, device="cuda")


# name, N, S, C, G: groups of whole vectors, over the border of two, and several to a vector (binary32 and 16 bits)
REGISTERS = [(16, 64, 128, 8), (16, 36, 96, 16), (16, 36, 64, 32), (9, 49, 80, 4), (5, 25, 24, 8)]
KERNELS = [(6, 1443, 250, 25), (3, 4000, 128, 8), (3, 5000, 64, 32), (4, 3025, 96, 8)]
# 256 rows to a thread: more samples than workgroups
MANY_ROWS = [(512, 16384, 16, 2, "fp32"), (512, 21760, 12, 2, "fp32"), (512, 16384, 16, 8, "fp32"), (512, 32768, 16, 8, "bf16")]


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("shape", REGISTERS + KERNELS)
def test_plain(ga, shape, x):
    N, S, C, G = shape
    check(ga, normal(N, S, C).to(DT[x]), G)


@pytest.mark.parametrize("shape", REGISTERS + KERNELS)
def test_beside_groups_of_another_size(ga, shape):
    """Each group's sums are about values of its own, whatever its neighbours in a vector hold."""
    N, S, C, G = shape
    x = normal(N, S, C).reshape(N, S, G, C // G)
    x[:, :, ::2] = 1e9 * (1 + 0.1 * x[:, :, ::2])
    x[:, :, 1::2] += 1000
    check(ga, x.reshape(N, S, C), G)


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("shape", REGISTERS + KERNELS)
def test_outliers(ga, shape, x):
    N, S, C, G = shape
    a = normal(N, S, C)
    a[0, 0, 0] = 1e4
    a[1, S // 2, C - 1] = -1e4
    a[2, 1] = 1e4 * a[2, 1]
    check(ga, a.clamp(-6e4, 6e4).to(DT[x]), G, rel=40)


@pytest.mark.parametrize("shape", MANY_ROWS)
def test_outliers_of_threads_with_many_rows(ga, shape):
    N, S, C, G, x = shape
    a = torch.empty(N, S, C, dtype=DT[x], device="cuda")
    for n in range(0, N, 64):
        a[n:n + 64] = normal(64, S, C, n)
    check(ga, a, G, 16, (0, 7, N - 1))
    a[0, 0, 0] = 1e4
    a[1, 3, C - 1] = -1e4
    a[2, :4] *= 1e4                            # the first values of four rows of threads
    a[N - 1, :, 0] += 1000                     # one channel apart
    check(ga, a, G, 40, (0, 1, 2, N - 1))
