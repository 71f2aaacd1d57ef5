"""How near group norm's statistics and outputs come to their definitions, with bounds
that hold for what the kernels claim and for little more: data far from zero, an outlier
among a thread's first values, groups beside ones of another size, several samples to a
workgroup, in every way that groups lie on vectors, held in registers and in two kernels.

U = 2^-24.  A mean is off by at most some roundings of the deviations that it is a mean
of, and of what its own rounding to binary32 left: the sums of thousands of roundings of
either sign, divided by the count, stay below 8 U.  1/deviation: 16 U where no value stands
out, 40 where one does: some tens of steps, each off by U of what a thread's values have
about their own mean.  test_groupnorm_model_host.py has a model in binary32 that keeps
these bounds, and leaves them where a step of the method is missing."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_groupnorm import DT, U, check_backward, check_forward, grouped, half_step, inputs, spread  # noqa: E402

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
def test_far_from_zero(ga, shape):
    N, S, C, G = shape
    noise = normal(N, S, C)
    for x in (1000 + noise, -1e4 + 1e-2 * noise, 1e4 + 1e-3 * noise, 1e6 + noise):
        check(ga, x, G)


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


# several samples to a workgroup, the last one with fewer: groups of whole vectors, and over the border of two
SEVERAL = [(130, 16, 1024, 32), (131, 16, 640, 32), (1030, 4, 320, 32), (2100, 2, 96, 8), (1031, 9, 64, 4)]


@pytest.mark.parametrize("x", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("shape", SEVERAL)
def test_several_samples_to_a_workgroup(ga, shape, x):
    N, S, C, G = shape
    check(ga, normal(N, S, C).to(DT[x]), G, samples=(0, 1, 2, 3, N // 2, N - 3, N - 2, N - 1))
    a, dy, gamma, beta = inputs(N, S, C, x, "fp32", "plain")
    check_forward(ga, a, gamma, beta, G, "silu")
    check_backward(ga, dy, a, gamma, beta, G, "silu", 1)
    # no weight gradients: dx as above, but for the order in which the two means are added
    gn = ga.GroupNorm(C, G, DT[x], activation="silu")
    mean, rstd = torch.empty(2, N, G, device="cuda")
    y, d1, d2 = torch.empty_like(a), torch.empty_like(a), torch.full_like(a, float("nan"))
    gn.forward(a, gamma, beta, y, mean, rstd)
    dg, db = torch.empty(2, 1, C, device="cuda")
    gn.backward(dy, a, gamma, beta, mean, rstd, d1, dg, db)
    gn.backward(dy, a, gamma, beta, mean, rstd, d2)
    one = torch.empty_like(a[:1])
    assert bool(((d1.double() - d2.double()).abs() <= 2 * half_step(DT[x]) * d1.double().abs() + 2.0 ** -18).all())
    for n in (0, 1, N // 2, N - 2, N - 1):      # and each sample's as that of a call on it alone
        gn.backward(dy[n:n + 1], a[n:n + 1], gamma, beta, mean[n:n + 1], rstd[n:n + 1], one)
        assert bool(((one.double() - d2[n:n + 1].double()).abs() <= 2 * half_step(DT[x]) * one.double().abs() + 2.0 ** -18).all())


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("shape,per", [((390, 16, 1024, 32), 2), ((390, 16, 1024, 32), 3), ((200, 16, 640, 32), 2),
                                       ((1600, 4, 320, 32), 2), ((2700, 4, 96, 8), 3)])
def test_samples_of_a_worker_in_a_workgroup(ga, shape, per, x):
    """As many workers as leave each so few samples that a workgroup takes them all, weight gradients and all."""
    N, S, C, G = shape
    a, dy, gamma, beta = inputs(N, S, C, x, "fp32", "plain")
    check_backward(ga, dy, a, gamma, beta, G, "silu", N // per)


@pytest.mark.parametrize("shape,W", [((16, 64, 128, 8), 16), ((16, 36, 64, 32), 4), ((6, 1443, 250, 25), 3), ((3, 5000, 64, 32), 1),
                                     ((4, 3025, 96, 8), 2), ((520, 16384, 16, 2), 1), ((64, 4096, 24, 8), 8)])
def test_sums_of_the_backward_pass(ga, shape, W):
    """Sums of terms of either sign, in chains of at most r = 256 rows (2 to 4 vectors' terms a row for a group, and then
    trees): each addition's rounding is up to U of a partial sum that grows with the root of its terms, so that the sum's error
    has a deviation of U sqrt(r / 6) sqrt(sum of squares); the terms' own, 4 U each, add 4 U / sqrt(3) of it.  Six deviations:
    60 U; and 8 U of the sum itself, as for the means above."""
    N, S, C, G = shape
    a, dy, gamma, _ = inputs(N, S, C, "fp32", "fp32", "plain")
    gn = ga.GroupNorm(C, G)
    mean, rstd = torch.empty(2, N, G, device="cuda")
    y, dx = torch.empty_like(a), torch.empty_like(a)
    dg, db = torch.empty(2, W, C, device="cuda")
    gn.forward(a, gamma, None, y, mean, rstd)
    gn.backward(dy, a, gamma, None, mean, rstd, dx, dg, db, workers=W)
    sums = torch.zeros(4, W, C, dtype=torch.float64, device="cuda")
    for n in range(N):
        xh = (a[n:n + 1].double() - spread(mean[n:n + 1].double(), C)) * spread(rstd[n:n + 1].double(), C)
        d = dy[n:n + 1].double()
        w = n * W // N
        for k, t in enumerate((d * xh, d)):
            sums[k, w] += t.sum((0, 1))
            sums[2 + k, w] += t.square().sum((0, 1))
        if n > 8 and n < N - 2:
            continue
        h = d * gamma.double()
        R, count = spread(rstd[n:n + 1].double(), C), S * C // G
        m1, m2 = grouped(h, G), grouped(h * xh, G)
        e1, e2 = (60 * U * (grouped(t.square(), G) / count).sqrt() + 8 * U * m.abs() for t, m in ((h, m1), (h * xh, m2)))
        m1, m2, e1, e2 = (spread(t, C) for t in (m1, m2, e1, e2))
        want = R * (h - m1 - xh * m2)
        err = R * (e1 + xh.abs() * e2 + 8 * U * (h.abs() + m1.abs() + (xh * m2).abs()))
        assert bool(((dx[n:n + 1].double() - want).abs() <= err).all())
    for got, want, squares in ((dg, sums[0], sums[2]), (db, sums[1], sums[3])):
        assert bool(((got.double() - want).abs() <= 60 * U * squares.sqrt() + 8 * U * want.abs()).all())
