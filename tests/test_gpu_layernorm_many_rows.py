"""Layer norm of more rows than one sweep of the workgroups takes: every team
goes round its row loop two or three times, the last time with part of its
rows, in every element type, with outputs of their own and over their inputs."""
import math

import pytest

from test_gpu_training import DT, check_ln_bwd, check_ln_fwd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


# a row's columns and the rows of a workgroup of 1024 threads (backward) or of
# 256 and more (forward)
BWD32 = [(61, 64), (100, 32), (250, 16), (509, 8), (1001, 4), (2047, 2), (4093, 1), (8189, 1), (12289, 1)]
BWD16 = [(100, 64), (250, 32), (509, 16), (1001, 16), (2047, 4), (4093, 2), (8191, 1), (12289, 1)]
# and the workgroups of a sweep
FWD32 = [(61, 16, 2048), (100, 8, 2048), (250, 4, 2048), (509, 4, 2048), (1001, 4, 2048), (2047, 1, 2048), (4093, 1, 2048),
         (8189, 1, 1024), (12289, 1, 512), (16390, 1, 1024)]
FWD16 = [(100, 16, 2048), (250, 8, 2048), (509, 4, 2048), (1001, 4, 2048), (2047, 1, 2048), (4093, 1, 2048),
         (8191, 1, 1024), (12289, 1, 512), (16390, 1, 1024)]


def rows_of(sweep):
    return 2 * sweep + sweep // 3 + 1


def cases(binary32, others):
    return [(x,) + c for x in DT for c in (binary32 if x == "fp32" else others)]


@pytest.mark.parametrize("x,dim,at_once,blocks", cases(FWD32, FWD16))
def test_forward(ga, x, dim, at_once, blocks):
    check_ln_fwd(ga, rows_of(at_once * blocks), dim, DT[x], torch.float32, res=dim % 2 == 1)


@pytest.mark.parametrize("x,dim,at_once", cases(BWD32, BWD16))
def test_backward(ga, x, dim, at_once):
    check_ln_bwd(ga, rows_of(at_once * 256), dim, DT[x], torch.float32, dp_dtype=torch.float32, res=dim % 2 == 1)
    # 64 groups of 4 workgroups each
    per = rows_of(at_once * 4)
    check_ln_bwd(ga, 64 * per, dim, DT[x], DT[x], dp_dtype=DT[x], groups=64)


@pytest.mark.parametrize("x", list(DT))
def test_backward_of_long_rows(ga, x):
    check_ln_bwd(ga, 1030, 16391, DT[x], torch.float32, res=True, groups=2)


@pytest.mark.parametrize("x,dim,at_once,blocks", cases(FWD32, FWD16))
def test_forward_in_place(ga, x, dim, at_once, blocks):
    gen = torch.Generator(device="cuda").manual_seed(dim)
    rows = rows_of(at_once * blocks)
    a, r = (torch.randn(rows, dim, generator=gen, device="cuda").to(DT[x]) for _ in range(2))
    ln = ga.LayerNorm(dim, DT[x], torch.float32, backward=False)
    y, s = torch.empty_like(a), torch.empty_like(a)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ln.forward(a, None, None, y, mean, rstd, residual=r, sum_out=s)
    stats = mean.clone(), rstd.clone()
    for k in range(4):                                     # sum over x, over the residual; y over x, over the residual
        a2, r2, other = a.clone(), r.clone(), torch.empty_like(a)
        y2, s2 = [(other, a2), (other, r2), (a2, other), (r2, other)][k]
        ln.forward(a2, None, None, y2, mean, rstd, residual=r2, sum_out=s2)
        assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(mean, stats[0]) and torch.equal(rstd, stats[1])


@pytest.mark.parametrize("x,dim,at_once", cases(BWD32, BWD16))
def test_backward_in_place(ga, x, dim, at_once):
    gen = torch.Generator(device="cuda").manual_seed(dim)
    rows = rows_of(at_once * 256)
    t = [torch.randn(rows, dim, generator=gen, device="cuda").to(DT[x]) for _ in range(3)]      # dy, x, dsum
    gamma = torch.randn(dim, generator=gen, device="cuda")
    mean, rstd = torch.randn(rows, generator=gen, device="cuda"), 1 + torch.rand(rows, generator=gen, device="cuda")
    ln = ga.LayerNorm(dim, DT[x], torch.float32)
    dx, sums = torch.empty_like(t[0]), torch.empty(2, 1, dim, device="cuda")
    ln.backward(t[0], t[1], gamma, mean, rstd, dx, sums[0], sums[1], dsum=t[2])
    assert math.isfinite(float(sums.sum()))
    for k in range(3):
        c, again = [a.clone() for a in t], torch.empty_like(sums)
        ln.backward(c[0], c[1], gamma, mean, rstd, c[k], again[0], again[1], dsum=c[2])
        assert torch.equal(c[k], dx) and torch.equal(again, sums)
