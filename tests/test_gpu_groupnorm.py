"""Group norm with an activation on the GPU against its formulas in binary64.

Tolerances count roundings (u = 2^-24 of binary32, half a step of the output's
type).  A sum of many terms passes a value through at most CHAIN additions (a
thread's rows, then the tree over threads, then the parts)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
CHAIN = 512
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


def half_step(dt):
    return torch.finfo(dt).eps / 2


def act(z, name):
    return z if name is None else z.clamp_min(0) if name == "relu" else z * torch.sigmoid(z)


def slope(z, name):
    if name is None:
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def images(N, S, C, layout, dt, gen, fill=math.nan):
    """An [N][S][C] tensor of that memory layout; what lies around it is `fill`."""
    if layout == "plain":
        return torch.empty(N, S, C, dtype=dt, device="cuda")
    if layout == "wide":            # rows inside wider ones, at an odd offset
        return torch.full((N, S, C + 11), fill, dtype=dt, device="cuda")[:, :, 3:3 + C]
    if layout == "gaps":            # samples apart
        return torch.full((N, S + 2, C), fill, dtype=dt, device="cuda")[:, 1:1 + S]
    if layout == "mixed":           # samples interleaved
        return torch.empty(S, N, C, dtype=dt, device="cuda").transpose(0, 1)
    raise ValueError(layout)


def grouped(a, G):
    """[N][S][C] -> [N][G] mean over positions and the group's channels."""
    N, S, C = a.shape
    return a.reshape(N, S, G, C // G).mean((1, 3))


def spread(a, C):
    """[N][G] -> [N][1][C]"""
    return a.repeat_interleave(C // a.shape[1], 1)[:, None, :]


def check_forward(ga, x, gamma, beta, G, name, y_of=None, eps=EPS):
    N, S, C = x.shape
    dt, pdt = x.dtype, torch.float32 if gamma is None else gamma.dtype
    gn = ga.GroupNorm(C, G, dt, pdt, activation=name, backward=False)
    y = torch.empty(N, S, C, dtype=dt, device="cuda") if y_of is None else y_of
    mean, rstd = torch.empty(N, G, device="cuda"), torch.empty(N, G, device="cuda")
    xd = x.double()
    gn.forward(x, gamma, beta, y, mean, rstd, eps=eps)
    g = torch.ones(C, dtype=torch.float64, device="cuda") if gamma is None else gamma.double()
    b = torch.zeros(C, dtype=torch.float64, device="cuda") if beta is None else beta.double()
    m = grouped(xd, G)
    d = xd - spread(m, C)
    var = grouped(d.square(), G)
    r = (var + eps) ** -0.5
    # sums about a value of the data: the mean is off by the sum's roundings, of the deviations' size, and its own
    dev = grouped(d.abs(), G) + var.sqrt()
    mean_err = CHAIN * U * dev + 2 * U * m.abs()
    assert bool(((mean.double() - m).abs() <= mean_err).all())
    # var's relative error: the sum's; the deviations' (2 U of the values about the mean); the mean's square
    far = (mean_err * r).clamp_max(1e3)
    rel = (CHAIN + 8) * U + far * far + 2 * far * U
    assert bool(((rstd.double() / r - 1).abs() <= rel + 4 * U).all())
    xh, R = d * spread(r, C), spread(r, C)
    xh_err = spread(mean_err, C) * R + xh.abs() * (spread(rel, C) + 6 * U)
    z = xh * g + b
    z_err = g.abs() * xh_err + U * (2 * (xh * g).abs() + 2 * z.abs())
    want = act(z, name)
    err = 1.2 * z_err + (0 if name is None else U * (8 + 2 * z.abs()) * want.abs())
    tol = err + half_step(dt) * (want.abs() + err) + torch.finfo(dt).tiny
    assert bool(((y.double() - want).abs() <= tol).all())
    return y, mean, rstd


def check_backward(ga, dy, x, gamma, beta, G, name, W=1, dp=torch.float32, dx=None, chain=CHAIN):
    N, S, C = x.shape
    dt, pdt = x.dtype, torch.float32 if gamma is None else gamma.dtype
    xd = x.double()
    g = torch.ones(C, dtype=torch.float64, device="cuda") if gamma is None else gamma.double()
    b = torch.zeros(C, dtype=torch.float64, device="cuda") if beta is None else beta.double()
    m = grouped(xd, G)
    mean = m.float()
    rstd = ((grouped((xd - spread(m, C)).square(), G) + EPS) ** -0.5).float()
    xh = (xd - spread(mean.double(), C)) * spread(rstd.double(), C)
    z = xh * g + b
    z_err = U * (4 * (xh * g).abs() + 2 * z.abs())
    if name == "relu":              # the derivative jumps: no gradient where a rounding decides
        dy[z.abs() <= 4 * z_err + 1e-30] = 0
    dyd = dy.double()
    gn = ga.GroupNorm(C, G, dt, pdt, activation=name)
    dx = torch.empty(N, S, C, dtype=dt, device="cuda") if dx is None else dx
    dg, db = (torch.full((W, C), math.nan, dtype=dp, device="cuda") for _ in range(2))
    gn.backward(dy, x, gamma, beta, mean, rstd, dx, dg, db, workers=W)
    dz = dyd * slope(z, name)
    dz_err = torch.zeros_like(dz) if name is None else dyd.abs() * (0 if name == "relu" else 0.6 * z_err + 16 * U * (1 + z.abs()))
    h, h_err = dz * g, dz_err * g.abs()
    m1, m2 = grouped(h, G), grouped(h * xh, G)
    e1 = grouped(h_err + chain * U * h.abs(), G)
    e2 = grouped(h_err * xh.abs() + (chain + 4) * U * (h * xh).abs(), G)
    R = spread(rstd.double(), C)
    want = R * (h - spread(m1, C) - xh * spread(m2, C))
    err = R * (h_err + spread(e1, C) + xh.abs() * spread(e2, C) + 4 * U * (h.abs() + spread(m1.abs(), C) + (xh * spread(m2, C)).abs()))
    tol = err + half_step(dt) * (want.abs() + err) + torch.finfo(dt).tiny
    assert bool(((dx.double() - want).abs() <= tol).all())
    per = (W, N // W * S, C)

    def worker(a):
        return a.reshape(per).sum(1)

    for got, terms, e in ((dg, dz * xh, dz_err * xh.abs() + 4 * U * (dz * xh).abs()), (db, dz, dz_err)):
        want = worker(terms)
        err = worker(e) + 2 * chain * U * worker(terms.abs())
        assert bool(((got.double() - want).abs() <= err + half_step(dp) * (want.abs() + err) + torch.finfo(dp).tiny).all())
    return dx, dg, db


SHAPES = [
    # N, S, C, G
    (1, 1, 1, 1), (2, 1, 8, 8), (3, 1, 64, 4), (1, 5, 6, 2), (2, 7, 12, 4), (5, 9, 20, 4), (3, 64, 32, 32), (2, 36, 1024, 32),
    (4, 169, 384, 32), (2, 100, 96, 32), (3, 33, 250, 25), (2, 49, 1001, 7), (1, 300, 40, 1), (2, 17, 2049, 3),
    (1, 1024, 320, 32), (2, 3025, 96, 8), (1, 4099, 64, 16), (1, 10007, 16, 4), (2, 2500, 640, 32), (1, 700, 1280, 32),
    (33, 16, 128, 32), (1, 64, 4100, 4), (2, 3, 9000, 1), (1, 20011, 24, 8), (300, 4, 48, 16), (1, 130, 16384, 2),
]
TYPES = [("fp32", "fp32"), ("fp16", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")]


def inputs(N, S, C, x, p, layout, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(N * 7 + S * 3 + C + seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    a, dy = images(N, S, C, layout, DT[x], gen), images(N, S, C, layout, DT[x], gen)
    a.copy_(normal(N, S, C) * (0.5 + normal(C).abs()) + normal(N, 1, C))
    dy.copy_(normal(N, S, C))
    gamma, beta = (1 + 0.3 * normal(C)).to(DT[p]), (0.3 * normal(C)).to(DT[p])
    return a, dy, gamma, beta


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_forward(ga, i, shape):
    N, S, C, G = shape
    for j, (x, p) in enumerate(TYPES):
        a, _, gamma, beta = inputs(N, S, C, x, p, "plain")
        check_forward(ga, a, gamma, beta, G, [None, "relu", "silu"][(i + j) % 3])


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_backward(ga, i, shape):
    N, S, C, G = shape
    for j, (x, p) in enumerate(TYPES):
        a, dy, gamma, beta = inputs(N, S, C, x, p, "plain", 1)
        W = [w for w in (N, 2, 3, 1) if N % w == 0][(i + j) % (2 if N > 1 else 1)]
        check_backward(ga, dy, a, gamma, beta, G, [None, "silu", "relu"][(i + j) % 3], W, DT[["fp32", x][j % 2]])


@pytest.mark.parametrize("layout", ["wide", "gaps", "mixed"])
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 5, 6, 2), (2, 33, 250, 25), (4, 100, 96, 32), (2, 700, 200, 8), (3, 2111, 41, 41)])
def test_layouts(ga, shape, x, layout):
    """The bits of the plain layout; nothing beside the images is read into a result or written."""
    N, S, C, G = shape
    a, dy, gamma, beta = inputs(N, S, C, x, "fp32", layout)
    y, dx = (images(N, S, C, layout, DT[x], None) for _ in range(2))
    got = check_forward(ga, a, gamma, beta, G, "silu", y)
    got2 = check_backward(ga, dy, a, gamma, beta, G, "silu", N, dx=dx)
    want = check_forward(ga, a.contiguous(), gamma, beta, G, "silu")
    want2 = check_backward(ga, dy.contiguous(), a.contiguous(), gamma, beta, G, "silu", N)
    assert all(torch.equal(p, q) for p, q in zip(got + got2, want + want2))
    for t, inner in ((y, slice(3, 3 + C)), (dx, slice(3, 3 + C))):
        whole = t._base
        if layout == "wide":
            assert bool(whole[:, :, :3].isnan().all()) and bool(whole[:, :, 3 + C:].isnan().all())
        elif layout == "gaps":
            assert bool(whole[:, 0].isnan().all()) and bool(whole[:, -1].isnan().all())


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 5, 6, 2), (3, 33, 250, 25), (2, 64, 1280, 32), (2, 2111, 41, 41), (1, 9000, 320, 32), (3, 2500, 640, 32)])
def test_in_place(ga, shape, x):
    """y over x, dx over dy or x: the bits of the calls with outputs of their own."""
    N, S, C, G = shape
    a, dy, gamma, beta = inputs(N, S, C, x, "fp32", "plain")
    gn = ga.GroupNorm(C, G, DT[x], activation="silu")
    mean, rstd = torch.empty(2, N, G, device="cuda")
    y = torch.empty_like(a)
    gn.forward(a, gamma, beta, y, mean, rstd)
    b = a.clone()
    gn.forward(b, gamma, beta, b)
    assert torch.equal(b, y)
    outs = []
    for k in range(3):
        t = [dy.clone(), a.clone(), torch.empty_like(a)]
        dg, db = torch.empty(2, N, C, device="cuda")
        gn.backward(t[0], t[1], gamma, beta, mean, rstd, t[k], dg, db, workers=N)
        outs.append((t[k], dg, db))
    assert all(torch.equal(p, q) for o in outs[:2] for p, q in zip(o, outs[2]))


@pytest.mark.parametrize("name", [None, "relu", "silu"])
def test_without_weights(ga, name):
    a, dy, _, beta = inputs(3, 50, 24, "bf16", "fp32", "plain")
    check_forward(ga, a, None, None, 8, name)
    check_forward(ga, a, None, beta, 8, name)
    check_backward(ga, dy, a, None, None, 8, name, 3)
    check_backward(ga, dy, a, None, beta, 8, name, 1)


@pytest.mark.parametrize("shape", [(3, 20, 16, 2), (2, 5000, 64, 4), (2, 1024, 640, 32)])
@pytest.mark.parametrize("x", ["fp32", "fp16"])
def test_far_from_zero(ga, shape, x):
    """Groups whose mean is far past their deviation, constant ones among them, and one spike in a group."""
    N, S, C, G = shape
    gen = torch.Generator(device="cuda").manual_seed(S)
    noise = torch.randn(N, S, C, generator=gen, device="cuda")
    a = (1000 + noise).to(DT[x])
    a[0, :, : C // G] = 1000.0
    check_forward(ga, a, None, None, G, None)
    # a copy: the spikes times 1e15 below would be 3e19, whose square, 9e38, is past binary32
    b = noise.to(DT[x]).clone()
    b[0, 0, 0] = 30000.0
    b[N - 1, S // 2, C - 1] = -30000.0
    check_forward(ga, b, None, None, G, None)
    if x == "fp32":
        check_forward(ga, noise * 1e-3 + 1e4, None, None, G, "silu", eps=1e-12)
        check_forward(ga, noise * 1e15, None, None, G, None)
        check_forward(ga, noise * 1e-20, None, None, G, None)


def test_constant_group_gives_the_bias(ga):
    a = torch.full((2, 77, 32), 123.456, device="cuda")
    beta = torch.randn(32, device="cuda")
    y, mean, rstd = check_forward(ga, a, None, beta, 4, None)
    assert torch.equal(y, beta.expand(2, 77, 32)) and bool((rstd - EPS ** -0.5).abs().max() < 1e-3)
    assert bool((mean == 123.456).all()) or float((mean.double() - float(a[0, 0, 0])).abs().max()) == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("shape", [(3, 20, 16, 2), (2, 5000, 64, 4), (3, 300, 40, 4)])
def test_not_finite_stays_in_its_group(ga, shape, bad):
    N, S, C, G = shape
    a, dy, gamma, beta = inputs(N, S, C, "fp32", "fp32", "plain")
    gn = ga.GroupNorm(C, G, activation="silu")
    outs = []
    for k in range(2):
        mean, rstd = torch.empty(2, N, G, device="cuda")
        y, dx = torch.empty_like(a), torch.empty_like(a)
        dg, db = torch.empty(2, N, C, device="cuda")
        gn.forward(a, gamma, beta, y, mean, rstd)
        gn.backward(dy, a, gamma, beta, mean, rstd, dx, dg, db, workers=N)
        outs.append((y, dx, dg, db))
        a[1, S // 2, C // G] = bad                                # sample 1, group 1
    inside = torch.zeros(N, C, dtype=torch.bool, device="cuda")
    inside[1, C // G:2 * (C // G)] = True
    for k, (p, q) in enumerate(zip(*outs)):
        m = inside[:, None, :].expand_as(p) if k < 2 else inside
        assert torch.equal(p[~m], q[~m])
        if k < 3:
            assert bool(q[m].isnan().all())


def test_differences(ga):
    """The gradients against differences of the forward pass's formula."""
    N, S, C, G = 2, 5, 12, 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, dy = torch.randn(2, N, S, C, generator=gen, device="cuda")
    gamma, beta = torch.randn(2, C, generator=gen, device="cuda")
    gn = ga.GroupNorm(C, G, activation="silu")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(2, N, G, device="cuda")
    dg, db = torch.empty(2, 1, C, device="cuda")
    gn.forward(x, gamma, beta, y, mean, rstd)
    gn.backward(dy, x, gamma, beta, mean, rstd, dx, dg, db)

    def loss(x, gamma, beta):
        m = grouped(x, G)
        d = x - spread(m, C)
        z = d * spread((grouped(d.square(), G) + EPS) ** -0.5, C) * gamma + beta
        return float((act(z, "silu") * dy.double()).sum())

    args = [x.double(), gamma.double(), beta.double()]
    for k, got in enumerate((dx, dg[0], db[0])):
        for i in range(0, got.numel(), 7):
            step, ends = 1e-5, []
            for s in (step, -step):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += s
                ends.append(loss(*moved))
            want = (ends[0] - ends[1]) / (2 * step)
            # the difference is off by step^2 times a third derivative; the kernel by some 100 roundings of its terms
            assert abs(float(got.reshape(-1)[i]) - want) <= 2e-5 * (1 + abs(want))


@pytest.mark.parametrize("shape", [(2, 36, 1024, 32), (2, 5000, 320, 32), (64, 36, 64, 8), (1, 64, 1280, 32)])
def test_repeats_streams_and_graphs(ga, shape):
    """Equal bits on every call, on another stream, and replayed from a graph with work between."""
    N, S, C, G = shape
    a, dy, gamma, beta = inputs(N, S, C, "bf16", "fp32", "plain")
    gn = ga.GroupNorm(C, G, torch.bfloat16, activation="silu")
    y, dx = torch.empty_like(a), torch.empty_like(a)
    mean, rstd = torch.empty(2, N, G, device="cuda")
    dg, db = torch.empty(2, N, C, device="cuda")

    def both():
        gn.forward(a, gamma, beta, y, mean, rstd)
        gn.backward(dy, a, gamma, beta, mean, rstd, dx, dg, db, workers=N)

    outs = (y, mean, rstd, dx, dg, db)
    both()
    want = [t.clone() for t in outs]

    def same():
        ok = all(torch.equal(p, q) for p, q in zip(outs, want))
        for t in outs:
            t.fill_(math.nan)
        return ok

    for _ in range(3):
        both()
        assert same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        graph.replay()
        assert same()
        a.copy_(a.flip(0))                    # other inputs between the replays, and back
        both()
        a.copy_(a.flip(0))
        torch.cuda.synchronize()
        both()
        assert same()


def test_nothing_to_do(ga):
    gn = ga.GroupNorm(16, 4)
    for shape in ((0, 5, 16), (3, 0, 16)):
        x = torch.empty(shape, device="cuda")
        mean, rstd = torch.full((2, shape[0], 4), 7.0, device="cuda")
        gn.forward(x, None, None, x, mean, rstd)
        assert bool((mean == 7).all())
        dg, db = torch.full((2, 3, 16), 7.0, device="cuda")
        gn.backward(x, x, None, None, mean, rstd, x, dg, db, workers=3)
        assert not bool(dg.any()) and not bool(db.any())


def test_refusals(ga):
    gn = ga.GroupNorm(16, 4, torch.bfloat16)
    x = torch.zeros(2, 3, 16, dtype=torch.bfloat16, device="cuda")
    mean, rstd = torch.zeros(2, 2, 4, device="cuda")
    for bad in (x.float(), x.cpu(), x[..., :8], x[0, 0]):
        with pytest.raises((ValueError, TypeError)):
            gn.forward(bad, None, None, bad)
    with pytest.raises(ValueError):
        gn.forward(x, None, None, x[:, :2])
    with pytest.raises(ValueError):
        gn.forward(x, torch.ones(8, device="cuda"), None, x)
    with pytest.raises(ValueError):
        gn.forward(x, None, None, x, mean[:1], rstd)
    with pytest.raises(ga.GAError):
        gn.forward(x, None, None, x, eps=0.0)
    dg, db = torch.zeros(2, 3, 16, device="cuda")
    with pytest.raises(ga.GAError):
        gn.backward(x, x, None, None, mean, rstd, x, dg, db, workers=3)
    with pytest.raises(ga.GAError):
        gn.backward(x, x, None, None, mean, rstd, x, dg, None)
    with pytest.raises(ga.GAError):
        gn.backward(x, x, None, None, None, rstd, x)
    with pytest.raises(ga.GAError):
        ga.GroupNorm(16, 4, torch.bfloat16, backward=False).backward(x, x, None, None, mean, rstd, x)


def test_offsets_past_32_bits(ga):
    """The last sample starts past 2^32 bytes."""
    big = torch.empty(1 << 32, dtype=torch.int8, device="cuda").view(torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(3)
    N, S, C, G = 2, 40, 96, 8
    gap = big.numel() - S * C
    x = big.as_strided((N, S, C), (gap, C, 1))
    x.copy_(torch.randn(N, S, C, generator=gen, device="cuda"))
    check_forward(ga, x, None, None, G, "silu")
    dy = torch.randn(N, S, C, generator=gen, device="cuda").bfloat16()
    check_backward(ga, dy, x, None, None, G, "silu", 2)
