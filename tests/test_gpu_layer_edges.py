"""Edges of group norm and the router on the GPU: more samples, workers and workgroups
than one launch or the workspace takes at once, rows shorter than a vector, groups that
several of them share, offsets past 32 bits, two streams at once."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import test_gpu_groupnorm as gnt  # noqa: E402
import test_gpu_router as rt  # noqa: E402
from test_gpu_groupnorm import DT, inputs  # noqa: E402


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 500, 3, 1), (2, 70, 7, 7), (1, 2000, 2, 2), (4, 1, 5, 1), (2, 2500, 40, 40), (1, 5000, 12, 6),
                                   (3, 1111, 30, 10), (2, 4000, 36, 4), (2, 1500, 68, 4), (1, 3000, 264, 8)])
def test_short_rows_and_shared_vectors(ga, shape, x):
    N, S, C, G = shape
    for k, name in enumerate((None, "silu")):
        a, dy, gamma, beta = inputs(N, S, C, x, "fp32", "plain", k)
        gnt.check_forward(ga, a, gamma, beta, G, name)
        gnt.check_backward(ga, dy, a, gamma, beta, G, name, N if k else 1)


@pytest.mark.parametrize("shape,W", [((70000, 2, 32, 32), 1), ((140000, 1, 20, 20), 2), ((2048, 3, 16, 4), 1024), ((1030, 5, 24, 8), 515),
                                     ((70000, 3, 20, 20), 1)])
def test_more_samples_than_at_once(ga, shape, W):
    """The backward pass's partial sums in several launches, of a part of a worker's samples or of some of the workers.
    The weight gradients of 70000 samples add up in chains of up to 70000 / 512 samples and 512 rows."""
    N, S, C, G = shape
    a, dy, gamma, beta = inputs(N, S, C, "bf16", "fp32", "plain")
    gnt.check_forward(ga, a, gamma, beta, G, "silu")
    gnt.check_backward(ga, dy, a, gamma, beta, G, "silu", W)
    # and with no weight gradients
    gn = ga.GroupNorm(C, G, torch.bfloat16, activation="silu")
    mean, rstd = torch.empty(2, N, G, device="cuda")
    y, d1, d2 = torch.empty_like(a), torch.empty_like(a), torch.empty_like(a)
    gn.forward(a, gamma, beta, y, mean, rstd)
    gn.backward(dy, a, gamma, beta, mean, rstd, d1)
    dg, db = torch.empty(2, W, C, device="cuda")
    gn.backward(dy, a, gamma, beta, mean, rstd, d2, dg, db, workers=W)
    # the means of h and h * xh are added in other orders: two roundings of the type apart at most
    assert bool(((d1.float() - d2.float()).abs() <= 2 * torch.finfo(torch.bfloat16).eps * (d1.float().abs() + 1e-3)).all())


def test_more_workgroups_than_a_launch(ga):
    """64 slabs of 16400 samples are more than 2^20 workgroups: the samples around where the second launch starts."""
    N, S, C, G = 16400, 40, 2048, 512
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(N, S, C, dtype=torch.bfloat16, device="cuda")
    for n in range(0, N, 2050):
        x[n:n + 2050] = torch.randn(2050, S, C, generator=gen, device="cuda", dtype=torch.bfloat16)
    y = torch.full_like(x, math.nan)
    mean, rstd = torch.full((2, N, G), math.nan, device="cuda")
    gn = ga.GroupNorm(C, G, torch.bfloat16, activation="silu", backward=False)
    gn.forward(x, None, None, y, mean, rstd)
    for n in (0, 1, 16383, 16384, 16399):
        one, m, r = torch.empty_like(x[n:n + 1]), torch.empty(1, G, device="cuda"), torch.empty(1, G, device="cuda")
        gn.forward(x[n:n + 1], None, None, one, m, r)
        assert torch.equal(one[0], y[n]) and torch.equal(m[0], mean[n]) and torch.equal(r[0], rstd[n])
    assert not bool(mean.isnan().any()) and not bool(y[::37].isnan().any())
    gnt.check_forward(ga, x[16380:16390], None, None, G, "silu")


@pytest.mark.parametrize("bias", [0.0, 100.0])
def test_long_groups(ga, bias):
    """A group of 8.4 million values, in pieces and parts: sums of 256 rows to a thread at most."""
    N, S, C, G = 1, 1 << 16, 256, 2
    gen = torch.Generator(device="cuda").manual_seed(2)
    a = (torch.randn(N, S, C, generator=gen, device="cuda") + bias).contiguous()
    dy = torch.randn(N, S, C, generator=gen, device="cuda")
    gnt.check_forward(ga, a, None, None, G, None)
    gnt.check_backward(ga, dy, a, None, None, G, "silu")


def test_router_offsets_past_32_bits(ga):
    """5.4 GB of logits: the last tokens as in a call on them alone."""
    T, E, k, W = 1310720, 2048 // 2, 4, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    l = torch.empty(T, 2 * E, dtype=torch.bfloat16, device="cuda")[:, E // 2:E // 2 + E]
    for t in range(0, T, 131072):
        l[t:t + 131072] = torch.randn(131072, E, generator=gen, device="cuda", dtype=torch.bfloat16)
    router = ga.Router(E, k, torch.bfloat16, workers=W, scope="worker")
    r, load = router.empty_routing(T), router.empty_load()
    router.forward(l, r, load)
    assert load.tokens.tolist() == [T // 2] * 2 and load.counts.sum(1).tolist() == [T // 2 * k] * 2
    last = l[-64:].contiguous()
    r2, load2 = router.empty_routing(64), router.empty_load()
    router.forward(last, r2, load2)
    assert torch.equal(r.experts[-64:], r2.experts) and torch.equal(r.gates[-64:], r2.gates) and torch.equal(r.lse[-64:], r2.lse)
    counts = torch.bincount(r.experts[T // 2:].reshape(-1).long(), minlength=E)
    assert torch.equal(load.counts[1].long(), counts)
    d = torch.empty(T, 2 * E, dtype=torch.bfloat16, device="cuda")[:, E // 2:E // 2 + E]
    dgates = torch.randn(T, k, generator=gen, device="cuda")
    router.backward(l, r, load, d, dgates=dgates, balance=0.5, z=0.1)
    load2.slope.copy_(load.slope[1])                      # both workers' tokens by the second's slope
    d2 = torch.empty_like(last)
    router.backward(last, r2, load2, d2, dgates=dgates[-64:].contiguous(), balance=0.5, z=0.1)
    assert torch.equal(d[-64:], d2)


@pytest.mark.parametrize("T,E,k,W", [(262144, 16, 2, 8), (100000, 384, 12, 5), (30000, 1024, 32, 3), (65536, 64, 16, 1024)])
def test_router_many_tokens(ga, T, E, k, W):
    """Many rows to a lane and many partial loads; k above a quarter of the team's lanes.  A probability's sum passes
    through as many additions as a lane takes tokens."""
    T = T // W * W
    l = rt.logits(T, E, "bf16", 3)
    old = rt.CHAIN
    rt.CHAIN = max(old, 4 * T // (256 * 16))
    try:
        router, r, load, o = rt.check_forward(ga, l, k, W, True, "worker")
        rt.check_backward(ga, l, router, r, load, o, torch.randn(T, k, device="cuda"))
    finally:
        rt.CHAIN = old


def test_two_handles_on_two_streams(ga):
    """Each with its own workspace: the bits of calls one after the other."""
    N, S, C, G, T, E, k = 8, 3000, 320, 32, 40000, 64, 6
    jobs = []
    for i in range(2):
        a, dy, gamma, beta = inputs(N, S, C, "bf16", "fp32", "plain", i)
        gn, router = ga.GroupNorm(C, G, DT["bf16"], activation="silu"), ga.Router(E, k, torch.bfloat16, workers=4)
        l, r, load, d = rt.logits(T, E, "bf16", i), router.empty_routing(T), router.empty_load(), None
        d = torch.empty_like(l)
        y, dx = torch.empty_like(a), torch.empty_like(a)
        mean, rstd = torch.empty(2, N, G, device="cuda")
        dg, db = torch.empty(2, 2, C, device="cuda")

        def run(a=a, dy=dy, gamma=gamma, beta=beta, gn=gn, router=router, l=l, r=r, load=load, d=d, y=y, dx=dx, mean=mean,
                rstd=rstd, dg=dg, db=db):
            gn.forward(a, gamma, beta, y, mean, rstd)
            gn.backward(dy, a, gamma, beta, mean, rstd, dx, dg, db, workers=2)
            router.forward(l, r, load)
            router.backward(l, r, load, d, balance=0.1, z=0.1)

        jobs.append((run, [y, mean, rstd, dx, dg, db, d] + list(vars(r).values()) + list(vars(load).values())))
    want = []
    for run, outs in jobs:
        run()
        want.append([t.clone() for t in outs])
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s, (run, _) in zip(streams, jobs):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    for (_, outs), w in zip(jobs, want):
        assert all(torch.equal(p, q) for p, q in zip(outs, w))


@pytest.mark.parametrize("C,G,S", [(65536, 65536, 1 << 18), (32768, 16384, 9 << 16)])
def test_long_images_of_many_groups(ga, C, G, S):
    """More partial sums than the workspace holds, were a thread to add 256 rows at most: 34 GB, 64 rows repeated, in place."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows = torch.randn(64, C, generator=gen, device="cuda").bfloat16()
    x = torch.empty(1, S, C, dtype=torch.bfloat16, device="cuda")
    x.view(S // 64, 64, C).copy_(rows)
    gn = ga.GroupNorm(C, G, torch.bfloat16, activation="relu")
    mean, rstd = torch.full((2, 1, G), math.nan, device="cuda")
    want = rows.double().reshape(64, G, C // G)
    m = want.mean((0, 2))
    d = want - m[:, None]
    r = (d.square().mean((0, 2)) + 1e-5) ** -0.5
    # a thread adds S / (16 * 32) rows or fewer; the roundings of so many equal terms add up
    chain = S // 512 + 512
    dev = d.abs().mean((0, 2)) + d.square().mean((0, 2)).sqrt()
    gn.forward(x, None, None, x, mean, rstd)
    assert bool(((mean[0].double() - m).abs() <= 2.0 ** -24 * (chain * dev + 2 * m.abs())).all())
    assert bool(((rstd[0].double() / r - 1).abs() <= 2.0 ** -24 * (chain + 16)).all())
    y = ((want - mean[0].double()[:, None]) * rstd[0].double()[:, None]).clamp_min(0).reshape(64, C)
    for s in range(0, S, S // 8):
        got = x[0, s:s + 64].double()
        assert bool(((got - y).abs() <= (2.0 ** -8 + 2.0 ** -20) * y + 2.0 ** -20).all())
    del x
    # the gradient: every 64 rows alike again
    x = torch.empty(1, S, C, dtype=torch.bfloat16, device="cuda")
    x.view(S // 64, 64, C).copy_(rows)
    dy = torch.empty_like(x)
    grad = torch.randn(64, C, generator=gen, device="cuda").bfloat16()
    dy.view(S // 64, 64, C).copy_(grad)
    dg, db = torch.empty(2, 1, C, device="cuda")
    xh = (want - mean[0].double()[:, None]) * rstd[0].double()[:, None]
    h = torch.where(xh > 0, grad.double().reshape(64, G, C // G), torch.zeros_like(xh))
    gn.backward(dy, x, None, None, mean, rstd, dy, dg, db)
    part = (64, G, C // G)
    for got, term in ((db, h), (dg, h * xh)):
        want_sum = term.sum(0).reshape(C) * (S // 64)
        size = term.abs().sum(0).reshape(C) * (S // 64)
        assert bool(((got[0].double() - want_sum).abs() <= 2.0 ** -24 * (chain + 16) * size).all())
    R = rstd[0].double()[:, None]
    dx = R * (h - h.mean((0, 2))[:, None] - xh * (h * xh).mean((0, 2))[:, None])
    err = 2.0 ** -24 * (chain + 16) * R * (h.abs().mean((0, 2))[:, None] + xh.abs() * (h * xh).abs().mean((0, 2))[:, None] + h.abs())
    for s in range(0, S, S // 8):
        got = dy[0, s:s + 64].double().reshape(part)
        assert bool(((got - dx).abs() <= err + 2.0 ** -8 * (dx.abs() + err)).all())


@pytest.mark.parametrize("x", ["fp32", "bf16"])
def test_widest_slabs(ga, x):
    """Groups that fill a workgroup's rows: the most shared memory that either pass takes."""
    for N, S, C, G in ((3, 3, 4096, 1), (2, 8, 4096, 1), (2, 1, 4096, 2), (2, 4, 2048, 1), (3, 5, 8192, 2), (2, 600, 2048, 1)):
        a, dy, gamma, beta = inputs(N, S, C, x, "fp32", "plain", S)
        gnt.check_forward(ga, a, gamma, beta, G, "silu")
        gnt.check_backward(ga, dy, a, gamma, beta, G, "silu", N)
        gnt.check_backward(ga, dy, a, gamma, beta, G, "silu", 1)
