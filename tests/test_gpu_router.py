"""The expert router, its counts and its balance loss on the GPU against their
formulas in binary64.

Tolerances count roundings of binary32 (U = 2^-24): a probability exp(l - lse)
is off by the roundings of its argument (a few U of |l - max|, of lse and of the
sum's logarithm) and some of its own; sums by CHAIN additions."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
CHAIN = 512
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
INF = math.inf


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


def oracle(l, mask, given, k, W, norm, scope):
    """The definitions, token by token where no vector form says it as plainly (binary64, finite or -inf logits)."""
    T, E = l.shape
    l = l.double()
    absent = (l == -INF).all(1)
    if mask is not None:
        absent = absent | ~mask.bool()
    safe = torch.where(absent[:, None], torch.zeros_like(l), l)
    lse = torch.logsumexp(safe, 1)
    p = torch.softmax(safe, 1)          # exp(l - lse) would lose log(E) beside an lse of 1e38
    p[absent] = 0
    lse = torch.where(absent, torch.zeros_like(lse), lse)
    if given is None:
        order = torch.sort(safe, dim=1, descending=True, stable=True).indices[:, :k]
        experts = torch.where(safe.gather(1, order) == -INF, -1, order)
        experts[absent] = -1
    else:
        experts = given.long()
    valid = (experts >= 0) & (experts < E) & ~absent[:, None]
    at = experts.clamp(0, E - 1)
    logit = torch.where(valid, safe.gather(1, at), torch.full_like(lse, -INF)[:, None].expand(T, k))
    if norm:
        none = (logit == -INF).all(1, keepdim=True)
        gates = torch.where(none, torch.zeros_like(logit), torch.softmax(torch.where(none, torch.zeros_like(logit), logit), 1))
    else:
        gates = torch.where(valid, p.gather(1, at), torch.zeros_like(logit))
    worker = torch.arange(T, device=l.device) // max(1, T // W)
    flat = (worker[:, None] * E + at)[valid]
    counts = torch.bincount(flat, minlength=W * E).reshape(W, E)
    probs = torch.zeros(W, E, dtype=torch.float64, device=l.device).index_add_(0, worker, p)
    tokens = torch.bincount(worker[~absent], minlength=W)
    squares = torch.zeros(W, dtype=torch.float64, device=l.device).index_add_(0, worker, lse.square())
    F, P, n, Z = counts.double(), probs, tokens.double(), squares
    if scope == "all":
        F, P, n, Z = F.sum(0, keepdim=True), P.sum(0, keepdim=True), n.sum(0, keepdim=True), Z.sum(0, keepdim=True)
    S = F.shape[0]
    m = n.clamp_min(1)[:, None]
    slope = E * F / (k * m * m) / S
    loss = torch.stack([(slope * P).sum(), (Z / m[:, 0]).sum() / S])
    last = torch.where(n > 0, 2 / m[:, 0] / S, torch.zeros_like(n))
    return dict(experts=experts, gates=gates, lse=lse, counts=counts, probs=probs, tokens=tokens, loss=loss,
                slope=torch.cat([slope, last[:, None]], 1), p=p, absent=absent, valid=valid)


def arg_err(l):
    """Error of the exponentials' argument, in units of U: |l - max| and the logits' size enter it, each rounded."""
    l = l.double()
    top = l.amax(1, keepdim=True).clamp_min(-1e300)
    far = torch.where(l == -INF, torch.zeros_like(l), (l - top).abs())
    return 4 * far + 48


def check_forward(ga, l, k, W=1, norm=True, scope="all", mask=None, given=None, router=None):
    T, E = l.shape
    router = router or ga.Router(E, k, l.dtype, workers=W, normalize=norm, scope=scope)
    r, load = router.empty_routing(T), router.empty_load()
    r.gates.fill_(7)
    r.lse.fill_(7)
    for t in (load.probs, load.loss, load.slope):
        t.fill_(math.nan)
    load.counts.fill_(-5)
    load.tokens.fill_(-5)
    if given is not None:
        r.experts.copy_(given)
    router.forward(l, r, load, mask=mask, select=given is None)
    o = oracle(l, mask, given, k, W, norm, scope)
    assert torch.equal(r.experts.long(), o["experts"])
    assert torch.equal(load.counts.long(), o["counts"]) and torch.equal(load.tokens.long(), o["tokens"])
    arg = arg_err(l)
    at = o["experts"].clamp(0, E - 1)
    gate_err = (arg.gather(1, at) + 48) * U * o["gates"] * 2 + 2.0 ** -126
    assert bool(((r.gates.double() - o["gates"]).abs() <= gate_err).all())
    lse_err = U * (4 * o["lse"].abs() + 64)
    assert bool(((r.lse.double() - o["lse"]).abs() <= lse_err).all())
    worker = torch.arange(T, device=l.device) // max(1, T // W)
    p_err = torch.zeros_like(o["probs"]).index_add_(0, worker, o["p"] * (arg + 8 + CHAIN) * U) + T * 2.0 ** -126
    assert bool(((load.probs.double() - o["probs"]).abs() <= p_err).all())
    assert bool(((load.slope.double() - o["slope"]).abs() <= 4 * U * o["slope"].abs()).all())
    S = o["slope"].shape[0]
    balance_err = (o["slope"][:, :E] * (p_err.sum(0, keepdim=True) if S == 1 else p_err)).sum() + 4 * U * o["loss"][0]
    assert abs(float(load.loss[0]) - float(o["loss"][0])) <= float(balance_err) + 1e-30
    z_err = float((2 * lse_err * o["lse"].abs()).max()) + (CHAIN + 4) * U * float(o["loss"][1])
    if math.isinf(float(o["loss"][1].float())):        # past binary32: the squares of logits of 1e38
        assert float(load.loss[1]) == INF
    else:
        assert abs(float(load.loss[1]) - float(o["loss"][1])) <= z_err + 1e-30
    # without a load, and without gates and lse: the same routing
    r2 = router.empty_routing(T)
    if given is not None:
        r2.experts.copy_(given)
    router.forward(l, r2, None, mask=mask, select=given is None)
    assert torch.equal(r2.experts, r.experts) and torch.equal(r2.gates, r.gates) and torch.equal(r2.lse, r.lse)
    r3 = ga.Routing(torch.zeros_like(r.experts) if given is None else r.experts.clone())
    router.forward(l, r3, None, mask=mask, select=given is None)
    assert torch.equal(r3.experts, r.experts)
    return router, r, load, o


def check_backward(ga, l, router, r, load, o, dgates, mask=None, balance=0.3, z=0.2, dlogits=None):
    T, E = l.shape
    k, W, norm = router.k, router.workers, router.normalize
    dlogits = torch.full((T, E), math.nan, dtype=l.dtype, device="cuda") if dlogits is None else dlogits
    ld = l.double()
    arg = arg_err(l)
    router.backward(l, r, load, dlogits, dgates=dgates, mask=mask, balance=balance, z=z)
    slope = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
    if load is not None:
        S = load.slope.shape[0]
        slope = load.slope.double().repeat_interleave(max(1, T // S), 0)[:T]
    # from the routing that the call was given: lse and gates in binary32
    absent, lse = o["absent"], r.lse.double()
    p = torch.exp(torch.where(absent[:, None], torch.full_like(ld, -INF), ld) - lse[:, None])
    h = float(torch.tensor(balance)) * slope[:, :E]
    h_abs = h.abs()
    direct = torch.zeros_like(p)
    direct_abs = torch.zeros_like(p)
    if dgates is not None:
        at = o["experts"].clamp(0, E - 1)
        dg = torch.where(o["valid"], dgates.double(), torch.zeros_like(o["gates"]))
        if norm:
            gates = r.gates.double()
            inner = (gates * dg).sum(1, keepdim=True)
            inner_abs = (gates * dg).abs().sum(1, keepdim=True)
            direct = direct.scatter_add(1, at, torch.where(o["valid"], gates * (dg - inner), torch.zeros_like(dg)))
            direct_abs = direct_abs.scatter_add(1, at, torch.where(o["valid"], gates * (dg.abs() + inner_abs), torch.zeros_like(dg)))
        else:
            h = h.scatter_add(1, at, dg)
            h_abs = h_abs.scatter_add(1, at, dg.abs())
    dot = (h * p).sum(1, keepdim=True)
    dot_abs = (h_abs * p).sum(1, keepdim=True)
    dot_err = (h_abs * p * (arg + 96) * U).sum(1, keepdim=True)
    zpart = float(torch.tensor(z)) * slope[:, E:] * lse[:, None]
    want = p * (h - dot + zpart) + direct
    size = p * (h_abs + dot_abs + zpart.abs())
    err = U * (arg + 64) * size + p * dot_err + (k + 8) * U * direct_abs
    want[absent], err[absent] = 0, 0
    dt = l.dtype
    # a result below the type's normal range is off by half of its least step
    tol = err + torch.finfo(dt).eps / 2 * (want.abs() + err) + torch.finfo(dt).tiny * torch.finfo(dt).eps + 2.0 ** -126
    assert bool(((dlogits.double() - want).abs() <= tol).all())
    return dlogits


def logits(T, E, x, seed=0, width=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed + T * 31 + E)
    return (width * torch.randn(T, E, generator=gen, device="cuda") + torch.randn(E, generator=gen, device="cuda")).to(DT[x])


SHAPES = [
    # T, E, k, W
    (1, 1, 1, 1), (1, 8, 2, 1), (3, 2, 2, 3), (4, 5, 3, 2), (64, 8, 2, 1), (17, 9, 9, 1), (100, 16, 4, 4), (33, 17, 5, 3),
    (66, 32, 32, 2), (999, 60, 4, 1), (500, 64, 6, 2), (128, 64, 8, 16), (70, 65, 7, 7), (300, 100, 3, 1), (40, 127, 10, 5), (256, 128, 1, 8),
    (65, 129, 2, 5), (120, 200, 12, 3), (512, 256, 8, 2), (31, 257, 4, 1), (90, 500, 20, 9), (60, 512, 8, 1), (24, 513, 3, 4),
    (20, 1000, 32, 2), (12, 1024, 10, 12), (4096, 8, 2, 4), (20000, 64, 6, 16), (5000, 256, 8, 1), (2048, 32, 3, 1024), (2050, 40, 5, 1),
]


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_both_passes(ga, i, shape, x):
    T, E, k, W = shape
    l = logits(T, E, x)
    gen = torch.Generator(device="cuda").manual_seed(i)
    dgates = torch.randn(T, k, generator=gen, device="cuda")
    for j in range(2):
        norm, scope = (i + j) % 2 == 0, ["all", "worker"][(i // 2 + j) % 2]
        router, r, load, o = check_forward(ga, l, k, W, norm, scope)
        check_backward(ga, l, router, r, load, o, dgates if (i + j) % 4 else None)


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 8, 2, 1), (96, 8, 2, 3), (300, 60, 6, 4), (1000, 256, 8, 2), (64, 1024, 32, 1)])
def test_given_experts(ga, shape, x):
    """A selection made elsewhere: any experts, the same twice or more, and some that are none."""
    T, E, k, W = shape
    l = logits(T, E, x)
    gen = torch.Generator(device="cuda").manual_seed(T)
    given = torch.randint(-2, E + 2, (T, k), generator=gen, device="cuda").int()
    given[::3] = given[::3, :1]
    given[0] = 2 ** 31 - 1
    given[-1] = -2 ** 31
    dgates = torch.randn(T, k, generator=gen, device="cuda")
    for norm in (False, True):
        router, r, load, o = check_forward(ga, l, k, W, norm, "all", given=given)
        check_backward(ga, l, router, r, load, o, dgates)


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("below", [100.0, 400.0, 3e4])
def test_given_experts_far_below_the_largest(ga, below, norm, x):
    """Gates that sum to 1 come from the given experts' logits, however small their probabilities are."""
    for T, E, k in ((70, 8, 2), (300, 60, 4), (50, 512, 32)):
        l = logits(T, E, x, 3)
        half = E // 2
        l[:, :half] -= below
        gen = torch.Generator(device="cuda").manual_seed(E)
        given = torch.argsort(torch.rand(T, half, generator=gen, device="cuda"), dim=1)[:, :k].int()
        l[3, given[3, 0].long()] = -INF             # one of a token's experts, and all of another's
        l[5, given[5].long()] = -INF
        given[7, 1] = -1
        router, r, load, o = check_forward(ga, l, k, W=1, norm=norm, given=given)
        if norm:
            sums = r.gates.sum(1)
            assert bool(((sums - 1).abs() <= (k + 4) * 2 * U)[torch.arange(T, device="cuda") != 5].all()) and float(sums[5]) == 0


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("E,k", [(4, 4), (8, 3), (40, 10), (64, 6), (256, 8), (300, 16), (1024, 32)])
def test_ties_go_to_the_lowest_index(ga, E, k, x):
    T = 64
    gen = torch.Generator(device="cuda").manual_seed(E)
    few = torch.randint(-2, 3, (T, E), generator=gen, device="cuda").to(DT[x])
    few[0] = 0
    few[1] = -torch.arange(E, device="cuda") // 4
    few[2, ::2] = -0.0
    few[2, 1::2] = 0.0
    check_forward(ga, few, k)


@pytest.mark.parametrize("x", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("E,k", [(4, 3), (8, 2), (60, 6), (256, 8), (600, 20)])
def test_masked_experts_and_tokens(ga, E, k, x):
    """Logits of -infinity and of the type's lowest value, rows of nothing else, and tokens masked out whatever they hold."""
    T, W = 96, 4
    l = logits(T, E, x)
    gen = torch.Generator(device="cuda").manual_seed(E + 1)
    l[torch.rand(T, E, generator=gen, device="cuda") < 0.5] = -INF
    l[3] = -INF
    l[4] = -INF
    l[4, E - 1] = 2.0                                  # one expert left
    l[5] = torch.finfo(DT[x]).min
    l[6] = torch.finfo(DT[x]).min
    l[6, 1] = torch.finfo(DT[x]).max
    l[7, :] = torch.finfo(DT[x]).max
    mask = torch.rand(T, generator=gen, device="cuda") < 0.7
    mask[3:8] = True
    mask[24:48] = False                                # a worker without tokens
    mask[0] = mask[1] = mask[2] = False
    clean = torch.where(mask[:, None], l, torch.zeros_like(l))
    l[0], l[1], l[2] = math.nan, INF, -INF
    dgates = torch.randn(T, k, generator=gen, device="cuda")
    for scope in ("all", "worker"):
        for norm in (False, True):
            for m in (mask, mask.to(torch.uint8) * 7):
                router, r, load, o = check_forward(ga, torch.where(mask[:, None], l, clean), k, W, norm, scope, mask=m)
            r2, load2 = router.empty_routing(T), router.empty_load()
            router.forward(l, r2, load2, mask=mask)
            for a, b in ((r, r2), (load, load2)):
                assert all(torch.equal(p, q) for p, q in zip(vars(a).values(), vars(b).values()))
            l2 = l.clone()
            l2[3:8] = 0.5                              # sums of 60000s are no gradients of interest
            router.forward(l2, r2, load2, mask=mask)
            o = oracle(torch.where(mask[:, None], l2, clean), mask, None, k, W, norm, scope)
            want = check_backward(ga, torch.where(mask[:, None], l2, clean), router, r2, load2, o, dgates, mask)
            got = torch.full_like(l2, math.nan)
            router.backward(l2, r2, load2, got, dgates=dgates, mask=mask, balance=0.3, z=0.2)
            assert torch.equal(got, want) and not bool(got[~mask].any())


def test_no_tokens_at_all(ga):
    for T in (0, 8):
        router = ga.Router(6, 2, workers=2)
        r, load = router.empty_routing(T), router.empty_load()
        for t in vars(load).values():
            t.fill_(9)
        l = torch.zeros(T, 6, device="cuda")
        router.forward(l, r, load, mask=torch.zeros(T, dtype=torch.bool, device="cuda"))
        for t in vars(load).values():
            assert not bool(t.any())
        d = torch.full_like(l, math.nan)
        router.backward(l, r, load, d, mask=torch.zeros(T, dtype=torch.bool, device="cuda"), balance=1.0, z=1.0)
        assert not bool(d.any())


@pytest.mark.parametrize("bad", [math.nan, INF])
@pytest.mark.parametrize("E,k", [(8, 2), (100, 6), (256, 8)])
def test_not_finite_spoils_its_token_alone(ga, bad, E, k):
    T = 40
    l = logits(T, E, "fp32")
    l[11, E // 2] = bad
    for norm in (False, True):
        router = ga.Router(E, k, normalize=norm)
        r, load = router.empty_routing(T), router.empty_load()
        router.forward(l, r, load)
        assert bool(r.gates[11].isnan().all()) and bool(r.lse[11].isnan()) and bool(load.loss.isnan().all())
        rest = [t for t in range(T) if t != 11]
        clean, r2 = l[rest].contiguous(), router.empty_routing(T - 1)
        router.forward(clean, r2)
        assert torch.equal(r.gates[rest], r2.gates) and torch.equal(r.experts[rest], r2.experts)
        order = torch.sort(torch.where(l[11].isnan(), -INF, l[11]), descending=True, stable=True).indices[:k]
        assert torch.equal(r.experts[11].long(), order)
        d = torch.empty_like(l)
        load.slope.fill_(1.0)
        router.backward(l, r, load, d, balance=1.0)
        assert bool(d[11].isnan().all()) and not bool(d[rest].isnan().any())


@pytest.mark.parametrize("x", ["fp32", "fp16"])
@pytest.mark.parametrize("E", [7, 60, 256])
def test_rows_inside_wider_ones(ga, E, x):
    T, k = 50, min(E, 6)
    wide = torch.full((T, E + 5), math.nan, dtype=DT[x], device="cuda")
    l = wide[:, 3:3 + E]
    l.copy_(logits(T, E, x))
    out = torch.full((T, E + 5), math.nan, dtype=DT[x], device="cuda")
    router, r, load, o = check_forward(ga, l, k)
    dgates = torch.randn(T, k, device="cuda")
    check_backward(ga, l, router, r, load, o, dgates, dlogits=out[:, 3:3 + E])
    assert bool(out[:, :3].isnan().all()) and bool(out[:, 3 + E:].isnan().all())
    d = check_backward(ga, l, router, r, load, o, dgates)
    assert torch.equal(d, out[:, 3:3 + E])
    c = l.contiguous()
    router.backward(c, r, load, c, dgates=dgates, balance=0.3, z=0.2)      # over the logits
    assert torch.equal(c, d)


def test_differences(ga):
    """The gradient against differences of the losses' and gates' formulas."""
    T, E, k, W = 12, 7, 3, 3
    l = logits(T, E, "fp32")
    dgates = torch.randn(T, k, device="cuda")
    for norm in (False, True):
        for scope in ("all", "worker"):
            router = ga.Router(E, k, workers=W, normalize=norm, scope=scope)
            r, load = router.empty_routing(T), router.empty_load()
            router.forward(l, r, load)
            d = torch.empty_like(l)
            router.backward(l, r, load, d, dgates=dgates, balance=0.7, z=0.4)
            given = r.experts

            def loss(l):
                # the counts, and so the slope, are constants of the gradient
                o = oracle(l, None, given, k, W, norm, scope)
                return float(0.7 * o["loss"][0] + 0.4 * o["loss"][1] + (o["gates"] * dgates.double()).sum())

            for i in range(0, T * E, 5):
                ends = []
                for s in (1e-5, -1e-5):
                    m = l.double()
                    m.view(-1)[i] += s
                    ends.append(loss(m))
                want = (ends[0] - ends[1]) / 2e-5
                assert abs(float(d.view(-1)[i]) - want) <= 1e-5 * (1 + abs(want))


@pytest.mark.parametrize("shape", [(64, 8, 2, 1), (8192, 64, 6, 16), (4000, 256, 8, 8)])
def test_repeats_streams_and_graphs(ga, shape):
    T, E, k, W = shape
    l = logits(T, E, "bf16")
    router = ga.Router(E, k, torch.bfloat16, workers=W)
    r, load, d = router.empty_routing(T), router.empty_load(), torch.empty_like(l)
    dgates = torch.randn(T, k, device="cuda")

    def both():
        router.forward(l, r, load)
        router.backward(l, r, load, d, dgates=dgates, balance=0.1, z=0.1)

    outs = list(vars(r).values()) + list(vars(load).values()) + [d]
    both()
    want = [t.clone() for t in outs]

    def same():
        ok = all(torch.equal(p, q) for p, q in zip(outs, want))
        for t in outs:
            t.fill_(3)
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
    for _ in range(3):
        graph.replay()
        assert same()
        l.copy_(l.flip(0))
        both()
        l.copy_(l.flip(0))
        torch.cuda.synchronize()
        both()
        assert same()


def test_refusals(ga):
    router = ga.Router(8, 2, workers=2)
    l = torch.zeros(4, 8, device="cuda")
    r, load = router.empty_routing(4), router.empty_load()
    for bad in (l.half(), l.cpu(), l[:, :7]):
        with pytest.raises((ValueError, TypeError)):
            router.forward(bad, r, load)
    with pytest.raises(ga.GAError):
        router.forward(l[:3], r, load)                 # 3 tokens of 2 workers
    with pytest.raises(ValueError):
        router.forward(l, router.empty_routing(3), load)
    with pytest.raises(ValueError):
        router.forward(l, r, load, mask=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        router.forward(l, r, load, mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(ga.GAError):
        router.backward(l, r, None, torch.empty_like(l), balance=0.1)
    with pytest.raises(ga.GAError):
        router.backward(l, ga.Routing(r.experts, None, r.lse), load, torch.empty_like(l), dgates=r.gates)
    with pytest.raises(ValueError):
        router.backward(l, r, load, torch.empty_like(l), dgates=r.gates.double())
