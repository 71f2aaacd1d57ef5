"""8-bit first moments rounded at random, on the GPU: the codes of one step
against their definition, and many steps against the exact recurrence.  The
update at the largest eps."""
import math

import pytest

import adamw8_model as model
from test_gpu_training import (DT, HYPER, LISTS, U, adamw_reference, code_step as normal_step, codes_of, f32, gradients,
                               mean_of, spread_decay, start)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


def code_step(a):
    """Spacing of the codes at magnitude a: 3 mantissa bits from 2^-6 on, 2^-9
    below.  Exact (a power taken on the device is not)."""
    return normal_step(a.clamp_min(2.0 ** -6))


@pytest.mark.parametrize("dtype,W,t", [("fp32", 1, 1), ("fp16", 1, 3), ("bf16", 1, 1 << 40), ("bf16", 2, 12345),
                                       ("fp16", 16, 77), ("fp16", 300, 2)])
@pytest.mark.parametrize("case", list(LISTS))
def test_codes_of_one_step(ga, dtype, W, case, t):
    numels = LISTS[case]
    P = sum(numels)
    nb = -(-P // 256)
    flags, decay = spread_decay(numels)
    buf, table, rows = gradients(W, numels, DT[dtype], seed=P + W, shift=lambda w, l: w + 3 * l)
    w, m, s = start(P, seed=P)
    pad = lambda a: torch.nn.functional.pad(a, (0, nb * 256 - P)).reshape(nb, 256)
    (mc, ms), (vc, vs) = codes_of(pad(m)), codes_of(pad(s))
    m64, s64 = ((c.double() * sc.double()[:, None]).reshape(-1)[:P] for c, sc in ((mc, ms), (vc, vs)))
    g, tol_g = mean_of(rows)
    _, (mn, tol_m), _ = adamw_reference(w.double(), m64, s64 * s64, g, tol_g, t, decay, **HYPER)
    tol_m = tol_m + f32(HYPER["beta1"]) * U * m64.abs()          # the code times its scale is rounded
    opt = ga.AdamW(numels, W=W, grad_dtype=DT[dtype], state_bits=8, decay=flags)
    other = [a.clone() for a in (w, mc, vc, ms, vs)]
    opt.step(table, w, ga.AdamWState(mc, vc, ms, vs, m_rounding="random"), t=t, **HYPER)
    # to nearest: everything but m's codes is the same
    opt.step(table, other[0], ga.AdamWState(*other[1:], m_rounding="nearest"), t=t, **HYPER)
    for k, a in enumerate((w, mc, vc, ms, vs)):
        assert k == 1 or torch.equal(a.view(torch.uint8), other[k].view(torch.uint8))

    x, tol = pad(mn).abs(), pad(tol_m)
    low, tol_top = x.amax(1, keepdim=True).clamp_min(2.0 ** -100), tol.amax(1, keepdim=True)
    y = x * (448 / low)
    # x's and the block maximum's error, and three roundings: 1/maximum, times 448, times m
    tol_y = tol * (448 / low) + y * (tol_top / low) + 3 * U * y
    up = (model.random_bits(nb * 256, model.step_counter(t) + model.SEED_M).double() / 2 ** 20).cuda().reshape(nb, 256)
    # the lifted value is rounded to 2^-20 of a step
    grid = lambda a: torch.floor(a / code_step(a) + up) * code_step(a)
    small = tol_y + 2.0 ** -9 * 2.0 ** -20
    lo, hi = (y - small).clamp(0, 448), (y + small).clamp(0, 448)
    got = mc.double()
    bad = ~((got.abs() >= grid(lo)) & (got.abs() <= grid(hi)))
    assert not bad.any(), "%d codes" % int(bad.sum())
    assert (torch.sign(got) * torch.sign(pad(mn)) >= 0)[got.abs() > grid(tol_y)].all()
    assert not mc.view(torch.uint8).reshape(-1)[P:].any(), "codes past P are zero"
    opt.close()


def test_zero_moments_stay_zero(ga):
    n = 512
    opt = ga.AdamW([n], state_bits=8)
    g = torch.zeros(n, device="cuda")
    g[::2] = torch.randn(n // 2, device="cuda")
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    w, state = torch.zeros(n, device="cuda"), opt.empty_state()
    for t in range(1, 51):
        opt.step(table, w, state, t=t, lr=0.1)
    assert not state.m.view(torch.uint8).reshape(-1)[1::2].any() and not w[1::2].any()
    assert bool(state.m.float().reshape(-1)[::2].any())


@pytest.mark.parametrize("factor,noise,beta1,beta2", model.TURNS)
def test_turned_gradients(ga, factor, noise, beta1, beta2):
    """Weights that share blocks with steady ones, and whose gradient turns,
    falls or goes, move as the exact recurrence says."""
    n = 4096
    turn = model.Turn(n, factor, noise, device="cuda")
    want = model.exact(turn, n, turn.steps, beta1, beta2, watch=(turn.BEFORE,), device="cuda")
    opt = ga.AdamW([n], state_bits=8)
    g, w, state = torch.empty(n, device="cuda"), torch.zeros(n, device="cuda"), opt.empty_state()
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    got = []
    for t in range(1, turn.steps + 1):
        g.copy_(turn(t))
        opt.step(table, w, state, t=t, lr=1.0, beta1=beta1, beta2=beta2, eps=1e-8)
        if t in (turn.BEFORE, turn.steps):
            got.append((w.double(),))
    assert abs(turn.moved(got) - turn.moved(want)) <= turn.bound(beta1, want)
    # the weights whose gradient stayed: the same bound
    steady = [float(((b[0] - a[0]) * turn.base.double().sign())[::2].mean()) for a, b in (got, want)]
    assert abs(steady[0] - steady[1]) <= (turn.steps - turn.BEFORE) / 8 + turn.bound(beta1, want)
    assert math.isfinite(float(w.abs().sum()))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rounding", ["random", "nearest"])
def test_a_gradient_that_is_not_finite_stays_in_its_block(ga, bad, rounding):
    """It spoils the block's moments, and of the weights its own at once."""
    n = 1024
    gen = torch.Generator().manual_seed(5)
    values = torch.randn(3, n, generator=gen)
    runs = []
    for x in (0.0, bad):
        g = values.clone().cuda()
        g[1, 300] = x
        opt = ga.AdamW([n], state_bits=8)
        w, state = torch.zeros(n, device="cuda"), opt.empty_state()
        state.m_rounding = rounding
        for t in (1, 2):
            table = torch.tensor([g[t - 1].data_ptr()], dtype=torch.int64, device="cuda")
            opt.step(table, w, state, t=t, lr=0.1)
        runs.append((w, state))
    (w0, s0), (w1, s1) = runs
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[300] = False
    assert torch.equal(w0[others], w1[others]) and not math.isfinite(float(w1[300]))
    for k in ("m", "v"):
        a, b = ((getattr(s, k).float() * getattr(s, k + "_scale")[:, None]) for s in (s0, s1))
        assert torch.equal(a[[0, 2, 3]], b[[0, 2, 3]]) and not bool(torch.isfinite(b[1]).any())


@pytest.mark.parametrize("factor", [0.7, 0.5])
def test_second_moments_of_changed_gradients(ga, factor):
    """Second moments that move by far less than a code's step per step, while
    the largest of their block stays."""
    n = 4096
    turn = model.Turn(n, factor, device="cuda")
    want = model.exact(turn, n, turn.steps, 0.9, 0.999, device="cuda")[-1]
    opt = ga.AdamW([n], state_bits=8)
    g, w, state = torch.empty(n, device="cuda"), torch.zeros(n, device="cuda"), opt.empty_state()
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    for t in range(1, turn.steps + 1):
        g.copy_(turn(t))
        opt.step(table, w, state, t=t, lr=0.0, beta1=0.9, beta2=0.999)
    v = (state.v.double() * state.v_scale.double()[:, None]).square().reshape(-1)
    assert abs(turn.second((w, v), want) - 1) <= turn.second_bound()


@pytest.mark.parametrize("eps", [8e37, 9e37, 3e38])
def test_an_eps_whose_reciprocal_is_denormal(ga, eps):
    """m / (root + eps) where 1/eps is below the normal range."""
    n = 700
    g, w = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    m = (torch.linspace(-1, 1, n) * 3e38).cuda()
    opt = ga.AdamW([n])
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    want = 1 - 0.25 * m.double() / f32(eps)                  # beta1 = 1/2 at t = 1: half of m over one half
    opt.step(table, w, ga.AdamWState(m, torch.ones(n, device="cuda")), t=1, lr=0.25, beta1=0.5, beta2=0.5, eps=eps)
    # lr's factor, a reciprocal of 2 units, three products and the difference
    off = float((w.double() - want).abs().max())
    assert off <= 8 * U * (1 + 0.25 * 3e38 / 8e37)
