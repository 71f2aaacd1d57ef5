"""The training-step operators on the GPU against their formulas in binary64.

Tolerances are counted in roundings.  u is the most that rounding to the
nearest binary32 value is off, relative to the value (2^-24); a square root or
quotient may be one unit in the last place off (2u).  A sum of n binary32
values in any order is at most (n - 1) u times the sum of their magnitudes off;
the constants below count the longest chain of additions in a lane, then in
the tree over the lanes."""
import math

import numpy as np
import pytest

import oracle
from helpers import device_layers

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TINY = 2.0 ** -126
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half the spacing of the smallest values
LEAST = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


def within(got, ref, tol, name):
    """|got - ref| <= tol elementwise, in binary64; a NaN fails."""
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        pick = lambda a: float((a if isinstance(a, torch.Tensor) else torch.tensor(a)).expand(got.shape).reshape(-1)[i])
        raise AssertionError("%s: %d of %d off, first at %d: %r, not %r (tolerance %r)" % (
            name, int(bad.sum()), bad.numel(), i, float(got.reshape(-1)[i]), float(ref.reshape(-1)[i]), pick(tol)))


def gradients(W, numels, dtype, seed, shift=lambda w, l: 0):
    """Random per-layer gradients of W workers at odd places of one buffer, the
    table of their addresses, and their values [W][P] in binary64."""
    gen = torch.Generator().manual_seed(seed)
    P = sum(numels)
    rows = (torch.randn(W, P, generator=gen) * 10.0 ** (4 * torch.rand(P, generator=gen) - 4)).to(dtype)
    bits = rows.view(torch.int32 if dtype == torch.float32 else torch.int16).numpy()
    buf, table = device_layers(bits, numels, shift)
    return buf, table, rows.double().cuda()


def mean_of(rows):
    """Mean gradient and its rounding error's bound: at most 11 levels of the
    tree, and the factor 1/W with the product."""
    W = rows.shape[0]
    depth = max(0, math.ceil(math.log2(W))) + (2 if W > 1 else 0)
    return rows.mean(0), depth * U * rows.abs().mean(0)


LISTS = {
    "one": [1], "seven": [7], "two tiles": [1024], "odd": [513, 1, 255, 2, 3001],
    "many small": [1, 2, 3, 1, 1, 5, 1, 1, 8, 700, 1, 1, 1, 1, 4, 9] * 5, "straddled": [510, 4, 600, 511, 1, 512, 513],
    "aligned": [4096, 64, 2048, 1000],
}
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def f32(x):
    return float(np.float32(x))


def adamw_reference(w, m, v, g, tol_g, t, decay, lr, beta1, beta2, eps, weight_decay):
    """New w, m, v in binary64 from binary32 hyper-parameters, each with its
    tolerance."""
    lr, b1, b2, eps, wd = (f32(a) for a in (lr, beta1, beta2, eps, weight_decay))
    c1, c2 = 1 - b1, 1 - b2
    mn = b1 * m + c1 * g
    vn = b2 * v + c2 * g * g
    # m: the factor c1, the product with g and the sum are rounded
    tol_m = c1 * tol_g + U * (2 * c1 * g.abs() + b1 * m.abs() + mn.abs()) + TINY
    # v: the factor c2, two products and the sum are rounded
    tol_v = c2 * (2 * g.abs() * tol_g + tol_g ** 2) + U * (4 * c2 * g * g + b2 * v + vn) + TINY
    bc1, bc2 = 1 - b1 ** t, 1 - b2 ** t
    root = vn.sqrt()
    tol_root = torch.minimum(tol_v / root.clamp_min(1e-300), tol_v.sqrt()) + 2 * U * root
    den = root / math.sqrt(bc2) + eps
    tol_den = (tol_root + 2 * U * root) / math.sqrt(bc2) + U * den
    low = (den - tol_den).clamp_min(eps * (1 - U))
    up = mn / den
    tol_up = tol_m / low + mn.abs() * (1 / low - 1 / den).abs() + 5 * U * up.abs()
    keep = torch.where(decay, 1 - lr * wd, 1.0)
    wn = w * keep - lr / bc1 * up
    # w: the factors lr/bc1 and keep, their products and the difference are rounded
    tol_w = lr / bc1 * (tol_up + 2 * U * up.abs()) + 2 * U * w.abs() + U * wn.abs() + TINY
    return (wn, tol_w), (mn, tol_m), (vn, tol_v)


def start(P, seed):
    gen = torch.Generator().manual_seed(seed)
    w = torch.randn(P, generator=gen)
    scale = 10.0 ** (4 * torch.rand(P, generator=gen) - 4)
    return w.cuda(), (torch.randn(P, generator=gen) * scale).cuda(), (scale * (0.5 + torch.rand(P, generator=gen))).cuda()


def spread_decay(numels):
    flags = [l % 3 != 1 for l in range(len(numels))]
    return flags, torch.tensor(flags).repeat_interleave(torch.tensor(numels)).cuda()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", list(LISTS))
@pytest.mark.parametrize("W", [1, 2, 5])
def test_adamw_layer_lists(ga, dtype, case, W):
    numels = LISTS[case]
    check_adamw32(ga, W, numels, DT[dtype], shift=lambda w, l: w + 3 * l, t=7)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
@pytest.mark.parametrize("W", [3, 7, 8, 31, 32, 33, 64, 65, 255, 256, 300, 1024])
def test_adamw_worker_counts(ga, dtype, W):
    check_adamw32(ga, W, [1500, 3, 517], DT[dtype], t=1)


@pytest.mark.parametrize("copy", ["fp16", "bf16"])
@pytest.mark.parametrize("clip", [None, 1.0, 0.03125])
def test_adamw_copy_and_clip(ga, copy, clip):
    check_adamw32(ga, 2, [5000, 333], torch.bfloat16, copy=DT[copy], clip=clip, t=100000)


def check_adamw32(ga, W, numels, dtype, shift=lambda w, l: 0, t=1, copy=None, clip=None):
    P = sum(numels)
    flags, decay = spread_decay(numels)
    buf, table, rows = gradients(W, numels, dtype, seed=P + W, shift=shift)
    w, m, v = start(P, seed=P)
    v = v * v
    g, tol_g = mean_of(rows)
    record = None
    opt = ga.AdamW(numels, W=W, grad_dtype=dtype, decay=flags)
    if clip is not None:
        record = opt.empty_clip()
        record.scale.fill_(clip)
        tol_g = clip * tol_g + U * clip * g.abs()
        g = clip * g
    want = adamw_reference(w.double(), m.double(), v.double(), g, tol_g, t, decay, **HYPER)
    out = None if copy is None else torch.empty(P, dtype=copy, device="cuda")
    state = ga.AdamWState(m, v)
    opt.step(table, w, state, t=t, clip=record, copy=out, **HYPER)
    for name, got, (ref, tol) in zip("wmv", (w, m, v), want):
        within(got, ref, tol, name)
    if out is not None:
        assert torch.equal(out, w.to(copy)), "the copy is the rounded weights"
    opt.close()


def test_adamw_first_step_from_zero_state(ga):
    """From a zero state the first step moves every weight with a gradient by
    lr, and leaves the others (decay aside) where they are."""
    numels = [1000, 24]
    opt = ga.AdamW(numels, grad_dtype=torch.float32)
    g = torch.zeros(1024, device="cuda")
    g[::2] = torch.randn(512, device="cuda")
    table = torch.tensor([g.data_ptr(), g.data_ptr() + 4000], dtype=torch.int64, device="cuda")
    w = torch.zeros(1024, device="cuda")
    state = opt.empty_state()
    opt.step(table, w, state, t=1, lr=0.5, eps=1e-12)
    within(w[::2], -0.5 * g[::2].sign().double(), 0.5 * (1e-12 / g[::2].abs().double() + 12 * U), "w")
    assert not w[1::2].any() and not state.m[1::2].any() and not state.v[1::2].any()


# ---- 8-bit states ------------------------------------------------------------

def codes_of(x):
    top = x.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100)
    return (x * (448.0 / top)).to(torch.float8_e4m3fn), (top / 448.0).reshape(-1).float()


def code_step(a):
    """Spacing of the codes at magnitude a >= 2^-6 (3 mantissa bits), exact: a
    over its mantissa in [1/2, 1) is a power of two."""
    return a / torch.frexp(a)[0] / 16


def random_units(n, t):
    """The rounding bits as a fraction of a code's step, from their definition."""
    i = np.arange(n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        x = ((i >> np.uint64(1)) + np.uint64((t * 0x9E3779B9 + 0x7F4A7C15) % 2 ** 32)).astype(np.uint32)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0xB7E15163)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x6A09E667)
        x = x ^ (x >> np.uint32(16))
    r = np.where(i % 2 == 1, x >> np.uint32(16), x & np.uint32(0xffff))
    return torch.from_numpy((r.astype(np.float64) * 16 + 8) / 2 ** 20).cuda()


def check_adamw8(ga, W, numels, dtype, t=3, copy=None, shift=lambda w, l: 0, zero_block=False):
    P = sum(numels)
    nb = -(-P // 256)
    flags, decay = spread_decay(numels)
    buf, table, rows = gradients(W, numels, dtype, seed=P + W, shift=shift)
    w, m, s = start(P, seed=P)
    if zero_block and P >= 256:
        buf.zero_()
        rows = torch.zeros_like(rows)
        m[:256] = 0
        s[:256] = 0
    pad = lambda a: torch.nn.functional.pad(a, (0, nb * 256 - P)).reshape(nb, 256)
    (mc, ms), (vc, vs) = codes_of(pad(m)), codes_of(pad(s))
    held = lambda c, sc: (c.double() * sc.double()[:, None]).reshape(-1)
    m64 = (c_m := held(mc, ms))[:P]
    s64 = held(vc, vs)[:P]
    g, tol_g = mean_of(rows)
    # codes times scales, and the root's square, are rounded
    want = adamw_reference(w.double(), m64, s64 * s64, g, tol_g, t, decay, **HYPER)
    b1, b2, lr, eps = (f32(HYPER[k]) for k in ("beta1", "beta2", "lr", "eps"))
    (wn, tol_w), (mn, tol_m), (vn, tol_v) = want
    extra_m, extra_v = b1 * U * m64.abs(), 3 * U * b2 * s64 * s64
    tol_m, tol_v = tol_m + extra_m, tol_v + extra_v
    root = vn.sqrt()
    tol_root = torch.minimum(tol_v / root.clamp_min(1e-300), tol_v.sqrt()) + 2 * U * root
    den = root / math.sqrt(1 - b2 ** t) + eps
    tol_w = tol_w + 2 * lr / (1 - b1 ** t) * (extra_m / den + mn.abs() / den * 3 * U)

    opt = ga.AdamW(numels, W=W, grad_dtype=dtype, state_bits=8, decay=flags)
    out = None if copy is None else torch.empty(P, dtype=copy, device="cuda")
    state = ga.AdamWState(mc, vc, ms, vs)
    opt.step(table, w, state, t=t, copy=out, **HYPER)
    within(w, wn, tol_w, "w")
    if out is not None:
        assert torch.equal(out, w.to(copy))

    up = random_units(nb * 256, t).reshape(nb, 256)
    for name, codes, scale, x, tol in (("m", mc, ms, pad(mn), pad(tol_m)), ("v", vc, vs, pad(root), pad(tol_root))):
        top, at = x.abs().max(1)
        tol_top = tol.amax(1)
        low = top.clamp_min(2.0 ** -100)
        within(scale, low / 448, tol_top / 448 + 2 * U * low / 448, name + "_scale")
        got = codes.double()
        assert torch.isfinite(got).all()
        # a code stands for x * 448/top: its error is x's and top's, and two roundings
        y = x * (448 / low)[:, None]
        tol_y = (tol * (448 / low)[:, None] + y.abs() * (tol_top / low)[:, None] + 3 * U * y.abs())
        if name == "m":
            step = code_step((y.abs() + tol_y).clamp_min(2.0 ** -6))
            within(got, y, step / 2 + tol_y, "m codes")
        else:
            y = torch.where(x > 0, y.clamp(2.0 ** -6, 448), y)
            # between the codes that the two ends of the interval round to
            grid = lambda a: torch.where(a > 0, (lambda st: torch.floor(a / st + up) * st)(
                code_step(a.clamp_min(2.0 ** -6))), 0.0)
            lo = torch.where(x > 0, (y - tol_y).clamp(2.0 ** -6, 448), torch.zeros_like(y))
            hi = torch.where(x > 0, (y + tol_y).clamp(2.0 ** -6, 448), torch.zeros_like(y))
            assert ((got >= grid(lo)) & (got <= grid(hi))).all(), "v codes"
            assert (got[x > 0] > 0).all(), "a second moment never rounds to zero"
        assert not codes.view(torch.uint8).reshape(-1)[P:].any(), "codes past P are zero"
    opt.close()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", list(LISTS))
def test_adamw8_layer_lists(ga, dtype, case):
    check_adamw8(ga, 1, LISTS[case], DT[dtype], shift=lambda w, l: w + 3 * l)


@pytest.mark.parametrize("dtype,W", [("bf16", 2), ("fp16", 16), ("fp32", 33), ("fp16", 300)])
def test_adamw8_worker_counts(ga, dtype, W):
    check_adamw8(ga, W, [1500, 3, 517, 256], DT[dtype], t=12345, copy=torch.bfloat16)


def test_adamw8_block_of_zeros(ga):
    check_adamw8(ga, 1, [256, 300], torch.float32, zero_block=True)


def test_adamw8_second_moment_moves_on_average(ga):
    """A second moment whose change per step is far below a code's step still
    follows its average: 512 steps at beta2 = 0.999 with a steady gradient."""
    n, steps = 4096, 512
    opt = ga.AdamW([n], grad_dtype=torch.float32, state_bits=8)
    g = torch.full((n,), 1.0, device="cuda")
    g[::256] = 2.0                              # the block's largest: the others' codes are not the top one
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    w, state = torch.zeros(n, device="cuda"), opt.empty_state()
    for t in range(1, steps + 1):
        opt.step(table, w, state, t=t, lr=0.0, beta2=0.999)
    v = (state.v.double() * state.v_scale.double()[:, None]).square().reshape(-1)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[::256] = False
    want = 1 - f32(0.999) ** steps
    # a step's rounding error has a variance of at most (step/2)^2 on the root, so at most (1/8)^2 v on v;
    # the errors of earlier steps fade by beta2: over 1/(2 (1 - beta2)) of them at most add up
    one = want / 8 * math.sqrt(steps)
    assert abs(float(v[keep].mean()) - want) < 5 * one / math.sqrt(n) + 0.02 * want


# ---- gradient norm ----------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("W,case", [(1, "one"), (1, "odd"), (1, "many small"), (2, "straddled"), (16, "aligned"),
                                    (33, "odd"), (300, "seven")])
def test_grad_norm(ga, dtype, W, case):
    numels = LISTS[case]
    buf, table, rows = gradients(W, numels, DT[dtype], seed=5, shift=lambda w, l: 5 * w + l)
    opt = ga.AdamW(numels, W=W, grad_dtype=DT[dtype])
    clip, grad = opt.empty_clip(), torch.full((sum(numels),), math.nan, device="cuda")
    g, tol_g = mean_of(rows)
    norm = float(g.norm())
    opt.grad_norm(table, clip, max_norm=0.5 * norm, grad=grad)
    within(grad, g, tol_g + TINY, "mean gradient")
    tol = float(tol_g.norm()) + U * norm + TINY
    within(clip.norm, torch.tensor([norm]).cuda(), tol, "norm")
    within(clip.scale, torch.tensor([0.5]).cuda(), 0.5 * (tol / norm + 3 * U), "scale")
    assert int(clip.skip) == 0
    opt.grad_norm(table, clip, max_norm=4 * norm)
    assert float(clip.scale) == 1.0
    opt.grad_norm(table, clip)
    assert float(clip.scale) == 1.0 and int(clip.skip) == 0


@pytest.mark.parametrize("W", [1, 5, 16, 40])
@pytest.mark.parametrize("fp16", [False, True])
def test_mean_gradient_is_the_tree_s(ga, W, fp16):
    numels = [3000, 5, 511, 8, 2049]
    dtype = torch.float16 if fp16 else torch.float32
    buf, table, rows = gradients(W, numels, dtype, seed=9)
    P = sum(numels)
    a, b = torch.empty(P, device="cuda"), torch.empty(P, device="cuda")
    ga.Plan(W, numels, fp16).tree_reduce_layers(table, a)
    opt = ga.AdamW(numels, W=W, grad_dtype=dtype)
    opt.grad_norm(table, opt.empty_clip(), grad=b)
    assert torch.equal(a, b)
    ref = oracle.dense_step(rows.to(dtype).cpu().numpy().view(np.uint16 if fp16 else np.float32), P, fp16, 0.0, 0.0,
                            None, None)
    assert np.array_equal(ref, b.cpu().numpy())


def test_grad_norm_many_workgroups(ga):
    """More tiles than one sweep of the workgroups takes, ending in a ragged tile."""
    numels = [5_000_000, 77, 3_000_001]
    g = torch.randn(sum(numels), device="cuda")
    starts = np.cumsum([0] + numels[:-1]) * 4 + g.data_ptr()
    table = torch.tensor(starts.tolist(), dtype=torch.int64, device="cuda")
    opt = ga.AdamW(numels)
    clip = opt.empty_clip()
    opt.grad_norm(table, clip)
    norm = float(g.double().norm())
    assert abs(float(clip.norm) - norm) <= norm * (U + 1e-12)


@pytest.mark.parametrize("size", [1e30, 1e-30, 0.0])
def test_grad_norm_range(ga, size):
    g = torch.full((1000,), size, device="cuda")
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    opt = ga.AdamW([1000])
    clip = opt.empty_clip()
    opt.grad_norm(table, clip, max_norm=1.0)
    norm = float(np.float32(size)) * math.sqrt(1000)
    assert abs(float(clip.norm) - norm) <= 2 * U * norm
    assert int(clip.skip) == 0
    assert abs(float(clip.scale) - min(1.0, 1.0 / norm if norm else 1.0)) <= 4 * U


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_that_is_not_finite_skips_the_step(ga, bad, bits):
    numels = [700, 300]
    g = torch.randn(1000, device="cuda")
    g[713] = bad
    table = torch.tensor([g.data_ptr(), g.data_ptr() + 2800], dtype=torch.int64, device="cuda")
    opt = ga.AdamW(numels, state_bits=bits)
    clip, state, w = opt.empty_clip(), opt.empty_state(), torch.randn(1000, device="cuda")
    copy = torch.zeros(1000, dtype=torch.bfloat16, device="cuda")
    opt.grad_norm(table, clip, max_norm=1.0)
    assert int(clip.skip) == 1
    before = w.clone()
    opt.step(table, w, state, t=1, clip=clip, copy=copy, **HYPER)
    assert torch.equal(w, before) and not copy.any()
    assert not state.m.view(torch.uint8).any() and not state.v.view(torch.uint8).any()
    g[713] = 0.0
    opt.grad_norm(table, clip, max_norm=1.0)
    opt.step(table, w, state, t=1, clip=clip, copy=copy, **HYPER)
    assert int(clip.skip) == 0 and not torch.equal(w, before) and torch.isfinite(w).all()


# ---- layer norm --------------------------------------------------------------

def chain(dim):
    """Additions in a row's sum: the longest chain of a lane, then the lanes."""
    return min(dim, max(64, dim // 128)) + 26


def ln_reference(s, gamma, beta, eps, dtype):
    """y, mean, rstd in binary64 with tolerances, of rows s."""
    dim = s.shape[1]
    k = chain(dim)
    mean = s.mean(1, keepdim=True)
    d = s - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    tol_mean = (k + 1) * U * s.abs().mean(1, keepdim=True) + TINY
    tol_d = tol_mean + U * d.abs()
    # the squares' errors: the deviations' own cancel to first order but for their rounding
    tol_var = (k + 4) * U * var + tol_mean ** 2 + 2 * U * (d.abs() * d.abs()).mean(1, keepdim=True)
    tol_rstd = rstd * (0.5 * tol_var / (var + eps) * 1.01 + 5 * U)
    y = d * rstd * gamma + beta
    tol_y = gamma.abs() * (tol_d * rstd + d.abs() * tol_rstd + U * (d * rstd).abs()) + U * y.abs()
    tol_y = tol_y * 1.01 + HALF_STEP[dtype] * (y.abs() + tol_y) + LEAST[dtype]
    return (y, tol_y), (mean[:, 0], tol_mean[:, 0]), (rstd[:, 0], tol_rstd[:, 0])


def strided(x, extra, offset=0):
    """A copy of x whose rows lie x.shape[1] + extra apart, `offset` elements
    into a buffer of NaN."""
    buf = torch.full((x.shape[0] * (x.shape[1] + extra) + offset,), math.nan, dtype=x.dtype, device="cuda")
    view = buf[offset:].view(x.shape[0], x.shape[1] + extra)[:, :x.shape[1]]
    view.copy_(x)
    return view


def check_ln_fwd(ga, rows, dim, x_dtype, p_dtype, res=False, keep_sum=True, affine=True, centre=0.0, extra=0, offset=0,
                 in_place=False):
    gen = torch.Generator().manual_seed(rows * 7919 + dim)
    x = (torch.randn(rows, dim, generator=gen) + centre).to(x_dtype).cuda()
    r = torch.randn(rows, dim, generator=gen).to(x_dtype).cuda() if res else None
    gamma = (1 + 0.2 * torch.randn(dim, generator=gen)).to(p_dtype).cuda() if affine else None
    beta = torch.randn(dim, generator=gen).to(p_dtype).cuda() if affine else None
    s = x if r is None else (x.float() + r.float()).to(x_dtype)
    one = torch.ones(dim, dtype=torch.float64, device="cuda")
    want = ln_reference(s.double(), one if gamma is None else gamma.double(), 0 * one if beta is None else beta.double(),
                        f32(1e-5), x_dtype)
    if extra or offset:
        x = strided(x, extra, offset)
        r = None if r is None else strided(r, extra + 3, offset + 1)
    y = x if in_place else strided(torch.zeros_like(s), extra, offset) if extra else torch.full_like(s, math.nan)
    total = torch.full_like(s, math.nan) if res and keep_sum else None
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ln = ga.LayerNorm(dim, x_dtype, p_dtype, backward=False)
    ln.forward(x, gamma, beta, y, mean, rstd, residual=r, sum_out=total, eps=1e-5)
    for name, got, (ref, tol) in zip(("y", "mean", "rstd"), (y, mean, rstd), want):
        within(got, ref, tol, name)
    if total is not None:
        assert torch.equal(total, s), "the sum, rounded once"
    if extra:
        assert torch.isnan(y.as_strided((rows - 1, extra), (dim + extra, 1), offset + dim)).all(), "gaps untouched"
    ln.close()


DIMS = [1, 2, 3, 7, 8, 48, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 1001, 1024, 1025, 2047, 2048, 2049, 4096,
        4097, 5120, 8192, 8193, 12288, 16383, 16384, 16385, 20001]
TYPES = [("fp32", "fp32"), ("fp16", "fp32"), ("fp16", "fp16"), ("bf16", "fp32"), ("bf16", "bf16")]


@pytest.mark.parametrize("x,p", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_ln_forward_widths(ga, dim, x, p):
    check_ln_fwd(ga, 5, dim, DT[x], DT[p])
    check_ln_fwd(ga, 3, dim, DT[x], DT[p], res=True)


@pytest.mark.parametrize("rows", [1, 2, 63, 64, 8193])
@pytest.mark.parametrize("dim", [96, 1001, 1536])
def test_ln_forward_rows(ga, rows, dim):
    check_ln_fwd(ga, rows, dim, torch.bfloat16, torch.float32, res=True)


@pytest.mark.parametrize("dim", [100, 1001, 4096, 20001])
@pytest.mark.parametrize("x", list(DT))
def test_ln_forward_forms(ga, dim, x):
    check_ln_fwd(ga, 6, dim, DT[x], DT[x], affine=False)
    check_ln_fwd(ga, 6, dim, DT[x], DT[x], res=True, keep_sum=False)
    check_ln_fwd(ga, 6, dim, DT[x], DT[x], res=True, extra=5, offset=1)
    check_ln_fwd(ga, 6, dim, DT[x], DT[x], in_place=True)
    check_ln_fwd(ga, 6, dim, DT[x], DT[x], res=True, in_place=True)


@pytest.mark.parametrize("dim", [64, 1001, 4096, 20001])
def test_ln_forward_far_from_zero(ga, dim):
    check_ln_fwd(ga, 9, dim, torch.float32, torch.float32, centre=1000.0)


def ln_bwd_reference(dy, x, gamma, mean, rstd, dsum, groups, dtype, dp_dtype):
    rows, dim = x.shape
    k = chain(dim)
    mean, rstd = mean[:, None], rstd[:, None]
    xh = (x - mean) * rstd
    tol_xh = 2 * U * xh.abs()
    h = dy * gamma
    m1 = h.mean(1, keepdim=True)
    m2 = (h * xh).mean(1, keepdim=True)
    tol_m1 = (k + 3) * U * h.abs().mean(1, keepdim=True)
    tol_m2 = (k + 6) * U * (h * xh).abs().mean(1, keepdim=True)
    inner = h - m1 - xh * m2
    tol_in = U * h.abs() + tol_m1 + xh.abs() * tol_m2 + 3 * U * (xh * m2).abs() + 2 * U * ((xh * m2).abs() + m1.abs()) + \
        U * inner.abs()
    dx = rstd * inner + (dsum if dsum is not None else 0.0)
    tol_dx = rstd * tol_in + U * dx.abs() + TINY
    tol_dx = tol_dx * 1.01 + HALF_STEP[dtype] * (dx.abs() + tol_dx) + LEAST[dtype]
    per = rows // groups if groups else 0
    split = lambda a: a.reshape(groups, per, dim)
    out = [(dx, tol_dx)]
    for term, own in ((dy * xh, (dy * xh).abs() * 3 * U), (dy, 0 * dy)):
        # any order of the group's rows: at most per - 1 additions each
        s = split(term).sum(1)
        tol = per * U * split(term).abs().sum(1) + split(own).sum(1) + TINY
        tol = tol * 1.01 + HALF_STEP[dp_dtype] * (s.abs() + tol) + LEAST[dp_dtype]
        out.append((s, tol))
    return out


def check_ln_bwd(ga, rows, dim, x_dtype, p_dtype, dp_dtype=torch.float32, groups=1, res=False, affine=True, extra=0,
                 offset=0, alias=None, weights=True):
    gen = torch.Generator().manual_seed(rows * 104729 + dim + groups)
    rand = lambda *shape: torch.randn(*shape, generator=gen)
    x = (rand(rows, dim) * 2 + 0.5).to(x_dtype).cuda()
    dy = (0.1 * rand(rows, dim)).to(x_dtype).cuda()
    gamma = (1 + 0.2 * rand(dim)).to(p_dtype).cuda() if affine else None
    dsum = (0.1 * rand(rows, dim)).to(x_dtype).cuda() if res else None
    x64 = x.double()
    mean = x64.mean(1).float()
    rstd = ((x64.var(1, unbiased=False) + 1e-5) ** -0.5).float()
    want = ln_bwd_reference(dy.double(), x64, gamma.double() if affine else torch.ones(dim).double().cuda(),
                            mean.double(), rstd.double(), dsum.double() if res else None, groups, x_dtype, dp_dtype)
    if extra or offset:
        x, dy = strided(x, extra, offset), strided(dy, extra + 2, offset)
        dsum = None if dsum is None else strided(dsum, extra + 1, offset + 1)
    dx = {"x": x, "dy": dy, "dsum": dsum}[alias] if alias else torch.full((rows, dim), math.nan, dtype=x_dtype,
                                                                        device="cuda")
    dg = db = None
    if weights:
        dg, db = (torch.full((groups, dim), math.nan, dtype=dp_dtype, device="cuda") for _ in range(2))
    ln = ga.LayerNorm(dim, x_dtype, p_dtype)
    ln.backward(dy, x, gamma, mean, rstd, dx, dg, db, dsum=dsum, groups=groups)
    for name, got, (ref, tol) in zip(("dx", "dgamma", "dbeta"), (dx, dg, db), want):
        if got is not None:
            within(got, ref, tol, name)
    ln.close()


@pytest.mark.parametrize("x,p", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_ln_backward_widths(ga, dim, x, p):
    check_ln_bwd(ga, 6, dim, DT[x], DT[p], dp_dtype=DT[x])
    check_ln_bwd(ga, 9, dim, DT[x], DT[p], res=True, groups=3)


@pytest.mark.parametrize("rows,groups", [(1, 1), (2, 2), (64, 1), (513, 1), (4100, 1), (4100, 4), (1024, 1024),
                                         (1026, 513), (2000, 500)])
@pytest.mark.parametrize("dim", [96, 1001, 2500, 20001])
@pytest.mark.parametrize("dp", ["fp32", "fp16"])
def test_ln_backward_rows_and_groups(ga, rows, groups, dim, dp):
    if dim > 10000 and rows > 1100:
        rows, groups = rows // 4 // groups * groups or groups, groups
    check_ln_bwd(ga, rows, dim, torch.bfloat16, torch.float32, dp_dtype=DT[dp], groups=groups)


@pytest.mark.parametrize("dim", [100, 1001, 4096, 20001])
@pytest.mark.parametrize("x", list(DT))
def test_ln_backward_forms(ga, dim, x):
    check_ln_bwd(ga, 6, dim, DT[x], DT[x], affine=False, dp_dtype=torch.bfloat16)
    check_ln_bwd(ga, 6, dim, DT[x], DT[x], weights=False)
    check_ln_bwd(ga, 6, dim, DT[x], DT[x], res=True, extra=5, offset=1, groups=2)
    for alias in ("x", "dy", "dsum"):
        check_ln_bwd(ga, 6, dim, DT[x], DT[x], res=True, alias=alias)


def test_ln_backward_against_differences(ga):
    """dx, dgamma and dbeta against central differences of the forward formula
    in binary64 (step h: their own error is O(h^2), about 1e-9 here)."""
    rows, dim, h = 3, 17, 1e-5
    gen = torch.Generator().manual_seed(3)
    x, dy = torch.randn(rows, dim, generator=gen), torch.randn(rows, dim, generator=gen)
    gamma, beta = 1 + 0.2 * torch.randn(dim, generator=gen), torch.randn(dim, generator=gen)

    def loss(x, gamma, beta):
        d = x - x.mean(1, keepdim=True)
        return float((dy.double() * (d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * gamma + beta)).sum())

    def slope(k):
        args = [x.double(), gamma.double(), beta.double()]
        out = torch.zeros_like(args[k])
        for i in range(out.numel()):
            both = []
            for sign in (1, -1):
                moved = args[k].clone()
                moved.view(-1)[i] += sign * h
                both.append(loss(*[moved if j == k else a for j, a in enumerate(args)]))
            out.view(-1)[i] = (both[0] - both[1]) / (2 * h)
        return out

    xd, mean, rstd = x.cuda(), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y, dx = torch.empty_like(xd), torch.empty_like(xd)
    dg, db = torch.empty(1, dim, device="cuda"), torch.empty(1, dim, device="cuda")
    ln = ga.LayerNorm(dim)
    ln.forward(xd, gamma.cuda(), beta.cuda(), y, mean, rstd, eps=1e-5)
    ln.backward(dy.cuda(), xd, gamma.cuda(), mean, rstd, dx, dg, db)
    for k, got in enumerate((dx, dg[0], db[0])):
        within(got.cpu(), slope(k), 1e-7 + 200 * U, "gradient %d" % k)


def test_ln_no_rows(ga):
    x = torch.empty(0, 65, device="cuda")
    ln = ga.LayerNorm(65)
    ln.forward(x, None, None, torch.empty_like(x))
    dg, db = torch.full((2, 65), math.nan, device="cuda"), torch.full((2, 65), math.nan, device="cuda")
    ln.backward(x, x, None, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), torch.empty_like(x), dg, db,
                groups=2)
    assert not dg.any() and not db.any()


def test_ln_higher_dimensions_and_refusals(ga):
    ln = ga.LayerNorm(24, torch.float16, torch.float32, backward=False)
    x = torch.randn(2, 3, 4, 24, device="cuda").half()
    y, flat = torch.empty_like(x), torch.empty(24, 24, device="cuda", dtype=torch.float16)
    ln.forward(x, None, None, y)
    ln.forward(x.reshape(24, 24), None, None, flat)
    assert torch.equal(y.reshape(24, 24), flat)
    wide = torch.randn(2, 3, 40, device="cuda").half()[:, :, 8:32]       # evenly spaced rows
    out = torch.empty(2, 3, 24, dtype=torch.float16, device="cuda")
    same = torch.empty_like(out)
    ln.forward(wide, None, None, out)
    ln.forward(wide.contiguous(), None, None, same)
    assert torch.equal(out, same)
    for bad in (torch.randn(4, 25, device="cuda").half(), torch.randn(4, 24, device="cuda"),
                torch.randn(24, 4, device="cuda").half().t(), torch.randn(4, 6, 24, device="cuda").half()[:, :3],
                torch.randn(4, 24).half()):
        with pytest.raises((ValueError, ga.GAError)):
            ln.forward(bad, None, None, torch.empty_like(bad))
    with pytest.raises(ga.GAError):                                       # made without a backward pass
        ln.backward(x, x, None, torch.zeros(24, device="cuda"), torch.zeros(24, device="cuda"), y)
    with pytest.raises(ValueError):
        ln.forward(x, torch.ones(23, device="cuda"), None, y)
    with pytest.raises(ValueError):
        ln.forward(x, torch.ones(24, device="cuda").half(), None, y)


# ---- streams, graphs, repeats --------------------------------------------------

def whole_step(ga, seed):
    """A layer norm forward and backward, the norm of its weight gradients over
    4 workers, and the update, as closures over one set of buffers."""
    gen = torch.Generator().manual_seed(seed)
    rows, dim, W = 64, 520, 4
    b = {}
    b["x"], b["res"], b["dy"] = (torch.randn(rows, dim, generator=gen).bfloat16().cuda() for _ in range(3))
    b["gamma"], b["beta"] = torch.ones(dim, device="cuda"), torch.zeros(dim, device="cuda")
    b["y"], b["s"], b["dx"] = (torch.zeros_like(b["x"]) for _ in range(3))
    b["mean"], b["rstd"] = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    b["grads"] = torch.zeros(2, W, dim, dtype=torch.float16, device="cuda")
    ptrs = [b["grads"].data_ptr() + 2 * (k * W + w) * dim for w in range(W) for k in range(2)]
    b["table"] = torch.tensor(ptrs, dtype=torch.int64, device="cuda")
    b["w"] = torch.cat((b["gamma"], b["beta"]))
    b["copy"] = torch.zeros(2 * dim, dtype=torch.bfloat16, device="cuda")
    ln, opt = ga.LayerNorm(dim, torch.bfloat16, torch.float32), ga.AdamW([dim, dim], W=W, grad_dtype=torch.float16,
                                                                       state_bits=8, decay=[False, True])
    state, clip = opt.empty_state(), opt.empty_clip()
    b.update(m=state.m, v=state.v, ms=state.m_scale, vs=state.v_scale, clip=clip.record)

    def run():
        ln.forward(b["x"], b["w"][:dim], b["w"][dim:], b["y"], b["mean"], b["rstd"], residual=b["res"], sum_out=b["s"])
        ln.backward(b["dy"], b["s"], b["w"][:dim], b["mean"], b["rstd"], b["dx"], b["grads"][0], b["grads"][1],
                    dsum=b["dy"], groups=W)
        opt.grad_norm(b["table"], clip, max_norm=0.1)
        opt.step(b["table"], b["w"], state, t=5, lr=1e-2, weight_decay=0.1, clip=clip, copy=b["copy"])

    run.keep = (ln, opt)
    return b, run


def bits(b):
    return {k: t.clone().view(torch.uint8) for k, t in b.items() if k != "table"}


def test_repeats_streams_and_graphs_agree(ga):
    """The same buffers through the current stream, another stream and a graph
    replayed with eager work between the replays: the same bits, step by step."""
    want = []
    b, run = whole_step(ga, 11)
    for _ in range(4):
        run()
        want.append(bits(b))

    b, run = whole_step(ga, 11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for ref in want:
            run()
            got = bits(b)
            side.synchronize()
            assert all(torch.equal(ref[k], got[k]) for k in ref)

    b, run = whole_step(ga, 11)
    start_bits = {k: t.clone() for k, t in b.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k, t in b.items():
        t.copy_(start_bits[k])
    for ref in want:
        graph.replay()
        got = bits(b)
        torch.randn(1000, device="cuda").sum()
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(ref[k], got[k]), k


def test_binding_refuses_arguments(ga):
    opt = ga.AdamW([100], W=2)
    w, state, clip = torch.zeros(100, device="cuda"), opt.empty_state(), opt.empty_clip()
    table = torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (lambda: opt.step(table[:1], w, state, t=1, lr=0.1), lambda: opt.step(table, w[:99], state, t=1, lr=0.1),
                 lambda: opt.step(table, w.double(), state, t=1, lr=0.1),
                 lambda: opt.step(table, w, state, t=1, lr=0.1, copy=torch.zeros(99, dtype=torch.float16, device="cuda")),
                 lambda: opt.step(table.cpu(), w, state, t=1, lr=0.1),
                 lambda: opt.grad_norm(table, clip, grad=torch.zeros(50, device="cuda")),
                 lambda: ga.AdamW([100], state_bits=8).step(table, w, state, t=1, lr=0.1)):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: opt.step(table, w, state, t=0, lr=0.1), ga.GA_ERR_INVALID),
                         (lambda: opt.step(table, w, state, t=1, lr=0.1, copy=w), ga.GA_ERR_INVALID),
                         (lambda: opt.grad_norm(table, clip, max_norm=0.0), ga.GA_ERR_INVALID),
                         (lambda: ga.AdamW([100], state_bits=4), ga.GA_ERR_INVALID)):
        with pytest.raises(ga.GAError) as e:
            call()
        assert e.value.status == status
    both = torch.zeros(101, device="cuda")
    with pytest.raises(ga.GAError) as e:
        opt.step(table, both[1:], state, t=1, lr=0.1)
    assert e.value.status == ga.GA_ERR_ALIGN
