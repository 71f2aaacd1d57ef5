"""Edges of the training-step operators on the GPU: tensors written over their
inputs at widths whose last vector crosses a wavefront, workgroup counts around
the norm's second kernel, moments below the normal range, offsets past 32 bits,
and the example that runs the operators together."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ga():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gradient_aggregation_amd as ga
    return ga


# One element past a wavefront's columns, of each team size: the last vector is
# read from where it ends at the row's end, which another wavefront writes.
WIDTHS = [9, 129, 257, 513, 515, 1025, 1030, 1281, 2049, 2055, 4097, 8193, 8200, 12289]


@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("dim", WIDTHS)
def test_ln_in_place(ga, dim, x):
    """y or the sum over x or the residual, and dx over dy, x or dsum: the bits
    of the calls with outputs of their own."""
    gen = torch.Generator().manual_seed(dim)
    rows, dt = 37, DT[x]
    a, r, dy, ds = (torch.randn(rows, dim, generator=gen).to(dt).cuda() for _ in range(4))
    gamma, beta = torch.randn(dim, generator=gen).cuda(), torch.randn(dim, generator=gen).cuda()
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ln = ga.LayerNorm(dim, dt, torch.float32)
    y, s = torch.empty_like(a), torch.empty_like(a)
    ln.forward(a, gamma, beta, y, mean, rstd, residual=r, sum_out=s)
    stats = mean.clone(), rstd.clone()
    for k in range(4):                                     # sum over x, over the residual; y over x, over the residual
        a2, r2, other = a.clone(), r.clone(), torch.empty_like(a)
        y2, s2 = [(other, a2), (other, r2), (a2, other), (r2, other)][k]
        ln.forward(a2, gamma, beta, y2, mean, rstd, residual=r2, sum_out=s2)
        assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(mean, stats[0]) and torch.equal(rstd, stats[1])
    plain = torch.empty_like(a)
    ln.forward(a, gamma, beta, plain)
    own = a.clone()
    ln.forward(own, gamma, beta, own)
    assert torch.equal(own, plain)

    dx, dg, db = torch.empty_like(a), torch.empty(1, dim, device="cuda"), torch.empty(1, dim, device="cuda")
    ln.backward(dy, s, gamma, mean, rstd, dx, dg, db, dsum=ds)
    sums = dg.clone(), db.clone()
    for k in range(3):
        t = [dy.clone(), s.clone(), ds.clone()]
        ln.backward(t[0], t[1], gamma, mean, rstd, t[k], dg, db, dsum=t[2])
        assert torch.equal(t[k], dx) and torch.equal(dg, sums[0]) and torch.equal(db, sums[1])


@pytest.mark.parametrize("x", ["fp32", "fp16"])
@pytest.mark.parametrize("dim", [1, 7, 8, 9, 65, 130, 511, 1001, 2050])
def test_ln_neighbours_stay(ga, dim, x):
    """Rows inside wider ones: the columns beside them are neither read into a
    result nor written."""
    gen = torch.Generator().manual_seed(dim)
    rows, dt = 19, DT[x]
    wide = torch.full((5, rows, dim + 5), math.nan, dtype=dt).cuda()
    a, dy, y, dx, out = (w[:, 3:3 + dim] for w in wide)
    a.copy_(torch.randn(rows, dim, generator=gen))
    dy.copy_(torch.randn(rows, dim, generator=gen))
    ln = ga.LayerNorm(dim, dt)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dg, db = torch.empty(1, dim, device="cuda"), torch.empty(1, dim, device="cuda")
    ln.forward(a, None, None, y, mean, rstd)
    ln.backward(dy, a, None, mean, rstd, dx, dg, db)
    same = [torch.empty(rows, dim, dtype=dt, device="cuda") for _ in range(2)]
    sums = torch.empty(2, 1, dim, device="cuda")
    ln.forward(a.contiguous(), None, None, same[0])
    ln.backward(dy.contiguous(), a.contiguous(), None, mean, rstd, same[1], sums[0], sums[1])
    assert torch.equal(y, same[0]) and torch.equal(dx, same[1])
    assert torch.equal(dg, sums[0]) and torch.equal(db, sums[1]) and bool(torch.isfinite(dg).all())
    assert bool(wide[:, :, :3].isnan().all()) and bool(wide[:, :, 3 + dim:].isnan().all())


@pytest.mark.parametrize("W", [1, 3])
@pytest.mark.parametrize("blocks", [1, 2, 255, 256, 257, 300])
def test_grad_norm_around_the_second_kernel(ga, blocks, W):
    """A workgroup takes 2048 elements: one launch up to 256 of them, two
    beyond.  Calls in a row find the counter as they need it."""
    n = blocks * 2048 - 5
    gen = torch.Generator().manual_seed(n)
    rows = torch.randn(W, n, generator=gen).cuda()
    table = torch.tensor([rows[w].data_ptr() for w in range(W)], dtype=torch.int64, device="cuda")
    opt = ga.AdamW([n], W=W)
    clip = opt.empty_clip()
    got = []
    for _ in range(3):
        clip.record.fill_(-1.0)
        opt.grad_norm(table, clip, max_norm=2.0)
        got.append(clip.record.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    want = float(rows.double().mean(0).norm())
    # the mean of W values: W - 1 additions and the product with 1/W, itself rounded; then one rounding of the norm
    tol = (0 if W == 1 else (W + 1) * U * float(rows.double().abs().mean(0).norm())) + U * want
    assert abs(float(got[0][0]) - want) <= tol
    assert abs(float(got[0][1]) - 2.0 / want) <= 2.0 / want * (tol / want + 2 * U)


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-30])
def test_adamw_second_moments_below_the_normal_range(ga, eps):
    """v down to the least denormal: its root is 2^-74.5, far above eps.  With
    m = v = 0 the weight keeps its value for any eps above 0."""
    v = torch.tensor([2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126, 2.0 ** -100, 2.0 ** -64, 1.0, 0.0], device="cuda")
    v = v.repeat(65)
    m = v.double().sqrt().float()
    w, g = torch.ones_like(v), torch.zeros_like(v)
    opt = ga.AdamW([v.numel()])
    table = torch.tensor([g.data_ptr()], dtype=torch.int64, device="cuda")
    # beta1 = beta2 = 0.5 at t = 1: m/2 over 1/2, the root of (v/2) over (1/2)
    vn = (v * 0.5).double()
    state = ga.AdamWState(m.clone(), v.clone())
    opt.step(table, w, state, t=1, lr=0.25, beta1=0.5, beta2=0.5, eps=eps)
    assert torch.equal(state.m, m * 0.5) and torch.equal(state.v, v * 0.5)
    some = vn > 0
    want = 1 - 0.25 * m.double() / ((2 * vn).sqrt() + eps)
    # a root and a reciprocal of 2 units each, the factors of t and four products and sums
    assert float((w.double() - want)[some].abs().max()) <= 12 * U
    if eps > 0:
        still = (v == 0)
        assert bool((w[still] == 1).all())


def test_offsets_past_32_bits(ga):
    """A layer of 2^31 + 1000 elements: its last ones against a handle of their
    own; then rows that far apart."""
    n, tail = (1 << 31) + 1000, 3000
    base = (n - tail) // 512 * 512                        # a tile boundary (and a block's)
    k = n - base
    gen = torch.Generator().manual_seed(3)
    g = torch.zeros(n, dtype=torch.float16, device="cuda")
    g[base:] = torch.randn(k, generator=gen).half().cuda()
    w, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    w[base:] = torch.randn(k, generator=gen).cuda()
    small = [t[base:].clone() for t in (g, w, m, v)]
    norms = []
    for grads, wt, mt, vt in ((g, w, m, v), small):
        opt = ga.AdamW([grads.numel()], grad_dtype=torch.float16)
        table = torch.tensor([grads.data_ptr()], dtype=torch.int64, device="cuda")
        clip = opt.empty_clip()
        opt.grad_norm(table, clip, max_norm=math.inf)
        norms.append(float(clip.norm))
        opt.step(table, wt, ga.AdamWState(mt, vt), t=1, lr=0.1, clip=clip)
        opt.close()
    for a, b in zip((w, m, v), small[1:]):
        assert torch.equal(a[base:], b)
    assert abs(norms[0] - norms[1]) <= 2 * U * norms[1] and not m[:base].any()   # each rounded once
    del w, m, v, small
    # two rows of a tensor whose stride passes 2^32 bytes
    ld = (1 << 31) + 200
    big = torch.zeros(ld + 130, dtype=torch.float16, device="cuda").as_strided((2, 130), (ld, 1))
    big.copy_(torch.randn(2, 130, generator=gen))
    ln = ga.LayerNorm(130, torch.float16)
    y, same = torch.empty(2, 130, dtype=torch.float16, device="cuda"), torch.empty(2, 130, dtype=torch.float16, device="cuda")
    ln.forward(big.contiguous(), None, None, same)
    ln.forward(big, None, None, y)
    assert torch.equal(y, same)
    ln.forward(big, None, None, big)
    assert torch.equal(big, same)


@pytest.mark.parametrize("bits", [8, 32])
def test_example_learns(ga, bits):
    spec = importlib.util.spec_from_file_location("train_mlp", os.path.join(ROOT, "examples", "train_mlp.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.train(steps=60, W=4, batch=32, state_bits=bits)
    assert all(math.isfinite(a) for a in losses)
    # from chance, log(10), to half of it
    assert sum(losses[:3]) / 3 > 2.0 and sum(losses[-10:]) / 10 < 1.2
