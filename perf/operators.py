"""Cases of the training-step operators: AdamW over a layer list with 32- or
8-bit states, the global gradient norm, and layer norm forward and backward.

`run` computes each operator in its plain form (elementary torch operations in
binary32) where `own` is false, and through gradient_aggregation_amd where it
is true.  The layer lists are those of the library's CNN workloads and generic
ones; layer norm takes generic widths.

Gradients of W workers lie in one [W][ld] buffer whose rows hold the layers in
fused order; w, m, v and the low-precision copy are flat vectors of P elements
(8-bit states: one scale per 256 consecutive elements)."""
import math
import random

import torch

own = False

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ESZ = {"fp32": 4, "fp16": 2, "bf16": 2}
BLOCK = 256             # elements per scale of the 8-bit states
E4M3_MAX = 448.0
E4M3_MIN = 2.0 ** -6    # smallest normal
FLOOR = 2.0 ** -100     # least block maximum
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 1e-3, 0.05
LN_EPS = 1e-5

# element counts of the layers, in fused order
NETS = {
    # the small listed network of the library's tests: 29,354 elements
    "tiny": [432, 16, 4608, 32, 18432, 64, 5760, 10],
    # 12 convolutions and their biases: 7.6M elements
    "nin": [34848, 96, 9216, 96, 9216, 96, 614400, 256, 65536, 256, 65536, 256, 884736, 384, 147456, 384, 147456, 384,
            3538944, 1024, 1048576, 1024, 1024000, 1000],
    # 5 convolutions, 3 matrices and their biases: 61M elements
    "alexnet": [34848, 96, 307200, 256, 884736, 384, 663552, 384, 442368, 256, 37748736, 4096, 16777216, 4096,
                4096000, 1000],
}


def layers(case):
    """Element counts of the case's layers (a drawn list: matrices, vectors and odd sizes adding up to about P)."""
    if case["net"] in NETS:
        return NETS[case["net"]]
    rng, left, out = random.Random(case["mix"]), case["P"], []
    for k in range(case["L"] - 1):
        n = min(left - (case["L"] - 1 - k), max(1, int(left * rng.uniform(0.05, 0.6)) if k % 2 == 0 else rng.randint(1, 4096)))
        out.append(max(1, n))
        left -= out[-1]
    return out + [max(1, left)]


def listed():
    return [
        # a small model's whole update: launch latency is all
        {"name": "adamw tiny fp32", "op": "adamw", "bits": 32, "net": "tiny", "W": 1, "grad": "fp32", "clip": False, "copy": "none"},
        # one worker's bf16 gradients, clipped, with the bf16 weights of the next forward pass
        {"name": "adamw nin bf16 clip", "op": "adamw", "bits": 32, "net": "nin", "W": 1, "grad": "bf16", "clip": True, "copy": "bf16"},
        # the data-parallel step: 16 workers' binary16 gradients averaged and applied in one go
        {"name": "adamw alexnet W16 fp16", "op": "adamw", "bits": 32, "net": "alexnet", "W": 16, "grad": "fp16", "clip": False, "copy": "none"},
        # the same update with states in 8 bits, smallest and largest
        {"name": "adamw8 tiny bf16", "op": "adamw", "bits": 8, "net": "tiny", "W": 1, "grad": "bf16", "clip": False, "copy": "none"},
        {"name": "adamw8 alexnet bf16 clip", "op": "adamw", "bits": 8, "net": "alexnet", "W": 1, "grad": "bf16", "clip": True, "copy": "bf16"},
        # the norm that clips them: one small model, one large one, and four workers' mean gradient kept
        {"name": "grad_norm tiny fp32", "op": "norm", "net": "tiny", "W": 1, "grad": "fp32", "keep": False},
        {"name": "grad_norm alexnet bf16", "op": "norm", "net": "alexnet", "W": 1, "grad": "bf16", "keep": False},
        # one token of a decoder layer
        {"name": "ln_fwd 1x4096 bf16", "op": "ln_fwd", "rows": 1, "dim": 4096, "x": "bf16", "p": "bf16", "res": False},
        # a training batch of a residual block: the sum and its norm
        {"name": "ln_fwd 16384x4096 bf16 res", "op": "ln_fwd", "rows": 16384, "dim": 4096, "x": "bf16", "p": "fp32", "res": True},
        # a short sequence of a small encoder, one worker
        {"name": "ln_bwd 128x512 fp32", "op": "ln_bwd", "rows": 128, "dim": 512, "x": "fp32", "p": "fp32", "dp": "fp32", "W": 1, "res": False},
        # an odd width and a ragged number of rows
        {"name": "ln_bwd 6151x1001 fp16", "op": "ln_bwd", "rows": 6151, "dim": 1001, "x": "fp16", "p": "fp32", "dp": "fp32", "W": 1, "res": False},
        # a training batch of 16 workers, each worker's weight gradients in its own row
        {"name": "ln_bwd 16384x4096 bf16 W16", "op": "ln_bwd", "rows": 16384, "dim": 4096, "x": "bf16", "p": "fp32", "dp": "fp16", "W": 16, "res": True},
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "norm", "ln_fwd", "ln_bwd"])
    if op in ("adamw", "norm"):
        W = rng.choice([1, 1, 1, 2, 3, 5, 8, 16])
        P = min(spread(rng, 1000, 60_000_000), 400_000_000 // W)
        c = {"op": op, "net": "drawn", "P": P, "L": rng.randint(1, 40), "mix": rng.randint(0, 1 << 30), "W": W,
             "grad": rng.choice(["fp32", "fp16", "bf16"])}
        if op == "adamw":
            c.update(bits=rng.choice([32, 8]), clip=rng.random() < 0.5, copy=rng.choice(["none", "bf16", "fp16"]))
        else:
            c["keep"] = rng.random() < 0.5
        return c
    dim = spread(rng, 48, 12288) if rng.random() < 0.5 else rng.choice([64, 128, 512, 768, 1024, 2048, 4096, 5120, 8192])
    W = 1 if op == "ln_fwd" else rng.choice([1, 1, 2, 4, 16])
    x = rng.choice(["fp32", "fp16", "bf16"])
    rows = max(W, min(spread(rng, 1, 60000), 130_000_000 // (dim * ESZ[x])) // W * W)
    c = {"op": op, "rows": rows, "dim": dim, "x": x, "p": rng.choice(["fp32", x]), "res": rng.random() < 0.5}
    if op == "ln_bwd":
        c.update(W=W, dp=rng.choice(["fp32", "fp16", "bf16"]))
    return c


def work(case):
    if case["op"] in ("adamw", "norm"):
        P, W = sum(layers(case)), case["W"]
        read = W * P * ESZ[case["grad"]]
        if case["op"] == "norm":
            return {"bytes": read + (4 * P if case["keep"] else 0) + 16, "flops": (W + 2) * P}
        state = 16 * P if case["bits"] == 32 else 4 * P + 16 * ((P + BLOCK - 1) // BLOCK)
        return {"bytes": read + 8 * P + state + (2 * P if case["copy"] != "none" else 0), "flops": (W + 20) * P}
    n, b = case["rows"] * case["dim"], ESZ[case["x"]]
    if case["op"] == "ln_fwd":
        return {"bytes": n * b * (4 if case["res"] else 2) + 2 * case["dim"] * ESZ[case["p"]] + 8 * case["rows"], "flops": 8 * n}
    return {"bytes": n * b * (4 if case["res"] else 3) + case["dim"] * (ESZ[case["p"]] + 2 * case["W"] * ESZ[case["dp"]]) + 8 * case["rows"],
            "flops": 14 * n}


def nearest_codes(x):
    """8-bit codes and scales of x [n_blocks][256], rounded to nearest."""
    top = x.abs().amax(1, keepdim=True).clamp_min(FLOOR)
    return (x * (E4M3_MAX / top)).to(torch.float8_e4m3fn), (top * (1.0 / E4M3_MAX)).reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st = {"case": case}
    if case["op"] in ("adamw", "norm"):
        numels, W, gdt = layers(case), case["W"], DT[case["grad"]]
        P = sum(numels)
        ld = (P + 63) // 64 * 64
        scale = (10.0 ** (2 * torch.rand(len(numels), generator=gen, device="cuda") - 1)).repeat_interleave(
            torch.tensor(numels, device="cuda"), output_size=P) * 1e-3       # per-layer gradient size
        grads = torch.zeros(W, ld, dtype=gdt, device="cuda")
        for w in range(W):
            grads[w, :P] = normal(P) * scale
        st.update(P=P, grads=grads)
        if own:
            import gradient_aggregation_amd as ga
            starts = torch.tensor([0] + numels[:-1], dtype=torch.int64).cumsum(0) * grads.element_size()
            rows = torch.arange(W, dtype=torch.int64) * (ld * grads.element_size()) + grads.data_ptr()
            st["table"] = (rows[:, None] + starts[None, :]).reshape(-1).cuda()
        if case["op"] == "norm":
            st["max_norm"] = 1.0
            if case["keep"]:
                st["mean"] = torch.zeros(P, device="cuda")
            if own:
                st["opt"] = ga.AdamW(numels, W=W, grad_dtype=gdt)
                st["clip"] = st["opt"].empty_clip()
            return st
        # vectors (biases, norm weights) are not decayed
        st["decays"] = [n > 4096 for n in numels]
        st["w"] = normal(P) * 0.05
        m, s = normal(P) * scale * 0.3, scale * (0.5 + torch.rand(P, generator=gen, device="cuda"))
        st["t"] = 1000
        st["copy"] = None if case["copy"] == "none" else st["w"].to(DT[case["copy"]])
        if case["bits"] == 32:
            st["m"], st["v"] = m, s * s
        else:
            pad = (-P) % BLOCK
            m, s = (torch.nn.functional.pad(a, (0, pad)).reshape(-1, BLOCK) for a in (m, s))
            st["m"], st["m_scale"] = nearest_codes(m)
            st["v"], st["v_scale"] = nearest_codes(s)
        # the record that a norm over these gradients left: clipped to a quarter
        st["clip_scale"] = torch.tensor([0.25], device="cuda") if case["clip"] else None
        if own:
            st["opt"] = ga.AdamW(numels, W=W, grad_dtype=gdt, state_bits=case["bits"], decay=st["decays"])
            st["state"] = ga.AdamWState(st["m"], st["v"], st.get("m_scale"), st.get("v_scale"))
            st["clip"] = None
            if case["clip"]:
                st["clip"] = st["opt"].empty_clip()
                st["clip"].scale.copy_(st["clip_scale"])
        else:
            st["decay"] = torch.tensor([DECAY if d else 0.0 for d in st["decays"]], device="cuda").repeat_interleave(
                torch.tensor(numels, device="cuda"), output_size=P)
        return st
    rows, dim, xdt, pdt = case["rows"], case["dim"], DT[case["x"]], DT[case["p"]]
    st["x"] = (normal(rows, dim) + 0.3 * normal(rows, 1)).to(xdt)
    st["gamma"], st["beta"] = (1 + 0.1 * normal(dim)).to(pdt), (0.1 * normal(dim)).to(pdt)
    st["res"] = normal(rows, dim).to(xdt) if case["res"] else None
    if case["op"] == "ln_bwd":
        x = st["x"].double()
        st["mean"] = x.mean(1).float()
        st["rstd"] = (1 / (x.var(1, unbiased=False) + LN_EPS).sqrt()).float()
        st["dy"] = (1e-2 * normal(rows, dim)).to(xdt)
        if case["res"]:
            st["res"] = 1e-2 * st["res"]          # the gradient that reaches the sum directly
    if own:
        import gradient_aggregation_amd as ga
        st["ln"] = ga.LayerNorm(dim, xdt, pdt)
    return st


def mean_gradient(st):
    g = st["grads"][:, :st["P"]]
    return g[0].float() if g.shape[0] == 1 else g.sum(0, dtype=torch.float32) * (1.0 / g.shape[0])


def random_bits(n, seed):
    """20 random bits for each of n elements from the counter (element // 2, seed): a multiply and xor-shift mixer
    gives 32 bits to a pair, 16 to each, centred in their interval."""
    mask = 0xFFFFFFFF
    x = (torch.arange((n + 1) // 2, device="cuda") + (seed * 0x9E3779B9 + 0x7F4A7C15)) & mask
    x = ((x ^ (x >> 16)) * 0xB7E15163) & mask
    x = ((x ^ (x >> 15)) * 0x6A09E667) & mask
    x = x ^ (x >> 16)
    r = torch.stack((x & 0xFFFF, x >> 16), 1).reshape(-1)[:n]
    return ((r << 4) | 8).to(torch.int32)


def plain_adamw(st):
    P, t, w = st["P"], st["t"], st["w"]
    # the hyper-parameters are binary32 values, their combinations are rounded once
    b1, b2, lr, eps = (torch.tensor(a, dtype=torch.float32).item() for a in (BETA1, BETA2, LR, EPS))
    g = mean_gradient(st)
    if st["clip_scale"] is not None:
        g = g * st["clip_scale"]
    if st["case"]["bits"] == 32:
        m, v = st["m"], st["v"]
    else:
        m = (st["m"].float() * st["m_scale"][:, None]).reshape(-1)[:P]
        s = (st["v"].float() * st["v_scale"][:, None]).reshape(-1)[:P]
        v = s * s
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * (1 - b2)) * g
    s = v.sqrt()
    w.copy_(w * (1 - lr * st["decay"]) - (lr / (1 - b1 ** t)) * (m / (s * (1 / math.sqrt(1 - b2 ** t)) + eps)))
    if st["copy"] is not None:
        st["copy"].copy_(w)
    if st["case"]["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return [st[k] for k in ("w", "m", "v", "copy") if st[k] is not None]
    pad = (-P) % BLOCK
    m, s = (torch.nn.functional.pad(a, (0, pad)).reshape(-1, BLOCK) for a in (m, s))
    codes, scales = nearest_codes(m)
    st["m"].copy_(codes)
    st["m_scale"].copy_(scales)
    top = s.amax(1, keepdim=True).clamp_min(FLOOR)
    x = s * (E4M3_MAX / top)
    x = torch.where(x > E4M3_MAX, E4M3_MAX, x)
    x = torch.where((s > 0) & (x < E4M3_MIN), E4M3_MIN, x)
    # three mantissa bits stay: the random bits are added to the 20 that go
    x = ((x.view(torch.int32) + random_bits(x.numel(), t).reshape(x.shape)) & -0x100000).view(torch.float32)
    st["v"].copy_(x.to(torch.float8_e4m3fn))
    st["v_scale"].copy_((top * (1.0 / E4M3_MAX)).reshape(-1))
    return [st[k] for k in ("w", "m", "v", "m_scale", "v_scale", "copy") if st[k] is not None]


def plain_norm(st):
    g = mean_gradient(st)
    norm = g.double().square().sum().sqrt().float().reshape(1)
    out = [norm, torch.clamp(st["max_norm"] / norm, max=1.0), (~torch.isfinite(norm)).to(torch.int32)]
    if st["case"]["keep"]:
        st["mean"].copy_(g)
        out.append(st["mean"])
    return out


def plain_ln_fwd(st):
    x, s = st["x"], None
    if st["res"] is not None:
        x = s = (x.float() + st["res"].float()).to(x.dtype)
    f = x.float()
    mean = f.mean(1)
    c = f - mean[:, None]
    rstd = 1 / ((c * c).mean(1) + LN_EPS).sqrt()
    y = (c * rstd[:, None] * st["gamma"].float() + st["beta"].float()).to(x.dtype)
    return [y, mean, rstd] + ([s] if s is not None else [])


def plain_ln_bwd(st):
    case, x, dy = st["case"], st["x"].float(), st["dy"].float()
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    h = dy * st["gamma"].float()
    dx = st["rstd"][:, None] * (h - h.mean(1, keepdim=True) - xh * (h * xh).mean(1, keepdim=True))
    if st["res"] is not None:
        dx = dx + st["res"].float()
    shape, gdt = (case["W"], case["rows"] // case["W"], case["dim"]), DT[case["dp"]]
    return [dx.to(st["x"].dtype), (dy * xh).reshape(shape).sum(1).to(gdt), dy.reshape(shape).sum(1).to(gdt)]


def run(st):
    case = st["case"]
    if case["op"] == "adamw":
        if not own:
            out = plain_adamw(st)
        else:
            st["opt"].step(st["table"], st["w"], st["state"], t=st["t"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                           weight_decay=DECAY, clip=st["clip"], copy=st["copy"])
            out = [st[k] for k in ("w", "m", "v", "m_scale", "v_scale", "copy") if st.get(k) is not None]
        st["t"] += 1
        return out
    if case["op"] == "norm":
        if not own:
            return plain_norm(st)
        clip, mean = st["clip"], st.get("mean")
        st["opt"].grad_norm(st["table"], clip, max_norm=st["max_norm"], grad=mean)
        return [clip.norm, clip.scale, clip.skip] + ([mean] if mean is not None else [])
    if case["op"] == "ln_fwd":
        if not own:
            return plain_ln_fwd(st)
        x = st["x"]
        y, mean, rstd = torch.empty_like(x), x.new_empty(x.shape[0], dtype=torch.float32), x.new_empty(x.shape[0], dtype=torch.float32)
        s = torch.empty_like(x) if st["res"] is not None else None
        st["ln"].forward(x, st["gamma"], st["beta"], y, mean, rstd, residual=st["res"], sum_out=s, eps=LN_EPS)
        return [y, mean, rstd] + ([s] if s is not None else [])
    if not own:
        return plain_ln_bwd(st)
    x, shape, gdt = st["x"], (case["W"], case["dim"]), DT[case["dp"]]
    dx, dg, db = torch.empty_like(x), x.new_empty(shape, dtype=gdt), x.new_empty(shape, dtype=gdt)
    st["ln"].backward(st["dy"], x, st["gamma"], st["mean"], st["rstd"], dx, dg, db, dsum=st["res"], groups=case["W"])
    return [dx, dg, db]


def exact(case, seed):
    """The same outputs from the definitions, in binary64."""
    st = prepare(case, seed)
    if case["op"] in ("adamw", "norm"):
        P, W = st["P"], case["W"]
        g = torch.zeros(P, dtype=torch.float64, device="cuda")
        for w in range(W):
            g += st["grads"][w, :P].double()
        g /= W
        if case["op"] == "norm":
            norm = torch.linalg.vector_norm(g).view(1)
            return [norm, (st["max_norm"] / norm).clamp(max=1.0), ((norm != norm) | (norm.abs() == math.inf)).int()] + ([g] if case["keep"] else [])
        if case["clip"]:
            g *= 0.25
        b1, b2, lr, eps = (float(torch.tensor(a, dtype=torch.float32)) for a in (BETA1, BETA2, LR, EPS))
        wd = torch.cat([torch.full((n,), float(torch.tensor(DECAY)) if d else 0.0, dtype=torch.float64, device="cuda")
                        for n, d in zip(layers(case), st["decays"])])
        if case["bits"] == 32:
            m, v = st["m"].double(), st["v"].double()
        else:
            m = (st["m"].double() * st["m_scale"].double()[:, None]).flatten()[:P]
            v = (st["v"].double() * st["v_scale"].double()[:, None]).flatten()[:P] ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        mhat, vhat = m / (1 - b1 ** st["t"]), v / (1 - b2 ** st["t"])
        w = st["w"].double()
        w = w - lr * wd * w - lr * mhat / (vhat ** 0.5 + eps)
        if case["bits"] == 32:
            return [w, m, v] + ([w] if st["copy"] is not None else [])
        nb = -(-P // BLOCK)

        def blocks(a):
            full = torch.zeros(nb * BLOCK, dtype=torch.float64, device="cuda")
            full[:P] = a
            return full.view(nb, BLOCK)

        def held(a, up):
            """a of magnitude <= 448 on the e4m3 grid: 3 mantissa bits above 2^-6, steps of 2^-9 below; up in [0, 1)
            is added to the position between two grid values before it is cut."""
            step = 2.0 ** (torch.floor(torch.log2(a.abs().clamp_min(E4M3_MIN))) - 3)
            q = a.abs() / step
            return torch.sign(a) * (torch.round(q) if up is None else torch.floor(q + up)) * step

        m, s = blocks(m), blocks(v ** 0.5)
        mt, vt = (a.abs().amax(1).clamp_min(FLOOR) for a in (m, s))
        u = 448 / vt[:, None] * s
        u = torch.where(s > 0, u.clamp(E4M3_MIN, 448), u)
        up = random_bits(nb * BLOCK, st["t"]).double().view(nb, BLOCK) / 2 ** 20
        return [w, held(448 / mt[:, None] * m, None), held(u, up), mt / 448, vt / 448] + ([w] if st["copy"] is not None else [])
    x, gamma = st["x"].double(), st["gamma"].double()
    if case["op"] == "ln_fwd":
        s = None
        if st["res"] is not None:
            s = x + st["res"].double()
            x = s.to(st["x"].dtype).double()
        var, mean = torch.var_mean(x, 1, correction=0)
        y = (x - mean[:, None]) / torch.sqrt(var + LN_EPS)[:, None] * gamma + st["beta"].double()
        return [y, mean, (var + LN_EPS) ** -0.5] + ([s] if s is not None else [])
    dy, mean, rstd = st["dy"].double(), st["mean"].double()[:, None], st["rstd"].double()[:, None]
    xh = (x - mean) * rstd
    dxh = dy * gamma
    dx = dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True)
    dx = dx * rstd + (st["res"].double() if st["res"] is not None else 0)
    rows = torch.arange(case["rows"], device="cuda") // (case["rows"] // case["W"])
    dgamma, dbeta = (torch.zeros(case["W"], case["dim"], dtype=torch.float64, device="cuda").index_add_(0, rows, a) for a in (dy * xh, dy))
    return [dx, dgamma, dbeta]
