"""Cases of the operators of image networks and mixtures of experts: group norm
with an activation, channels last, forward and backward, and the expert router
with its per-expert counts and balance loss, forward and backward.

`run` computes each operator in its plain form (elementary torch operations in
binary32) where `own` is false, and through gradient_aggregation_amd where it
is true.  Image sizes are those of the library's CNN workloads (55 x 55 and 6 x 6
positions) and generic ones; the routers' are generic.

Images are [samples][positions][channels]; W workers own consecutive runs of
samples, or of tokens, and each has its own weight gradients or counts."""
import math

import torch

own = False

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ESZ = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-5
BALANCE, ZLOSS = 1e-2, 1e-3     # coefficients of the two losses
MOST_IMAGE = 67_108_864         # elements of the largest forward image batch
MOST_LOGITS = 33_554_432


def listed():
    return [
        # one small feature map of a wide network: launch latency is all
        {"name": "gn_fwd 1x64x1280 bf16 silu", "op": "gn_fwd", "N": 1, "S": 64, "C": 1280, "G": 32, "x": "bf16", "p": "bf16", "act": "silu", "wide": 0},
        # a training batch in the middle of such a network
        {"name": "gn_fwd 16x1024x640 bf16 silu", "op": "gn_fwd", "N": 16, "S": 1024, "C": 640, "G": 32, "x": "bf16", "p": "fp32", "act": "silu", "wide": 0},
        # the first convolution's 55 x 55 positions, 96 channels
        {"name": "gn_fwd 64x3025x96 fp16 relu", "op": "gn_fwd", "N": 64, "S": 3025, "C": 96, "G": 8, "x": "fp16", "p": "fp32", "act": "relu", "wide": 0},
        # few large images
        {"name": "gn_fwd 4x65536x256 bf16 silu", "op": "gn_fwd", "N": 4, "S": 65536, "C": 256, "G": 32, "x": "bf16", "p": "fp32", "act": "silu", "wide": 0},
        # the last convolution's 6 x 6 positions, one sample for each of four workers
        {"name": "gn_bwd 4x36x1024 fp32 W4", "op": "gn_bwd", "N": 4, "S": 36, "C": 1024, "G": 32, "x": "fp32", "p": "fp32", "act": "none", "wide": 0, "W": 4, "dp": "fp32"},
        # odd sizes, groups of 10 channels, rows inside wider ones
        {"name": "gn_bwd 6x1443x250 fp32 silu W3", "op": "gn_bwd", "N": 6, "S": 1443, "C": 250, "G": 25, "x": "fp32", "p": "fp32", "act": "silu", "wide": 6, "W": 3, "dp": "fp32"},
        # a training batch of 16 workers, each worker's weight gradients in its own row
        {"name": "gn_bwd 16x16384x128 bf16 silu W16", "op": "gn_bwd", "N": 16, "S": 16384, "C": 128, "G": 32, "x": "bf16", "p": "fp32", "act": "silu", "wide": 0, "W": 16, "dp": "bf16"},
        # the tokens of one short sequence and few experts
        {"name": "router_fwd 64x8 k2 fp32", "op": "router_fwd", "T": 64, "E": 8, "k": 2, "x": "fp32", "W": 1, "norm": True, "scope": "all", "given": False, "absent": 0.0},
        # a batch of 16 workers with padding
        {"name": "router_fwd 65536x64 k6 bf16 W16", "op": "router_fwd", "T": 65536, "E": 64, "k": 6, "x": "bf16", "W": 16, "norm": True, "scope": "all", "given": False, "absent": 0.1},
        # many experts, logits in binary32
        {"name": "router_fwd 131072x256 k8 fp32 W8", "op": "router_fwd", "T": 131072, "E": 256, "k": 8, "x": "fp32", "W": 8, "norm": False, "scope": "worker", "given": False, "absent": 0.0},
        # a small batch, an odd number of experts, the selection made elsewhere
        {"name": "router_bwd 999x60 k4 fp16", "op": "router_bwd", "T": 999, "E": 60, "k": 4, "x": "fp16", "W": 1, "norm": True, "scope": "all", "given": True, "absent": 0.1},
        # a batch of 8 workers, many experts
        {"name": "router_bwd 131072x256 k8 bf16 W8", "op": "router_bwd", "T": 131072, "E": 256, "k": 8, "x": "bf16", "W": 8, "norm": False, "scope": "all", "given": False, "absent": 0.0},
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.55:
        op = rng.choice(["gn_fwd", "gn_bwd"])
        G = rng.choice([1, 4, 8, 16, 25, 32, 32, 32])
        C = G * rng.choice([c for c in (1, 2, 3, 4, 8, 10, 12, 16, 20, 24, 40, 64, 128) if 16 <= c * G <= 2560])
        N = spread(rng, 1, 128)
        W = 1
        if op == "gn_bwd":
            W = rng.choice([1, 1, 2, 4, 16])
            N = max(1, N // W) * W
        most = MOST_IMAGE // (1 if op == "gn_fwd" else 2)
        x = rng.choice(["fp32", "fp16", "bf16", "bf16"])
        S = max(1, min(spread(rng, 1, 65536), most * 2 // ESZ[x] // (N * C)))
        c = {"op": op, "N": N, "S": S, "C": C, "G": G, "x": x, "p": rng.choice(["fp32", x]), "wide": rng.choice([0, 0, 0, 8, 13])}
        if op == "gn_fwd":
            c["act"] = rng.choice(["silu", "silu", "relu", "none"])
        else:
            # relu's derivative jumps where z is 0: an element within a rounding of it has either value
            c.update(act=rng.choice(["silu", "silu", "none"]), W=W, dp=rng.choice(["fp32", x]))
        return c
    E = rng.choice([8, 16, 64, 128, 256]) if rng.random() < 0.6 else spread(rng, 4, 512)
    W = rng.choice([1, 1, 4, 8, 16])
    x = rng.choice(["fp32", "fp16", "bf16"])
    T = max(W, min(spread(rng, 16, 262144), MOST_LOGITS * 4 // ESZ[x] // 2 // E) // W * W)
    return {"op": rng.choice(["router_fwd", "router_bwd"]), "T": T, "E": E, "k": rng.randint(1, min(E, 10)), "x": x, "W": W,
            "norm": rng.random() < 0.5, "scope": rng.choice(["all", "worker"]), "given": rng.random() < 0.3,
            "absent": rng.choice([0.0, 0.0, 0.1, 0.5])}


def work(case):
    if case["op"].startswith("gn"):
        n, b = case["N"] * case["S"] * case["C"], ESZ[case["x"]]
        params, stats = 2 * case["C"] * ESZ[case["p"]], 8 * case["N"] * case["G"]
        if case["op"] == "gn_fwd":
            return {"bytes": 2 * n * b + params + stats, "flops": 16 * n}
        return {"bytes": 3 * n * b + params + stats + 2 * case["W"] * case["C"] * ESZ[case["dp"]], "flops": 30 * n}
    T, E, k, b = case["T"], case["E"], case["k"], ESZ[case["x"]]
    mask = T if case["absent"] else 0
    if case["op"] == "router_fwd":
        chosen = 8 * T * k      # experts (read where given) and gates
        return {"bytes": T * E * b + chosen + 4 * T + mask + 8 * case["W"] * E, "flops": (8 + k) * T * E}
    return {"bytes": 2 * T * E * b + 12 * T * k + 4 * T + mask + 4 * E, "flops": 12 * T * E}


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st = {"case": case}
    xdt = DT[case["x"]]
    if case["op"].startswith("gn"):
        N, S, C, G = (case[k] for k in "NSCG")

        def images(values):
            rows = torch.zeros(N, S, C + case["wide"], dtype=xdt, device="cuda")
            rows[:, :, :C] = values
            return rows[:, :, :C]

        # channels of different size and mean, as a convolution leaves them
        st["x"] = images(normal(N, S, C) * (0.5 + torch.rand(C, generator=gen, device="cuda")) + 0.5 * normal(C) + 0.2 * normal(N, 1, C))
        pdt = DT[case["p"]]
        st["gamma"], st["beta"] = (1 + 0.2 * normal(C)).to(pdt), (0.2 * normal(C)).to(pdt)
        if case["op"] == "gn_bwd":
            st["dy"] = images(1e-2 * normal(N, S, C))
            st["mean"], st["rstd"] = torch.empty(N, G, device="cuda"), torch.empty(N, G, device="cuda")
            per = max(1, (1 << 26) // (S * C))          # samples whose binary64 values are formed together
            for n in range(0, N, per):
                v = st["x"][n:n + per].double().reshape(-1, S, G, C // G)
                mean = v.mean((1, 3))
                st["mean"][n:n + per] = mean
                st["rstd"][n:n + per] = ((v - mean[:, None, :, None]).square().mean((1, 3)) + EPS).rsqrt()
        if own:
            import gradient_aggregation_amd as ga
            st["gn"] = ga.GroupNorm(C, G, xdt, pdt, activation=case["act"])
            if case["op"] == "gn_fwd":
                st["out"] = [torch.empty(N, S, C, dtype=xdt, device="cuda"), torch.empty(N, G, device="cuda"), torch.empty(N, G, device="cuda")]
            else:
                st["out"] = [torch.empty(N, S, C, dtype=xdt, device="cuda")] + [torch.empty(case["W"], C, dtype=DT[case["dp"]], device="cuda") for _ in range(2)]
        return st
    T, E, k, W = (case[a] for a in "TEkW")
    # some experts are preferred, and more so by some workers
    taste = 0.7 * normal(E) + 0.3 * normal(W, 1, E)
    st["logits"] = (1.5 * normal(W, T // W, E) + taste).reshape(T, E).to(xdt)
    st["mask"] = (torch.rand(T, generator=gen, device="cuda") >= case["absent"]) if case["absent"] else None
    st["given"] = None
    if case["given"]:
        # selected elsewhere, by the logits and a bias for each expert
        st["given"] = (st["logits"].float() + 0.5 * normal(E)).topk(k, 1).indices.int()
    if case["op"] == "router_bwd":
        # what the forward pass left, in binary64, rounded once
        experts, gates, lse, _, _, _, _, slope = route(st["logits"].double(), st["mask"], st["given"], case)
        st["experts"], st["gates"], st["lse"], st["slope"] = experts, gates.float(), lse.float(), slope.float()
        st["dgates"] = 1e-2 * normal(T, k)
    if own:
        import gradient_aggregation_amd as ga
        st["router"] = ga.Router(E, k, xdt, workers=W, normalize=case["norm"], scope=case["scope"])
        st["load"] = st["router"].empty_load()
        st["routing"] = st["router"].empty_routing(T)
        if case["op"] == "router_bwd":
            st["load"].slope.copy_(st["slope"])
            for name in ("experts", "gates", "lse"):
                getattr(st["routing"], name).copy_(st[name])
            st["dlogits"] = torch.empty(T, E, dtype=xdt, device="cuda")
        elif case["given"]:
            st["routing"].experts.copy_(st["given"])
    return st


# ---- plain forms -----------------------------------------------------------

def plain_gn_fwd(st):
    case, x = st["case"], st["x"]
    N, S, C, G = (case[k] for k in "NSCG")
    f = x.float().reshape(N, S, G, C // G)
    mean = f.mean((1, 3))
    c = f - mean[:, None, :, None]
    rstd = 1 / (c.square().mean((1, 3)) + EPS).sqrt()
    z = (c * rstd[:, None, :, None]).reshape(N, S, C) * st["gamma"].float() + st["beta"].float()
    if case["act"] == "relu":
        z = z.clamp_min(0)
    elif case["act"] == "silu":
        z = z / (1 + (-z).exp())
    return [z.to(x.dtype), mean, rstd]


def plain_gn_bwd(st):
    case = st["case"]
    N, S, C, G, W = (case[k] for k in "NSCGW")
    grouped = (N, S, G, C // G)
    rstd = st["rstd"][:, None, :, None]
    xh = (st["x"].float().reshape(grouped) - st["mean"][:, None, :, None]) * rstd
    gamma, dz = st["gamma"].float(), st["dy"].float()
    if case["act"] == "silu":
        z = xh.reshape(N, S, C) * gamma + st["beta"].float()
        s = 1 / (1 + (-z).exp())
        dz = dz * (s * (1 + z * (1 - s)))
    h = (dz * gamma).reshape(grouped)
    m1, m2 = h.mean((1, 3), keepdim=True), (h * xh).mean((1, 3), keepdim=True)
    dx = rstd * (h - m1 - xh * m2)
    per = (W, N // W * S, C)
    dgamma, dbeta = (dz * xh.reshape(N, S, C)).reshape(per).sum(1), dz.reshape(per).sum(1)
    return [dx.reshape(N, S, C).to(st["x"].dtype), dgamma.to(DT[case["dp"]]), dbeta.to(DT[case["dp"]])]


def route(l, mask, given, case):
    """Experts, gates, lse, counts, sums of probabilities, tokens, losses and slope of logits l."""
    T, E, k, W = (case[a] for a in "TEkW")
    top = l.amax(1, keepdim=True)
    e = (l - top).exp()
    total = e.sum(1, keepdim=True)
    p, lse = e / total, (top + total.log()).reshape(T)
    if given is None:
        experts = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]     # ties: the lowest index
    else:
        experts = given.long()
    gates = p.gather(1, experts)
    if case["norm"]:
        gates = gates / gates.sum(1, keepdim=True)
    chosen = torch.zeros(T, E, dtype=torch.int32, device=l.device).scatter_(1, experts, 1)
    present = torch.ones(T, dtype=torch.bool, device=l.device) if mask is None else mask
    if mask is not None:
        absent = ~mask[:, None]
        gates = gates.masked_fill(absent, 0)
        if given is None:
            experts = experts.masked_fill(absent, -1)
        p, chosen, lse = p.masked_fill(absent, 0), chosen.masked_fill(absent, 0), lse.masked_fill(~mask, 0)
    counts = chosen.reshape(W, T // W, E).sum(1, dtype=torch.int32)
    probs = p.reshape(W, T // W, E).sum(1)
    tokens = present.reshape(W, T // W).sum(1, dtype=torch.int32)
    squares = lse.square().reshape(W, T // W).sum(1)
    # in binary64: products of counts of many tokens
    F, P, n, Z = counts.double(), probs.double(), tokens.double(), squares.double()
    if case["scope"] == "all":
        F, P, n, Z = (a.sum(0, keepdim=True) for a in (F, P, n, Z))
    share = (1 / n.clamp_min(1) / n.shape[0])[:, None]      # of a token in the mean over tokens, then workers
    slope = F * (E / k) * share / n.clamp_min(1)[:, None]
    loss = torch.stack([(slope * P).sum(), (Z[:, None] * share).sum()])
    slope = torch.cat([slope, 2 * share], 1)
    return [experts.int(), gates, lse, counts, probs, tokens, loss.to(l.dtype), slope.to(l.dtype)]


def plain_router_bwd(st):
    case, l = st["case"], st["logits"].float()
    T, E, k, W = (case[a] for a in "TEkW")
    slope = st["slope"].repeat_interleave(T // st["slope"].shape[0], 0)
    p = (l - st["lse"][:, None]).exp()
    h = BALANCE * slope[:, :E]
    at, gates, dgates = st["experts"].long().clamp_min(0), st["gates"], st["dgates"]
    if not case["norm"]:
        h = h.scatter_add(1, at, dgates)
    dl = p * (h - (h * p).sum(1, keepdim=True) + ZLOSS * (slope[:, E] * st["lse"])[:, None])
    if case["norm"]:
        dl = dl.scatter_add(1, at, gates * (dgates - (gates * dgates).sum(1, keepdim=True)))
    if st["mask"] is not None:
        dl = dl.masked_fill(~st["mask"][:, None], 0)
    return [dl.to(st["logits"].dtype)]


def run(st):
    op = st["case"]["op"]
    if not own:
        if op == "gn_fwd":
            return plain_gn_fwd(st)
        if op == "gn_bwd":
            return plain_gn_bwd(st)
        if op == "router_fwd":
            return route(st["logits"].float(), st["mask"], st["given"], st["case"])
        return plain_router_bwd(st)
    if op == "gn_fwd":
        y, mean, rstd = st["out"]
        st["gn"].forward(st["x"], st["gamma"], st["beta"], y, mean, rstd, eps=EPS)
        return [y, mean, rstd]
    if op == "gn_bwd":
        dx, dgamma, dbeta = st["out"]
        st["gn"].backward(st["dy"], st["x"], st["gamma"], st["beta"], st["mean"], st["rstd"], dx, dgamma, dbeta, workers=st["case"]["W"])
        return [dx, dgamma, dbeta]
    r, load = st["routing"], st["load"]
    if op == "router_fwd":
        st["router"].forward(st["logits"], r, load, mask=st["mask"], select=st["given"] is None)
        return [r.experts, r.gates, r.lse, load.counts, load.probs, load.tokens, load.loss, load.slope]
    st["router"].backward(st["logits"], r, load, st["dlogits"], dgates=st["dgates"], mask=st["mask"], balance=BALANCE, z=ZLOSS)
    return [st["dlogits"]]


# ---- definitions in binary64 -------------------------------------------------

def exact(case, seed):
    """The same outputs from the definitions, in binary64."""
    st = prepare(case, seed)
    if case["op"].startswith("gn"):
        N, S, C, G = (case[k] for k in "NSCG")
        out, per = [], max(1, (1 << 26) // (S * C))
        sums = torch.zeros(2, case.get("W", 1), C, dtype=torch.float64, device="cuda")
        for n in range(N):
            x = st["x"][n].double()
            xg = x.reshape(S, G, -1).transpose(0, 1).reshape(G, -1)         # a row per group
            if case["op"] == "gn_fwd":
                var, mean = torch.var_mean(xg, 1, correction=0)
                xh = ((xg - mean[:, None]) / torch.sqrt(var + EPS)[:, None]).reshape(G, S, -1).transpose(0, 1).reshape(S, C)
                z = xh * st["gamma"].double() + st["beta"].double()
                y = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z)}[case["act"]]()
                out.append((y, mean, (var + EPS) ** -0.5))
                continue
            mean, rstd = (st[k][n].double().repeat_interleave(C // G) for k in ("mean", "rstd"))
            xh = (x - mean) * rstd
            g = st["dy"][n].double()
            if case["act"] == "silu":
                z = xh * st["gamma"].double() + st["beta"].double()
                s = torch.sigmoid(z)
                g = g * (s + z * s * torch.sigmoid(-z))
            w = n // (N // case["W"])
            sums[0, w] += (g * xh).sum(0)
            sums[1, w] += g.sum(0)
            h = g * st["gamma"].double()
            groups = [a.reshape(S, G, -1).mean((0, 2)).repeat_interleave(C // G) for a in (h, h * xh)]
            out.append(((h - groups[0] - xh * groups[1]) * rstd,))
        out = [torch.stack(a) for a in zip(*out)]
        return out + ([sums[0], sums[1]] if case["op"] == "gn_bwd" else [])
    T, E, k, W = (case[a] for a in "TEkW")
    l = st["logits"].double()
    here = torch.ones(T, dtype=torch.float64, device="cuda") if st["mask"] is None else st["mask"].double()
    if case["op"] == "router_bwd":
        # the gradient of the two losses and of the gates' product with dgates, by the chain rule
        p = torch.softmax(l, 1)
        slope = st["slope"].double()[torch.arange(T, device="cuda") // (T // st["slope"].shape[0])]
        dp = BALANCE * slope[:, :E]
        rows = torch.arange(T, device="cuda")
        gates, dgates = st["gates"].double(), st["dgates"].double()
        inner = (gates * dgates).sum(1)
        dg, direct = torch.zeros_like(l), torch.zeros_like(l)
        for j in range(k):
            at = st["experts"][:, j].long().clamp_min(0)
            dg[rows, at] += dgates[:, j]
            direct[rows, at] += gates[:, j] * (dgates[:, j] - inner)
        if not case["norm"]:
            dp, direct = dp + dg, 0
        dl = p * dp - p * (p * dp).sum(1, keepdim=True) + ZLOSS * (slope[:, E] * torch.logsumexp(l, 1))[:, None] * p + direct
        return [dl * here[:, None]]
    logp = torch.log_softmax(l, 1)
    # an order without ties: by logit, then by index
    if st["given"] is None:
        levels = torch.unique(l)
        rank = torch.searchsorted(levels, l)
        experts = (rank * E + (E - 1 - torch.arange(E, device="cuda"))).topk(k, 1).indices
    else:
        experts = st["given"].long()
    logg = logp.gather(1, experts)
    gates = torch.softmax(logg, 1) if case["norm"] else logg.exp()
    lse = torch.logsumexp(l, 1) * here
    worker = torch.arange(T, device="cuda") // (T // W)
    probs = torch.zeros(W, E, dtype=torch.float64, device="cuda").index_add_(0, worker, logp.exp() * here[:, None])
    counts = torch.bincount((worker[:, None] * E + experts)[here > 0].reshape(-1), minlength=W * E).reshape(W, E)
    tokens = torch.bincount(worker[here > 0], minlength=W)
    if st["given"] is None:
        experts = torch.where(here[:, None] > 0, experts, -1)
    squares = torch.zeros(W, dtype=torch.float64, device="cuda").index_add_(0, worker, lse ** 2)
    if case["scope"] == "all":
        n = max(1, int(tokens.sum()))
        slope = E * counts.sum(0, keepdim=True) / (k * n * n)
        loss = [(slope * probs.sum(0)).sum(), squares.sum() / n]
        last = torch.full((1, 1), 2 / n, dtype=torch.float64, device="cuda")
    else:
        n = tokens.clamp_min(1).double()[:, None]
        slope = E * counts / (k * n * n) / W
        loss = [(slope * probs).sum(), (squares / n[:, 0]).mean()]
        last = 2 / n / W
    return [experts.int(), gates * here[:, None], lse, counts.int(), probs, tokens.int(), torch.stack(loss), torch.cat([slope, last], 1)]
