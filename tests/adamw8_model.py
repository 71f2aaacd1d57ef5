"""The AdamW recurrence with 8-bit states on the CPU, as include/gradagg.h
specifies it, with the roundings of m and of v's root as arguments: "random",
"nearest" or "down".  It says what a test of many steps can tell apart."""
import math

import numpy as np
import torch

SEED_M = 0xBB67AE85


def random_bits(n, counter):
    """20 random bits (16 of them, centred) for each of n elements."""
    i = np.arange(n, dtype=np.uint64)
    with np.errstate(over="ignore"):
        x = ((i >> np.uint64(1)) + np.uint64(counter % 2 ** 32)).astype(np.uint32)
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0xB7E15163)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x6A09E667)
        x = x ^ (x >> np.uint32(16))
    r = np.where(i % 2 == 1, x >> np.uint32(16), x & np.uint32(0xffff))
    return torch.from_numpy(r.astype(np.int32) * 16 + 8)


def step_counter(t):
    return t * 0x9E3779B9 + 0x7F4A7C15


def rounded(y, how, bits):
    """y (binary32, of magnitude <= 448) on the e4m3 grid."""
    if how == "nearest":
        return y.to(torch.float8_e4m3fn).float()
    lift = torch.where(y.abs() < 2.0 ** -6, 2.0 ** -6, 0.0).float()
    z = (y.abs() + lift).view(torch.int32) + (bits if how == "random" else 0)
    return torch.copysign((z & -0x100000).view(torch.float32) - lift, y)


def run(gradient, n, steps, beta1, beta2, m_how="random", v_how="random", lr=1.0, eps=1e-8, watch=()):
    """Weights from 0 after each step of `watch` (and the last), and v: a list
    of (w, v) in binary64.  n: a multiple of 256."""
    b1, b2 = (float(np.float32(b)) for b in (beta1, beta2))
    mc, vc = torch.zeros(n // 256, 256), torch.zeros(n // 256, 256)
    ms, vs = torch.zeros(n // 256, 1), torch.zeros(n // 256, 1)
    w, out = torch.zeros(n, dtype=torch.float64), []
    for t in range(1, steps + 1):
        g = gradient(t).reshape(-1, 256)
        m = b1 * (mc * ms) + float(np.float32(1 - b1)) * g
        v = b2 * (vc * vs).square() + float(np.float32(1 - b2)) * g * g
        root = v.sqrt()
        w -= lr * (m / (1 - b1 ** t) / (root / math.sqrt(1 - b2 ** t) + eps)).double().reshape(-1)
        top_m, top_v = (a.abs().amax(1, keepdim=True).clamp_min(2.0 ** -100) for a in (m, root))
        ms, vs = top_m / 448, top_v / 448
        c = step_counter(t)
        mc = rounded((m * (448 / top_m)).clamp(-448, 448), m_how, random_bits(n, c + SEED_M).view(-1, 256))
        y = (root * (448 / top_v)).clamp(2.0 ** -6, 448)
        vc = torch.where(root > 0, rounded(y, v_how, random_bits(n, c).view(-1, 256)), 0.0)
        if t in watch or t == steps:
            out.append((w.clone(), (vc * vs).double().square().reshape(-1)))
    return out


def exact(gradient, n, steps, beta1, beta2, lr=1.0, eps=1e-8, watch=(), device="cpu"):
    """The same recurrence in binary64 with unrounded states: a list of (w, v,
    path), path the sum of the updates' magnitudes so far."""
    b1, b2 = (float(np.float32(b)) for b in (beta1, beta2))
    m, v, w, path = (torch.zeros(n, dtype=torch.float64, device=device) for _ in range(4))
    out = []
    for t in range(1, steps + 1):
        g = gradient(t).double()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        up = lr * m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + eps)
        w, path = w - up, path + up.abs()
        if t in watch or t == steps:
            out.append((w, v, path))
    return out


class Turn:
    """Gradients of n weights: steady, and from step 201 on every second one is
    `factor` times what it was."""
    BEFORE, AFTER = 200, 800

    def __init__(self, n, factor, noise=0.0, device="cpu"):
        gen = torch.Generator().manual_seed(n)
        size = 10.0 ** (2 * torch.rand(n, generator=gen) - 1)
        self.base = (size * torch.randn(n, generator=gen).sign()).to(device)
        self.turned = self.base.clone()
        self.turned[1::2] *= factor
        self.noise, self.gen = noise, gen
        self.steps = self.BEFORE + (self.AFTER if factor else 2800)
        self.drawn = {}

    def __call__(self, t):
        g = self.base if t <= self.BEFORE else self.turned
        if self.noise:
            if t not in self.drawn:
                self.drawn[t] = torch.randn(g.numel(), generator=self.gen).to(g.device)
            g = g + self.noise * self.base.abs() * self.drawn[t]
        return g

    def moved(self, states):
        """Mean movement of the turned weights against their first gradient's sign after step 200."""
        return float(((states[1][0] - states[0][0]) * self.base.double().sign())[1::2].mean())

    def bound(self, beta1, states):
        """What the mean movement may differ by from the exact recurrence's (`states`).

        v's root is held on codes that lie a step, at most an eighth of the value, apart: an eighth of the updates'
        magnitudes.  m: rounding a value that moves by d per step to neighbours a step s apart has a variance of at
        most d s, d = (1 - beta1) s where m is a step from its gradient; each error acts for 1/(1 - beta1) updates, so
        T steps leave a standard deviation of at most sqrt(T / (1 - beta1)) / 8 updates on one weight.  Five of those
        over the root of the number of weights."""
        path = float((states[1][2] - states[0][2])[1::2].mean())
        T = self.steps - self.BEFORE
        return path / 8 + 5 * math.sqrt(T / (1 - beta1)) / 8 / math.sqrt(self.base.numel() / 2)


    def second(self, state, want):
        """Mean ratio of the turned weights' second moments at the end to the exact ones."""
        return float((state[1] / want[1])[1::2].mean())

    def second_bound(self):
        """What that may differ from 1 by.  A root a distance d from the code c that it is rounded to, of a step s <= c/8,
        has a variance of at most |d| s, which the square adds to its drift 2 c d: a sixteenth of the drift, so of v
        where it moves by at most itself.  And five standard deviations of the mean of values that lie on codes around
        their expectation: at most a step, a quarter of v, each."""
        return 1 / 16 + 5 / 4 / math.sqrt(self.base.numel() / 2)


TURNS = [  # factor, noise, beta1, beta2
    (-1.0, 0.0, 0.9, 0.999), (-1.0, 0.0, 0.95, 0.95), (-1.0, 0.0, 0.99, 0.999), (-1.0, 0.1, 0.95, 0.95),
    (0.7, 0.0, 0.9, 0.999), (0.0, 0.0, 0.9, 0.95), (0.0, 0.0, 0.99, 0.999),
]
