#!/usr/bin/env python3
"""A small image classifier with a mixture of experts, trained by W data-parallel
workers on one GPU.

A 3 x 3 convolution - group norm with silu - mean over the positions - router - two
of E expert matrices - linear, in bf16, on synthetic images.  Images are channels
last throughout.  Each worker's part of the batch gives its own weight gradients;
the router's counts are those of all workers' images, and its balance loss keeps the
experts in use.  The optimizer reads all gradients in place, averages and clips them
and updates the binary32 weights and the bf16 copy of the next forward pass.

    python examples/train_moe.py --steps 100
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_aggregation_amd as ga  # noqa: E402


class Moe:
    """Weights as slices of one flat vector, in the order of `shapes`."""

    def __init__(self, size=9, channels=48, groups=8, experts=8, k=2, classes=10, W=4, dtype=torch.bfloat16, seed=0):
        self.size, self.W, self.k, self.dtype = size, W, k, dtype
        C, E = channels, experts
        self.shapes = [(27, C), (C,), (C,), (C, E), (E, C, C), (C, classes)]
        self.numels = [torch.Size(s).numel() for s in self.shapes]
        gen = torch.Generator().manual_seed(seed)
        parts = [torch.randn(27 * C, generator=gen) / 27 ** 0.5, torch.ones(C), torch.zeros(C),
                 torch.randn(C * E, generator=gen) / C ** 0.5, torch.randn(E * C * C, generator=gen) / C ** 0.5,
                 torch.randn(C * classes, generator=gen) / C ** 0.5]
        self.w = torch.cat(parts).cuda()
        self.copy = self.w.to(dtype)
        self.weights = [p.view(s) for p, s in zip(self.copy.split(self.numels), self.shapes)]
        # every worker's gradient of every tensor, and the table of their addresses
        self.grads = [torch.zeros((W,) + s, dtype=dtype, device="cuda") for s in self.shapes]
        self.table = torch.tensor([g[w].data_ptr() for w in range(W) for g in self.grads], dtype=torch.int64, device="cuda")
        self.norm = ga.GroupNorm(C, groups, dtype, dtype, activation="silu")
        self.router = ga.Router(E, k, dtype, workers=W, normalize=True, scope="all")
        self.load = self.router.empty_load()
        self.opt = ga.AdamW(self.numels, W=W, grad_dtype=dtype, state_bits=32, decay=[len(s) > 1 for s in self.shapes])
        self.state, self.clip, self.t = self.opt.empty_state(), self.opt.empty_clip(), 0

    def gradients(self, x, target, balance=1e-2, z=1e-3):
        """Every worker's weight gradients of its own mean loss into self.grads; x
        [W * B][size][size][3], each worker's B images together.  Returns the mean
        classification loss (on the device)."""
        dt, W, (conv, gamma, beta, gate, experts, head) = self.dtype, self.W, self.weights
        rows, S, C = x.shape[0], self.size * self.size, gamma.numel()
        B = rows // W
        # the convolution as a product with the 27 values around each position
        pad = torch.nn.functional.pad(x, (0, 0, 1, 1, 1, 1))
        around = torch.stack([pad[:, i:i + self.size, j:j + self.size] for i in range(3) for j in range(3)], 3).reshape(rows * S, 27)
        h = (around @ conv).view(rows, S, C)
        y, mean, rstd = torch.empty_like(h), h.new_empty(rows, self.norm.groups, dtype=torch.float32), \
            h.new_empty(rows, self.norm.groups, dtype=torch.float32)
        self.norm.forward(h, gamma, beta, y, mean, rstd)
        f = y.float().mean(1).to(dt)
        logits = f @ gate
        routing = self.router.empty_routing(rows)
        self.router.forward(logits, routing, self.load)
        at = routing.experts.long()
        u = torch.stack([(f[:, None] @ experts[at[:, j]].contiguous())[:, 0] for j in range(self.k)], 1)      # [rows][k][C]
        v = (u.float() * routing.gates[:, :, None]).sum(1).to(dt)
        logp = torch.log_softmax((v @ head).float(), 1)
        loss = -logp.gather(1, target[:, None]).mean()

        dz = logp.exp()
        dz[torch.arange(rows, device=x.device), target] -= 1
        dz = (dz / B).to(dt)                                # each worker's own mean loss
        dv = (dz @ head.t().contiguous()).float()
        dgates = (dv[:, None] * u.float()).sum(2)
        dlogits = torch.empty_like(logits)
        # the losses are means over all workers' images: a worker's share of the mean gradient is W times its part
        self.router.backward(logits, routing, self.load, dlogits, dgates=dgates, balance=balance * W, z=z * W)
        du = (routing.gates[:, :, None] * dv[:, None]).to(dt)
        df = dlogits @ gate.t().contiguous()
        df = df.float() + sum((du[:, j, None] @ experts[at[:, j]].transpose(1, 2).contiguous())[:, 0].float() for j in range(self.k))
        dy = (df / S).to(dt)[:, None].expand(rows, S, C).contiguous()
        dh = torch.empty_like(h)
        dconv, dgamma, dbeta, dgate, dexperts, dhead = self.grads
        self.norm.backward(dy, h, gamma, beta, mean, rstd, dh, dgamma, dbeta, workers=W)
        for w in range(W):
            part = slice(w * B, (w + 1) * B)
            torch.mm(around[w * B * S:(w + 1) * B * S].t().contiguous(), dh[part].reshape(B * S, C), out=dconv[w])
            torch.mm(f[part].t().contiguous(), dlogits[part], out=dgate[w])
            torch.mm(v[part].t().contiguous(), dz[part], out=dhead[w])
            outer = (f[part, None, :, None].float() * du[part, :, None, :].float()).reshape(B * self.k, C * C)
            chosen = (at[part].reshape(1, -1) == torch.arange(experts.shape[0], device=x.device)[:, None]).float()
            dexperts[w].copy_((chosen @ outer).view(experts.shape))
        return loss

    def step(self, x, target, lr):
        loss = self.gradients(x, target)
        self.t += 1
        self.opt.grad_norm(self.table, self.clip, max_norm=1.0)
        self.opt.step(self.table, self.w, self.state, t=self.t, lr=lr, weight_decay=0.01, clip=self.clip, copy=self.copy)
        return loss


def train(steps=100, W=4, batch=64, lr=3e-3, seed=0, dtype=torch.bfloat16):
    """Losses of the steps: the labels are those of a fixed random map of the images."""
    gen = torch.Generator().manual_seed(seed + 1)
    net = Moe(W=W, seed=seed, dtype=dtype)
    teacher = torch.randn(3, 10, generator=gen).cuda()
    losses = []
    for _ in range(steps):
        x = torch.randn(W * batch, net.size, net.size, 3, generator=gen).cuda()
        losses.append(net.step(x.to(dtype), ((x + 0.3 * x * x).mean((1, 2)) @ teacher).argmax(1), lr))
    return torch.stack(losses).tolist(), net


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=64, help="images per worker")
    a = ap.parse_args()
    losses, net = train(a.steps, a.workers, a.batch)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %5d  loss %.4f" % (k + 1, losses[k]))
    print("step %5d  loss %.4f" % (len(losses), losses[-1]))
    print("experts' use (all workers):", net.load.counts.sum(0).tolist())


if __name__ == "__main__":
    main()
