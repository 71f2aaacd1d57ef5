#!/usr/bin/env python3
"""A small classifier trained by W data-parallel workers on one GPU.

Linear - layer norm - ReLU - linear, in bf16, on synthetic data.  Each worker's
part of the batch gives its own weight gradients (the layer norm's backward pass
takes the workers as groups); the optimizer reads all of them in place through
a table of addresses, averages them, clips the mean by its norm and updates the
binary32 weights, their moments (8 or 32 bits) and the bf16 copy that the next
forward pass uses.

    python examples/train_mlp.py --steps 200 --state-bits 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gradient_aggregation_amd as ga  # noqa: E402


class Mlp:
    """Weights as slices of one flat vector, in the order of `numels`."""

    def __init__(self, inputs, hidden, classes, W, state_bits, seed):
        self.shapes = [(inputs, hidden), (hidden,), (hidden,), (hidden, classes)]
        self.numels = [inputs * hidden, hidden, hidden, hidden * classes]
        self.W, bf16 = W, torch.bfloat16
        gen = torch.Generator().manual_seed(seed)
        parts = [torch.randn(inputs * hidden, generator=gen) / inputs ** 0.5, torch.ones(hidden), torch.zeros(hidden),
                 torch.randn(hidden * classes, generator=gen) / hidden ** 0.5]
        self.w = torch.cat(parts).cuda()
        self.copy = self.w.to(bf16)
        self.w1, self.gamma, self.beta, self.w2 = (
            p.view(s) for p, s in zip(self.copy.split(self.numels), self.shapes))
        # every worker's gradient of every tensor, and the table of their addresses
        self.grads = [torch.zeros((W,) + s, dtype=bf16, device="cuda") for s in self.shapes]
        self.table = torch.tensor([g[w].data_ptr() for w in range(W) for g in self.grads], dtype=torch.int64,
                                  device="cuda")
        self.norm = ga.LayerNorm(hidden, bf16, bf16)
        # only the matrices decay
        self.opt = ga.AdamW(self.numels, W=W, grad_dtype=bf16, state_bits=state_bits,
                            decay=[len(s) == 2 for s in self.shapes])
        self.state, self.clip, self.t = self.opt.empty_state(), self.opt.empty_clip(), 0

    def step(self, x, target, lr):
        """One training step; x [W * B][inputs] with each worker's B rows
        together.  Returns the loss before it (on the device)."""
        rows, W = x.shape[0], self.W
        B = rows // W
        h = x @ self.w1
        y, mean, rstd = torch.empty_like(h), h.new_empty(rows, dtype=torch.float32), h.new_empty(rows, dtype=torch.float32)
        self.norm.forward(h, self.gamma, self.beta, y, mean, rstd)
        a = y.relu()
        logp = torch.log_softmax((a @ self.w2).float(), 1)
        loss = -logp.gather(1, target[:, None]).mean()

        dz = logp.exp()
        dz[torch.arange(rows, device=x.device), target] -= 1
        dz = (dz / B).to(x.dtype)                       # each worker's own mean loss
        dw1, dgamma, dbeta, dw2 = self.grads
        dy = (dz @ self.w2.t().contiguous()) * (y > 0)
        dh = torch.empty_like(h)
        self.norm.backward(dy, h, self.gamma, mean, rstd, dh, dgamma, dbeta, groups=W)
        for w in range(W):
            part = slice(w * B, (w + 1) * B)
            torch.mm(x[part].t().contiguous(), dh[part], out=dw1[w])
            torch.mm(a[part].t().contiguous(), dz[part], out=dw2[w])

        self.t += 1
        self.opt.grad_norm(self.table, self.clip, max_norm=1.0)
        self.opt.step(self.table, self.w, self.state, t=self.t, lr=lr, weight_decay=0.01, clip=self.clip,
                      copy=self.copy)
        return loss


def train(steps=200, W=4, batch=64, state_bits=8, inputs=64, hidden=520, classes=10, lr=3e-3, seed=0):
    """Losses of the steps: the labels are those of a fixed random linear map."""
    gen = torch.Generator().manual_seed(seed + 1)
    teacher = torch.randn(inputs, classes, generator=gen).cuda()
    net = Mlp(inputs, hidden, classes, W, state_bits, seed)
    losses = []
    for _ in range(steps):
        x = torch.randn(W * batch, inputs, generator=gen).cuda()
        losses.append(net.step(x.bfloat16(), (x @ teacher).argmax(1), lr))
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=64, help="rows per worker")
    ap.add_argument("--state-bits", type=int, choices=[8, 32], default=8)
    a = ap.parse_args()
    losses = train(a.steps, a.workers, a.batch, a.state_bits)
    for k in range(0, len(losses), max(1, len(losses) // 10)):
        print("step %5d  loss %.4f" % (k + 1, losses[k]))
    print("step %5d  loss %.4f" % (len(losses), losses[-1]))


if __name__ == "__main__":
    main()
