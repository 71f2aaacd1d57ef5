"""Group norm, router, gradient norm and AdamW together, as examples/train_moe.py uses
them: it runs, repeats itself, and its gradients are those of the model by differentiation
in binary64."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_moe", os.path.join(ROOT, "examples", "train_moe.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(moe):
    losses, net = moe.train(steps=5, W=2, batch=16)
    assert len(losses) == 5 and all(math.isfinite(x) for x in losses)
    assert int(net.load.counts.sum()) == 2 * 16 * net.k and net.load.tokens.tolist() == [16, 16]
    assert bool(torch.isfinite(net.w).all()) and int(net.clip.skip) == 0
    again, net2 = moe.train(steps=5, W=2, batch=16)
    assert losses == again and torch.equal(net.w, net2.w)


def test_gradients_are_the_model_s(moe):
    """In binary32, against the same model differentiated in binary64 on the CPU (selection and counts held)."""
    W, B = 3, 4
    net = moe.Moe(size=5, channels=12, groups=3, experts=5, k=2, classes=4, W=W, dtype=torch.float32)
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(W * B, 5, 5, 3, generator=gen)
    target = torch.randint(0, 4, (W * B,), generator=gen)
    net.gradients(x.cuda(), target.cuda(), balance=0.5, z=0.25)
    got = [g.cpu().double() for g in net.grads]

    weights = [p.cpu().double().requires_grad_() for p in net.weights]
    conv, gamma, beta, gate, experts, head = weights
    xd, rows, k, E = x.double(), W * B, 2, 5
    pad = torch.nn.functional.pad(xd, (0, 0, 1, 1, 1, 1))
    around = torch.stack([pad[:, i:i + 5, j:j + 5] for i in range(3) for j in range(3)], 3).reshape(rows, 25, 27)
    h = (around @ conv).transpose(1, 2)
    y = torch.nn.functional.silu(torch.nn.functional.group_norm(h, 3, gamma, beta, 1e-5))
    f = y.mean(2)
    logits = f @ gate
    top = logits.topk(k, 1)
    gates = torch.softmax(top.values, 1)
    v = sum(gates[:, j, None] * (f[:, None] @ experts[top.indices[:, j]])[:, 0] for j in range(k))
    ce = torch.nn.functional.cross_entropy(v @ head, target, reduction="none")
    counts = torch.bincount(top.indices.reshape(-1), minlength=E).double()
    p = torch.softmax(logits, 1)
    balance = E / (k * rows * rows) * (counts * p.sum(0)).sum()
    zloss = torch.logsumexp(logits, 1).square().mean()
    assert abs(float(net.load.loss[0]) - float(balance.detach())) < 1e-5 and abs(float(net.load.loss[1]) - float(zloss.detach())) < 1e-4
    for w in range(W):
        # a worker's mean loss, and W times its tokens' part of the losses of all
        part = slice(w * B, (w + 1) * B)
        mine = ce[part].mean() + W * (0.5 * E / (k * rows * rows) * (counts * p[part].sum(0)).sum()
                                      + 0.25 * torch.logsumexp(logits[part], 1).square().sum() / rows)
        want = torch.autograd.grad(mine, weights, retain_graph=True)
        for a, b in zip(got, want):
            # some hundred binary32 roundings of terms of the gradient's size, in products of up to 25 * 4 of them
            assert float((a[w] - b).abs().max()) <= 1e-5 * (1 + float(b.abs().max()))
