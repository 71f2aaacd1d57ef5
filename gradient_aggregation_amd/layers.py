"""Binding of the layer operators: group norm with an activation over images,
and the router of a mixture of experts with its counts and balance loss.

Argument marshalling only, like the rest of the binding: the operators are the
HIP kernels behind ga_groupnorm_forward, ga_groupnorm_backward, ga_router_forward
and ga_router_backward, specified in include/gradagg.h.  Calls run on the current
stream, allocate nothing and do not synchronize.

A handle owns one workspace.  Both passes of a GroupNorm use it, and a
Router.forward with a load: two such calls on one handle must not run at the same
time.  Give each stream that runs them a handle of its own, or order the streams
with events.  A captured call uses its handle's memory at every replay: keep the
handle.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _VP, Images, LoadPtrs, RoutingPtrs, _check, _stream_ptr, lib
from . import _dev as _address
from .training import _dtype, _rows

ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2}
BALANCES = {"all": 0, "worker": 1}
MAX_CHANNELS = 65536
MAX_EXPERTS = 1024
MAX_TOPK = 32


def _dev(t, dtype, min_numel: int, name: str, device: int):
    """Address of a contiguous tensor on the handle's device (None stays None)."""
    at = _address(t, dtype, min_numel, name)
    if at is not None and t.get_device() != device:
        raise ValueError("%s is on cuda:%d, the handle on cuda:%d" % (name, t.get_device(), device))
    return at


def _images(t, like, name: str):
    """ga_images of a tensor of x's shape and type, [samples] first and channels
    last, whose positions are evenly spaced."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError("%s must be %s %s, got %s %s" % (name, like.dtype, tuple(like.shape), t.dtype, tuple(t.shape)))
    if t.get_device() != like.get_device():
        raise ValueError("%s is on %s, x on %s" % (name, t.device, like.device))
    C = t.shape[-1]
    if t.is_contiguous():
        return Images(t.data_ptr(), C, t.numel() // max(1, t.shape[0]))
    if t.stride(-1) != 1 and C > 1:
        raise ValueError("%s must have contiguous channels" % name)
    # one stride has to lead from every position to the next
    ld, positions = None, 1
    for n, s in zip(reversed(t.shape[1:-1]), reversed(t.stride()[1:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * positions:
            raise ValueError("%s must have evenly spaced positions" % name)
        positions *= n
    return Images(t.data_ptr(), C if ld is None else ld, t.stride(0))


class GroupNorm:
    """Group norm over the last dimension's `channels` channels (of x_dtype) in
    `groups` groups of consecutive ones, with weight and bias of p_dtype (float32
    or x_dtype), and an activation: None, "relu" or "silu".

    x is [samples][...][channels]: the dimensions between are positions.  A tensor
    [N][C][H][W] in torch.channels_last memory is x.permute(0, 2, 3, 1), a view.
    backward=False makes a handle without what the backward pass needs."""

    def __init__(self, channels: int, groups: int, x_dtype=torch.float32, p_dtype=torch.float32,
                 activation: Optional[str] = None, backward: bool = True):
        xd, pd = _dtype(x_dtype, "x_dtype"), _dtype(p_dtype, "p_dtype")
        if activation not in ACTIVATIONS:
            raise ValueError("activation must be None, \"relu\" or \"silu\", got %r" % (activation,))
        if not torch.cuda.is_available():
            raise RuntimeError("no GPU: the layer operators run on the GPU only")
        h = _VP()
        _check(lib().ga_groupnorm_create(int(channels), int(groups), xd, pd, ACTIVATIONS[activation],
                                         int(bool(backward)), ctypes.byref(h)))
        self._h, self.device = h, torch.cuda.current_device()
        self.channels, self.groups, self.x_dtype, self.p_dtype = int(channels), int(groups), x_dtype, p_dtype
        self.activation = activation

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().ga_groupnorm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _sizes(self, x):
        if not isinstance(x, torch.Tensor):
            raise TypeError("x must be a torch.Tensor")
        if x.dim() < 2 or x.shape[-1] != self.channels or x.dtype != self.x_dtype:
            raise ValueError("x must be %s [samples][...][%d], got %s %s" % (self.x_dtype, self.channels, x.dtype,
                                                                            tuple(x.shape)))
        if x.get_device() != self.device:
            raise ValueError("x is on %s, the handle on cuda:%d" % (x.device, self.device))
        positions = 1
        for n in x.shape[1:-1]:
            positions *= n
        return x.shape[0], positions

    def forward(self, x, gamma, beta, y, mean=None, rstd=None, eps: float = 1e-5) -> None:
        """y = activation(group norm of x); the groups' mean and 1/deviation into
        mean, rstd (float32 [samples][groups]).  gamma, beta: [channels] or None.
        y may be x."""
        N, S = self._sizes(x)
        C, G, d = self.channels, self.groups, self.device
        _check(lib().ga_groupnorm_forward(
            self._h, N, S, _images(x, x, "x"), _dev(gamma, self.p_dtype, C, "gamma", d),
            _dev(beta, self.p_dtype, C, "beta", d), eps, _images(y, x, "y"), _dev(mean, torch.float32, N * G, "mean", d),
            _dev(rstd, torch.float32, N * G, "rstd", d), _stream_ptr()))

    def backward(self, dy, x, gamma, beta, mean, rstd, dx, dgamma=None, dbeta=None, workers: int = 1) -> None:
        """dx of the forward pass at x; dgamma, dbeta: [workers][channels] in any of
        the three types, each worker its own run of consecutive samples.  dx may
        be dy or x."""
        N, S = self._sizes(x)
        C, G, d = self.channels, self.groups, self.device
        pdt = torch.float32 if dgamma is None else dgamma.dtype
        _check(lib().ga_groupnorm_backward(
            self._h, N, S, _images(dy, x, "dy"), _images(x, x, "x"), _dev(gamma, self.p_dtype, C, "gamma", d),
            _dev(beta, self.p_dtype, C, "beta", d), _dev(mean, torch.float32, N * G, "mean", d),
            _dev(rstd, torch.float32, N * G, "rstd", d), _images(dx, x, "dx"), workers,
            _dev(dgamma, pdt, workers * C, "dgamma", d), _dev(dbeta, pdt, workers * C, "dbeta", d),
            _dtype(pdt, "dgamma"), _stream_ptr()))


class Routing:
    """Where tokens go (ga_routing): `experts` int32 [tokens][k], `gates` float32
    [tokens][k] and `lse` float32 [tokens], the logarithm of the sum of the logits'
    exponentials."""

    def __init__(self, experts, gates=None, lse=None):
        self.experts, self.gates, self.lse = experts, gates, lse


class RouterLoad:
    """The workers' use of the experts (ga_load): `counts` int32 and `probs` float32
    [workers][experts], `tokens` int32 [workers], `loss` float32 [2] (balance, z),
    and `slope`, which the backward pass reads."""

    def __init__(self, counts, probs, tokens, loss, slope):
        self.counts, self.probs, self.tokens, self.loss, self.slope = counts, probs, tokens, loss, slope


class Router:
    """Router of a mixture of experts: softmax over the experts, the k largest,
    their gates, the counts of `workers` workers, and a balance loss.

    dtype: of the logits (float32, float16, bfloat16).
    normalize: a token's gates sum to 1.
    scope: "all" (counts and means over all workers' tokens) or "worker" (each
        worker's own; the losses are averaged).
    """

    def __init__(self, experts: int, k: int, dtype=torch.float32, workers: int = 1, normalize: bool = True,
                 scope: str = "all"):
        xd = _dtype(dtype, "dtype")
        if scope not in BALANCES:
            raise ValueError("scope must be \"all\" or \"worker\", got %r" % (scope,))
        if not torch.cuda.is_available():
            raise RuntimeError("no GPU: the layer operators run on the GPU only")
        h = _VP()
        _check(lib().ga_router_create(int(experts), int(k), xd, int(workers), int(bool(normalize)), BALANCES[scope],
                                      ctypes.byref(h)))
        self._h, self.device = h, torch.cuda.current_device()
        self.experts, self.k, self.dtype, self.workers = int(experts), int(k), dtype, int(workers)
        self.normalize, self.scope = bool(normalize), scope
        self.slopes = (1 if scope == "all" else self.workers) * (self.experts + 1)

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().ga_router_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def empty_routing(self, tokens: int, device="cuda") -> Routing:
        return Routing(torch.full((tokens, self.k), -1, dtype=torch.int32, device=device),
                       torch.zeros((tokens, self.k), dtype=torch.float32, device=device),
                       torch.zeros(tokens, dtype=torch.float32, device=device))

    def empty_load(self, device="cuda") -> RouterLoad:
        W, E = self.workers, self.experts
        return RouterLoad(torch.zeros((W, E), dtype=torch.int32, device=device),
                          torch.zeros((W, E), dtype=torch.float32, device=device),
                          torch.zeros(W, dtype=torch.int32, device=device),
                          torch.zeros(2, dtype=torch.float32, device=device),
                          torch.zeros((self.slopes // (E + 1), E + 1), dtype=torch.float32, device=device))

    def _tokens(self, logits, mask):
        if not isinstance(logits, torch.Tensor):
            raise TypeError("logits must be a torch.Tensor")
        if logits.dim() < 1 or logits.shape[-1] != self.experts or logits.dtype != self.dtype:
            raise ValueError("logits must be %s with %d columns, got %s %s" % (self.dtype, self.experts, logits.dtype,
                                                                             tuple(logits.shape)))
        if logits.get_device() != self.device:
            raise ValueError("logits are on %s, the handle on cuda:%d" % (logits.device, self.device))
        T = logits.numel() // self.experts
        if mask is not None and isinstance(mask, torch.Tensor) and mask.dtype == torch.uint8:
            return T, _dev(mask, torch.uint8, T, "mask", self.device)
        return T, _dev(mask, torch.bool, T, "mask", self.device)

    def _routing(self, r: Routing, T: int):
        d = self.device
        return RoutingPtrs(_dev(r.experts, torch.int32, T * self.k, "experts", d),
                           _dev(r.gates, torch.float32, T * self.k, "gates", d), _dev(r.lse, torch.float32, T, "lse", d))

    def forward(self, logits, routing: Routing, load: Optional[RouterLoad] = None, mask=None,
                select: bool = True) -> None:
        """The tokens' experts, gates and lse into `routing` (select=False: its
        experts are read, a selection made elsewhere), the counts and losses into
        `load` where given.  logits: [...][experts]; mask: bool or uint8, one per
        token, false where a token is absent.  With a load, not at the same time as
        another such call on this handle (on another stream)."""
        T, m = self._tokens(logits, mask)
        W, E, d = self.workers, self.experts, self.device
        ptrs = None if load is None else LoadPtrs(
            _dev(load.counts, torch.int32, W * E, "counts", d), _dev(load.probs, torch.float32, W * E, "probs", d),
            _dev(load.tokens, torch.int32, W, "tokens", d), _dev(load.loss, torch.float32, 2, "loss", d),
            _dev(load.slope, torch.float32, self.slopes, "slope", d))
        _check(lib().ga_router_forward(self._h, T, _rows(logits, logits, "logits"), m, int(bool(select)),
                                       self._routing(routing, T), ptrs, _stream_ptr()))

    def backward(self, logits, routing: Routing, load: Optional[RouterLoad], dlogits, dgates=None, mask=None,
                 balance: float = 0.0, z: float = 0.0) -> None:
        """Gradient of balance * load.loss[0] + z * load.loss[1] + sum(dgates *
        gates) to the logits, into dlogits (which may be logits).  routing, load and
        mask: those of the forward pass; dgates: float32 [tokens][k] or None."""
        T, m = self._tokens(logits, mask)
        d, out = self.device, _rows(dlogits, logits, "dlogits")
        if out is not None and dlogits.get_device() != d:
            raise ValueError("dlogits are on %s, the handle on cuda:%d" % (dlogits.device, d))
        _check(lib().ga_router_backward(
            self._h, T, _rows(logits, logits, "logits"), m, self._routing(routing, T),
            None if load is None else _dev(load.slope, torch.float32, self.slopes, "slope", d),
            _dev(dgates, torch.float32, T * self.k, "dgates", d), balance, z, out, _stream_ptr()))
