"""Binding of the training-step operators: gradient norm, AdamW and layer norm.

Argument marshalling only, like the rest of the binding: the operators are the
HIP kernels behind ga_grad_norm, ga_adamw_step, ga_layernorm_forward and
ga_layernorm_backward, specified in include/gradagg.h.  Calls run on the
current stream, allocate nothing and do not synchronize.

A handle owns one workspace.  AdamW.grad_norm and LayerNorm.backward use it: two
such calls on one handle must not run at the same time.  Give each stream that
runs them a handle of its own, or order the streams with events.  Calls that did
overlap can leave the handle's count of ended workgroups wrong, and later calls
on it without a result: make a new handle then.  The other calls may overlap.
A captured call uses its handle's memory at every replay: keep the handle.
"""
from __future__ import annotations

import ctypes
import warnings
from typing import Optional, Sequence

import torch

from . import _VP, GA_BF16, AdamWParamsLayout, AdamWStatePtrs, Rows, _check, _dev, _stream_ptr, lib

STATE_BLOCK = 256
MAX_GROUPS = 1024
MAX_DIM = 1 << 20
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: GA_BF16}
CODES = torch.float8_e4m3fn
ROUNDINGS = {"random": 0, "nearest": 1}


def _dtype(t, what: str) -> int:
    if t not in DTYPES:
        raise ValueError("%s must be float32, float16 or bfloat16, got %s" % (what, t))
    return DTYPES[t]


class Clip:
    """What a gradient norm leaves on the device (ga_clip): `norm`, `scale` (the
    factor that brings the norm to max_norm, at most 1) and `skip` (1 when the
    norm is not finite), one-element views of one record."""

    def __init__(self, device="cuda"):
        self.record = torch.zeros(4, dtype=torch.float32, device=device)
        self.record[1] = 1.0
        self.norm, self.scale = self.record[0:1], self.record[1:2]
        self.skip = self.record.view(torch.int32)[2:3]


class AdamWState:
    """Moments of the P parameters.  32 bits: m, v float32 [P].  8 bits: m, v
    float8_e4m3fn [n_blocks][256] codes with float32 scales [n_blocks]; v holds
    the square root of the second moment (see gradagg.h).

    m_rounding (8 bits): how the steps round m's codes, "random" as in the state
    of empty_state(), or "nearest", under which a moment that moves by less than
    half a code's step per step stays where it is.  A state made without saying
    which is rounded to nearest, as such states always were, and warns."""

    m_rounding = "nearest"      # of a state pickled before there was a choice

    def __init__(self, m, v, m_scale=None, v_scale=None, m_rounding: Optional[str] = None):
        if m_rounding is None:
            m_rounding = "nearest"
            if m_scale is not None:
                warnings.warn("8-bit first moments rounded to nearest do not follow slow changes of the gradient: "
                              "say m_rounding=\"random\" (or \"nearest\", to repeat earlier results)", stacklevel=2)
        if m_rounding not in ROUNDINGS:
            raise ValueError("m_rounding must be \"random\" or \"nearest\", got %r" % (m_rounding,))
        self.m, self.v, self.m_scale, self.v_scale, self.m_rounding = m, v, m_scale, v_scale, m_rounding


class AdamW:
    """Gradient norm and AdamW update over W workers' layer lists.

    layer_numels: element count of every layer, in fused order.
    grad_dtype: type of the workers' gradient tensors (float32, float16, bfloat16).
    state_bits: 32 or 8.
    decay: one truth value per layer, where weight decay applies (default: everywhere).
    """

    def __init__(self, layer_numels: Sequence[int], W: int = 1, grad_dtype=torch.float32, state_bits: int = 32,
                 decay: Optional[Sequence[bool]] = None):
        self.layer_numels = [int(n) for n in layer_numels]
        L = len(self.layer_numels)
        if decay is not None and len(decay) != L:
            raise ValueError("decay has %d entries for %d layers" % (len(decay), L))
        gdt = _dtype(grad_dtype, "grad_dtype")
        if not torch.cuda.is_available():
            raise RuntimeError("no GPU: the training-step operators run on the GPU only")
        flags = None if decay is None else (ctypes.c_uint8 * L)(*[1 if d else 0 for d in decay])
        h = _VP()
        _check(lib().ga_adamw_create(int(W), L, (ctypes.c_int64 * L)(*self.layer_numels), gdt, int(state_bits), flags,
                                     ctypes.byref(h)))
        self._h = h
        self.W, self.P, self.state_bits, self.grad_dtype = int(W), sum(self.layer_numels), int(state_bits), grad_dtype
        self.n_blocks = (self.P + STATE_BLOCK - 1) // STATE_BLOCK

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().ga_adamw_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def empty_clip(self, device="cuda") -> Clip:
        """A record that clips nothing."""
        return Clip(device)

    def empty_state(self, device="cuda") -> AdamWState:
        """The state before the first step (all zero)."""
        if self.state_bits == 32:
            return AdamWState(*(torch.zeros(self.P, dtype=torch.float32, device=device) for _ in range(2)))
        codes = [torch.zeros((self.n_blocks, STATE_BLOCK), dtype=torch.uint8, device=device).view(CODES)
                 for _ in range(2)]
        scales = [torch.zeros(self.n_blocks, dtype=torch.float32, device=device) for _ in range(2)]
        return AdamWState(*codes, *scales, m_rounding="random")

    def grad_norm(self, layer_ptrs, clip: Clip, max_norm: float = float("inf"), grad=None) -> None:
        """Norm of the workers' mean gradient into `clip`; the mean gradient
        itself into `grad` ([P] float32) where given.  layer_ptrs: int64 tensor
        of the W*L gradient tensors' addresses, worker-major.  Not at the same
        time as another grad_norm on this handle (on another stream)."""
        _check(lib().ga_grad_norm(self._h, _dev(layer_ptrs, torch.int64, self.W * len(self.layer_numels), "layer_ptrs"),
                                  max_norm, _dev(grad, torch.float32, self.P, "grad"),
                                  _dev(clip.record, torch.float32, 4, "clip"), _stream_ptr()))

    def step(self, layer_ptrs, w, state: AdamWState, t: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
             eps: float = 1e-8, weight_decay: float = 0.0, clip: Optional[Clip] = None, copy=None) -> None:
        """One update of w ([P] float32) and the state, step t counted from 1;
        the new weights also go into `copy` ([P] float16 or bfloat16).  `clip`:
        a record of grad_norm, whose scale multiplies the gradient and whose
        skip leaves everything unchanged."""
        n = self.P if self.state_bits == 32 else self.n_blocks * STATE_BLOCK
        sdt = torch.float32 if self.state_bits == 32 else CODES
        ptrs = AdamWStatePtrs(_dev(state.m, sdt, n, "m"), _dev(state.v, sdt, n, "v"))
        if self.state_bits == 8:
            ptrs.m_scale = _dev(state.m_scale, torch.float32, self.n_blocks, "m_scale")
            ptrs.v_scale = _dev(state.v_scale, torch.float32, self.n_blocks, "v_scale")
        cdt = 0
        if copy is not None:
            cdt = _dtype(copy.dtype, "copy")
        _check(lib().ga_adamw_step(
            self._h, _dev(layer_ptrs, torch.int64, self.W * len(self.layer_numels), "layer_ptrs"),
            AdamWParamsLayout(lr, beta1, beta2, eps, weight_decay, ROUNDINGS[state.m_rounding], t),
            _dev(w, torch.float32, self.P, "w"), ptrs,
            None if clip is None else _dev(clip.record, torch.float32, 4, "clip"),
            None if copy is None else _dev(copy, copy.dtype, self.P, "copy"), cdt, _stream_ptr()))


def _rows(t, like, name: str):
    """ga_rows of a tensor of x's shape and type whose rows are contiguous and
    evenly spaced (None stays None)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError("%s must be %s %s, got %s %s" % (name, like.dtype, tuple(like.shape), t.dtype, tuple(t.shape)))
    if t.is_contiguous():
        return Rows(t.data_ptr(), t.shape[-1])
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s must have contiguous rows" % name)
    # one stride has to lead from every row to the next
    ld, rows = None, 1
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            raise ValueError("%s must have evenly spaced rows" % name)
        rows *= n
    return Rows(t.data_ptr(), t.shape[-1] if ld is None else ld)


class LayerNorm:
    """Layer norm over the last dimension (`dim` elements of x_dtype), weight and
    bias of p_dtype (float32 or x_dtype).  backward=False makes a handle without
    the backward pass's workspace (2048 * dim bytes)."""

    def __init__(self, dim: int, x_dtype=torch.float32, p_dtype=torch.float32, backward: bool = True):
        xd, pd = _dtype(x_dtype, "x_dtype"), _dtype(p_dtype, "p_dtype")
        if not torch.cuda.is_available():
            raise RuntimeError("no GPU: the training-step operators run on the GPU only")
        h = _VP()
        _check(lib().ga_layernorm_create(int(dim), xd, pd, int(bool(backward)), ctypes.byref(h)))
        self._h = h
        self.dim, self.x_dtype, self.p_dtype = int(dim), x_dtype, p_dtype

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().ga_layernorm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _count(self, x) -> int:
        if not isinstance(x, torch.Tensor):
            raise TypeError("x must be a torch.Tensor")
        if x.dim() < 1 or x.shape[-1] != self.dim or x.dtype != self.x_dtype:
            raise ValueError("x must be %s with %d columns, got %s %s" % (self.x_dtype, self.dim, x.dtype,
                                                                        tuple(x.shape)))
        return x.numel() // self.dim

    def forward(self, x, gamma, beta, y, mean=None, rstd=None, residual=None, sum_out=None, eps: float = 1e-5) -> None:
        """y = layer norm of x (of x + residual, which also goes into sum_out);
        the rows' mean and 1/deviation into mean, rstd (float32, one per row).
        gamma, beta: [dim] or None."""
        n = self._count(x)
        _check(lib().ga_layernorm_forward(
            self._h, n, _rows(x, x, "x"), _rows(residual, x, "residual"), _dev(gamma, self.p_dtype, self.dim, "gamma"),
            _dev(beta, self.p_dtype, self.dim, "beta"), eps, _rows(y, x, "y"), _rows(sum_out, x, "sum_out"),
            _dev(mean, torch.float32, n, "mean"), _dev(rstd, torch.float32, n, "rstd"), _stream_ptr()))

    def backward(self, dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, dsum=None, groups: int = 1) -> None:
        """dx of the forward pass at x (its sum_out where it had a residual),
        plus dsum where given; dgamma, dbeta: [groups][dim] in any of the three
        types, each group its own run of consecutive rows.  Not at the same time
        as another backward on this handle (on another stream)."""
        n = self._count(x)
        pdt = torch.float32 if dgamma is None else dgamma.dtype
        _check(lib().ga_layernorm_backward(
            self._h, n, _rows(dy, x, "dy"), _rows(x, x, "x"), _dev(gamma, self.p_dtype, self.dim, "gamma"),
            _dev(mean, torch.float32, n, "mean"), _dev(rstd, torch.float32, n, "rstd"), _rows(dsum, x, "dsum"),
            _rows(dx, x, "dx"), groups, _dev(dgamma, pdt, groups * self.dim, "dgamma"),
            _dev(dbeta, pdt, groups * self.dim, "dbeta"), _dtype(pdt, "dgamma"), _stream_ptr()))
