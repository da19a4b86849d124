"""Operators on the residual stream, between a block and the next one or the loss
head: the root-mean-square norm with the residual's addition, and dropout from a
counter-based generator.

    y, h = flce_rms_norm_forward(x, weight, residual, rstd=rstd)
    dx, dresidual, dW = flce_rms_norm_backward(dy, h, weight, rstd, dh)
    y8, scale, h = flce_rms_norm_quantized(x, weight, residual, scales="row")
    y = flce_dropout(x, 0.1, seed, residual=residual)

``fused_rms_norm`` and ``fused_dropout`` are the autograd forms, ``FusedRMSNorm``
the module. As in the rest of the package the functions only check and marshal
arguments; every step runs in the library's kernels, on the current CUDA stream,
without a synchronisation.
"""
from __future__ import annotations

from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from ._lib import SCALES
from .block import _On, _calls

Seed = Union[int, torch.Tensor, None]


# --------------------------------------------------------------------- norm
def flce_rms_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor],
                          residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                          dropout: float = 0.0, seed: Seed = None, offset: int = 0, h=None,
                          rstd: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          stream=None):
    """(y, h): h = residual + D(x), y = weight h / sqrt(mean(h^2) + eps).

    x [..., H] is bf16, fp16 or fp32, contiguous or two-dimensional with rows of any
    pitch; H up to 32768. weight [H] (None: ones) is of x's type or fp32, and so is the
    residual, of x's shape; h has its type. Without a residual and dropout h is x. A
    tensor ``h`` receives the sum (it may be the residual itself, which it then
    replaces), False leaves it out (None is returned for it). ``out`` may be x.
    ``rstd`` ([rows] fp32) receives what flce_rms_norm_backward needs beside h.

    D is the dropout of flce_dropout, with its ``seed`` and ``offset``."""
    if stream is not None:
        with _On(x.device, stream):
            return _calls.rms_norm_forward(x, weight, residual, eps, dropout, seed, offset, h, rstd, out)
    return _calls.rms_norm_forward(x, weight, residual, eps, dropout, seed, offset, h, rstd, out)


def flce_rms_norm_quantized(x: torch.Tensor, weight: Optional[torch.Tensor],
                            residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                            scales: str = "row", dropout: float = 0.0, seed: Seed = None,
                            offset: int = 0, h=None, out: Optional[torch.Tensor] = None,
                            scale: Optional[torch.Tensor] = None, stream=None):
    """(y8, scale, h): flce_rms_norm_forward with y in 8 bits (float8_e4m3fn), y = y8 scale.

    ``scales``: "row", scale [...] fp32, or "block", one for each 128 columns, scale
    [..., ceil(H / 128)]; largest |y| / 448 either way. ``out`` and ``scale`` receive them."""
    if scales not in ("row", "block"):
        raise ValueError(f"flce: scales must be 'row' or 'block', got {scales!r}")
    block = SCALES[scales] == SCALES["block"]
    if stream is not None:
        with _On(x.device, stream):
            return _calls.rms_norm_quantized(x, weight, residual, eps, dropout, seed, offset, h, block,
                                             out, scale)
    return _calls.rms_norm_quantized(x, weight, residual, eps, dropout, seed, offset, h, block, out,
                                     scale)


def flce_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: Optional[torch.Tensor],
                           rstd: torch.Tensor, dh: Optional[torch.Tensor] = None, *,
                           dropout: float = 0.0, seed: Seed = None, offset: int = 0,
                           dW_dtype: torch.dtype = torch.float32, needs=(True, True, True),
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """dx in dy's type, dresidual in h's and dW [H] (fp32 or dy's type; None without a
    weight) of flce_rms_norm_forward, which gave h and ``rstd``. h is read as it is stored:
    in 16 bits its rounding reaches dW, about as much again as rounding dW to 16 bits.

    ``dh``: the gradient that reaches h along the residual stream, of h's type, or None.
    dropout, seed and offset are the forward's. Without dropout and with one type dx and
    dresidual are one tensor. ``needs``: which of (dx, dresidual, dW) to compute; the
    others are None."""
    if dW_dtype not in (torch.float32, dy.dtype):
        raise TypeError("flce: dW_dtype must be fp32 or dy's dtype")
    if stream is not None:
        with _On(dy.device, stream):
            return flce_rms_norm_backward(dy, h, weight, rstd, dh, dropout=dropout, seed=seed,
                                          offset=offset, dW_dtype=dW_dtype, needs=needs,
                                          workspace=workspace)
    need_dx, need_dr, need_dW = needs
    return _calls.rms_norm_backward(dy, h, weight, rstd, dh, dropout, seed, offset,
                                    dW_dtype is torch.float32, need_dx, need_dr, need_dW, workspace)


# ------------------------------------------------------------------ dropout
def flce_dropout(x: torch.Tensor, p: float, seed: Seed, *, offset: int = 0,
                 residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 like: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """residual + D(x): each element of x is dropped with probability p (taken to 2^-16),
    else divided by what is left of 1. The gradient of x is the same call on dy.

    x [..., H] is bf16, fp16 or fp32, contiguous or two-dimensional with rows of any
    pitch. y is of the type of ``out``, of the residual (x's shape), of ``like`` or
    of x; x's type, or one of the two is fp32. ``out`` may be x or the residual.

    The mask is a function of (seed, offset, row, column) alone and is stored nowhere: a
    training program keeps the seed and counts ``offset`` up by layers and steps. ``seed``
    is an int (its low 64 bits), or an int64 tensor of one element that is read when the
    kernel runs, so that a captured graph draws anew. A dropped element is 0 even where x
    is not finite."""
    if stream is not None:
        with _On(x.device, stream):
            return _calls.dropout(x, p, seed, offset, residual, out, like)
    return _calls.dropout(x, p, seed, offset, residual, out, like)


# ------------------------------------------------------------ autograd, modules
def _probability(p: float) -> float:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"flce: dropout must be a probability, got {p!r}")
    return float(p)


def _new_seed(device) -> torch.Tensor:
    """A seed from the device's generator: torch.manual_seed makes it repeatable, and a
    captured graph draws another at each replay."""
    return torch.empty(1, dtype=torch.int64, device=device).random_()


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t where the kernels can read its rows, else a dense copy."""
    if t.is_contiguous() or (t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return t
    return t.contiguous()


def _keep(ctx, seed, *tensors):
    """Keeps tensors and the seed; a seed tensor that is written before the backward is an error then."""
    ctx.seed = None if torch.is_tensor(seed) else seed
    ctx.save_for_backward(seed if torch.is_tensor(seed) else None, *tensors)


def _kept(ctx):
    seed, *tensors = ctx.saved_tensors
    return (ctx.seed if seed is None else seed, *tensors)


class FusedRMSNormFunction(torch.autograd.Function):
    """Autograd form of the norm: (y, h). It keeps h, one number for each row, and the seed."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, dropout, seed):
        rstd = None
        if any(ctx.needs_input_grad[:3]):
            rstd = torch.empty(x.shape[:-1].numel(), dtype=torch.float32, device=x.device)
        y, h = flce_rms_norm_forward(x, weight, residual, eps=eps, dropout=dropout, seed=seed, rstd=rstd)
        ctx.set_materialize_grads(False)
        ctx.dropout, ctx.x_dtype = dropout, x.dtype
        _keep(ctx, seed, h, weight, rstd)
        return y, (None if h is x else h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        seed, h, weight, rstd = _kept(ctx)
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        dx = dr = dW = None
        if dy is not None:
            dh = None if dh is None else _rows(dh)
            dx, dr, dW = flce_rms_norm_backward(
                _rows(dy), h, weight, rstd, dh, dropout=ctx.dropout, seed=seed,
                dW_dtype=torch.float32 if weight is None else weight.dtype,
                needs=(need_x, need_r, need_w))
        elif dh is not None:
            # Only the sum was used.
            dr = dh if need_r else None
            if need_x:
                like = torch.empty(0, dtype=ctx.x_dtype, device=dh.device)
                dx = flce_dropout(_rows(dh), ctx.dropout, seed, like=like)
            dW = torch.zeros_like(weight) if need_w else None
        return dx, dW, dr, None, None, None


class FusedDropoutFunction(torch.autograd.Function):
    """Autograd form of dropout with the residual's addition. It keeps the seed alone."""

    @staticmethod
    def forward(ctx, x, residual, p, seed):
        ctx.p, ctx.like = p, x.new_empty(0)
        _keep(ctx, seed)
        return flce_dropout(x, p, seed, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dx = None
        (seed,) = _kept(ctx)
        if ctx.needs_input_grad[0]:
            dx = flce_dropout(_rows(dy), ctx.p, seed, like=ctx.like)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None


def _drawn(p: float, seed: Seed, device) -> Seed:
    return _new_seed(device) if p > 0 and seed is None else seed


def fused_rms_norm(x, weight=None, residual=None, eps=1e-6, dropout=0.0, seed=None):
    """weight h / sqrt(mean(h^2) + eps) with h = residual + D(x), with gradients: y where h
    is x (no residual and no dropout), else (y, h), h being the residual stream to carry on.
    ``seed``: as in flce_dropout, by default drawn from the device's generator."""
    p = _probability(dropout)
    y, h = FusedRMSNormFunction.apply(_rows(x), weight, None if residual is None else _rows(residual),
                                      eps, p, _drawn(p, seed, x.device))
    return y if h is None else (y, h)


def fused_dropout(x, p=0.5, residual=None, seed=None):
    """residual + D(x) with gradients. ``seed``: as in flce_dropout, by default drawn from the
    device's generator."""
    p = _probability(p)
    return FusedDropoutFunction.apply(_rows(x), None if residual is None else _rows(residual), p,
                                      _drawn(p, seed, x.device))


class FusedRMSNorm(torch.nn.Module):
    """The norm with its weight: y = norm(x), or (y, h) = norm(x, residual) with
    h = residual + D(x), dropout with probability ``dropout`` in training."""

    def __init__(self, hidden: int, eps: float = 1e-6, dropout: float = 0.0, dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        self.eps, self.dropout = eps, _probability(dropout)
        self.weight = torch.nn.Parameter(torch.ones(hidden, dtype=dtype, device=device))

    def forward(self, x, residual=None):
        p = self.dropout if self.training else 0.0
        out = fused_rms_norm(x, self.weight, residual, self.eps, p)
        # With dropout the function returns the sum too; without a residual there is no stream to carry on.
        return out[0] if residual is None and p > 0 else out
