"""Layer operators around the loss head: a linear layer with bias, activation
and residual in its epilogue, the gated feed-forward projection, and the
global gradient norm with clipping.

    y = flce_linear_forward(x, W, b, residual, activation="gelu", pre=z)
    dx, dW, db = flce_linear_backward(dy, x, W, b, activation="gelu", pre=z)
    h = flce_gated_forward(x, Wg, Wu, activation="silu", pre=gu)
    dx, dWg, dWu = flce_gated_backward(dh, x, Wg, Wu, gu, activation="silu")
    norm = flce_clip_grads(grads, max_norm=1.0)

``fused_linear`` and ``gated_linear`` are the autograd forms, and
``GatedFeedForward`` the block made of them. As in the rest of the package
the functions only check and marshal arguments; every step runs in the
library's kernels, on the current CUDA stream, without a synchronisation.
"""
from __future__ import annotations

from typing import Iterable, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import ACTIVATIONS, KEEP


class _On:
    """A stream of the caller's choice: outputs and scratch are allocated on it too, so
    that none of them can be handed out again while its kernels still run."""

    def __init__(self, device, stream):
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        self.context = torch.cuda.stream(stream)

    def __enter__(self):
        self.context.__enter__()

    def __exit__(self, *exc):
        self.context.__exit__(*exc)


def _error_word(index: int) -> torch.Tensor:
    from . import device_error_word
    return device_error_word(torch.device("cuda", index))


class _Late:
    """The compiled calls, loaded at the first one."""

    def __getattr__(self, name):
        calls = _lib.calls(_error_word)
        for n in ("linear_forward", "linear_backward", "gated_forward", "gated_backward",
                  "clip_grads"):
            setattr(self, n, getattr(calls, n))
        return getattr(calls, name)


_calls = _Late()


# ------------------------------------------------------------------- linear
def flce_linear_forward(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor] = None,
                        residual: Optional[torch.Tensor] = None, *, activation: str = "none",
                        pre: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a(x W^T + b) + residual, [M, N] in x's type: one kernel from x to y.

    x [M, K] and W [N, K] are bf16 or fp16, K a multiple of 8; x's rows may be
    strided (a multiple of 8 elements). b [N]; residual and ``out`` [M, N] with
    rows of any pitch, ``out`` may be the residual itself. ``pre`` (an [M, N]
    tensor) receives what flce_linear_backward needs of a layer with an activation:
    the slopes a'(z), in a form of their own. An int16 tensor takes them with
    relative precision where units saturate (2^-10 of the slope); one of x's type (by
    its size alone) in fixed steps of 2^-15, in which slopes below 2^-16 are 0.
    ``workspace``: as in flce_forward."""
    if stream is not None:
        with _On(x.device, stream):
            return _calls.linear_forward(x, W, b, residual, activation, pre, out, workspace)
    return _calls.linear_forward(x, W, b, residual, activation, pre, out, workspace)


def flce_linear_backward(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor,
                         b: Optional[torch.Tensor] = None, *, activation: str = "none",
                         pre: Optional[torch.Tensor] = None,
                         dW_dtype: torch.dtype = torch.float32,
                         db_dtype: torch.dtype = torch.float32, needs=(True, True, True),
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """dx [M, K] in x's type, dW [N, K] (fp32 or x's type) and db [N] (None
    without a bias) of flce_linear_forward; the residual's gradient is dy.

    ``pre``: the forward's, with an activation. dz = dy a'(z) is rounded to x's
    type before the two products. ``needs``: which of (dx, dW, db) to compute;
    the others are None."""
    f32 = torch.float32
    for t in (dW_dtype, db_dtype):
        if t not in (f32, x.dtype):
            raise TypeError("flce: dW_dtype and db_dtype must be fp32 or x's dtype")
    if stream is not None:
        with _On(x.device, stream):
            return flce_linear_backward(dy, x, W, b, activation=activation, pre=pre,
                                        dW_dtype=dW_dtype, db_dtype=db_dtype, needs=needs,
                                        workspace=workspace)
    need_dx, need_dW, need_db = needs
    return _calls.linear_backward(dy, x, W, b, activation, pre, dW_dtype is f32, db_dtype is f32,
                                  need_dx, need_dW, need_db, workspace)


# -------------------------------------------------------------------- gated
def flce_gated_forward(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, *,
                       activation: str = "silu", pre: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a(x Wg^T) * (x Wu^T), [M, F] in x's type: both projections, the
    activation and the product in one kernel.

    x [M, K], Wg and Wu [F, K] are bf16 or fp16, K and F multiples of 8; the rows
    of x and ``out`` may be strided (a multiple of 8 elements). ``pre`` (a
    [2, M, F] tensor) receives what flce_gated_backward needs, in a form of its own:
    an int16 tensor takes it with relative precision (2^-11 of each value), one of
    x's type (by its size alone) to 2^-14 of the largest of 8 neighbouring columns.
    ``workspace``: as in flce_forward."""
    if stream is not None:
        with _On(x.device, stream):
            return _calls.gated_forward(x, Wg, Wu, activation, pre, out, workspace)
    return _calls.gated_forward(x, Wg, Wu, activation, pre, out, workspace)


def flce_gated_backward(dh: torch.Tensor, x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                        pre: torch.Tensor, *, activation: str = "silu",
                        dW_dtype: torch.dtype = torch.float32, needs=(True, True),
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """dx [M, K] in x's type, dWg and dWu [F, K] (fp32 or x's type) of
    flce_gated_forward, whose ``pre`` it takes. ``needs``: whether to compute dx,
    and the weight gradients; what is not computed is None."""
    if dW_dtype not in (torch.float32, x.dtype):
        raise TypeError("flce: dW_dtype must be fp32 or x's dtype")
    if stream is not None:
        with _On(x.device, stream):
            return flce_gated_backward(dh, x, Wg, Wu, pre, activation=activation,
                                       dW_dtype=dW_dtype, needs=needs, workspace=workspace)
    need_dx, need_dW = needs
    return _calls.gated_backward(dh, x, Wg, Wu, pre, activation, dW_dtype is torch.float32, need_dx,
                                 need_dW, workspace)


# ------------------------------------------------------ gradient norm, clipping
def _list(tensors) -> list:
    return [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)


def flce_grad_norm(grads: Iterable[torch.Tensor], *, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The global 2-norm of all elements of ``grads`` (dense bf16, fp16 and fp32
    CUDA tensors of any shapes) as a 0-dim fp32 tensor."""
    grads = _list(grads)
    if stream is not None and grads:
        with _On(grads[0].device, stream):
            return _calls.clip_grads(grads, None, None, 0.0, workspace)
    return _calls.clip_grads(grads, None, None, 0.0, workspace)


def flce_clip_grads(grads: Iterable[torch.Tensor], max_norm: float, *,
                    out: Optional[Sequence[torch.Tensor]] = None, eps: float = 1e-6,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scales ``grads`` by min(1, max_norm / (norm + eps)), in place or into
    ``out`` (tensors of the same shapes, types and strides), and returns their
    global norm before the scaling as a 0-dim fp32 tensor. Each tensor is given
    once. The scale is formed on the device: nothing is read back. A NaN norm
    makes every element NaN, an infinite one scales by 0."""
    grads = _list(grads)
    out = None if out is None else _list(out)
    if stream is not None and grads:
        with _On(grads[0].device, stream):
            return _calls.clip_grads(grads, out, float(max_norm), eps, workspace)
    return _calls.clip_grads(grads, out, float(max_norm), eps, workspace)


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0, *,
                    eps: float = 1e-6) -> torch.Tensor:
    """flce_clip_grads over the ``.grad`` of ``parameters`` (those that have
    one), in place; the norm before the scaling, 0 where there is no gradient.
    Positional arguments as torch.nn.utils.clip_grad_norm_ has them; ``norm_type``
    can only be 2. A parameter that is listed twice counts once."""
    if float(norm_type) != 2.0:
        raise ValueError(f"flce: clip_grad_norm_ clips by the 2-norm, got norm_type={norm_type!r}")
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    # A tied parameter that is listed twice is one: two blocks must not scale the same memory.
    grads = [p.grad for p in dict.fromkeys(parameters) if p.grad is not None]
    if not grads:
        return torch.zeros(())
    return flce_clip_grads(grads, max_norm, eps=eps)


# ------------------------------------------------------------ autograd, modules
def _usable(t: torch.Tensor) -> torch.Tensor:
    """t itself where the kernels can read its rows, else a dense copy."""
    if t.stride(1) == 1 and t.stride(0) >= t.shape[1] and t.stride(0) % 8 == 0 and \
            t.data_ptr() % 16 == 0:
        return t
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _kept_dtype(x: torch.Tensor, keep: str) -> torch.dtype:
    if keep not in KEEP:
        raise ValueError(f"flce: keep must be one of {sorted(KEEP)}, got {keep!r}")
    return torch.int16 if keep == "relative" else x.dtype


def _dense(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """A weight or bias itself where the kernels can read it, else a dense copy."""
    if t is None:
        return None
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class FusedLinearFunction(torch.autograd.Function):
    """Autograd form of the linear layer. It keeps x, and the slopes of an activation in the
    form ``keep``."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation, keep="fixed"):
        pre = None
        dtype = _kept_dtype(x, keep)
        if activation != "none" and any(ctx.needs_input_grad[:3]):
            pre = torch.empty(x.shape[0], weight.shape[0], dtype=dtype, device=x.device)
        y = flce_linear_forward(x, weight, bias, residual, activation=activation, pre=pre)
        ctx.save_for_backward(x, weight, bias, pre)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, pre = ctx.saved_tensors
        dx = dW = db = None
        if any(ctx.needs_input_grad[:3]):
            d = _usable(dy)
            dx, dW, db = flce_linear_backward(d, x, weight, bias, activation=ctx.activation,
                                              pre=pre, dW_dtype=weight.dtype, db_dtype=x.dtype,
                                              needs=ctx.needs_input_grad[:3])
        return dx, dW, db, dy if ctx.needs_input_grad[3] else None, None, None


class GatedLinearFunction(torch.autograd.Function):
    """Autograd form of the gated projection. It keeps x and 32 bits for each output,
    in the form ``keep``."""

    @staticmethod
    def forward(ctx, x, gate_weight, up_weight, activation, keep="relative"):
        pre = None
        dtype = _kept_dtype(x, keep)
        if any(ctx.needs_input_grad[:3]):
            pre = torch.empty(2, x.shape[0], gate_weight.shape[0], dtype=dtype, device=x.device)
        h = flce_gated_forward(x, gate_weight, up_weight, activation=activation, pre=pre)
        ctx.save_for_backward(x, gate_weight, up_weight, pre)
        ctx.activation = activation
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, Wg, Wu, pre = ctx.saved_tensors
        need_x, need_g, need_u = ctx.needs_input_grad[:3]
        dx, dWg, dWu = flce_gated_backward(_usable(dh), x, Wg, Wu, pre, activation=ctx.activation,
                                           dW_dtype=Wg.dtype, needs=(need_x, need_g or need_u))
        return dx, dWg if need_g else None, dWu if need_u else None, None, None


def fused_linear(x, weight, bias=None, residual=None, activation="none", keep="fixed"):
    """activation(x weight^T + bias) + residual with gradients; x [..., K], weight
    [N, K], residual [..., N]. Inputs whose rows the kernels cannot read as they
    are (flce_linear_forward) are copied first. ``keep``: how the slopes of the
    activation are kept for the backward, "fixed" (steps of 2^-15: a saturated
    unit's gradient is lost) or "relative" (2^-10 of the slope there); both take
    two bytes a value."""
    x2 = _usable(x.reshape(-1, x.shape[-1]))
    r2 = None
    if residual is not None:
        r2 = residual.reshape(-1, weight.shape[0])
        if r2.stride(1) != 1 or r2.stride(0) < r2.shape[1]:
            r2 = r2.contiguous()
    y = FusedLinearFunction.apply(x2, _dense(weight), _dense(bias), r2, activation, keep)
    return y.reshape(*x.shape[:-1], weight.shape[0])


def gated_linear(x, gate_weight, up_weight, activation="silu", keep="relative"):
    """activation(x gate_weight^T) * (x up_weight^T) with gradients; x [..., K],
    the weights [F, K]. ``keep``: what the backward needs is kept with "relative"
    precision, or "fixed": to 2^-14 of the largest of 8 neighbouring features, which
    is finer for features of one size and loses those beside an outlier."""
    x2 = _usable(x.reshape(-1, x.shape[-1]))
    h = GatedLinearFunction.apply(x2, _dense(gate_weight), _dense(up_weight), activation, keep)
    return h.reshape(*x.shape[:-1], gate_weight.shape[0])


class GatedFeedForward(torch.nn.Module):
    """x + W_down (a(W_gate x) * (W_up x)): the gated projection and the down
    projection that adds the residual stream, two kernels forward. ``inputs``
    (by default x) is what the block reads, such as the normed residual stream."""

    def __init__(self, hidden: int, features: int, activation: str = "silu",
                 dtype=torch.bfloat16, device=None):
        super().__init__()
        if activation not in ACTIVATIONS:
            raise ValueError(f"flce: activation must be one of {sorted(ACTIVATIONS)}, "
                             f"got {activation!r}")
        self.activation = activation

        def weight(rows, cols):
            w = torch.empty(rows, cols, dtype=dtype, device=device)
            return torch.nn.Parameter(w.normal_(std=cols ** -0.5))

        self.gate, self.up = weight(features, hidden), weight(features, hidden)
        self.down = weight(hidden, features)

    def forward(self, x, inputs=None):
        h = gated_linear(x if inputs is None else inputs, self.gate, self.up, self.activation)
        return fused_linear(h, self.down, residual=x)
