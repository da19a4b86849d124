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

import array
import ctypes
import operator
from typing import Iterable, Optional, Sequence

import torch

from . import _lib
from ._lib import ACTIVATIONS, FlceError, FlceGatedParams, FlceLinearParams

_OPERANDS = (torch.bfloat16, torch.float16)
_GRAD_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

# Parameter structs by their values (sizes, pitches and options only): (library,
# address, forward and backward workspace bytes, the struct that keeps the address
# alive). Bounded: emptied when it is full.
_params = {}
_PARAMS_MOST = 4096


def _struct(kind, *values):
    key = (kind, values)
    got = _params.get(key)
    if got is None:
        lib = _lib.load()
        p = kind(*[int(v) for v in values])
        at = ctypes.addressof(p)
        size = lib.flce_linear_workspace_size if kind is FlceLinearParams else \
            lib.flce_gated_workspace_size
        if len(_params) >= _PARAMS_MOST:
            _params.clear()
        got = _params[key] = (lib, at, int(size(at, 0)), int(size(at, 1)), p)
    return got[:4]


def _activation(name) -> int:
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"flce: activation must be one of {sorted(ACTIVATIONS)}, got {name!r}") from None


def _rows(t: torch.Tensor, rows: int, cols: int, dtype, name: str) -> int:
    """The row pitch (elements) of a [rows, cols] CUDA tensor whose rows are contiguous."""
    if t.dtype is not dtype or not t.is_cuda:
        raise TypeError(f"flce: {name} must be a CUDA tensor of type {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"flce: {name} must have shape [{rows}, {cols}], got {tuple(t.shape)}")
    if rows <= 1 or cols == 0:
        if cols > 1 and t.stride(1) != 1:
            raise ValueError(f"flce: the rows of {name} must be contiguous")
        return cols
    ld, step = t.stride()
    if (step != 1 and cols > 1) or ld < cols:
        raise ValueError(f"flce: the rows of {name} must be contiguous and must not overlap")
    return ld


def _dense(t: torch.Tensor, shape, dtype, name: str):
    if t.dtype is not dtype or not t.is_cuda:
        raise TypeError(f"flce: {name} must be a CUDA tensor of type {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"flce: {name} must be contiguous with shape {list(shape)}")


def _operand(x: torch.Tensor) -> None:
    if not x.is_cuda or x.dtype not in _OPERANDS:
        raise TypeError("flce: x must be a bf16 or fp16 CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"flce: x must be two-dimensional, got shape {tuple(x.shape)}")


class _On:
    """The device and stream of a call that names a stream or runs on another
    device than the current one. With a stream of its own, outputs and scratch are
    allocated on that stream too, so that none of them can be handed out again
    while its kernels still run."""

    def __init__(self, device, stream):
        self.contexts = [torch.cuda.device(device)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_error_words = {}


def _elsewhere(device, stream) -> bool:
    return stream is not None or device.index != _current_device()


def _error_word(index: int) -> int:
    """Address of the device's error word (which lives as long as the process)."""
    at = _error_words.get(index)
    if at is None:
        from . import device_error_word
        at = _error_words[index] = device_error_word(torch.device("cuda", index)).data_ptr()
    return at


def _scratch(workspace, need: int, device):
    """The caller's workspace where it is large enough, else a new one (None: none needed)."""
    if need == 0:
        return None
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
            raise TypeError("flce: workspace must be a contiguous uint8 CUDA tensor")
        if workspace.numel() >= need:
            return workspace
    return torch.empty(need, dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _done(status: int, what: str) -> None:
    if status != _lib.FLCE_OK:
        raise FlceError(status, what)


# ------------------------------------------------------------------- linear
def _weight(W: torch.Tensor) -> None:
    if W.dim() != 2:
        raise ValueError(f"flce: weights must be two-dimensional, got shape {tuple(W.shape)}")


def _linear_params(x, W, b, res, y, activation, dW_fp32, db_fp32):
    """(library, address of the parameters, forward and backward workspace bytes) of a
    linear call; y: the output, or the backward's dy."""
    M, K = x.shape
    N = W.shape[0]
    dtype = x.dtype
    if W.shape[1] != K:
        raise ValueError(f"flce: W must have shape [N, {K}], got {tuple(W.shape)}")
    _dense(W, (N, K), dtype, "W")
    if b is not None:
        _dense(b, (N,), dtype, "b")
    return _struct(FlceLinearParams, M, K, N, _rows(x, M, K, dtype, "x"),
                   0 if res is None else _rows(res, M, N, dtype, "residual"),
                   _rows(y, M, N, dtype, "the output or its gradient"), _activation(activation),
                   b is not None, res is not None, dtype is torch.float16, dW_fp32, db_fp32)


def flce_linear_forward(x: torch.Tensor, W: torch.Tensor, b: Optional[torch.Tensor] = None,
                        residual: Optional[torch.Tensor] = None, *, activation: str = "none",
                        pre: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a(x W^T + b) + residual, [M, N] in x's type: one kernel from x to y.

    x [M, K] and W [N, K] are bf16 or fp16, K a multiple of 8; x's rows may be
    strided (a multiple of 8 elements). b [N]; residual and ``out`` [M, N] with
    rows of any pitch, ``out`` may be the residual itself. ``pre`` (an [M, N]
    tensor of x's type) receives z = x W^T + b for flce_linear_backward; a layer
    without an activation needs none. ``workspace``: as in flce_forward."""
    device = x.device
    if device.type == "cuda" and _elsewhere(device, stream):
        with _On(device, stream):
            return flce_linear_forward(x, W, b, residual, activation=activation, pre=pre, out=out,
                                       workspace=workspace)
    _operand(x)
    _weight(W)
    y = torch.empty((x.shape[0], W.shape[0]), dtype=x.dtype, device=device) if out is None else out
    lib, p, need, _ = _linear_params(x, W, b, residual, y, activation, False, False)
    if pre is not None:
        _dense(pre, y.shape, x.dtype, "pre")
    ws = None if need == 0 else _scratch(workspace, need, device)
    index = device.index
    st = lib.flce_linear_forward(p, x.data_ptr(), W.data_ptr(),
                                 None if b is None else b.data_ptr(),
                                 None if residual is None else residual.data_ptr(), y.data_ptr(),
                                 None if pre is None else pre.data_ptr(),
                                 None if ws is None else ws.data_ptr(), need, _error_word(index),
                                 _raw_stream(index))
    if st:
        raise FlceError(st, "flce_linear_forward")
    return y


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
    device = x.device
    if device.type == "cuda" and _elsewhere(device, stream):
        with _On(device, stream):
            return flce_linear_backward(dy, x, W, b, activation=activation, pre=pre,
                                        dW_dtype=dW_dtype, db_dtype=db_dtype, needs=needs,
                                        workspace=workspace)
    _operand(x)
    _weight(W)
    dtype, f32 = x.dtype, torch.float32
    if (dW_dtype is not f32 and dW_dtype is not dtype) or \
            (db_dtype is not f32 and db_dtype is not dtype):
        raise TypeError("flce: dW_dtype and db_dtype must be fp32 or x's dtype")
    lib, p, _, need = _linear_params(x, W, b, None, dy, activation, dW_dtype is f32,
                                     db_dtype is f32)
    z = None
    if activation != "none":
        if pre is None:
            raise ValueError("flce: the backward of a layer with an activation needs pre=")
        _dense(pre, dy.shape, dtype, "pre")
        z = pre.data_ptr()
    (M, K), N, index = x.shape, W.shape[0], device.index
    dx = torch.empty((M, K), dtype=dtype, device=device) if needs[0] else None
    dW = torch.empty((N, K), dtype=dW_dtype, device=device) if needs[1] else None
    db = torch.empty(N, dtype=db_dtype, device=device) if b is not None and needs[2] else None
    ws = _scratch(workspace, need, device)
    _done(lib.flce_linear_backward(p, dy.data_ptr(), x.data_ptr(), W.data_ptr(), z, _ptr(dx),
                                   _ptr(dW), _ptr(db), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _error_word(index), _raw_stream(index)),
          "flce_linear_backward")
    return dx, dW, db


# -------------------------------------------------------------------- gated
def _gated_params(x, Wg, Wu, h, activation, dW_fp32):
    """As _linear_params; h: the output, or the backward's dh."""
    M, K = x.shape
    F = Wg.shape[0]
    dtype = x.dtype
    if Wg.shape[1] != K:
        raise ValueError(f"flce: Wg must have shape [F, {K}], got {tuple(Wg.shape)}")
    _dense(Wg, (F, K), dtype, "Wg")
    _dense(Wu, (F, K), dtype, "Wu")
    return _struct(FlceGatedParams, M, K, F, _rows(x, M, K, dtype, "x"),
                   _rows(h, M, F, dtype, "h or its gradient"), _activation(activation),
                   dtype is torch.float16, dW_fp32)


def flce_gated_forward(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, *,
                       activation: str = "silu", pre: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a(x Wg^T) * (x Wu^T), [M, F] in x's type: both projections, the
    activation and the product in one kernel.

    x [M, K], Wg and Wu [F, K] are bf16 or fp16, K and F multiples of 8; the rows
    of x and ``out`` may be strided (a multiple of 8 elements). ``pre`` (a
    [2, M, F] tensor of x's type) receives both projections for
    flce_gated_backward. ``workspace``: as in flce_forward."""
    device = x.device
    if device.type == "cuda" and _elsewhere(device, stream):
        with _On(device, stream):
            return flce_gated_forward(x, Wg, Wu, activation=activation, pre=pre, out=out,
                                      workspace=workspace)
    _operand(x)
    _weight(Wg)
    h = torch.empty((x.shape[0], Wg.shape[0]), dtype=x.dtype, device=device) if out is None else out
    lib, p, need, _ = _gated_params(x, Wg, Wu, h, activation, False)
    if pre is not None:
        _dense(pre, (2,) + tuple(h.shape), x.dtype, "pre")
    ws = None if need == 0 else _scratch(workspace, need, device)
    index = device.index
    st = lib.flce_gated_forward(p, x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), h.data_ptr(),
                                None if pre is None else pre.data_ptr(),
                                None if ws is None else ws.data_ptr(), need, _error_word(index),
                                _raw_stream(index))
    if st:
        raise FlceError(st, "flce_gated_forward")
    return h


def flce_gated_backward(dh: torch.Tensor, x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                        pre: torch.Tensor, *, activation: str = "silu",
                        dW_dtype: torch.dtype = torch.float32, needs=(True, True),
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """dx [M, K] in x's type, dWg and dWu [F, K] (fp32 or x's type) of
    flce_gated_forward, whose ``pre`` it takes. ``needs``: whether to compute dx,
    and the weight gradients; what is not computed is None."""
    device = x.device
    if device.type == "cuda" and _elsewhere(device, stream):
        with _On(device, stream):
            return flce_gated_backward(dh, x, Wg, Wu, pre, activation=activation,
                                       dW_dtype=dW_dtype, needs=needs, workspace=workspace)
    _operand(x)
    _weight(Wg)
    if dW_dtype not in (torch.float32, x.dtype):
        raise TypeError("flce: dW_dtype must be fp32 or x's dtype")
    lib, p, _, need = _gated_params(x, Wg, Wu, dh, activation, dW_dtype is torch.float32)
    _dense(pre, (2,) + tuple(dh.shape), x.dtype, "pre")
    (M, K), F, index = x.shape, Wg.shape[0], device.index
    dx = torch.empty((M, K), dtype=x.dtype, device=device) if needs[0] else None
    dWg = torch.empty((F, K), dtype=dW_dtype, device=device) if needs[1] else None
    dWu = torch.empty((F, K), dtype=dW_dtype, device=device) if needs[1] else None
    ws = _scratch(workspace, need, device)
    _done(lib.flce_gated_backward(p, dh.data_ptr(), x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                                  pre.data_ptr(), _ptr(dx), _ptr(dWg), _ptr(dWu), _ptr(ws),
                                  0 if ws is None else ws.numel(), _error_word(index),
                                  _raw_stream(index)), "flce_gated_backward")
    return dx, dWg, dWu


# ------------------------------------------------------ gradient norm, clipping
def _is_dense(t: torch.Tensor) -> bool:
    """Whether the elements fill one stretch of memory, in whatever order."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n > 1):
        if stride != step:
            return False
        step *= size
    return True


_data_ptr, _numel = torch.Tensor.data_ptr, torch.Tensor.numel
_get_device, _is_contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous
_dtype_of = operator.attrgetter("dtype")


def _grad_arrays(grads: Sequence[torch.Tensor], out):
    """(device index, HOST arrays of addresses, element counts, types, destinations)."""
    try:
        types = array.array("i", map(_GRAD_TYPES.__getitem__, map(_dtype_of, grads)))
    except KeyError:
        raise TypeError("flce: gradients must be bf16, fp16 or fp32 CUDA tensors") from None
    index = grads[0].get_device()
    if index < 0:
        raise TypeError("flce: gradients must be CUDA tensors")
    if set(map(_get_device, grads)) != {index}:
        raise ValueError("flce: gradients must be on one device")
    if not all(map(_is_contiguous, grads)) and not all(map(_is_dense, grads)):
        raise ValueError("flce: gradients must be dense")
    outs = None
    if out is not None:
        if len(out) != len(grads):
            raise ValueError(f"flce: out must hold {len(grads)} tensors, got {len(out)}")
        if list(map(_dtype_of, out)) != list(map(_dtype_of, grads)) or \
                set(map(_get_device, out)) != {index}:
            raise TypeError("flce: out must match the gradients' types and device")
        for g, o in zip(grads, out):
            if o.shape != g.shape or (o.stride() != g.stride() and
                                      not (o.is_contiguous() and g.is_contiguous())):
                raise ValueError("flce: out must match the gradients' shapes and strides")
        outs = array.array("Q", map(_data_ptr, out))
    return (index, array.array("Q", map(_data_ptr, grads)), array.array("q", map(_numel, grads)),
            types, outs)


def _at(a) -> int:
    return a.buffer_info()[0]


def _grad_list(grads) -> list:
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if not grads:
        raise ValueError("flce: no gradients given")
    return grads


def flce_grad_norm(grads: Iterable[torch.Tensor], *, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The global 2-norm of all elements of ``grads`` (dense bf16, fp16 and fp32
    CUDA tensors of any shapes) as a 0-dim fp32 tensor."""
    grads = _grad_list(grads)
    device = grads[0].device
    if device.type == "cuda" and _elsewhere(device, stream):
        with _On(device, stream):
            return flce_grad_norm(grads, workspace=workspace)
    index, ptrs, numels, types, _ = _grad_arrays(grads, None)
    lib, n = _lib.load(), len(grads)
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws = _scratch(workspace, lib.flce_grad_norm_workspace_size(n), device)
    _done(lib.flce_grad_norm(n, _at(ptrs), _at(numels), _at(types), norm.data_ptr(), ws.data_ptr(),
                             ws.numel(), _raw_stream(index)), "flce_grad_norm")
    return norm


def flce_clip_grads(grads: Iterable[torch.Tensor], max_norm: float, *,
                    out: Optional[Sequence[torch.Tensor]] = None, eps: float = 1e-6,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scales ``grads`` by min(1, max_norm / (norm + eps)), in place or into
    ``out`` (tensors of the same shapes, types and strides), and returns their
    global norm before the scaling as a 0-dim fp32 tensor. Each tensor is given
    once. The scale is formed on the device: nothing is read back. A NaN norm
    makes every element NaN, an infinite one scales by 0."""
    grads = _grad_list(grads)
    out = None if out is None else list(out)
    device = grads[0].device
    if device.type == "cuda" and _elsewhere(device, stream):
        with _On(device, stream):
            return flce_clip_grads(grads, max_norm, out=out, eps=eps, workspace=workspace)
    index, ptrs, numels, types, outs = _grad_arrays(grads, out)
    lib, n = _lib.load(), len(grads)
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws = _scratch(workspace, lib.flce_grad_norm_workspace_size(n), device)
    _done(lib.flce_clip_grads(n, _at(ptrs), None if outs is None else _at(outs), _at(numels),
                              _at(types), float(max_norm), float(eps), norm.data_ptr(),
                              ws.data_ptr(), ws.numel(), _raw_stream(index)), "flce_clip_grads")
    return norm


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """flce_clip_grads over the ``.grad`` of ``parameters`` (those that have
    one), in place; the norm before the scaling, 0 where there is no gradient."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
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


class FusedLinearFunction(torch.autograd.Function):
    """Autograd form of the linear layer. It keeps x, and z where there is an activation."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation):
        pre = None
        if activation != "none" and any(ctx.needs_input_grad[:3]):
            pre = torch.empty(x.shape[0], weight.shape[0], dtype=x.dtype, device=x.device)
        y = flce_linear_forward(x, weight, bias, residual, activation=activation, pre=pre)
        ctx.save_for_backward(x, weight, bias, pre)
        ctx.activation = activation
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, pre = ctx.saved_tensors
        dx = dW = db = None
        if any(ctx.needs_input_grad[:3]):
            d = _usable(dy)
            dx, dW, db = flce_linear_backward(d, x, weight, bias, activation=ctx.activation,
                                              pre=pre, dW_dtype=weight.dtype, db_dtype=x.dtype,
                                              needs=ctx.needs_input_grad[:3])
        return dx, dW, db, dy if ctx.needs_input_grad[3] else None, None


class GatedLinearFunction(torch.autograd.Function):
    """Autograd form of the gated projection. It keeps x and both projections."""

    @staticmethod
    def forward(ctx, x, gate_weight, up_weight, activation):
        pre = None
        if any(ctx.needs_input_grad[:3]):
            pre = torch.empty(2, x.shape[0], gate_weight.shape[0], dtype=x.dtype, device=x.device)
        h = flce_gated_forward(x, gate_weight, up_weight, activation=activation, pre=pre)
        ctx.save_for_backward(x, gate_weight, up_weight, pre)
        ctx.activation = activation
        return h

    @staticmethod
    def backward(ctx, dh):
        x, Wg, Wu, pre = ctx.saved_tensors
        need_x, need_g, need_u = ctx.needs_input_grad[:3]
        dx, dWg, dWu = flce_gated_backward(_usable(dh), x, Wg, Wu, pre, activation=ctx.activation,
                                           dW_dtype=Wg.dtype, needs=(need_x, need_g or need_u))
        return dx, dWg if need_g else None, dWu if need_u else None, None


def fused_linear(x, weight, bias=None, residual=None, activation="none"):
    """activation(x weight^T + bias) + residual with gradients; x [..., K], weight
    [N, K], residual [..., N]. Inputs whose rows the kernels cannot read as they
    are (flce_linear_forward) are copied first."""
    x2 = _usable(x.reshape(-1, x.shape[-1]))
    r2 = None
    if residual is not None:
        r2 = residual.reshape(-1, weight.shape[0])
        if r2.stride(1) != 1 or r2.stride(0) < r2.shape[1]:
            r2 = r2.contiguous()
    y = FusedLinearFunction.apply(x2, weight, bias, r2, activation)
    return y.reshape(*x.shape[:-1], weight.shape[0])


def gated_linear(x, gate_weight, up_weight, activation="silu"):
    """activation(x gate_weight^T) * (x up_weight^T) with gradients; x [..., K],
    the weights [F, K]."""
    x2 = _usable(x.reshape(-1, x.shape[-1]))
    h = GatedLinearFunction.apply(x2, gate_weight, up_weight, activation)
    return h.reshape(*x.shape[:-1], gate_weight.shape[0])


class GatedFeedForward(torch.nn.Module):
    """x + W_down (a(W_gate x) * (W_up x)): the gated projection and the down
    projection that adds the residual stream, two kernels forward. ``inputs``
    (by default x) is what the block reads, such as the normed residual stream."""

    def __init__(self, hidden: int, features: int, activation: str = "silu",
                 dtype=torch.bfloat16, device=None):
        super().__init__()
        _activation(activation)
        self.activation = activation

        def weight(rows, cols):
            w = torch.empty(rows, cols, dtype=dtype, device=device)
            return torch.nn.Parameter(w.normal_(std=cols ** -0.5))

        self.gate, self.up = weight(features, hidden), weight(features, hidden)
        self.down = weight(hidden, features)

    def forward(self, x, inputs=None):
        h = gated_linear(x if inputs is None else inputs, self.gate, self.up, self.activation)
        return fused_linear(h, self.down, residual=x)
