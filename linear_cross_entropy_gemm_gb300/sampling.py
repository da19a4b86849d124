"""From the head's logits to tokens: sampling with temperature, top-k, top-p and min-p
from given random numbers.

    tokens = flce_sample(logits, u, temperature=0.8, top_k=50, top_p=0.9)
    tokens = fused_linear_sample(hidden, W, top_p=0.95)   # the head's product, then the draw

The functions only check and marshal arguments; every step runs in the library's
kernels, on the current CUDA stream, without a synchronisation.
"""
from __future__ import annotations

from typing import Optional, Union

import torch

from .block import _On, _calls, flce_linear_forward

Setting = Union[float, torch.Tensor]


def flce_sample(logits: torch.Tensor, u: torch.Tensor, *, temperature: Setting = 1.0,
                top_k: Union[int, torch.Tensor] = 0, top_p: Setting = 1.0, min_p: Setting = 0.0,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A token (int64) for each row of logits [B, V], from a random number u [B] (fp32, in
    [0, 1)) for each.

    logits are bf16, fp16 or fp32 with rows of any pitch, V up to 2^20. With
    w = exp((z - max z) / temperature) and the words ordered by falling logit, equal ones
    by index: ``top_k`` keeps the first k (0: all), ``top_p`` those of them before which
    less than p of their sum lies (1: all), ``min_p`` those of them with w >= min_p. The
    token is the lowest index at which the w of the words kept, summed in the order of the
    vocabulary, exceed u times their sum. temperature 0 takes the first word of the order.

    Each setting is a number, or a tensor [B] with one for each row (fp32; top_k int32).
    A logit of -inf is never chosen; a row without any other, or with a NaN, gives -1. The
    sums are exact, so a row's token does not depend on the batch. Numbers
    of torch.rand are multiples of 2^-24: a word whose stretch of the sum holds none is never drawn."""
    if stream is not None:
        with _On(logits.device, stream):
            return _calls.sample(logits, u, temperature, top_k, top_p, min_p, out)
    return _calls.sample(logits, u, temperature, top_k, top_p, min_p, out)


def fused_linear_sample(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
                        u: Optional[torch.Tensor] = None, temperature: Setting = 1.0,
                        top_k: Union[int, torch.Tensor] = 0, top_p: Setting = 1.0,
                        min_p: Setting = 0.0, logit_scale: float = 1.0) -> torch.Tensor:
    """The loss head's serving side: tokens for the last hidden states x [B, H] of the
    distribution that FusedLinearCrossEntropyLoss trains with this weight, bias and
    ``logit_scale`` (above 0), sampled as in flce_sample. The logits are rounded to x's
    type. ``u``: by default drawn from the device's generator."""
    if not logit_scale > 0:
        raise ValueError(f"flce: sampling needs a logit_scale above 0, got {logit_scale!r}")
    logits = flce_linear_forward(x, weight, bias)
    if u is None:
        u = torch.rand(x.shape[0], dtype=torch.float32, device=x.device)
    if logit_scale != 1.0:
        temperature = temperature / logit_scale
    return flce_sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
