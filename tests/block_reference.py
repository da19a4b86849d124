"""Plain 64-bit forms of the layer operators and the error bounds of their kernels.

Bounds. Operands are exact 16-bit values, products are exact in fp32, and a sum
of n of them in fp32, in any order and with truncating adds, is off by at most
n 2^-23 times the sum of their absolute values. An output rounded to its type
adds u |value| (u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32), a little more where
that type is subnormal. Activations are Lipschitz with constant 1.2 and are
evaluated to 2^-18 of their argument's size.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
ADD = 2.0 ** -23
ACT = 2.0 ** -18
LIP = 1.2


def act(z, name):
    """a(z), a'(z)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z), (z > 0).to(z.dtype)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * c * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(z)
    return (z * p, p * (1 + z * (1 - p))) if name == "silu" else (p, p * (1 - p))


def rounded(value, off, dtype):
    """Bound of an output of `dtype` whose unrounded value is off by at most `off`."""
    u = UNIT[dtype]
    return off * (1 + u) + u * value.abs() + TINY[dtype]


def linear(x, W, b, r, name):
    """(z, bound), (y, bound)."""
    dt = x.dtype
    x64, W64 = x.double(), W.double()
    size = x64.abs() @ W64.abs().t()
    z = x64 @ W64.t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    off = (x.shape[1] + 1) * ADD * size
    y, _ = act(z, name)
    y_off = off if name == "none" else LIP * off + ACT * (z.abs() + (1.0 if name == "sigmoid" else 0.0))
    if r is not None:
        y_off = y_off + ADD * (y.abs() + r.double().abs())
        y = y + r.double()
    return (z, rounded(z, off, dt)), (y, rounded(y, y_off, dt))


def product(a, a_off, b, dtype):
    """a b with a known up to a_off (elementwise): value and bound as `dtype`."""
    n = a.shape[1]
    v = a @ b
    off = a_off @ b.abs() + n * ADD * ((a.abs() + a_off) @ b.abs())
    return v, rounded(v, off, dtype)


def linear_grad(dy, x, W, pre, name, dW_dtype, db_dtype):
    """(dx, bound), (dW, bound), (db, bound) from the kept z."""
    dt = x.dtype
    slope = act(pre.double(), name)[1] if name != "none" else 1.0
    dz = dy.double() * slope
    raw = torch.zeros_like(dz) if name == "none" else 4 * ACT * dy.double().abs() * LIP
    dz_off = torch.zeros_like(dz) if name == "none" else rounded(dz, raw, dt)
    dx = product(dz, dz_off, W.double(), dt)
    dW = product(dz.t().contiguous(), dz_off.t().contiguous(), x.double(), dW_dtype)
    db = dz.sum(0)
    db_off = raw.sum(0) + dz.shape[0] * ADD * dz.abs().sum(0)
    return dx, dW, (db, rounded(db, db_off, db_dtype))


def gated(x, Wg, Wu, name):
    """(g, bound), (u, bound), (h, bound)."""
    (g, gb), _ = linear(x, Wg, None, None, "none")
    (u, ub), _ = linear(x, Wu, None, None, "none")
    K = (x.shape[1] + 1) * ADD
    g_off, u_off = (K * (x.double().abs() @ w.double().abs().t()) for w in (Wg, Wu))
    a, _ = act(g, name)
    a_off = g_off if name == "none" else LIP * g_off + ACT * (g.abs() + (1.0 if name == "sigmoid" else 0.0))
    h = a * u
    off = a_off * u.abs() + (a.abs() + a_off) * u_off + ADD * h.abs()
    return (g, gb), (u, ub), (h, rounded(h, off, x.dtype))


def gated_grad(dh, x, Wg, Wu, pre, name, dW_dtype):
    """(dx, bound), (dWg, bound), (dWu, bound) from the kept projections."""
    dt = x.dtype
    g, u, d = pre[0].double(), pre[1].double(), dh.double()
    a, slope = act(g, name)
    dg, du = d * u * slope, d * a
    dg_off = rounded(dg, 4 * ACT * LIP * (d * u).abs(), dt)
    du_off = rounded(du, 2 * ACT * d.abs() * (g.abs() + 1), dt)
    both, both_off = torch.cat((dg, du), 1), torch.cat((dg_off, du_off), 1)
    dx = product(both, both_off, torch.cat((Wg, Wu), 0).double(), dt)
    dWg = product(dg.t().contiguous(), dg_off.t().contiguous(), x.double(), dW_dtype)
    dWu = product(du.t().contiguous(), du_off.t().contiguous(), x.double(), dW_dtype)
    return dx, dWg, dWu


def assert_within(got, want, what):
    value, bound = want
    assert got.shape == value.shape, f"{what}: shape {tuple(got.shape)}"
    d = (got.double() - value).abs()
    over = d - bound
    if not bool((over <= 0).all()):
        at = int(torch.nan_to_num(over, nan=math.inf).argmax())
        raise AssertionError(f"{what}: element {at}: got {got.reshape(-1)[at].item()}, want "
                             f"{value.reshape(-1)[at].item()} within {bound.reshape(-1)[at].item()}")
