"""Plain 64-bit forms of the layer operators and the error bounds of their kernels.

Bounds. Operands are exact 16-bit values, products are exact in fp32, and a sum
of n of them in fp32, in any order and with truncating adds, is off by at most
n 2^-23 times the sum of their absolute values. An output rounded to its type
adds u |value| (u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32), a little more where
that type is subnormal. Activations and their slopes are Lipschitz with constant 1.2 and are
evaluated to 2^-18 of their argument's size and of 1. What the forward keeps: slopes in
steps of 2^-15, and groups of 8 values within 2^-14 of the group's largest.
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


def sums(x, W, b=None):
    """x W^T + b and how far off it may be."""
    x64, W64 = x.double(), W.double()
    z, size = x64 @ W64.t(), x64.abs() @ W64.abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    return z, (x.shape[1] + 1) * ADD * size


def activated(z, off, name):
    """(a(z), its bound), (a'(z), its bound) of a z that is off by at most `off`."""
    v, slope = act(z, name)
    if name == "none":
        return (v, off), (slope, torch.zeros_like(z))
    v_off = LIP * off + ACT * (z.abs() + 1.0)
    s_off = LIP * off + 4 * ACT
    if name == "relu":
        s_off = (z.abs() <= off).double()
    return (v, v_off), (slope, s_off)


def linear(x, W, b, r, name):
    """(a'(z) as kept, bound), (y, bound)."""
    z, off = sums(x, W, b)
    (y, y_off), (slope, s_off) = activated(z, off, name)
    if r is not None:
        y_off = y_off + ADD * (y.abs() + r.double().abs())
        y = y + r.double()
    return (slope, s_off + 2.0 ** -15), (y, rounded(y, y_off, x.dtype))


def codes(pre):
    return pre.view(torch.int16).to(torch.int64) & 0xFFFF


def kept_slopes(pre):
    q = codes(pre)
    return torch.where(q == 65535, math.nan, q.double() / 32768 - 0.25)


def kept_groups(pre):
    c = codes(pre).reshape(-1, 8)
    eb = sum((c[:, j] & 1) << j for j in range(8))
    q = ((c ^ 0x8000) - 0x8000) >> 1
    unit = torch.where(eb == 255, math.nan, torch.ldexp(torch.full_like(eb, 1, dtype=torch.float64), eb - 140))
    return (q.double() * unit[:, None] * (16384 / 16383)).reshape(pre.shape)


def group_off(v, off):
    """Bound of kept values v that are off by at most `off` before they are kept."""
    most = (v.abs() + off).reshape(-1, 8).amax(1, keepdim=True).expand(-1, 8).reshape(v.shape)
    return off + 2.0 ** -14 * most + 2.0 ** -112


def product(a, a_off, b, dtype):
    """a b with a known up to a_off (elementwise): value and bound as `dtype`."""
    n = a.shape[1]
    v = a @ b
    off = a_off @ b.abs() + n * ADD * ((a.abs() + a_off) @ b.abs())
    return v, rounded(v, off, dtype)


def linear_grad(dy, x, W, slope, dW_dtype, db_dtype):
    """(dx, bound), (dW, bound), (db, bound) from the kept slopes (None: all 1)."""
    dt = x.dtype
    dz, raw = dy.double(), torch.zeros_like(dy, dtype=torch.float64)
    dz_off = raw
    if slope is not None:
        dz = dz * slope
        raw = ADD * dz.abs()
        dz_off = rounded(dz, raw, dt)
    dx = product(dz, dz_off, W.double(), dt)
    dW = product(dz.t().contiguous(), dz_off.t().contiguous(), x.double(), dW_dtype)
    db = dz.sum(0)
    db_off = raw.sum(0) + dz.shape[0] * ADD * dz.abs().sum(0)
    return dx, dW, (db, rounded(db, db_off, db_dtype))


def gated(x, Wg, Wu, name):
    """(a(g) as kept, bound), (u a'(g) as kept, bound), (h, bound)."""
    (g, g_off), (u, u_off) = sums(x, Wg), sums(x, Wu)
    (a, a_off), (slope, s_off) = activated(g, g_off, name)

    def times_u(v, off):
        p = v * u
        return p, off * u.abs() + (v.abs() + off) * u_off + ADD * p.abs()

    (h, h_off), (cross, c_off) = times_u(a, a_off), times_u(slope, s_off)
    return (a, group_off(a, a_off)), (cross, group_off(cross, c_off)), (h, rounded(h, h_off, x.dtype))


def gated_grad(dh, x, Wg, Wu, val, cross, dW_dtype):
    """(dx, bound), (dWg, bound), (dWu, bound) from the kept values."""
    dt, d = x.dtype, dh.double()
    dg, du = d * cross, d * val
    dg_off, du_off = (rounded(t, 2 * ADD * t.abs(), dt) for t in (dg, du))
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
