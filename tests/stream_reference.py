"""The operators on the residual stream, and sampling, in 64 bits, with bounds on what fp32
arithmetic and one rounding of each output may be off."""
import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ----------------------------------------------------------------- dropout
def philox(counter, key):
    """Philox4x32-10 on Python's whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def factors(M, H, p, seed, offset=0, row0=0):
    """D(x) = factor x, 64-bit on the GPU; the generator in numpy's 64-bit whole numbers."""
    t = math.floor(p * 65536 + 0.5)
    if t == 0:
        return torch.ones((), dtype=torch.float64, device="cuda")
    seed, offset = seed % 2 ** 64, offset % 2 ** 64
    groups, m = -(-H // 8), np.uint64(0xFFFFFFFF)
    c0 = np.broadcast_to(np.arange(groups, dtype=np.uint64)[None, :], (M, groups))
    c1 = np.broadcast_to((np.arange(M, dtype=np.uint64) + np.uint64(row0))[:, None], (M, groups))
    c2 = np.full((M, groups), offset & 0xFFFFFFFF, np.uint64)
    c3 = np.full((M, groups), offset >> 32, np.uint64)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    s = np.uint64(32)
    for _ in range(10):
        a, b = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = (b >> s) ^ c1 ^ np.uint64(k0), b & m, (a >> s) ^ c3 ^ np.uint64(k1), a & m
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    halves = [v for c in (c0, c1, c2, c3) for v in (c & np.uint64(0xFFFF), c >> np.uint64(16))]
    bits = np.stack(halves, -1).reshape(M, groups * 8)[:, :H]
    keep = torch.from_numpy((bits >= t).astype(np.float64)).cuda()
    return keep * (65536.0 / max(1, 65536 - t))


def dropped_sum(x, r, f):
    """(r + D(x), bound of its fp32 error): the scale's and the product's rounding, the sum's."""
    d = torch.where(f == 0, 0.0, x.double() * f)
    h = d if r is None else d + r.double()
    return h, 2 * U * d.abs() + U * h.abs()


# -------------------------------------------------------------------- norm
def norm(x, w, r, eps, f):
    """h, its error, rstd, y and y's error before the rounding to its type."""
    h, dh = dropped_sum(x, r, f)
    H = h.shape[-1]
    rstd = (h.square().mean(-1) + eps).rsqrt()
    w64 = torch.ones(H, dtype=torch.float64, device=h.device) if w is None else w.double()
    y = h * rstd[:, None] * w64
    # A thread adds at most 32 squares, the block ten times more: 42 roundings of a positive
    # sum, the errors of h twice in a square; half of that through the root; the division, eps,
    # the root (2 units in the last place = 4 half steps) and two products.
    rel = (42 + 4) / 2 * U + (1 + 1 + 4 + 2) * U
    return h, dh, rstd, y, rel * y.abs() + dh * (rstd[:, None] * w64.abs())


def norm_grad(dy, h, w, rstd, dh, f):
    """dresidual, dx, dW and their fp32 errors, from the given h and rstd."""
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    M, H = h.shape
    w64 = torch.ones(H, dtype=torch.float64, device=h.device) if w is None else w.double()
    g, xhat = dy * w64, h * rstd
    c = (g * xhat).mean(-1, keepdim=True)
    c_err = 46 * U * (g * xhat).abs().mean(-1, keepdim=True)
    e = rstd * (g - xhat * c)
    err = rstd * (3 * U * g.abs() + 5 * U * (xhat * c).abs() + xhat.abs() * c_err)
    if dh is not None:
        e = e + dh.double()
    err = err + 2 * U * e.abs()
    dW = (dy * xhat).sum(0)
    dW_err = (M + 2) * U * (dy * xhat).abs().sum(0)
    return e, err, e * f, (err + 2 * U * e.abs()) * f, dW, dW_err


def assert_near(got, want, err, what=""):
    """|got - want| within err and one rounding to got's type."""
    t = got.dtype
    tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps  # one step below the normal numbers
    limit = err + half_step(t) * (want.abs() + err) + tiny
    off = (got.double() - want).abs()
    bad = ~(off <= limit)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} values off, first at {i}: {float(got[i])} for "
                             f"{float(want[i])}, allowed {float(limit[i]):.3e}")


# ---------------------------------------------------------------- sampling
def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row by the definition, in 64 bits: z a list or tensor of logits as they are."""
    z = torch.as_tensor(z).double().cpu().numpy()
    V = len(z)
    if np.isnan(z).any() or not (z > -np.inf).any():
        return -1
    order = np.lexsort((np.arange(V), -z))
    order = order[z[order] > -np.inf]
    top = z[order[0]]
    if not temperature > 0 or top_k == 1 or not top_p > 0:
        return int(order[0])
    with np.errstate(invalid="ignore"):
        w = np.where(z[order] == top, 1.0, np.exp((z[order] - top) / float(temperature)))
    if 0 < top_k < len(order):
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        n = max(1, int((before < float(top_p) * w.sum()).sum()))
        order, w = order[:n], w[:n]
    keep = w >= min(max(float(min_p), 0.0), 1.0)
    order, w = order[keep], w[keep]
    at = np.argsort(order)
    order, w = order[at], w[at]
    sums = np.cumsum(w)
    target = min(max(float(u), 0.0), 1.0 - 2.0 ** -53) * sums[-1]
    return int(order[np.searchsorted(sums, target, side="right")])
