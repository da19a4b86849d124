"""Sampling where a comparison hangs on little: rows of infinities, distributions that the middles of
the histogram's bins misjudge, weights that cross a limit in their last bits. The same tokens as
the definition in 64 bits."""
import decimal
import math

import numpy as np
import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
import stream_reference as R

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")
UNWRITTEN = -7


def tokens_of(z, u, **kw):
    """The call's tokens, in a buffer that tells a token that was not written."""
    out = torch.full((z.shape[0],), UNWRITTEN, dtype=torch.int64, device="cuda")
    return F.flce_sample(z, u, out=out, **kw).tolist()


def check(z, u, **kw):
    zs = z.float().cpu()
    assert tokens_of(z, u, **kw) == [R.sample(zs[b], float(u[b]), **kw) for b in range(z.shape[0])]


def randoms(n, seed=0):
    return torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


# ---------------------------------------------------------------- infinities
def infinite_rows(B, V, infinities, dtype, seed=1):
    """Rows with so many +infinities at random places; and the rows whose weights they have."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(B, V, generator=g, device="cuda") * 3
    z[:, ::7] = -INF
    at = torch.stack([torch.randperm(V, generator=g, device="cuda")[:infinities] for _ in range(B)])
    z.scatter_(1, at, INF)
    return z.to(dtype), torch.where(z == INF, 0.0, -INF)


# One block for a row, and a cluster of them.
@pytest.mark.parametrize("B,V", [(1, 1), (4, 300), (2, 70000), (1, 1 << 18), (330, 2000)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_infinities_with_min_p(B, V, dtype):
    """+infinity leaves the others no weight, whatever min_p is."""
    for infinities in sorted({1, min(3, V), min(V, 1000)}):
        z, flat = infinite_rows(B, V, infinities, dtype)
        u = randoms(B, 2)
        for kw in (dict(min_p=0.05), dict(min_p=1.0), dict(min_p=1e-6, temperature=30.0)):
            want = tokens_of(flat, u)
            assert tokens_of(z, u, **kw) == want and UNWRITTEN not in want
        check(z[:4], u[:4], min_p=0.3, top_k=1200)


@pytest.mark.parametrize("infinities", [2, 40, 1500, 5000])
@pytest.mark.parametrize("B,V", [(330, 7000), (2, 131072)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_infinities_with_top_k_and_top_p(B, V, infinities, dtype):
    """They are equal weights: the limits keep the first ones of them."""
    z, flat = infinite_rows(B, V, infinities, dtype)
    u = randoms(B, 3)
    u[:2] = 1 - 2.0 ** -24
    for kw in (dict(top_p=0.5), dict(top_k=1200, top_p=0.5), dict(top_k=3000, top_p=0.25), dict(top_k=6000),
               dict(top_p=0.9, min_p=0.1), dict(top_p=0.01), dict(top_k=900, top_p=0.75)):
        check(z[:3], u[:3], **kw)
        want = tokens_of(flat, u, **kw)
        assert tokens_of(z, u, **kw) == want
        # A temperature above all changes nothing among equals.
        assert tokens_of(z, u, temperature=INF, **kw) == want


@pytest.mark.parametrize("B,V", [(330, 2000), (3, 70000)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_min_p_beside_masks(B, V, dtype):
    """min_p alone, from passes over the row: -infinity and the type's lowest value in most places, a row
    with one word left, one with nothing."""
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(B, V, generator=g, device="cuda") * 2
    z[torch.rand(B, V, generator=g, device="cuda") < 0.9] = -INF
    z[:, ::5] = torch.finfo(dtype).min
    z[0] = -INF
    z[1] = -INF
    z[1, V - 3] = -40.0
    z, u = z.to(dtype), randoms(B, 6)
    for kw in (dict(min_p=0.05), dict(min_p=1.0), dict(min_p=1e-9), dict(min_p=0.3, temperature=0.2)):
        check(z[:3], u[:3], **kw)
        got = tokens_of(z, u, **kw)
        assert got[:2] == [-1, V - 3] and UNWRITTEN not in got


# ---------------------------------------------------------- misjudged bins
def groups_row(groups, V, dtype, seed=4):
    """A row of (value, count) groups; the values of each at places of their own, in random order."""
    assert sum(n for _, n in groups) == V
    z = torch.cat([torch.full((n,), v, dtype=torch.float64) for v, n in groups]).to(dtype)
    assert all(float(torch.tensor(v, dtype=torch.float64).to(dtype).double()) == v for v, _ in groups) or dtype == FP32
    return z[torch.randperm(V, generator=torch.Generator().manual_seed(seed))].cuda()


def bins_apart(dtype):
    """Values in three neighbouring bins of 1/64 of a factor of 2, the first at its bin's low end, whose
    weight the bin's middle overestimates; (largest, the three, value of the rest, temperature)."""
    if dtype == FP32:
        b = math.log(2) / 64
        return 0.0, (-64.97 * b, -65.5 * b, -66.03 * b), -20.0, 1.0
    top, step, T = (1.0, 2.0 ** -8, 4.0) if dtype == BF16 else (8.0, 2.0 ** -8, 2.0)
    of_bin = {}
    for j in range(1, 100):
        of_bin.setdefault(int((top - (top - j * step)) * 64 / (T * math.log(2))), []).append(top - j * step)
    return top, (of_bin[3][-1], of_bin[4][len(of_bin[4]) // 2], of_bin[5][0]), -20.0 * T, T


@pytest.mark.parametrize("V,many,few", [(131072, 60000, 300), (8000, 3500, 100)], ids=str)
@pytest.mark.parametrize("top_k", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_a_bracket_that_is_too_high(dtype, top_k, V, many, few):
    """Between two groups of thousands lie a few words: the first guess of where the cut lies is just
    they, and the exact sums refute it. A few hundred of the second group are kept, not all."""
    top, (a, b, c), rest, T = bins_apart(dtype)
    groups = [(top, 1), (a, many), (b, few), (c, many), (rest, V - 1 - 2 * many - few)]
    z = groups_row(groups, V, dtype)
    k = 1 + 2 * many + few + (V - 1 - 2 * many - few) // 2 if top_k else 0
    value = [float(z.double().max()), *sorted(set(z.double().tolist()), reverse=True)[1:]]
    weights = [n * math.exp((v - value[0]) / T) for v, (_, n) in zip(value, groups)]
    if top_k:
        weights[-1] /= 2
    p = float(np.float32((sum(weights[:3]) + 0.001 * sum(weights)) / sum(weights)))
    u = torch.tensor([1 - 2.0 ** -24, 0.9999, 0.999, 0.75, 0.5, 0.25], device="cuda")
    check(z.expand(6, V).contiguous(), u, top_k=k, top_p=p, temperature=T)


def test_bins_narrower_than_a_step_of_the_logits():
    """Large logits at a small temperature: a step of fp32 is nearly two bins wide, and a bin's weight
    is that of its own middle, not of a logit rounded from it. The cut lies 32 words into the second group."""
    V, many, top, T = 131072, 10000, 127.0, 0.0003646422701422125
    step = 2.0 ** -17  # of fp32 in [64, 128)
    groups = [(top, 1), (top - 15 * step, many), (top - 16 * step, V - 1 - many)]
    z = torch.cat([torch.full((n,), v, dtype=FP32) for v, n in groups]).cuda()
    weights = [n * math.exp((v - top) / float(np.float32(T))) for v, n in groups]
    p = float(np.float32((weights[0] + 1.003 * weights[1]) / sum(weights)))
    u = torch.tensor([1 - 2.0 ** -24, 0.9995, 0.998, 0.5], device="cuda")
    check(z.expand(4, V).contiguous(), u, top_p=p, temperature=T)
    check(z.expand(4, V).contiguous(), u, top_k=V - 5, top_p=p, temperature=T)


def test_sums_by_2_to_the_x_far_from_0():
    """z / T of 2^25: the exponents of the words outside the list are off by up to 2, so their sum by
    the hardware's 2^x is not what decides. p is so near a multiple of one word's share that the others'
    weight of 2^-37 each keeps one word more."""
    V, listed = 1 << 20, 701
    top, T = np.float32(10.33804988861084), np.float32(4.428887336871412e-07)
    step = 2.0 ** -20  # of fp32 in [8, 16)
    low = float(top) - 12 * step
    z = torch.full((V,), low, dtype=FP32)
    at = torch.arange(listed) * (V // listed) + 5
    z[at] = float(top)
    others = (V - listed) * math.exp((low - float(top)) / float(T))
    # j words and a little less lie before p of the sum: word j is kept.
    found = [(j, p) for j in range(50, listed - 1) for p in [float(np.float32(j / (listed + 0.9 * others)))]
             if 0.03 * p * others < p * (listed + others) - j < 0.17 * p * others]
    assert len(found) >= 4
    u = torch.full((1,), 1 - 2.0 ** -24, device="cuda")
    for j, p in found[:8]:
        assert R.sample(z, float(u), temperature=float(T), top_p=p) == int(at[j])
        assert tokens_of(z.cuda()[None], u, temperature=float(T), top_p=p) == [int(at[j])]


# ------------------------------------------------------------ the weights
def nearly_equal(gap, most):
    """(m, n) up to `most` with m and n e^-gap nearly equal, and whether m is the larger: the best
    whose distance is above 2^-30 of them."""
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        r, best = (-decimal.Decimal(gap)).exp(), None
        x, (p0, q0), (p1, q1) = r, (0, 1), (1, 0)
        for _ in range(30):  # the continued fraction of e^-gap, and what lies between two of its terms
            a = int(x)
            for i in range(1, a + 1) if a < 50 else (1, a):
                m, n = i * p1 + p0, i * q1 + q0
                if m < 1 or m + n > most:
                    continue
                off = abs(m / (n * r) - 1)
                if off > decimal.Decimal(2) ** -30 and (best is None or off < best[0]):
                    best = off, m, n, m > n * r
            (p0, q0), (p1, q1) = (p1, q1), (a * p1 + p0, a * q1 + q0)
            if x == a or q1 > most:
                break
            x = 1 / (x - a)
    return best


@pytest.mark.parametrize("top,T", [(0.0, 1.0), (7.5, 1.0), (-3.25, 0.75), (900.0, 1.0), (9000.0, 1.0), (2.5, 0.000244140625)],
                         ids=str)
def test_a_weights_precision(top, T):
    """m words of one logit, then n of another, with sums apart by as little as 2^-30 of themselves: half
    of the whole lies on the right side. Each weight is right to 2^-32 of itself, two
    of them to 2^-31."""
    step = abs(float(np.spacing(np.float32(top if top else 1.0))))
    gaps = [round(g * T / step) * step for g in (0.011, 0.07, 0.3, 0.69, 0.7, 1.1, 1.9, 2.3)]
    tried = 0
    for gap in gaps:
        lower = np.float32(top - gap)
        found = nearly_equal(decimal.Decimal(float(top) - float(lower)) / decimal.Decimal(T), 1 << 20)
        if found is None or found[0] > decimal.Decimal(2) ** -26:
            continue
        tried += 1
        _, m, n, above = found
        z = torch.cat((torch.full((m,), top), torch.full((n,), float(lower)))).cuda()[None]
        got = tokens_of(z, torch.tensor([0.5], device="cuda"), temperature=T)
        assert got == [m - 1 if above else m], (gap, m, n)
        # The other way round.
        got = tokens_of(z.flip(1), torch.tensor([0.5], device="cuda"), temperature=T)
        assert got == [n if above else n - 1], (gap, m, n)
    assert tried >= 4
