"""The layer operators on whole numbers, where every sum is exact in fp32 and every output is the
correctly rounded one, bit for bit: a lost remainder, a partial sum rounded on its way, a tile
or slice added twice or left out shows in any shape. Every kernel form (block_plans.py) and the
long shapes; and sums of real numbers by their norm."""
import pytest
import torch

import block_plans as P
import linear_cross_entropy_gemm_gb300 as F
from test_gpu_block import LONG

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
# None of it may depend on how torch multiplies: its operands and sums are exact as well.
LONG_GATED = [(M, K, -(-N // 8) * 8) for M, K, N in LONG]


def whole(gen, *shape, most, dtype, density=1.0):
    t = torch.randint(-most, most + 1, shape, generator=gen, device="cuda").float()
    if density < 1.0:
        t *= torch.rand(shape, generator=gen, device="cuda") < density
    return t.to(dtype)


def equal(got, want, what):
    """want: exact in fp32; rounded once to the output's type."""
    want = want.to(got.dtype)
    if not torch.equal(got, want):
        bad = (got != want).nonzero()
        at = tuple(int(v) for v in bad[0])
        raise AssertionError(f"{what}: {len(bad)} of {got.numel()} differ, first at {at}: "
                             f"{got[at].item()}, not {want[at].item()}")


def check_linear(M, K, N, dtype, act):
    """|x|, |W|, |dy| <= 3: sums of 16384 products stay below 2^18, far beyond the 8 and 11 bits of
    the operands' types."""
    gen = torch.Generator(device="cuda").manual_seed(M + K + N)
    x, W, dy = (whole(gen, *s, most=3, dtype=dtype) for s in ((M, K), (N, K), (M, N)))
    b, r = whole(gen, N, most=9, dtype=dtype), whole(gen, M, N, most=9, dtype=dtype)
    z = x.float() @ W.float().t() + b.float()
    slope = (z > 0).float() if act == "relu" else torch.ones_like(z)
    dz = dy.float() * slope
    dx, dW, db = dz @ W.float(), dz.t() @ x.float(), dz.sum(0)
    for form in (dtype, torch.int16) if act == "relu" else (None,):
        pre = None if form is None else torch.empty(M, N, dtype=form, device="cuda")
        y = F.flce_linear_forward(x, W, b, r, activation=act, pre=pre)
        equal(y, z * slope + r.float(), "y")
        got = F.flce_linear_backward(dy, x, W, b, activation=act, pre=pre)
        for g, want, what in zip(got, (dx, dW, db), ("dx", "dW", "db")):
            equal(g, want, what)
    got = F.flce_linear_backward(dy, x, W, b, activation=act, pre=pre, dW_dtype=dtype, db_dtype=dtype)
    equal(got[1], dW, "dW in 16 bits")
    equal(got[2], db, "db in 16 bits")
    torch.cuda.synchronize()
    assert F.flce_read_device_error() == 0


def check_gated(M, K, N, dtype):
    """x of +-1 and W of 0, +-1 with so many zeros that |g| and |u| stay below 256: whole numbers
    that the fixed form keeps to 2^-14 of 256 and dg, du (dh of +-1, +-2) round to exactly."""
    gen = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = whole(gen, M, K, most=1, dtype=dtype)
    x[x == 0] = 1
    Wg, Wu = (whole(gen, N, K, most=1, dtype=dtype, density=min(1.0, 1500 / K)) for _ in range(2))
    dh = whole(gen, M, N, most=2, dtype=dtype)
    g, u = x.float() @ Wg.float().t(), x.float() @ Wu.float().t()
    assert float(g.abs().max()) <= 256 and float(u.abs().max()) <= 256
    a, slope = g.clamp(min=0), (g > 0).float()
    dg, du = dh.float() * u * slope, dh.float() * a
    want = (dg @ Wg.float() + du @ Wu.float(), dg.t() @ x.float(), du.t() @ x.float())
    for form in (dtype, torch.int16):
        pre = torch.empty(2, M, N, dtype=form, device="cuda")
        h = F.flce_gated_forward(x, Wg, Wu, activation="relu", pre=pre)
        equal(h, a * u, "h")
        got = F.flce_gated_backward(dh, x, Wg, Wu, pre, activation="relu")
        for v, w, what in zip(got, want, ("dx", "dWg", "dWu")):
            equal(v, w, what)
    equal(F.flce_gated_forward(x, Wg, Wu, activation="relu"), a * u, "h without kept values")
    got = F.flce_gated_backward(dh, x, Wg, Wu, pre, activation="relu", dW_dtype=dtype)
    equal(got[1], want[1], "dWg in 16 bits")
    equal(got[2], want[2], "dWu in 16 bits")
    torch.cuda.synchronize()
    assert F.flce_read_device_error() == 0


@pytest.mark.parametrize("shape", P.LINEAR + LONG, ids=str)
@pytest.mark.parametrize("act", ["none", "relu"])
def test_linear_is_exact_on_whole_numbers(shape, act):
    check_linear(*shape, BF16 if sum(shape) % 2 else FP16, act)


@pytest.mark.parametrize("shape", P.GATED + LONG_GATED, ids=str)
def test_gated_is_exact_on_whole_numbers(shape):
    check_gated(*shape, BF16 if sum(shape) % 16 else FP16)


@pytest.mark.parametrize("shape", P.LINEAR + LONG, ids=str)
def test_sums_of_real_numbers_by_their_norm(shape):
    """dW in fp32 without an activation has no rounding but its sum's: 2^-23 of the running sum for
    each step of 16 products at most. y and dx add one rounding."""
    M, K, N = shape
    gen = torch.Generator(device="cuda").manual_seed(M * 3 + K + N)
    x, W, dy = (torch.randn(*s, generator=gen, device="cuda").to(BF16) for s in ((M, K), (N, K), (M, N)))
    y = F.flce_linear_forward(x, W)
    dx, dW, _ = F.flce_linear_backward(dy, x, W)
    x64, W64, d64 = x.double(), W.double(), dy.double()
    for got, want, n, u in ((y, x64 @ W64.t(), K, 2.0 ** -8), (dx, d64 @ W64, N, 2.0 ** -8),
                            (dW, d64.t() @ x64, M, 2.0 ** -24)):
        limit = u + 2.0 ** -23 * (n / 16 + 2)
        assert float((got.double() - want).norm() / want.norm()) <= limit


@pytest.mark.parametrize("shape", [(37, 544, 232), (300, 2056, 96), (513, 96, 1032), (2049, 512, 1048)], ids=str)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("form", ["fixed", "relative"])
def test_gradients_end_to_end_by_their_norm(shape, dtype, form):
    """Forward and backward against 64 bits throughout. dz (dg, du) is off by its rounding u and by
    the kept value: slopes 2^-16 (1.13 at most), groups 2^-14 of their largest, which is at most 4 of
    their root mean square here, or 2^-11; dx by u more."""
    M, K, N = shape
    gen = torch.Generator(device="cuda").manual_seed(M)

    def normal(*s, std=1.0):
        return (torch.randn(s, generator=gen, device="cuda") * std).to(dtype)

    x, W, Wu, b, dy = normal(M, K), normal(N, K, std=K ** -0.5), normal(N, K, std=K ** -0.5), \
        normal(N, std=0.3), normal(M, N)
    u, sums = 2.0 ** -8 if dtype is BF16 else 2.0 ** -11, 2.0 ** -23 * (max(shape) / 8 + 2)
    store = dtype if form == "fixed" else torch.int16
    leaves = [t.double().requires_grad_() for t in (x, W, b)]
    z = leaves[0] @ leaves[1].t() + leaves[2]
    (torch.nn.functional.gelu(z)).backward(dy.double())
    pre = torch.empty(M, N, dtype=store, device="cuda")
    F.flce_linear_forward(x, W, b, activation="gelu", pre=pre)
    got = F.flce_linear_backward(dy, x, W, b, activation="gelu", pre=pre)
    for g, leaf, own in zip(got, leaves, (2 * u, u, 0.0)):
        err = float((g.double() - leaf.grad).norm() / leaf.grad.norm())
        assert err <= own + 2.0 ** -14 + sums, err
    leaves = [t.double().requires_grad_() for t in (x, W, Wu)]
    (torch.nn.functional.silu(leaves[0] @ leaves[1].t()) * (leaves[0] @ leaves[2].t())).backward(dy.double())
    pre = torch.empty(2, M, N, dtype=store, device="cuda")
    F.flce_gated_forward(x, W, Wu, pre=pre)
    got = F.flce_gated_backward(dy, x, W, Wu, pre)
    for g, leaf, own in zip(got, leaves, (2 * u, u, u)):
        err = float((g.double() - leaf.grad).norm() / leaf.grad.norm())
        assert err <= own + (2.0 ** -12 if form == "fixed" else 2.0 ** -11) + sums, err
