"""The layer operators where they could go wrong unseen: outputs that nothing writes, saturated
activations, features of very different size, infinities, what a call leaves to autograd."""
import ctypes

import pytest
import torch

import block_reference as R
import linear_cross_entropy_gemm_gb300 as F
from linear_cross_entropy_gemm_gb300 import _lib

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def randn(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape, std=1.0, dtype=BF16: (
        torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# ------------------------------------------------------------------ empty lists
@pytest.mark.parametrize("count", [0, 1, 3, 70, 300, 1100])
def test_clip_writes_the_norm_of_no_elements(count):
    """Through the C ABI, into a norm that holds NaN before the call."""
    lib = _lib.load()
    ptrs, numel = (ctypes.c_void_p * max(count, 1))(), (ctypes.c_int64 * max(count, 1))()
    types = (ctypes.c_int32 * max(count, 1))()
    ws = torch.empty(lib.flce_grad_norm_workspace_size(count), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for clip in (False, True):
        norm = torch.full((), float("nan"), device="cuda")
        tail = (norm.data_ptr(), ws.data_ptr(), ws.numel(), stream)
        if clip:
            status = lib.flce_clip_grads(count, ptrs, None, numel, types, 1.0, 1e-6, *tail)
        else:
            status = lib.flce_grad_norm(count, ptrs, numel, types, *tail)
        assert status == 0 and float(norm) == 0.0


def test_clip_of_empty_tensors_returns_zero():
    """The allocator's small blocks hold NaN when the call takes one for its result."""
    empty = torch.empty(0, device="cuda")
    blocks = [torch.full((128,), float("nan"), device="cuda") for _ in range(64)]
    del blocks
    assert float(F.flce_clip_grads([empty, empty], 1.0)) == 0.0
    p = torch.nn.Parameter(torch.empty(0, 4, device="cuda"))
    p.grad = torch.empty(0, 4, device="cuda")
    blocks = [torch.full((128,), float("nan"), device="cuda") for _ in range(64)]
    del blocks
    assert float(F.clip_grad_norm_([p], 1.0)) == 0.0


# -------------------------------------------------------- saturated activations
def one_by_one(z, dtype):
    """x and W whose product holds exactly the values z (rounded to dtype) in column 0."""
    x = torch.zeros(z.numel(), 8, dtype=dtype, device="cuda")
    x[:, 0] = z.to(dtype)
    return x, torch.eye(8, dtype=dtype, device="cuda")


def gelu64(z):
    """z Phi(z), with Phi's tail from erfcx."""
    x = -z / 2 ** 0.5
    return z * 0.5 * torch.special.erfcx(x) * torch.exp(-x * x)


@pytest.mark.parametrize("rows", ["few", "many"])
def test_gelu_keeps_its_negative_tail(rows):
    """bf16 holds gelu(-12) = -2e-32: relative to the output's rounding of 2^-8 (it is below
    2^-126 only under z = -13), the fit is off by 8e-5 and e^(-z^2 / 2) by the fp32 rounding of
    an exponent of at most 104, 104 2^-24."""
    z = torch.linspace(-12, -2, 60 if rows == "few" else 600, device="cuda")
    x, W = one_by_one(z, BF16)
    y = F.flce_linear_forward(x, W, activation="gelu")[:, 0].double()
    want = gelu64(x[:, 0].double())
    assert bool(((y - want).abs() <= (2.0 ** -8 + 8e-5 + 2 * 104 * 2.0 ** -24) * want.abs()).all())


# Kept slopes in the relative form: off by 2^-10 of the slope (where it is above 2^-6 by 2^-16),
# by 2^-54 below 2^-44. An activation's slope at a given z is evaluated to 2^-14 of itself there
# (gelu's fit 8e-5 of a part of it; exponents up to 200 in fp32).
KEPT, FLOOR, EVAL = 2.0 ** -10, 2.0 ** -54, 2.0 ** -14
SATURATED = [("silu", -30.0, -2.5), ("sigmoid", -30.0, -2.5), ("sigmoid", 2.5, 30.0), ("gelu", -9.0, -2.5),
             ("gelu_tanh", -9.0, -2.5)]


def slope64(z, act):
    """a'(z), every term formed without cancellation for z below -1.5 (and for sigmoid anywhere)."""
    if act == "sigmoid":
        return torch.sigmoid(z) * torch.sigmoid(-z)
    if act == "silu":
        return torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        x = -z / 2 ** 0.5
        return torch.exp(-x * x) * (0.5 * torch.special.erfcx(x) + z / (2 * torch.pi) ** 0.5)
    c = (2 / torch.pi) ** 0.5
    w = 2 * c * (z + 0.044715 * z ** 3)
    p, q = torch.sigmoid(w), torch.sigmoid(-w)
    return p * (1 + z * q * 2 * c * (1 + 3 * 0.044715 * z * z))


@pytest.mark.parametrize("act,lo,hi", SATURATED)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M", [40, 700])
def test_saturated_units_keep_their_gradients(act, lo, hi, dtype, M):
    x, W = one_by_one(torch.linspace(lo, hi, M, device="cuda"), dtype)
    z = x[:, 0].double()
    scale = 512.0  # keeps fp16's gradients away from its smallest numbers
    dy = torch.full((M, 8), scale, dtype=dtype, device="cuda")
    want = scale * slope64(z, act)
    u = R.UNIT[dtype]
    size, floor = want.abs(), scale * FLOOR
    pre = torch.empty(M, 8, dtype=torch.int16, device="cuda")
    F.flce_linear_forward(x, W, W[0], activation=act, pre=pre)
    x0 = x.clone()
    x0[:, 0] -= 1  # the bias is 1 in column 0
    F.flce_linear_forward(x0, W, W[0], activation=act, pre=pre)
    z0 = x0[:, 0].double() + 1
    want0 = scale * slope64(z0, act)
    db = F.flce_linear_backward(dy, x0, W, W[0], activation=act, pre=pre)[2]
    total = want0.sum()
    assert abs(float(db[0]) - float(total)) <= float(
        (KEPT + EVAL + M * 2.0 ** -23) * want0.abs().sum() + M * floor)
    leaf = x.clone().requires_grad_()
    y = F.fused_linear(leaf, W, activation=act, keep="relative")
    y.backward(dy)
    got = leaf.grad[:, 0].double()
    # dz, then dx, is rounded.
    bound = (2 * u + KEPT + EVAL) * (1 + u) * size + floor + 2 * R.TINY[dtype]
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu_tanh"])
@pytest.mark.parametrize("M", [9, 300])
def test_units_far_below_zero_train(act, M):
    """Biases of -14 to -5: dz, dW and db against 64 bits, relative to their own size. z is off by
    its fp32 sum, and the slope of these activations by at most 12 times as much of itself."""
    n = randn(M)
    K, N = 64, 72
    x, W, dy = n(M, K), n(N, K, std=0.01), n(M, N)
    b = torch.linspace(-14 if act != "gelu_tanh" else -6, -5, N, device="cuda").to(BF16)
    pre = torch.empty(M, N, dtype=torch.int16, device="cuda")
    F.flce_linear_forward(x, W, b, activation=act, pre=pre)
    dx, dW, db = F.flce_linear_backward(dy, x, W, b, activation=act, pre=pre)
    z, z_off = R.sums(x, W, b)
    dz = dy.double() * slope64(z, act)
    off = (KEPT + EVAL + 12 * z_off) * dz.abs() + FLOOR * dy.double().abs()
    u = R.UNIT[BF16]
    assert bool(((db.double() - dz.sum(0)).abs() <= off.sum(0) + M * R.ADD * dz.abs().sum(0)).all())
    off = off * (1 + u) + u * dz.abs()
    R.assert_within(dW, R.product(dz.t(), off.t(), x.double(), FP32), "dW")
    R.assert_within(dx, R.product(dz, off, W.double(), BF16), "dx")


def test_kept_forms_agree_where_units_are_not_saturated():
    """The relative form's codes are the fixed form's, and with them every gradient."""
    n = randn(3)
    x, W, dy = n(300, 64), n(77, 64, std=0.125), n(300, 77)
    x[7, 3] = float("nan")
    for act in ("silu", "gelu", "gelu_tanh", "relu", "none"):
        fixed, relative = (torch.empty(300, 77, dtype=t, device="cuda") for t in (BF16, torch.int16))
        F.flce_linear_forward(x, W, activation=act, pre=fixed)
        F.flce_linear_forward(x, W, activation=act, pre=relative)
        slopes = R.kept_slopes(fixed)
        same = ~((slopes.abs() < 2.0 ** -6) & (x.double() @ W.double().t() < -1.9))
        assert torch.equal(fixed.view(torch.int16)[same], relative[same]) and bool(same.any())
        assert bool(R.kept_slopes(relative)[7].isnan().all()) == (act not in ("relu", "none"))


# ---------------------------------------------------- infinities in kept values
@pytest.mark.parametrize("M", [5, 50, 300])
@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=str)
@pytest.mark.parametrize("form", [BF16, torch.int16], ids=["fixed", "relative"])
def test_a_bad_feature_stays_in_its_row_of_the_weight_gradients(M, value, form):
    """A weight row with an infinity or NaN makes u a'(g) of its own feature non-finite in every
    token, and nothing of its seven neighbours'. Those are compared with 64 bits: each dg and
    du is off by its rounding and the kept value's 2^-14 of the group's largest (the relative
    form's 2^-11 of its own size)."""
    n = randn(M)
    x, Wg, Wu, dh = n(M, 64), n(72, 64, std=0.125), n(72, 64, std=0.125), n(M, 72)
    Wu[11, 5] = value
    pre = torch.empty(2, M, 72, dtype=form, device="cuda")
    F.flce_gated_forward(x, Wg, Wu, pre=pre)
    dx, dWg, dWu = F.flce_gated_backward(dh, x, Wg, Wu, pre)
    good = torch.arange(72, device="cuda") != 11
    assert not bool(dx.isfinite().any()) and not bool(dWg[11].isfinite().any())
    x64, d64 = x.double(), dh.double()
    g, u = x64 @ Wg.double().t(), x64 @ Wu.double().t()
    p = torch.sigmoid(g)
    u[:, 11] = 0
    most = [t.abs().reshape(M, 9, 8).amax(2).repeat_interleave(8, 1)
            for t in (u * p * (1 + g * (1 - p)), g * p)]
    for got, kept, size, rows in ((dWg, u * p * (1 + g * (1 - p)), most[0], good),
                                  (dWu, g * p, most[1], torch.ones_like(good))):
        d = d64 * kept
        kept_off = 2.0 ** -14 * size if form is BF16 else 2.0 ** -11 * kept.abs() + 2.0 ** -24 * size
        off = 2.0 ** -8 * d.abs() + 1.01 * d64.abs() * kept_off + 2.0 ** -16 * d64.abs()
        bound = off.t() @ x64.abs() + M * 2.0 ** -23 * (d.abs().t() @ x64.abs())
        err = (got.double() - d.t() @ x64).abs()
        assert bool((err <= bound)[rows].all())


# ------------------------------------------- kept values of very different size
def relative_off(v, off):
    """Bound of a kept value v of the relative form that is off by at most `off` before."""
    size = v.abs() + off
    most = size.reshape(-1, 8).amax(1, keepdim=True).expand(-1, 8).reshape(v.shape)
    return off + 2.0 ** -11 * size + 2.0 ** -24 * most + 2.0 ** -140


def gated_relative(x, Wg, Wu, act):
    """(a(g), bound), (u a'(g), bound) of the kept values in the relative form."""
    (g, g_off), (u, u_off) = R.sums(x, Wg), R.sums(x, Wu)
    (a, a_off), (slope, s_off) = R.activated(g, g_off, act)
    cross = u * slope
    c_off = s_off * u.abs() + (slope.abs() + s_off) * u_off + R.ADD * cross.abs()
    return (a, relative_off(a, a_off)), (cross, relative_off(cross, c_off))


def check_gated_gradients(got, x, Wg, Wu, dh, act, dW_dtype):
    """Against 64 bits, not against what the kernels kept."""
    dt, d = x.dtype, dh.double()
    (a, a_off), (cross, c_off) = gated_relative(x, Wg, Wu, act)
    dg, du = d * cross, d * a
    dg_off = R.rounded(dg, d.abs() * c_off + R.ADD * dg.abs(), dt)
    du_off = R.rounded(du, d.abs() * a_off + R.ADD * du.abs(), dt)
    both, both_off = torch.cat((dg, du), 1), torch.cat((dg_off, du_off), 1)
    R.assert_within(got[0], R.product(both, both_off, torch.cat((Wg, Wu)).double(), dt), "dx")
    R.assert_within(got[1], R.product(dg.t(), dg_off.t(), x.double(), dW_dtype), "dWg")
    R.assert_within(got[2], R.product(du.t(), du_off.t(), x.double(), dW_dtype), "dWu")
    return dg.t() @ x.double(), du.t() @ x.double()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
@pytest.mark.parametrize("M,K,N", [(1, 64, 8), (5, 64, 72), (50, 136, 264), (300, 200, 136)])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_gated_gradients_of_the_relative_form(act, M, K, N, dtype):
    n = randn(M + K + N)
    x, Wg, Wu = n(M, K, dtype=dtype), n(N, K, std=K ** -0.5, dtype=dtype), n(N, K, std=K ** -0.5, dtype=dtype)
    dh = n(M, N, std=0.1, dtype=dtype)
    pre = torch.empty(2, M, N, dtype=torch.int16, device="cuda")
    h = F.flce_gated_forward(x, Wg, Wu, activation=act, pre=pre)
    assert torch.equal(h, F.flce_gated_forward(x, Wg, Wu, activation=act))
    got = F.flce_gated_backward(dh, x, Wg, Wu, pre, activation=act, dW_dtype=dtype)
    check_gated_gradients(got, x, Wg, Wu, dh, act, dtype)
    leaves = [t.clone().requires_grad_() for t in (x, Wg, Wu)]
    F.gated_linear(*leaves, activation=act).backward(dh)
    for leaf, g in zip(leaves, got):
        assert torch.equal(leaf.grad, g)


@pytest.mark.parametrize("scale", [30.0, 100.0, 1000.0])
@pytest.mark.parametrize("M", [6, 400])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_features_beside_an_outlier_keep_their_gradients(scale, M, dtype):
    """One feature in eight has weights `scale` times as large. Of every other feature each dg and
    du is off by u and 2^-11 of itself; over the tokens these add like their squares at worst,
    so a row of dWg or dWu is off by that share of its size. 2^-13 more: a' in fp32, and
    2^-24 of a neighbour."""
    n = randn(M)
    x, dh = n(M, 64, dtype=dtype), n(M, 72, std=0.1, dtype=dtype)
    Wg, Wu = n(72, 64, std=0.125, dtype=dtype), n(72, 64, std=0.125, dtype=dtype)
    Wg[2::8] *= scale / 10
    Wu[5::8] *= scale
    pre = torch.empty(2, M, 72, dtype=torch.int16, device="cuda")
    F.flce_gated_forward(x, Wg, Wu, pre=pre)
    got = F.flce_gated_backward(dh, x, Wg, Wu, pre)
    if dtype is BF16:
        want = check_gated_gradients(got, x, Wg, Wu, dh, "silu", FP32)
    else:
        g, u, d = x.double() @ Wg.double().t(), x.double() @ Wu.double().t(), dh.double()
        p = torch.sigmoid(g)
        want = (d * u * p * (1 + g * torch.sigmoid(-g))).t() @ x.double(), (d * g * p).t() @ x.double()
    index = torch.arange(72, device="cuda") % 8
    limit = R.UNIT[dtype] + 2.0 ** -11 + 2.0 ** -13
    for w, v, out in ((got[1], want[0], 5), (got[2], want[1], 2)):
        rows = (index != out) & (index != 2)  # a unit with huge g is saturated: its size is its own
        err = (w.double() - v).norm(dim=1) / v.norm(dim=1)
        assert float(err[rows].max()) <= limit, float(err[rows].max())


@pytest.mark.parametrize("exponent", [-100, -20, 20, 100, 125])
@pytest.mark.parametrize("M", [5, 200])
def test_relative_form_at_any_size(exponent, M):
    """u from 2^-100 to near the largest fp32 number."""
    n = randn(M)
    x, Wg, dh = n(M, 64), n(72, 64, std=0.125), n(M, 72, std=0.01)
    Wu = (n(72, 64, std=0.1, dtype=FP32) * 2.0 ** exponent).to(BF16)
    pre = torch.empty(2, M, 72, dtype=torch.int16, device="cuda")
    F.flce_gated_forward(x, Wg, Wu, pre=pre)
    got = F.flce_gated_backward(dh, x, Wg, Wu, pre)
    check_gated_gradients(got, x, Wg, Wu, dh, "silu", FP32)


# ------------------------------------------------------------- clip_grad_norm_
def test_clip_grad_norm_scales_as_torchs_does():
    """The third positional argument is the norm's type: the same gradients as torch's, within the
    rounding of the norm (2^-20) and of the product."""
    n = randn(12)
    ours = [torch.nn.Parameter(n(*s, dtype=FP32)) for s in ((40, 7), (3,), (1000,))]
    torchs = [torch.nn.Parameter(p.detach().clone()) for p in ours]
    for p, q in zip(ours, torchs):
        p.grad = n(*p.shape, dtype=FP32)
        q.grad = p.grad.clone()
    norm = F.clip_grad_norm_(ours, 0.5, 2.0)
    want = torch.nn.utils.clip_grad_norm_(torchs, 0.5, 2.0)
    assert abs(float(norm) - float(want)) <= 2.0 ** -20 * float(want)
    for p, q in zip(ours, torchs):
        assert bool(((p.grad - q.grad).abs() <= 2.0 ** -19 * q.grad.abs()).all())


# --------------------------------------------- writes that autograd has to know of
def test_written_tensors_raise_their_version():
    n = randn(21)
    x, W, Wu, r, out = n(4, 64), n(16, 64), n(16, 64), n(4, 16), n(4, 16)
    pre, both = torch.empty(4, 16, dtype=BF16, device="cuda"), torch.empty(2, 4, 16, dtype=torch.int16, device="cuda")
    grads = [n(50, dtype=FP32), n(7, 3)]
    copies = [torch.empty_like(g) for g in grads]

    def raised(call, written, kept=()):
        before = [t._version for t in written], [t._version for t in kept]
        call()
        assert all(t._version > v for t, v in zip(written, before[0]))
        assert [t._version for t in kept] == before[1]

    raised(lambda: F.flce_linear_forward(x, W, None, r, activation="silu", pre=pre, out=out),
           [pre, out], [x, W, r])
    raised(lambda: F.flce_linear_forward(x, W, None, r, out=r), [r], [x, W])
    raised(lambda: F.flce_gated_forward(x, W, Wu, pre=both, out=out), [both, out], [x, W, Wu])
    raised(lambda: F.flce_grad_norm(grads), [], grads)
    raised(lambda: F.flce_clip_grads(grads, 0.1, out=copies), copies, grads)
    raised(lambda: F.flce_clip_grads(grads, 0.1), grads)
    p = torch.nn.Parameter(n(9, dtype=FP32))
    p.grad = n(9, dtype=FP32)
    raised(lambda: F.clip_grad_norm_([p], 0.1), [p.grad], [p])
    with torch.inference_mode():
        t = torch.ones(9, device="cuda")
    F.flce_clip_grads([t], 0.5)  # has no version
    assert bool((t < 1).all())


def test_autograd_refuses_an_overwritten_saved_residual():
    n = randn(22)
    x, W, leaf = n(4, 64), n(16, 64), n(4, 16).requires_grad_()
    r = leaf * 2
    s = r.square()  # saves r
    with torch.no_grad():
        F.flce_linear_forward(x, W, None, r.detach(), out=r.detach())
    with pytest.raises(RuntimeError, match="inplace"):
        s.sum().backward()


# ------------------------------------------------------ scratch of the backward
@pytest.mark.parametrize("offset", [0, 8])
@pytest.mark.parametrize("M,K,N", [(5, 64, 24), (300, 264, 80), (2048, 1032, 1032), (15, 16384, 64)])
def test_backward_of_an_aligned_dy_stays_inside_the_smaller_workspace(M, K, N, offset):
    """Without an activation, with exactly the bytes that an aligned dy needs, at any address."""
    lib, n = _lib.load(), randn(M)
    x, W, b, dy = n(M, K), n(N, K), n(N), n(M, N)
    want = F.flce_linear_backward(dy, x, W, b, dW_dtype=BF16, db_dtype=BF16)
    p = _lib.FlceLinearParams(M=M, K=K, N=N, has_bias=1)
    at = ctypes.addressof(p)
    need = lib.flce_linear_workspace_size(at, 2)
    buf = torch.full((need + offset + 64,), 7, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(x), torch.empty_like(W), torch.empty_like(b)
    rest = (x.data_ptr(), W.data_ptr(), None, *(t.data_ptr() for t in got), buf.data_ptr() + offset,
            need, F.device_error_word("cuda:0").data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert lib.flce_linear_backward(at, dy.data_ptr(), *rest) == 0
    assert bool((buf[:offset] == 7).all()) and bool((buf[offset + need:] == 7).all())
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    big = torch.empty(M * N + 8, dtype=BF16, device="cuda")
    shifted = big[1:1 + M * N].view(M, N).copy_(dy)
    assert lib.flce_linear_backward(at, shifted.data_ptr(), *rest) == \
        (0 if need == lib.flce_linear_workspace_size(at, 1) else 3)
    for g, w in zip(F.flce_linear_backward(shifted, x, W, b, dW_dtype=BF16, db_dtype=BF16), want):
        assert torch.equal(g, w)
    torch.cuda.synchronize()
    assert F.flce_read_device_error() == 0


def test_backward_without_an_activation_holds_no_copy_of_dy():
    x, W, dy = (torch.zeros(s, dtype=BF16, device="cuda") for s in ((8192, 512), (4096, 512), (8192, 4096)))
    F.flce_linear_backward(dy, x, W)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    outputs = F.flce_linear_backward(dy, x, W)
    size = sum(t.numel() * t.element_size() for t in outputs if t is not None)
    assert torch.cuda.max_memory_allocated() - held - size < 8192 * 4096 * 2 // 8


# ------------------------------------- weights and biases the kernels cannot read
@pytest.mark.parametrize("M", [4, 300])
def test_autograd_forms_copy_weights_and_biases_too(M):
    """A transposed weight, and ones that start off the 16-byte boundaries, as views of a flat
    buffer do: the same results and gradients as of dense copies."""
    n = randn(M)
    x = n(M, 64)
    flat = n(1 + 16 * 64 + 16)
    cases = [(n(64, 16).t(), n(16)), (flat[1:1 + 16 * 64].view(16, 64), flat[1 + 16 * 64:]),
             (n(16, 72)[:, :64], n(32)[::2])]
    for W, b in cases:
        W, b = W.detach().requires_grad_(), b.detach().requires_grad_()
        dense = [t.detach().clone(memory_format=torch.contiguous_format).requires_grad_() for t in (W, b)]
        dy = n(M, 16)
        for weights in ((W, b), dense):
            y = F.fused_linear(x, *weights, activation="silu")
            y.backward(dy)
            h = F.gated_linear(x, weights[0], weights[0])
            h.backward(dy)
            if weights[0] is W:
                want_y, want_h = y, h
        assert torch.equal(want_y, y) and torch.equal(want_h, h)
        assert torch.equal(W.grad, dense[0].grad) and torch.equal(b.grad, dense[1].grad)


# ------------------------------------------------------------ tensors given twice
def test_clip_refuses_tensors_that_share_memory():
    n = randn(31)
    flat = n(100, dtype=FP32)
    kept = flat.clone()
    with pytest.raises(ValueError, match="overlap"):
        F.flce_clip_grads([flat, flat], 0.1)
    with pytest.raises(ValueError, match="overlap"):
        F.flce_clip_grads([flat[:60], flat[59:]], 0.1)
    with pytest.raises(ValueError, match="overlap"):
        F.flce_clip_grads([flat, kept], 0.1, out=[torch.empty_like(flat)] * 2)
    assert torch.equal(flat, kept)
    twice = F.flce_grad_norm([flat, flat])  # the norm only reads
    assert abs(float(twice) - 2 ** 0.5 * float(flat.double().norm())) <= 1e-5 * float(twice)
    empty = flat[:0]
    one = F.flce_clip_grads([flat[:60], flat[60:], empty, empty], 0.1)
    p = torch.nn.Parameter(kept.clone())
    p.grad = kept.clone()
    tied = F.clip_grad_norm_([p, p], 0.1)
    want = float(kept.double().norm())
    for norm, g in ((one, flat), (tied, p.grad)):
        assert abs(float(norm) - want) <= 1e-5 * want
        assert bool(((g.double() - kept.double() * (0.1 / (want + 1e-6))).abs() <= 1e-5 * kept.double().abs()).all())


# ------------------------------------------------------------ signs of relu's inputs
def relu_signs(M, K, N, dtype, gated, seed):
    """(kept slopes above 0, z in 64 bits)."""
    n = randn(seed)
    x, W = n(M, K, dtype=dtype), n(N, K, std=K ** -0.5, dtype=dtype)
    z = x.double() @ W.double().t()
    if gated:
        # u = 1 everywhere: the kept u a'(g) is the slope.
        x[:, 0] = 1
        Wu = torch.zeros(N, K, dtype=dtype, device="cuda")
        Wu[:, 0] = 1
        z = x.double() @ W.double().t()
        pre = torch.empty(2, M, N, dtype=torch.int16, device="cuda")
        F.flce_gated_forward(x, W, Wu, activation="relu", pre=pre)
        return (pre[1] & 0x3FFF) > 0, z
    b = n(N, std=0.1, dtype=dtype)
    pre = torch.empty(M, N, dtype=dtype, device="cuda")
    F.flce_linear_forward(x, W, b, activation="relu", pre=pre)
    return R.kept_slopes(pre) > 0.5, z + b.double()


@pytest.mark.parametrize("M,K,N", [(2048, 16384, 2048), (1000, 8192, 4100), (64, 16384, 16384), (20, 12808, 30000)])
@pytest.mark.parametrize("gated", [False, True], ids=["linear", "gated"])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_relu_takes_the_sign_of_an_accurate_sum(M, K, N, gated, dtype):
    """z has size 1. The tensor core's sums are off by 1e-5 to 2e-5 here (root mean square), fp32 adds
    of K / 128 products and then of 128 partial sums by 3.4e-7: ten times that, 2^-18, leaves no
    wrong sign, of which the tensor core's sums alone have several in each of these."""
    above, z = relu_signs(M, K, -(-N // 8) * 8 if gated else N, dtype, gated, 5)
    wrong = (above != (z > 0)) & (z.abs() > 2.0 ** -18)
    assert int(wrong.sum()) == 0


def test_relu_with_rows_and_weights_far_smaller_than_their_neighbours():
    """Zero tokens, zero weights and tiny weights: more sums near 0 than are looked at again.
    Outside the tensor core's error (2^-24 of the row's largest sum for each 16 products, four
    times) every sign is right."""
    n = randn(6)
    M, K, N = 600, 4096, 520
    x, W = n(M, K), n(N, K, std=K ** -0.5)
    x[::3] = 0
    W[::5] = 0
    W[1::5] = (W[1::5].float() * 2.0 ** -14).to(BF16)
    pre = torch.empty(M, N, dtype=BF16, device="cuda")
    y = F.flce_linear_forward(x, W, activation="relu", pre=pre)
    z = x.double() @ W.double().t()
    error = 4 * (K / 16 + 8) * 2.0 ** -24 * z.abs().amax(1, keepdim=True)
    above = R.kept_slopes(pre) > 0.5
    assert bool((above == (z > 0))[z.abs() > error].all())
    assert not bool(above[::3].any()) and not bool(above[:, ::5].any())
    assert torch.equal(y, F.flce_linear_forward(x, W, activation="relu"))


@pytest.mark.parametrize("M,K,N", [(5942, 6456, 1408), (64, 11112, 12368)])
def test_relu_gradients_are_those_of_an_accurate_sum(M, K, N):
    """fp16: dz without a wrong sign is exact, so dx and dW are off by their rounding alone, and by
    what signs inside 2^-18 can do: a share of 2^-18 of the elements, sqrt(2^-17) if all were wrong,
    of which the fp32 sum's 3.4e-7 leaves a tenth of the share."""
    n = randn(9)
    x, W, dy = n(M, K, dtype=FP16), n(N, K, std=K ** -0.5, dtype=FP16), n(M, N, std=0.01, dtype=FP16)
    pre = torch.empty(M, N, dtype=FP16, device="cuda")
    F.flce_linear_forward(x, W, activation="relu", pre=pre)
    dx, dW, _ = F.flce_linear_backward(dy, x, W, activation="relu", pre=pre)
    dz = dy.double() * (x.double() @ W.double().t() > 0)
    for got, want, u in ((dx, dz @ W.double(), 2.0 ** -11), (dW, dz.t() @ x.double(), 0.0)):
        err = float((got.double() - want).norm() / want.norm())
        assert err <= u + 2.0 ** -23 * (max(M, N) / 16) + (0.1 * 2.0 ** -17) ** 0.5, err


# ------------------------------------------------ the autograd functions by themselves
def test_autograd_functions_take_their_arguments_without_a_form():
    """`keep` is the last argument of both and may be left out."""
    n = randn(41)
    x, W, Wu, b, r = (t.requires_grad_() for t in (n(9, 64), n(16, 64), n(16, 64), n(16), n(9, 16)))
    dy = n(9, 16)
    F.FusedLinearFunction.apply(x, W, b, r, "silu").backward(dy)
    F.GatedLinearFunction.apply(x, W, Wu, "silu").backward(dy)
    short = [t.grad for t in (x, W, Wu, b, r)]
    for t in (x, W, Wu, b, r):
        t.grad = None
    F.FusedLinearFunction.apply(x, W, b, r, "silu", "fixed").backward(dy)
    F.GatedLinearFunction.apply(x, W, Wu, "silu", "relative").backward(dy)
    for t, g in zip((x, W, Wu, b, r), short):
        assert torch.equal(t.grad, g)
