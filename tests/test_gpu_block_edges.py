"""The layer operators where they could go wrong unseen: outputs that nothing writes, saturated
activations, features of very different size, infinities, what a call leaves to autograd."""
import ctypes

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
from linear_cross_entropy_gemm_gb300 import _lib

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


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


# ---------------------------------------------------- infinities in kept values
def randn(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape, std=1.0, dtype=BF16: (
        torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("M", [5, 50, 300])
@pytest.mark.parametrize("value", [float("inf"), float("nan")], ids=str)
def test_a_bad_feature_stays_in_its_row_of_the_weight_gradients(M, value):
    """A weight row with an infinity or NaN makes u a'(g) of its own feature non-finite in every
    token, and nothing of its seven neighbours'. Those are compared with 64 bits: each dg and
    du is off by its rounding and the kept value's 2^-14 of the group's largest."""
    n = randn(M)
    x, Wg, Wu, dh = n(M, 64), n(72, 64, std=0.125), n(72, 64, std=0.125), n(M, 72)
    Wu[11, 5] = value
    pre = torch.empty(2, M, 72, dtype=BF16, device="cuda")
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
        off = 2.0 ** -8 * d.abs() + 1.01 * 2.0 ** -14 * d64.abs() * size + 2.0 ** -16 * d64.abs()
        bound = off.t() @ x64.abs() + M * 2.0 ** -23 * (d.abs().t() @ x64.abs())
        err = (got.double() - d.t() @ x64).abs()
        assert bool((err <= bound)[rows].all())
