"""RMS norm with the residual's addition, its 8-bit output, and dropout, against 64 bits."""
import ctypes
import itertools

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
import stream_reference as R
from linear_cross_entropy_gemm_gb300 import _lib

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP16, FP32), (FP32, FP32)]  # of x, of the stream
# One row to many; one column; around the widths of a group of 8, a warp, a block, and the number
# of groups that a thread holds; the widest.
SHAPES = [(1, 1), (3, 7), (2, 8), (5, 9), (7, 256), (4, 264), (9, 1111), (33, 2048), (1, 4096), (300, 136),
          (2, 8192), (3, 8200), (2, 16384), (2, 16392), (3, 20001), (2, 32768), (700, 512)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def problem(M, H, x_type, stream, res=True, seed=0):
    g = gen(seed + 31 * M + H)
    x = normal(g, M, H, dtype=x_type)
    r = normal(g, M, H, std=3.0, dtype=stream) if res else None
    w = normal(g, H, std=0.3, dtype=x_type) + 1
    return x, w, r, normal(g, M, H, std=0.1, dtype=x_type), normal(g, M, H, std=0.1, dtype=stream)


def check_forward(x, w, r, eps=1e-5, p=0.0, seed=5, offset=0, **kw):
    """The call's results, held to the reference."""
    rstd = torch.full((x.shape[0],), float("nan"), device="cuda")
    y, h = F.flce_rms_norm_forward(x, w, r, eps=eps, dropout=p, seed=seed, offset=offset, rstd=rstd, **kw)
    f = R.factors(*x.shape, p, seed, offset)
    h64, h_err, rstd64, y64, y_err = R.norm(x, w, r, eps, f)
    R.assert_near(y, y64, y_err, "y")
    R.assert_near(h, h64, h_err, "h")
    R.assert_near(rstd, rstd64, 32 * R.U * rstd64, "rstd")
    return y, h, rstd, f


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_norm(shape, types):
    x, w, r, dy, dh = problem(*shape, *types)
    y, h, rstd, _ = check_forward(x, w, r)
    assert y.dtype == types[0] and h.dtype == types[1]
    dx, dr, dW = F.flce_rms_norm_backward(dy, h, w, rstd, dh)
    e, e_err, _, _, dW64, dW_err = R.norm_grad(dy, h, w, rstd, dh, 1.0)
    R.assert_near(dr, e, e_err, "dresidual")
    R.assert_near(dx, e, e_err, "dx")
    R.assert_near(dW, dW64, dW_err, "dW")
    assert dx.dtype == types[0] and dr.dtype == types[1] and dW.dtype == FP32
    assert (dx is dr) == (types[0] == types[1])


@pytest.mark.parametrize("shape", [(1, 8), (5, 100), (40, 4096), (3, 8200), (2, 32768), (1025, 264)], ids=str)
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_norm_with_dropout(shape, types, p):
    x, w, r, dy, dh = problem(*shape, *types)
    seed, offset = -(2 ** 62) + 12345, 2 ** 40 + 3
    y, h, rstd, f = check_forward(x, w, r, p=p, seed=seed, offset=offset)
    dx, dr, dW = F.flce_rms_norm_backward(dy, h, w, rstd, dh, dropout=p, seed=seed, offset=offset,
                                          dW_dtype=dy.dtype)
    e, e_err, d, d_err, dW64, dW_err = R.norm_grad(dy, h, w, rstd, dh, f)
    R.assert_near(dr, e, e_err, "dresidual")
    R.assert_near(dx, d, d_err, "dx")
    R.assert_near(dW, dW64, dW_err, "dW")
    assert bool((dx[f == 0] == 0).all())


@pytest.mark.parametrize("H", [24, 999, 5000])
def test_norm_without_residual_or_weight(H):
    x, w, _, dy, _ = problem(6, H, BF16, BF16, res=False)
    y, h, rstd, _ = check_forward(x, w, None)
    assert h is x
    dx, dr, dW = F.flce_rms_norm_backward(dy, h, w, rstd, needs=(True, False, True))
    assert dr is None
    e, e_err, _, _, dW64, dW_err = R.norm_grad(dy, x, w, rstd, None, 1.0)
    R.assert_near(dx, e, e_err, "dx")
    R.assert_near(dW, dW64, dW_err, "dW")
    # Dropout without a residual: the sum is a tensor of its own.
    _, h, _, f = check_forward(x, w, None, p=0.25)
    assert h is not x
    # Without a weight.
    y, h, rstd, _ = check_forward(x, None, None)
    dx, _, dW = F.flce_rms_norm_backward(dy, h, None, rstd, needs=(True, False, True))
    assert dW is None
    e, e_err, _, _, _, _ = R.norm_grad(dy, x, None, rstd, None, 1.0)
    R.assert_near(dx, e, e_err, "dx")


@pytest.mark.parametrize("types", [(BF16, FP32), (FP16, FP32)], ids=str)
def test_norm_weight_in_fp32(types):
    x, w, r, dy, dh = problem(20, 640, *types)
    w = w.float() + 2.0 ** -13
    y, h, rstd, _ = check_forward(x, w, r)
    dx, dr, dW = F.flce_rms_norm_backward(dy, h, w, rstd, dh)
    e, e_err, _, _, dW64, dW_err = R.norm_grad(dy, h, w, rstd, dh, 1.0)
    R.assert_near(dx, e, e_err, "dx")
    R.assert_near(dW, dW64, dW_err, "dW")


@pytest.mark.parametrize("needs", list(itertools.product((True, False), repeat=3)), ids=str)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_norm_gradients_that_are_asked_for(needs, p):
    x, w, r, dy, dh = problem(11, 320, BF16, BF16)
    rstd = torch.empty(11, device="cuda")
    _, h = F.flce_rms_norm_forward(x, w, r, dropout=p, seed=1, rstd=rstd)
    full = F.flce_rms_norm_backward(dy, h, w, rstd, dh, dropout=p, seed=1)
    some = F.flce_rms_norm_backward(dy, h, w, rstd, dh, dropout=p, seed=1, needs=needs)
    for need, a, b in zip(needs, full, some):
        assert b is None if not need else torch.equal(a, b)


def poisoned(rows, cols, ld, offset, dtype):
    """A view of `rows` rows, `ld` apart, inside a buffer of NaN; and the buffer."""
    buf = torch.full((offset + rows * ld + 64,), float("nan"), dtype=dtype, device="cuda")
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols], buf


@pytest.mark.parametrize("H,pad,offset", [(256, 8, 8), (256, 8, 1), (256, 3, 0), (250, 6, 0), (100, 0, 5),
                                          (8192, 24, 16)])
@pytest.mark.parametrize("types", [(BF16, BF16), (FP16, FP32)], ids=str)
def test_norm_strides_and_alignment(H, pad, offset, types):
    """Rows of any pitch at any element; nothing outside the outputs is written."""
    M = 9
    x0, w, r0, dy0, dh0 = problem(M, H, *types)
    views = []
    for t in (x0, r0, dy0, dh0):
        v, _ = poisoned(M, H, H + pad, offset, t.dtype)
        views.append(v.copy_(t))
    x, r, dy, dh = views
    wbuf = torch.full((H + 8,), float("nan"), dtype=w.dtype, device="cuda")
    w1 = wbuf[offset % 8:offset % 8 + H].copy_(w)
    out, out_buf = poisoned(M, H, H + pad + 5, offset + 3, types[0])
    h_out, h_buf = poisoned(M, H, H + pad, offset, types[1])
    y, h, rstd, _ = check_forward(x, w1, r, out=out, h=h_out)
    assert y.data_ptr() == out.data_ptr() and h.data_ptr() == h_out.data_ptr()
    for view, buf in ((out, out_buf), (h_out, h_buf)):
        assert int(buf.isnan().sum()) == buf.numel() - view.numel()
    dense = F.flce_rms_norm_forward(x0, w, r0, eps=1e-5)
    # The sum is elementwise; the order of the squares' sum goes by the rows' alignment.
    assert torch.equal(dense[1], h)
    _, _, _, y64, y_err = R.norm(x0, w, r0, 1e-5, R.factors(M, H, 0.0, 0))
    R.assert_near(dense[0], y64, y_err, "y of dense rows")
    got = F.flce_rms_norm_backward(dy, h, w1, rstd, dh)
    e, e_err, _, _, dW64, dW_err = R.norm_grad(dy, h, w1, rstd, dh, 1.0)
    R.assert_near(got[0], e, e_err, "dx")
    R.assert_near(got[2], dW64, dW_err, "dW")


@pytest.mark.parametrize("H", [1000, 1001])
def test_norm_in_place(H):
    """y in x's buffer, the sum in the residual's."""
    x, w, r, _, _ = problem(13, H, BF16, BF16)
    y, h = F.flce_rms_norm_forward(x, w, r, dropout=0.2, seed=9)
    x1, r1 = x.clone(), r.clone()
    versions = x1._version, r1._version
    y1, h1 = F.flce_rms_norm_forward(x1, w, r1, dropout=0.2, seed=9, out=x1, h=r1)
    assert y1.data_ptr() == x1.data_ptr() and torch.equal(y1, y) and torch.equal(h1, h)
    assert x1._version > versions[0] and r1._version > versions[1]
    # Without the sum.
    y2, h2 = F.flce_rms_norm_forward(x, w, r, dropout=0.2, seed=9, h=False)
    assert torch.equal(y2, y)
    # Halves of one buffer lie next to each other.
    both = torch.cat((x, x), 1)
    F.flce_rms_norm_forward(both[:, :H], w, r, out=both[:, H:])
    assert torch.equal(both[:, :H], x) and torch.equal(both[:, H:], F.flce_rms_norm_forward(x, w, r)[0])


def test_norm_refuses_shared_memory():
    x, w, r, _, _ = problem(8, 64, BF16, BF16)
    buf = torch.zeros(8 * 64 + 64, dtype=BF16, device="cuda")
    a, b = buf[:512].view(8, 64), buf[8:520].view(8, 64)
    for call in (lambda: F.flce_rms_norm_forward(a, w, r, out=b), lambda: F.flce_rms_norm_forward(x, w, a, h=b),
                 lambda: F.flce_rms_norm_forward(x, w, r, out=a, h=a), lambda: F.flce_dropout(a, 0.5, 1, out=b),
                 lambda: F.flce_dropout(x, 0.5, 1, residual=a, out=b),
                 lambda: F.flce_rms_norm_forward(x, a[0], r, out=a)):
        with pytest.raises(ValueError, match="overlap"):
            call()


@pytest.mark.parametrize("scales", ["row", "block"])
@pytest.mark.parametrize("shape", [(1, 4096), (7, 128), (5, 129), (3, 7), (45, 1000), (2, 20001), (2, 32768),
                                   (300, 264)], ids=str)
@pytest.mark.parametrize("types", [(BF16, BF16), (FP16, FP32), (FP32, FP32)], ids=str)
def test_norm_in_8_bits(shape, types, scales):
    M, H = shape
    x, w, r, _, _ = problem(M, H, *types)
    w = w * torch.exp2(torch.arange(H, device="cuda") % 11 - 5.0).to(w.dtype)
    y8, scale, h = F.flce_rms_norm_quantized(x, w, r, eps=1e-5, scales=scales, dropout=0.1, seed=4)
    h64, h_err, _, y64, y_err = R.norm(x, w, r, 1e-5, R.factors(M, H, 0.1, 4))
    R.assert_near(h, h64, h_err, "h")
    blocks = -(-H // 128)
    if scales == "row":
        want = y64.abs().amax(-1) / 448
        each, err = scale[:, None].expand(M, H), y_err.amax(-1) / 448
        assert scale.shape == (M,)
    else:
        padded = torch.zeros(M, blocks * 128, dtype=torch.float64, device="cuda")
        padded[:, :H] = y64
        want = padded.view(M, blocks, 128).abs().amax(-1) / 448
        padded[:, :H] = y_err
        err = padded.view(M, blocks, 128).amax(-1) / 448
        each = scale.repeat_interleave(128, 1)[:, :H]
        assert scale.shape == (M, blocks)
    R.assert_near(scale, want, err, "scale")
    # y / scale: the scale's inverse and the product round once each, and e4m3 by half a step
    # of 2^-3, or of its smallest number.
    each = each.double()
    off = (y8.double() * each - y64).abs()
    limit = y_err + (2.0 ** -4 + 4 * R.U) * (y64.abs() + y_err) + each * 2.0 ** -10
    assert bool((off <= limit).all()), float((off / limit).max())
    assert y8.dtype == torch.float8_e4m3fn and bool((y8.float().abs() <= 448).all())


def test_norm_in_8_bits_edges():
    H = 256
    x = torch.zeros(5, H, dtype=FP32, device="cuda")
    x[1] = 1.0
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    x[4] = 1e-42
    w = torch.ones(H, device="cuda")
    y8, scale, _ = F.flce_rms_norm_quantized(x, w, scales="row")
    assert bool((y8[0].float() == 0).all()) and float(scale[0]) == 0.0
    assert bool((y8[1].float() == 448).all())
    assert bool(scale[2:4].isnan().all()) and bool(y8[2].float().isnan().all())
    # (1e-42)^2 is 0 in 32 bits: y is 1e-39, whose scale would be below the normal numbers.
    assert float(scale[4]) == 0.0 and bool((y8[4].float() == 0).all())
    out, buf = torch.empty(5, H, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(5, 2, device="cuda")
    y, s, h = F.flce_rms_norm_quantized(x, w, scales="block", out=out, scale=buf)
    assert y.data_ptr() == out.data_ptr() and s.data_ptr() == buf.data_ptr() and h is x


def test_norm_non_finite_and_zero_rows():
    """A row's infinity or NaN stays in its row; a row of zeros is normed to zeros."""
    x, w, r, dy, dh = problem(6, 512, BF16, BF16)
    clean = F.flce_rms_norm_forward(x, w, r)
    x[1, 5], x[3, 9], x[4], r[4] = float("inf"), float("nan"), 0, 0
    rstd = torch.empty(6, device="cuda")
    y, h = F.flce_rms_norm_forward(x, w, r, rstd=rstd)
    for i in (0, 2, 5):
        assert torch.equal(y[i], clean[0][i])
    assert bool(y[1, 5].isnan()) and bool((y[1, 6:] == 0).all()) and bool(y[3].isnan().all())
    assert bool((y[4] == 0).all()) and float(rstd[4]) == pytest.approx(1e3, rel=1e-6)
    dx, _, _ = F.flce_rms_norm_backward(dy, h, w, rstd, dh)
    assert bool(dx[[0, 2, 4, 5]].isfinite().all())
    # Dropped elements are 0 whatever they held.
    bad = torch.full((4, 64), float("nan"), dtype=BF16, device="cuda")
    kept = R.factors(4, 64, 0.5, 3) != 0
    out = F.flce_dropout(bad, 0.5, 3)
    assert torch.equal(out.isnan(), kept) and bool((out[~kept] == 0).all())


def test_norm_empty():
    x, w = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    y, h = F.flce_rms_norm_forward(x, w, x.clone())
    assert y.shape == (0, 64)
    dx, dr, dW = F.flce_rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and bool((dW == 0).all())
    assert F.flce_rms_norm_quantized(x, w, scales="block")[1].shape == (0, 1)
    assert F.flce_dropout(x, 0.5, 1).shape == (0, 64)


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (5, 8), (2, 1000), (17, 1111), (1000, 96)], ids=str)
@pytest.mark.parametrize("types", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP16, FP16), (FP16, FP32),
                                   (FP32, FP16), (FP32, FP32)], ids=str)
def test_dropout(shape, types):
    g = gen(2)
    x, r = normal(g, *shape, dtype=types[0]), normal(g, *shape, dtype=types[1])
    f = R.factors(*shape, 0.3, 77, 5)
    y = F.flce_dropout(x, 0.3, 77, offset=5, residual=r)
    want, err = R.dropped_sum(x, r, f)
    R.assert_near(y, want, err, "y")
    y = F.flce_dropout(x, 0.3, 77, offset=5, like=r)
    want, err = R.dropped_sum(x, None, f)
    R.assert_near(y, want, err, "y without a residual")
    assert y.dtype == types[1] and torch.equal(y != 0, (f != 0) & (x != 0))


def test_dropout_probabilities():
    """p is taken to 2^-16, the scale is exact for what is drawn, and the ends are exact."""
    x = torch.ones(512, 1024, device="cuda")
    assert torch.equal(F.flce_dropout(x, 0.0, None), x)
    assert bool((F.flce_dropout(x, 1.0, 1) == 0).all())
    r = torch.full_like(x, 2.0)
    assert torch.equal(F.flce_dropout(x, 1.0, 1, residual=r), r)
    assert torch.equal(F.flce_dropout(x, 2.0 ** -18, 1), x)
    for p in (2.0 ** -16, 0.1, 0.5, 0.9):
        y = F.flce_dropout(x, p, 123)
        t = int(p * 65536 + 0.5)
        kept = float((y != 0).double().mean())
        q = 1 - t / 65536
        # 2^19 draws: five standard deviations.
        assert abs(kept - q) <= 5 * (q * (1 - q) / 2 ** 19) ** 0.5
        assert float(y.max()) == pytest.approx(65536 / (65536 - t), rel=2 ** -23)


def test_dropout_masks_differ_and_repeat():
    x = torch.ones(64, 256, device="cuda")
    base = F.flce_dropout(x, 0.5, 3, offset=7) != 0
    assert torch.equal(base, F.flce_dropout(x.bfloat16(), 0.5, 3, offset=7) != 0)
    for kw in (dict(seed=4, offset=7), dict(seed=3, offset=8), dict(seed=3 + 2 ** 32, offset=7),
               dict(seed=3, offset=7 + 2 ** 32)):
        other = F.flce_dropout(x, 0.5, kw["seed"], offset=kw["offset"]) != 0
        # 2^14 independent pairs of bits.
        assert abs(float((base == other).double().mean()) - 0.5) <= 5 * 0.5 / 2 ** 7
    # The mask goes by row and column alone: a slice's, and a wider tensor's, are the same.
    assert torch.equal(base[:, :100], F.flce_dropout(x[:, :100], 0.5, 3, offset=7) != 0)
    three = F.flce_dropout(x.view(4, 16, 256), 0.5, 3, offset=7)
    assert torch.equal(base, three.view(64, 256) != 0)
    seed = torch.tensor([3], device="cuda")
    assert torch.equal(base, F.flce_dropout(x, 0.5, seed, offset=7) != 0)
    negative = F.flce_dropout(x, 0.5, -5) != 0
    assert torch.equal(negative, F.flce_dropout(x, 0.5, torch.tensor([-5], device="cuda")) != 0)
    y, h = F.flce_rms_norm_forward(x, None, None, dropout=0.5, seed=3, offset=7)
    assert torch.equal(base, h != 0)


def test_dropout_beyond_32_bits():
    """More than 2^32 elements, the last rows against the generator."""
    M, H, tail = (1 << 16) + 40, 1 << 16, 4
    x = torch.ones(M, H, dtype=BF16, device="cuda")
    y = F.flce_dropout(x, 0.25, 11, out=x)
    f = R.factors(tail, H, 0.25, 11, row0=M - tail)
    assert torch.equal(y[-tail:] != 0, f != 0)
    del x, y
    x = torch.full((M, H), 0.5, dtype=BF16, device="cuda")
    y, _ = F.flce_rms_norm_forward(x[:, :32768], None, out=x[:, 32768:], eps=0.0)
    assert bool((y[-tail:] == 1).all()) and bool((x[-tail:, :32768] == 0.5).all())


def test_dropout_in_place_and_strided():
    g = gen(8)
    x, r = normal(g, 30, 136), normal(g, 30, 136)
    want = F.flce_dropout(x, 0.4, 2, residual=r)
    for target in ("x", "r"):
        a, b = x.clone(), r.clone()
        F.flce_dropout(a, 0.4, 2, residual=b, out=a if target == "x" else b)
        assert torch.equal(a if target == "x" else b, want)
    for H, pad, offset in ((136, 8, 8), (136, 3, 1), (131, 1, 0)):
        v, buf = poisoned(30, H, H + pad, offset, BF16)
        v.copy_(x[:, :H])
        out, out_buf = poisoned(30, H, H + pad, offset, BF16)
        F.flce_dropout(v, 0.4, 2, residual=r[:, :H], out=out)
        assert torch.equal(out, want[:, :H]) and int(out_buf.isnan().sum()) == out_buf.numel() - out.numel()


def test_refusals():
    x, w, r, dy, dh = problem(4, 64, BF16, BF16)
    rstd = torch.ones(4, device="cuda")
    with pytest.raises(TypeError, match="seed"):
        F.flce_dropout(x, 0.1, None)
    with pytest.raises(TypeError, match="seed"):
        F.flce_rms_norm_forward(x, w, r, dropout=0.1)
    for bad in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                torch.zeros(1, dtype=torch.int64)):
        with pytest.raises(ValueError, match="seed"):
            F.flce_dropout(x, 0.1, bad)
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises((F.FlceError, ValueError)):
            F.flce_dropout(x, p, 1) if p == p else F.flce_rms_norm_forward(x, w, r, dropout=p, seed=1)
    with pytest.raises(TypeError, match="residual"):
        F.flce_rms_norm_forward(x, w, r.half())
    with pytest.raises(TypeError, match="weight"):
        F.flce_rms_norm_forward(x, w.half(), r)
    with pytest.raises(ValueError, match="weight"):
        F.flce_rms_norm_forward(x, w[:-8], r)
    with pytest.raises(ValueError, match="residual"):
        F.flce_rms_norm_forward(x, w, r[:3])
    with pytest.raises(ValueError, match="rows"):
        F.flce_rms_norm_forward(x[:, ::2], w[::2].contiguous(), r[:, ::2])
    with pytest.raises(ValueError, match="rows"):
        F.flce_rms_norm_forward(x[:1].expand(4, 64), w, r)
    with pytest.raises(TypeError, match="h"):
        F.flce_rms_norm_forward(x, w, r, h=torch.empty(4, 64, device="cuda"))
    with pytest.raises(TypeError, match="dh"):
        F.flce_rms_norm_backward(dy, x, w, rstd, dh.float())
    with pytest.raises(ValueError, match="rstd"):
        F.flce_rms_norm_backward(dy, x, w, rstd[:3], dh)
    with pytest.raises(F.FlceError):
        F.flce_rms_norm_forward(torch.zeros(1, 32776, dtype=BF16, device="cuda"), None)
    with pytest.raises(TypeError):
        F.flce_rms_norm_forward(x.double(), None)
    with pytest.raises(TypeError, match="type"):
        F.flce_dropout(x, 0.1, 1, like=r.half())


# ----------------------------------------------------- streams, graphs, autograd
def test_streams_and_repeatability():
    x, w, r, dy, dh = problem(600, 2056, BF16, BF16)
    rstd = torch.empty(600, device="cuda")
    want = F.flce_rms_norm_forward(x, w, r, dropout=0.1, seed=1, rstd=rstd)
    grads = F.flce_rms_norm_backward(dy, want[1], w, rstd, dh, dropout=0.1, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.flce_rms_norm_forward(x, w, r, dropout=0.1, seed=1, rstd=rstd, stream=side)
    again = F.flce_rms_norm_backward(dy, got[1], w, rstd, dh, dropout=0.1, seed=1, stream=side.cuda_stream)
    d = F.flce_dropout(x, 0.1, 1, stream=side)
    q = F.flce_rms_norm_quantized(x, w, r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want + grads, got + again):
        assert torch.equal(a, b)
    assert torch.equal(d, F.flce_dropout(x, 0.1, 1))
    assert torch.equal(q[1], F.flce_rms_norm_quantized(x, w, r)[1])


def test_captured_calls_share_a_workspace_and_draw_anew():
    """Two graphs over one workspace, replayed in turn, with a seed in device memory."""
    x, w, r, dy, dh = problem(40, 520, BF16, BF16)
    p = _lib.FlceRmsNormParams(M=40, H=520, eps=1e-6)
    ws = torch.empty(_lib.load().flce_rms_norm_workspace_size(ctypes.byref(p)), dtype=torch.uint8, device="cuda")
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    rstd = torch.empty(40, device="cuda")

    def step(scale):
        y, h = F.flce_rms_norm_forward(x, w, r, dropout=0.3, seed=seed, rstd=rstd)
        return (y, h) + F.flce_rms_norm_backward(dy * scale, h, w, rstd, dh, dropout=0.3, seed=seed, workspace=ws)

    step(1.0)
    torch.cuda.synchronize()
    graphs, results = [], []
    for scale in (1.0, 3.0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(step(scale))
        graphs.append(g)
    seen = []
    for s in (1, 2):
        seed.fill_(s)
        for g, got, scale in zip(graphs, results, (1.0, 3.0)):
            g.replay()
            for a, b in zip(got, step(scale)):
                assert torch.equal(a, b)
        seen.append(results[0][0].clone())
    assert not torch.equal(*seen)


def reference_module(x, r, w, f, eps):
    h = r + x * f
    return h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w, h


@pytest.mark.parametrize("uses", ["y", "h", "both"])
@pytest.mark.parametrize("types", [(FP32, FP32), (BF16, FP32)], ids=str)
def test_autograd_of_the_norm(uses, types):
    x, w, r, dy, dh = problem(24, 200, *types)
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, h = F.fused_rms_norm(leaves[0].view(4, 6, 200), leaves[1], leaves[2].view(4, 6, 200), eps=1e-5,
                            dropout=0.2, seed=42)
    f = R.factors(24, 200, 0.2, 42)
    want = [t.double().requires_grad_() for t in (x, w, r)]
    y64, h64 = reference_module(want[0], want[2], want[1], f, 1e-5)
    total, total64 = 0, 0
    if uses != "h":
        total, total64 = (y * dy.view_as(y)).sum(), (y64 * dy.double()).sum()
    if uses != "y":
        total, total64 = total + (h * dh.view_as(h)).sum(), total64 + (h64 * dh.double()).sum()
    total.backward()
    total64.backward()
    for got, ref in zip(leaves, want):
        if uses == "h" and got is leaves[1]:
            assert bool((got.grad == 0).all())
            continue
        rel = float((got.grad.double() - ref.grad).norm() / ref.grad.norm())
        # Each gradient is rounded once, and bf16's products of them before.
        assert rel <= (2.0 ** -7 if types[0] == BF16 else 2.0 ** -18), rel


def test_autograd_of_expanded_and_transposed_gradients():
    x = torch.randn(12, 64, device="cuda").requires_grad_()
    F.fused_rms_norm(x).sum().backward()  # a gradient without strides
    a = x.grad.clone()
    x.grad = None
    (F.fused_rms_norm(x).t().contiguous().t() * 1.0).sum().backward()
    assert torch.allclose(a, x.grad, rtol=1e-5, atol=1e-6)
    x.grad = None
    F.fused_dropout(x, 0.25, seed=6).sum().backward()
    assert torch.equal(x.grad.double(), R.factors(12, 64, 0.25, 6).float().double())


def test_seeds_come_from_the_generator():
    x = torch.ones(64, 64, device="cuda")
    torch.manual_seed(5)
    a, b = F.fused_dropout(x, 0.5), F.fused_dropout(x, 0.5)
    torch.manual_seed(5)
    assert torch.equal(a, F.fused_dropout(x, 0.5)) and not torch.equal(a, b)
    norm = F.FusedRMSNorm(64, dropout=0.5, dtype=FP32, device="cuda")
    assert not torch.equal(norm(x, x)[1], norm(x, x)[1])
    norm.eval()
    assert torch.equal(norm(x, x)[1], x + x)


def test_a_captured_training_step_draws_anew():
    """Forward and backward of the block with norm and dropout in a graph; gradients as an eager
    step of the same seed gives them, and other masks at each replay."""
    torch.manual_seed(0)
    block = F.GatedFeedForward(64, 96, device="cuda", norm_eps=1e-6, dropout=0.5)
    x = torch.randn(32, 64, device="cuda").bfloat16()
    params = list(block.parameters())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            torch.autograd.grad(block(x).float().square().sum(), params)
    torch.cuda.current_stream().wait_stream(stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = block(x)
        grads = torch.autograd.grad(y.float().square().sum(), params)
    outs = []
    for _ in range(3):
        g.replay()
        outs.append((y.clone(), grads[0].clone()))
    assert not torch.equal(outs[0][0], outs[1][0]) and not torch.equal(outs[1][1], outs[2][1])
    # Half of the elements come from the stream alone.
    for out, _ in outs:
        assert 0.4 < float((out == x).double().mean()) < 0.6


def test_block_with_norm_and_dropout():
    """The block's gradients against 64 bits, with the mask that its seed gives."""
    torch.manual_seed(3)
    block = F.GatedFeedForward(128, 192, device="cuda", norm_eps=1e-5, dropout=0.25)
    with torch.no_grad():
        block.norm.weight.copy_(1 + 0.1 * torch.randn(128, device="cuda"))
    x = torch.randn(50, 128, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(50, 128, device="cuda").bfloat16()
    state = torch.cuda.get_rng_state()
    y = block(x)
    y.backward(dy)
    torch.cuda.set_rng_state(state)
    seed = int(torch.empty(1, dtype=torch.int64, device="cuda").random_())
    f = R.factors(50, 128, 0.25, seed)
    p64 = {n: p.detach().double().requires_grad_() for n, p in block.named_parameters()}
    x64 = x.detach().double().requires_grad_()
    n = x64 * (x64.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * p64["norm.weight"]
    h = torch.nn.functional.silu(n @ p64["gate"].t()) * (n @ p64["up"].t())
    y64 = x64 + (h @ p64["down"].t()) * f
    y64.backward(dy.double())
    pairs = [(y.detach(), y64.detach(), "y"), (x.grad, x64.grad, "x")] + \
        [(p.grad, p64[n].grad, n) for n, p in block.named_parameters()]
    for got, want, name in pairs:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 1.5e-2, (name, rel)  # five roundings to bf16 in a row, 2^-8 of a value at most each
    block.eval()
    with torch.no_grad():
        assert torch.equal(block(x), F.fused_linear(F.gated_linear(block.norm(x), block.gate, block.up),
                                                    block.down, residual=x))


def test_training_step_through_norm_and_loss_head():
    """Block, dropout + residual + norm, loss head and clipping, in a row."""
    torch.manual_seed(1)
    M, H, V = 96, 64, 300
    block = F.GatedFeedForward(H, 96, device="cuda", norm_eps=1e-6)
    norm = F.FusedRMSNorm(H, dropout=0.1, device="cuda")
    head = torch.nn.Parameter(torch.randn(V, H, device="cuda").mul_(H ** -0.5).bfloat16())
    x = torch.randn(M, H, device="cuda").bfloat16().requires_grad_()
    t = torch.randint(0, V, (M,), device="cuda")
    branch = block(x)
    state = torch.cuda.get_rng_state()
    y, stream = norm(branch, x)
    loss = F.FusedLinearCrossEntropyLoss()(y, t, head)
    loss.backward()
    torch.cuda.set_rng_state(state)
    f = R.factors(M, H, 0.1, int(torch.empty(1, dtype=torch.int64, device="cuda").random_()))
    x64, b64 = x.detach().double().requires_grad_(), branch.detach().double().requires_grad_()
    h64 = x64 + b64 * f
    y64 = h64 * (h64.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    l64 = torch.nn.functional.cross_entropy(y64 @ head.detach().double().t(), t)
    l64.backward()
    loss, l64 = float(loss.detach()), float(l64.detach())
    assert abs(loss - l64) <= 2e-3 * l64
    params = [*block.parameters(), norm.weight, head]
    assert all(p.grad is not None and bool(p.grad.isfinite().all()) for p in params)
    total = sum(float(p.grad.double().square().sum()) for p in params) ** 0.5
    got = F.clip_grad_norm_(params, 1e-3)
    assert float(got) == pytest.approx(total, rel=1e-5)


def test_numbers_of_rows_share_no_memory_with_the_rows():
    buf = torch.zeros(8 * 64 + 8, dtype=FP32, device="cuda")
    x, tail = buf[:512].view(8, 64), buf[508:516]
    for call in (lambda: F.flce_rms_norm_forward(x, None, rstd=tail), lambda: F.flce_rms_norm_quantized(x, None, scale=tail),
                 lambda: F.flce_rms_norm_forward(torch.ones_like(x), None, out=x, rstd=tail)):
        with pytest.raises(ValueError, match="overlap"):
            call()
    F.flce_rms_norm_forward(x[:7], None, rstd=buf[512:519])


def test_a_seed_that_is_written_before_the_backward_is_an_error():
    """The gradients would be of another mask."""
    x = torch.randn(8, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda")
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    for call in (lambda: F.fused_dropout(x, 0.5, seed=seed), lambda: F.fused_rms_norm(x, w, dropout=0.5, seed=seed)[0]):
        y = call()
        seed.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        call().sum().backward()


@pytest.mark.parametrize("H", [257, 2049, 4100, 8193, 9000, 16388])
def test_wide_odd_rows_draw_the_same_masks(H):
    """Rows off 16-byte boundaries, of each number of threads and groups: the masks and sums of
    64 bits, in the norm, its backward and dropout by itself."""
    M, p, seed = 5, 0.25, 77
    g = torch.Generator(device="cuda").manual_seed(H)
    x, r, dy = (torch.randn(M, H, device="cuda", generator=g) for _ in range(3))
    f = R.factors(M, H, p, seed)
    rstd = torch.empty(M, device="cuda")
    y, h = F.flce_rms_norm_forward(x, None, r, dropout=p, seed=seed, rstd=rstd)
    h64 = r.double() + x.double() * f
    # One product and one sum, each rounded by half a step of up to 2 |x| + |r| < 16.
    assert float((h.double() - h64).abs().max()) <= 2 * 16 * 2.0 ** -24
    assert torch.equal(h, F.flce_dropout(x, p, seed, residual=r))
    n64 = h64 * (h64.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    # The root of the mean: a thread's sum of 32 terms, its tree and rsqrt, under 2^-18 together; |y| < 16.
    assert float((y.double() - n64).abs().max()) <= 16 * 2.0 ** -18
    dx, dr, _ = F.flce_rms_norm_backward(dy, h, None, rstd, dropout=p, seed=seed)
    assert torch.equal(dx == 0, f == 0)
    kept = f != 0
    scale = float(f.max())
    assert torch.equal(dx[kept], (dr * scale)[kept])


def test_equal_gradients_of_two_leaves_stay_apart():
    """dx and dresidual are one tensor where they are equal: the leaves' gradients are not, and a
    tensor that is both gets their sum."""
    x, w, r, dy, _ = problem(6, 64, FP32, FP32)
    x, r, w = (t.clone().requires_grad_() for t in (x, r, w))
    for times in (1, 2):
        y, h = F.fused_rms_norm(x, w, r)
        (y * dy + h).sum().backward()
        assert torch.equal(x.grad, r.grad)
    assert x.grad.data_ptr() != r.grad.data_ptr()
    kept = r.grad.clone()
    x.grad.zero_()
    assert torch.equal(r.grad, kept)
    y, h = F.fused_rms_norm(r, w, r)
    (both,) = torch.autograd.grad((y * dy + h).sum(), r)
    x2, r2 = r.detach().clone().requires_grad_(), r.detach().clone().requires_grad_()
    y, h = F.fused_rms_norm(x2, w, r2)
    (y * dy + h).sum().backward()
    assert torch.equal(both, x2.grad + r2.grad)
