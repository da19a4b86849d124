"""The layer operators against their plain 64-bit forms, within derived bounds."""
import ctypes

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
import block_reference as R
from linear_cross_entropy_gemm_gb300 import _lib

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]
# One token to several tiles of them; sizes around the 8-, 32-, 64-, 128- and 256-wide edges.
SHAPES = [(1, 64, 64), (1, 8, 1), (2, 72, 13), (7, 264, 40), (16, 512, 256), (17, 128, 127),
          (33, 200, 515), (64, 1024, 384), (65, 136, 8), (127, 72, 130), (128, 256, 256),
          (129, 64, 264), (200, 2056, 96), (256, 192, 1000), (257, 320, 513), (300, 640, 72),
          (513, 96, 136), (1000, 264, 300)]
# Long sums; more tiles than the GPU has places for them; few tiles of a long sum; rows that
# start between 32-byte sectors (K or N 8 modulo 16); operands that span little memory.
LONG = [(3, 16384, 520), (40, 8192, 1048), (150, 14336, 264), (700, 4096, 2304), (2049, 512, 4104),
        (267, 12808, 376), (600, 8200, 72), (2048, 4104, 4104), (2000, 4096, 8), (1100, 256, 3000)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def strided(t, pad, offset=0):
    """t's values in rows `pad` elements apart from dense, inside a poisoned buffer."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset + 64,), float("nan"), dtype=t.dtype, device=t.device)
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def poisoned(nbytes):
    return torch.full((max(nbytes, 1) + 512,), 255, dtype=torch.uint8, device="cuda")


def no_device_error():
    torch.cuda.synchronize()
    assert F.flce_read_device_error() == 0


def linear_problem(M, K, N, dtype, bias, res, seed=0):
    g = gen(seed + M * 7 + K * 3 + N)
    x, W = normal(g, M, K, dtype=dtype), normal(g, N, K, std=K ** -0.5, dtype=dtype)
    b = normal(g, N, std=0.5, dtype=dtype) if bias else None
    r = normal(g, M, N, dtype=dtype) if res else None
    return x, W, b, r, normal(g, M, N, std=0.1, dtype=dtype)


def check_linear(M, K, N, act, dtype=BF16, bias=True, res=True, dW_dtype=FP32, db_dtype=FP32):
    x, W, b, r, dy = linear_problem(M, K, N, dtype, bias, res)
    pre = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    y = F.flce_linear_forward(x, W, b, r, activation=act, pre=pre)
    lean = F.flce_linear_forward(x, W, b, r, activation=act)
    s_ref, y_ref = R.linear(x, W, b, r, act)
    slope = R.kept_slopes(pre)
    R.assert_within(y, y_ref, "y")
    R.assert_within(slope, s_ref, "kept slopes")
    assert torch.equal(y, lean)
    dx, dW, db = F.flce_linear_backward(dy, x, W, b, activation=act, pre=pre, dW_dtype=dW_dtype,
                                        db_dtype=db_dtype)
    want = R.linear_grad(dy, x, W, slope if act != "none" else None, dW_dtype, db_dtype)
    R.assert_within(dx, want[0], "dx")
    R.assert_within(dW, want[1], "dW")
    if bias:
        R.assert_within(db, want[2], "db")
    else:
        assert db is None
    no_device_error()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_shapes(shape, act):
    check_linear(*shape, act)


@pytest.mark.parametrize("shape", LONG, ids=str)
def test_linear_long(shape):
    check_linear(*shape, "gelu", dtype=FP16)


@pytest.mark.parametrize("M", [3, 130, 300])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_linear_activations(M, act, dtype):
    check_linear(M, 136, 264, act, dtype=dtype, dW_dtype=dtype, db_dtype=dtype)


@pytest.mark.parametrize("M", [5, 140])
@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True)])
def test_linear_parts(M, bias, res):
    check_linear(M, 96, 200, "none", bias=bias, res=res)
    check_linear(M, 96, 77, "relu", bias=bias, res=res)


@pytest.mark.parametrize("M,K,N", [(1, 64, 48), (50, 136, 77), (200, 72, 264), (300, 256, 128)])
@pytest.mark.parametrize("pad", [8, 24])
def test_linear_strides(M, K, N, pad):
    """Strided x, residual, output and dy; residual and output at any element offset."""
    x, W, b, r, dy = linear_problem(M, K, N, BF16, True, True)
    dense = F.flce_linear_forward(x, W, b, r, activation="gelu")
    for off in (0, 3):
        out_buf = torch.full((M * (N + pad) + 64,), 7.0, dtype=BF16, device="cuda")
        out = out_buf[off:off + M * (N + pad)].view(M, N + pad)[:, :N]
        got = F.flce_linear_forward(strided(x, pad), W, b, strided(r, pad - 1, off),
                                    activation="gelu", out=out)
        assert got is out and torch.equal(out, dense)
        rest = out_buf.clone()
        rest[off:off + M * (N + pad)].view(M, N + pad)[:, :N] = 7.0
        assert bool((rest == 7.0).all()), "wrote outside the output"
    ref = F.flce_linear_backward(dy, x, W, b)
    for off, p in ((0, pad), (1, pad - 1)):
        got = F.flce_linear_backward(strided(dy, p, off), strided(x, pad), W, b)
        for a, c in zip(got, ref):
            assert torch.equal(a, c)
    no_device_error()


@pytest.mark.parametrize("N", [66, 131, 258, 1025])
@pytest.mark.parametrize("M,dtype", [(135, BF16), (300, FP16), (1500, BF16)])
def test_linear_rows_off_the_16_byte_boundaries(M, N, dtype):
    """Even and odd counts of columns that are no multiple of 8: the output, the kept slopes and
    the residual, also when the output is the residual."""
    check_linear(M, 72, N, "gelu_tanh", dtype=dtype)
    x, W, b, r, _ = linear_problem(M, 72, N, dtype, True, True)
    want = F.flce_linear_forward(x, W, b, r, activation="gelu_tanh")
    for pad, off in ((0, 1), (0, 2), (1, 0), (2, 2), (3, 1)):
        own = strided(r, pad, off)
        around = own.as_strided((M, N + pad), (N + pad, 1), own.storage_offset())[:-1, N:].clone()
        got = F.flce_linear_forward(x, W, b, own, activation="gelu_tanh", out=own)
        assert got is own and torch.equal(own, want)
        after = own.as_strided((M, N + pad), (N + pad, 1), own.storage_offset())[:-1, N:]
        assert torch.equal(after.view(torch.int16), around.view(torch.int16)), "wrote between the rows"
    no_device_error()


def test_linear_output_may_be_the_residual():
    for M in (4, 300):
        x, W, b, r, _ = linear_problem(M, 128, 200, BF16, True, True)
        want = F.flce_linear_forward(x, W, b, r)
        got = F.flce_linear_forward(x, W, b, r, out=r)
        assert got is r and torch.equal(r, want)


@pytest.mark.parametrize("M", [6, 300])
def test_workspace_contents_do_not_matter(M):
    x, W, b, r, dy = linear_problem(M, 1032, 200, BF16, True, True)
    ws = poisoned(1 << 24)
    pre = torch.empty(M, 200, dtype=BF16, device="cuda")
    a = F.flce_linear_forward(x, W, b, r, activation="silu", pre=pre)
    assert torch.equal(a, F.flce_linear_forward(x, W, b, r, activation="silu", workspace=ws))
    one = F.flce_linear_backward(dy, x, W, b, activation="silu", pre=pre)
    two = F.flce_linear_backward(dy, x, W, b, activation="silu", pre=pre, workspace=poisoned(1 << 24))
    for p, q in zip(one, two):
        assert torch.equal(p, q)
    g = torch.empty(2, M, 200, dtype=BF16, device="cuda")
    h = F.flce_gated_forward(x, W, W, pre=g)
    assert torch.equal(h, F.flce_gated_forward(x, W, W, workspace=poisoned(1 << 24)))
    one = F.flce_gated_backward(dy, x, W, W, g)
    two = F.flce_gated_backward(dy, x, W, W, g, workspace=poisoned(1 << 24))
    for p, q in zip(one, two):
        assert torch.equal(p, q)


@pytest.mark.parametrize("offset", [0, 8])
@pytest.mark.parametrize("M,K,N", [(5, 64, 24), (300, 264, 77), (2048, 1032, 1032), (600, 8200, 72)])
def test_c_abi_stays_inside_its_workspace(M, K, N, offset):
    """The C entry points with a workspace of exactly the size they ask for, at any
    address, give what the Python calls give and write nothing behind it."""
    lib = _lib.load()
    x, W, b, r, dy = linear_problem(M, K, N, BF16, True, True)
    stream = torch.cuda.current_stream().cuda_stream
    word = F.device_error_word("cuda:0").data_ptr()

    def scratch(need):
        buf = torch.full((need + offset + 64,), 7, dtype=torch.uint8, device="cuda")
        return buf, buf.data_ptr() + offset

    def untouched(buf, need):
        return bool((buf[:offset] == 7).all()) and bool((buf[offset + need:] == 7).all())

    p = _lib.FlceLinearParams(M=M, K=K, N=N, activation=4, has_bias=1, has_residual=1)
    at = ctypes.addressof(p)
    y, pre = torch.empty_like(r), torch.empty_like(r)
    need = lib.flce_linear_workspace_size(at, 0)
    buf, ws = scratch(need)
    assert lib.flce_linear_forward(at, x.data_ptr(), W.data_ptr(), b.data_ptr(), r.data_ptr(),
                                   y.data_ptr(), pre.data_ptr(), ws, need, word, stream) == 0
    assert untouched(buf, need)
    want_pre = torch.empty_like(r)
    assert torch.equal(y, F.flce_linear_forward(x, W, b, r, activation="silu", pre=want_pre))
    assert torch.equal(pre.view(torch.int16), want_pre.view(torch.int16))
    dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty_like(b)
    need = lib.flce_linear_workspace_size(at, 1)
    buf, ws = scratch(need)
    assert lib.flce_linear_backward(at, dy.data_ptr(), x.data_ptr(), W.data_ptr(), pre.data_ptr(),
                                    dx.data_ptr(), dW.data_ptr(), db.data_ptr(), ws, need, word,
                                    stream) == 0
    assert untouched(buf, need)
    assert lib.flce_linear_backward(at, dy.data_ptr(), x.data_ptr(), W.data_ptr(), pre.data_ptr(),
                                    dx.data_ptr(), dW.data_ptr(), db.data_ptr(), ws, need - 1, word,
                                    stream) == 3
    for got, want in zip((dx, dW, db), F.flce_linear_backward(
            dy, x, W, b, activation="silu", pre=pre, dW_dtype=BF16, db_dtype=BF16)):
        assert torch.equal(got, want)
    if N % 8:
        return
    p = _lib.FlceGatedParams(M=M, K=K, F=N, activation=4)
    at = ctypes.addressof(p)
    pre = torch.empty(2, M, N, dtype=BF16, device="cuda")
    need = lib.flce_gated_workspace_size(at, 0)
    buf, ws = scratch(need)
    assert lib.flce_gated_forward(at, x.data_ptr(), W.data_ptr(), W.data_ptr(), y.data_ptr(),
                                  pre.data_ptr(), ws, need, word, stream) == 0
    assert untouched(buf, need) and torch.equal(y, F.flce_gated_forward(x, W, W))
    dWu = torch.empty_like(W)
    need = lib.flce_gated_workspace_size(at, 1)
    buf, ws = scratch(need)
    assert lib.flce_gated_backward(at, dy.data_ptr(), x.data_ptr(), W.data_ptr(), W.data_ptr(),
                                   pre.data_ptr(), dx.data_ptr(), dW.data_ptr(), dWu.data_ptr(), ws,
                                   need, word, stream) == 0
    assert untouched(buf, need)
    for got, want in zip((dx, dW, dWu),
                         F.flce_gated_backward(dy, x, W, W, pre, dW_dtype=BF16)):
        assert torch.equal(got, want)
    no_device_error()


def test_linear_needs():
    x, W, b, _, dy = linear_problem(70, 64, 96, BF16, True, False)
    full = F.flce_linear_backward(dy, x, W, b)
    for needs in [(True, False, False), (False, True, False), (False, False, True), (False,) * 3]:
        got = F.flce_linear_backward(dy, x, W, b, needs=needs)
        for want, have, need in zip(full, got, needs):
            assert (have is None) == (not need)
            assert have is None or torch.equal(have, want)


def test_no_tokens():
    W = normal(gen(1), 16, 64)
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert F.flce_linear_forward(x, W).shape == (0, 16)
    b = normal(gen(2), 16)
    dx, dW, db = F.flce_linear_backward(torch.empty(0, 16, dtype=BF16, device="cuda"), x, W, b)
    assert dx.shape == (0, 64) and not dW.any() and not db.any()
    assert F.flce_gated_forward(x, W, W).shape == (0, 16)
    pre = torch.empty(2, 0, 16, dtype=BF16, device="cuda")
    dx, dWg, dWu = F.flce_gated_backward(torch.empty(0, 16, dtype=BF16, device="cuda"), x, W, W, pre)
    assert dx.shape == (0, 64) and not dWg.any() and not dWu.any()


@pytest.mark.parametrize("M", [3, 40, 300])
def test_a_bad_token_stays_in_its_row(M):
    """NaN and infinity in one token's row leave the other rows as they were."""
    x, W, b, r, dy = linear_problem(M, 264, 136, BF16, True, True)
    clean = F.flce_linear_forward(x, W, b, r, activation="silu")
    h = F.flce_gated_forward(x, W, W)
    dx = F.flce_linear_backward(dy, x, W, b)[0]
    bad = x.clone()
    bad[1, 5], bad[1, 77] = float("nan"), float("inf")
    keep = torch.arange(M, device="cuda") != 1
    y = F.flce_linear_forward(bad, W, b, r, activation="silu")
    assert torch.equal(y[keep], clean[keep]) and bool(y[1].isnan().all())
    y = F.flce_gated_forward(bad, W, W)
    assert torch.equal(y[keep], h[keep]) and bool(y[1].isnan().all())
    bad = dy.clone()
    bad[1, 3] = float("nan")
    y = F.flce_linear_backward(bad, x, W, b)[0]
    assert torch.equal(y[keep], dx[keep]) and bool(y[1].isnan().all())
    pre, bad_pre = (torch.empty(2, M, 136, dtype=BF16, device="cuda") for _ in range(2))
    bad = x.clone()
    bad[1, 5] = float("inf")
    F.flce_gated_forward(x, W, W, pre=pre)
    F.flce_gated_forward(bad, W, W, pre=bad_pre)
    dx = F.flce_gated_backward(dy, x, W, W, pre)[0]
    y, dWg, dWu = F.flce_gated_backward(dy, bad, W, W, bad_pre)
    assert torch.equal(y[keep], dx[keep]) and not bool(y[1].isfinite().any())
    assert not bool(dWg.isfinite().any()) and not bool(dWu.isfinite().any())
    F.flce_linear_forward(bad, W, b, activation="silu", pre=pre[0])
    dW = F.flce_linear_backward(dy, bad, W, b, activation="silu", pre=pre[0])[1]
    assert not bool(dW.isfinite().all())


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("M", [5, 200])
def test_kept_groups_keep_their_precision_at_any_size(M, scale):
    """u from tiny to huge: the kept u a'(g) stays within 2^-14 of its group's largest."""
    x, Wg, Wu, dh = gated_problem(M, 64, 72, BF16)
    Wu = (Wu.double() * scale).to(BF16)
    pre = torch.empty(2, M, 72, dtype=BF16, device="cuda")
    h = F.flce_gated_forward(x, Wg, Wu, pre=pre)
    v_ref, c_ref, h_ref = R.gated(x, Wg, Wu, "silu")
    R.assert_within(h, h_ref, "h")
    R.assert_within(R.kept_groups(pre[1]), c_ref, "kept u a'(g)")
    got = F.flce_gated_backward(dh, x, Wg, Wu, pre)
    for a, want in zip(got, R.gated_grad(dh, x, Wg, Wu, R.kept_groups(pre[0]),
                                         R.kept_groups(pre[1]), FP32)):
        R.assert_within(a, want, "gradient")


@pytest.mark.parametrize("act", ACTS)
def test_activation_range(act):
    """z from far below to far above 0, where the exponentials overflow: finite everywhere."""
    z = torch.cat((torch.linspace(-300, 300, 513), torch.tensor([0.0, -0.0, 1e4, -1e4, 3e38, -3e38,
                                                                  1e-30])))
    x = z.to(BF16).cuda().view(-1, 1).repeat(1, 8)
    x[:, 1:] = 0
    W = torch.eye(8, dtype=BF16, device="cuda")
    pre = torch.empty_like(x)
    y = F.flce_linear_forward(x, W, activation=act, pre=pre)
    want, slope = R.act(x.double(), act)
    R.assert_within(R.kept_slopes(pre), (slope, torch.full_like(slope, 2.0 ** -15 + 4 * R.ACT)),
                    "kept slopes")
    bound = R.rounded(want, R.ACT * (x.double().abs() + 1), BF16)
    R.assert_within(y, (want, bound), "y")
    dy = torch.ones_like(x)
    dx = F.flce_linear_backward(dy, x, W, activation=act, pre=pre, needs=(True, False, False))[0]
    R.assert_within(dx, (slope, R.rounded(slope, torch.full_like(slope, 2.0 ** -15 + 4 * R.ACT), BF16)), "a'")


# -------------------------------------------------------------------- gated
def gated_problem(M, K, N, dtype, seed=0):
    g = gen(seed + M * 5 + K * 11 + N)
    x = normal(g, M, K, dtype=dtype)
    Wg, Wu = (normal(g, N, K, std=K ** -0.5, dtype=dtype) for _ in range(2))
    return x, Wg, Wu, normal(g, M, N, std=0.1, dtype=dtype)


def check_gated(M, K, N, act, dtype=BF16, dW_dtype=FP32):
    x, Wg, Wu, dh = gated_problem(M, K, N, dtype)
    pre = torch.full((2, M, N), float("nan"), dtype=dtype, device="cuda")
    h = F.flce_gated_forward(x, Wg, Wu, activation=act, pre=pre)
    assert torch.equal(h, F.flce_gated_forward(x, Wg, Wu, activation=act))
    v_ref, c_ref, h_ref = R.gated(x, Wg, Wu, act)
    val, cross = R.kept_groups(pre[0]), R.kept_groups(pre[1])
    R.assert_within(val, v_ref, "kept a(g)")
    R.assert_within(cross, c_ref, "kept u a'(g)")
    R.assert_within(h, h_ref, "h")
    got = F.flce_gated_backward(dh, x, Wg, Wu, pre, activation=act, dW_dtype=dW_dtype)
    for a, want, what in zip(got, R.gated_grad(dh, x, Wg, Wu, val, cross, dW_dtype),
                             ("dx", "dWg", "dWu")):
        R.assert_within(a, want, what)
    no_device_error()


@pytest.mark.parametrize("shape", [(M, K, -(-N // 8) * 8) for M, K, N in SHAPES], ids=str)
def test_gated_shapes(shape):
    check_gated(*shape, "silu")


@pytest.mark.parametrize("shape", LONG, ids=str)
def test_gated_long(shape):
    check_gated(*shape, "gelu", dtype=FP16)


@pytest.mark.parametrize("shape", LONG, ids=str)
def test_linear_long_without_activation(shape):
    check_linear(*shape, "none", bias=False)


@pytest.mark.parametrize("M", [3, 130])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_gated_activations(M, act, dtype):
    check_gated(M, 136, 264, act, dtype=dtype, dW_dtype=dtype)


@pytest.mark.parametrize("M", [1, 50, 300])
def test_gated_strides_and_needs(M):
    x, Wg, Wu, dh = gated_problem(M, 136, 72, BF16)
    pre = torch.empty(2, M, 72, dtype=BF16, device="cuda")
    want = F.flce_gated_forward(x, Wg, Wu, pre=pre)
    buf = torch.full((M, 96), 7.0, dtype=BF16, device="cuda")
    got = F.flce_gated_forward(strided(x, 8), Wg, Wu, out=buf[:, 8:80])
    assert torch.equal(got, want) and bool((buf[:, :8] == 7).all() and (buf[:, 80:] == 7).all())
    full = F.flce_gated_backward(dh, x, Wg, Wu, pre)
    for a, b in zip(F.flce_gated_backward(strided(dh, 8), strided(x, 16), Wg, Wu, pre), full):
        assert torch.equal(a, b)
    only_x = F.flce_gated_backward(dh, x, Wg, Wu, pre, needs=(True, False))
    only_w = F.flce_gated_backward(dh, x, Wg, Wu, pre, needs=(False, True))
    assert torch.equal(only_x[0], full[0]) and only_x[1] is None and only_x[2] is None
    assert only_w[0] is None and torch.equal(only_w[1], full[1]) and torch.equal(only_w[2], full[2])


# ------------------------------------------------- gradients against differences
def directional(f, t, d, h=1e-4):
    return float((f(t + h * d) - f(t - h * d)) / (2 * h))


@pytest.mark.parametrize("M", [9, 150])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "sigmoid"])
def test_gradients_against_differences(M, act):
    """<gradient, direction> against a central difference of the 64-bit definition.
    The kept slopes are off by 2^-15, the kept groups by 2^-14 of their largest; dz, dg, du
    and the gradients are rounded to u of their size. h^2 times the third derivative is
    far below that."""
    g = gen(M)
    x, W, b, r, dy = linear_problem(M, 72, 88, BF16, True, True)

    def loss(x_, W_, b_):
        return (R.act(x_ @ W_.t() + b_, act)[0] * dy.double()).sum()

    x64, W64, b64 = x.double(), W.double(), b.double()
    pre = torch.empty(M, 88, dtype=BF16, device="cuda")
    F.flce_linear_forward(x, W, b, r, activation=act, pre=pre)
    grads = F.flce_linear_backward(dy, x, W, b, activation=act, pre=pre)
    u = R.UNIT[BF16]
    dz_off = (1.2 * u + 2.0 ** -14) * dy.double().abs()
    offs = (dz_off @ W64.abs(), dz_off.t() @ x64.abs(), dz_off.sum(0))
    for i, (t, off) in enumerate(zip((x64, W64, b64), offs)):
        d = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)

        def f(v):
            return loss(*[v if k == i else q for k, q in enumerate((x64, W64, b64))])

        got = float((grads[i].double() * d).sum())
        bound = float(((off + u * grads[i].double().abs()) * d.abs()).sum())
        assert abs(got - directional(f, t, d)) <= bound

    Wu = normal(g, 88, 72, std=72 ** -0.5)
    Wu64 = Wu.double()

    def gated_loss(x_, Wg_, Wu_):
        return (R.act(x_ @ Wg_.t(), act)[0] * (x_ @ Wu_.t()) * dy.double()).sum()

    pre = torch.empty(2, M, 88, dtype=BF16, device="cuda")
    F.flce_gated_forward(x, W, Wu, activation=act, pre=pre)
    grads = F.flce_gated_backward(dy, x, W, Wu, pre, activation=act)
    val, cross = R.kept_groups(pre[0]), R.kept_groups(pre[1])
    d, none = dy.double().abs(), torch.zeros_like(val)
    dg_off = d * (u * cross.abs() + 2 * R.group_off(cross, none))
    du_off = d * (u * val.abs() + 2 * R.group_off(val, none))
    offs = (dg_off @ W64.abs() + du_off @ Wu64.abs(), dg_off.t() @ x64.abs(),
            du_off.t() @ x64.abs())
    for i, (t, off) in enumerate(zip((x64, W64, Wu64), offs)):
        d = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)

        def f(v):
            return gated_loss(*[v if k == i else q for k, q in enumerate((x64, W64, Wu64))])

        got = float((grads[i].double() * d).sum())
        bound = float(((off + u * grads[i].double().abs()) * d.abs()).sum())
        assert abs(got - directional(f, t, d)) <= bound


# ------------------------------------------------------- gradient norm, clipping
def grad_list(sizes, types, seed=0, offset=0):
    g = gen(seed)
    out = []
    for i, n in enumerate(sizes):
        t = types[i % len(types)]
        buf = torch.empty(n + offset + 8, dtype=t, device="cuda")
        buf[offset:offset + n].copy_(torch.randn(n, generator=g, device="cuda") * 10.0 ** (-(i % 4)))
        out.append(buf[offset:offset + n])
    return out


def norm64(grads):
    return sum(float(g.double().square().sum()) for g in grads) ** 0.5


LISTS = [[1], [7], [8], [1, 2, 3, 0, 5], [16384], [16385, 1, 8191], [100000, 3, 65536, 0, 12345],
         [1 << 21, 31], [5] * 70, [1000] * 300, [17] * 1100, [3000000, 9, 700001, 2500000]]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("types", [(BF16,), (FP16,), (FP32,), (BF16, FP32, FP16)],
                         ids=["bf16", "fp16", "fp32", "mixed"])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_and_clip(sizes, types, offset):
    grads = grad_list(sizes, types, offset=offset)
    want = norm64(grads)
    got = F.flce_grad_norm(grads)
    # 64 fp32 adds at most, then fp64, one rounding to fp32.
    tol = (64 * 2.0 ** -24 + 2.0 ** -23) * want
    assert got.shape == () and got.dtype == FP32 and abs(float(got) - want) <= tol
    max_norm = 0.37 * want
    c = max_norm / (want + 1e-6)
    for out_off in (offset, offset + 1):
        outs = [torch.full((g.numel() + 16,), 7.0, dtype=g.dtype, device="cuda") for g in grads]
        views = [o[out_off:out_off + g.numel()] for o, g in zip(outs, grads)]
        n = F.flce_clip_grads(grads, max_norm, out=views)
        assert torch.equal(n, got)
        for g, v, o in zip(grads, views, outs):
            ref = g.double() * c
            R.assert_within(v, (ref, R.rounded(ref, ref.abs() * 2.0 ** -17, g.dtype)), "clipped")
            assert bool((o[:out_off] == 7).all() and (o[out_off + g.numel():] == 7).all())
    places = [g.clone() for g in grads]
    F.flce_clip_grads(places, max_norm)
    for p, g in zip(places, grads):
        ref = g.double() * c
        R.assert_within(p, (ref, R.rounded(ref, ref.abs() * 2.0 ** -17, g.dtype)), "clipped in place")
    same = [g.clone() for g in grads]
    F.flce_clip_grads(same, 2 * want + 1)
    for a, b in zip(same, grads):
        assert torch.equal(a, b)


def test_norm_of_nothing_and_of_bad_values():
    empty = torch.empty(0, device="cuda")
    assert float(F.flce_grad_norm([empty])) == 0.0
    assert float(F.flce_clip_grads([empty, empty], 1.0)) == 0.0
    g = torch.ones(5000, device="cuda")
    h = g.clone()
    h[4999] = float("inf")
    assert float(F.flce_grad_norm([g, h])) == float("inf")
    F.flce_clip_grads([g, h], 1.0)
    assert not g.any() and bool(h[4999].isnan()) and not h[:4999].any()
    g = torch.ones(5000, dtype=BF16, device="cuda")
    g[17] = float("nan")
    assert bool(F.flce_grad_norm([g]).isnan())
    F.flce_clip_grads([g], 1.0)
    assert bool(g.isnan().all())


def test_norm_takes_any_dense_layout_and_repeats_bit_for_bit():
    a = torch.randn(300, 70, device="cuda")
    assert torch.equal(F.flce_grad_norm([a.t()]), F.flce_grad_norm([a]))
    b = torch.randn(5, 6, 7, device="cuda").permute(2, 0, 1)
    c = b.clone(memory_format=torch.preserve_format)
    F.flce_clip_grads([c], 1.0)
    torch.testing.assert_close(c, b * (1.0 / (b.norm() + 1e-6)), rtol=1e-5, atol=0)
    grads = grad_list([999, 123457, 31, 2000001], (BF16, FP32))
    first = F.flce_grad_norm(grads)
    for _ in range(5):
        assert torch.equal(F.flce_grad_norm(grads), first)


# ----------------------------------------------------- streams, graphs, autograd
def test_own_stream_and_graph():
    M = 20
    x, W, b, r, dy = linear_problem(M, 512, 264, BF16, True, True)
    want = F.flce_linear_forward(x, W, b, r, activation="gelu")
    hw = F.flce_gated_forward(x, W, W)
    grads = [torch.randn(5000, device="cuda")]
    nw = F.flce_grad_norm(grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = F.flce_linear_forward(x, W, b, r, activation="gelu", stream=s)
    h = F.flce_gated_forward(x, W, W, stream=s.cuda_stream)
    n = F.flce_grad_norm(grads, stream=s)
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(h, hw) and torch.equal(n, nw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = F.flce_linear_forward(x, W, b, r, activation="gelu")
        h = F.flce_gated_forward(x, W, W)
        n = F.flce_clip_grads(grads, 1e30)
    y.zero_(), h.zero_(), n.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, hw) and torch.equal(n, nw)


def test_feed_forward_block_head_and_clipping_together():
    """One training step of a block and the loss head, and its clipped gradients,
    against autograd in 64 bits over the same (16-bit) values."""
    torch.manual_seed(0)
    N, H, FF, V = 150, 128, 264, 500
    block = F.GatedFeedForward(H, FF, device="cuda")
    head = torch.nn.Parameter(torch.randn(V, H, device="cuda").mul_(0.1).to(BF16))
    x = torch.randn(3, N // 3, H, device="cuda").to(BF16).requires_grad_()
    y = torch.randint(0, V, (3, N // 3), device="cuda")
    loss = F.FusedLinearCrossEntropyLoss()(block(x), y, head)
    loss.backward()
    params = [block.gate, block.up, block.down, head]
    ref = [p.detach().double().requires_grad_() for p in params + [x]]
    x64 = ref[4].reshape(N, H)
    out = x64 + (torch.nn.functional.silu(x64 @ ref[0].t()) * (x64 @ ref[1].t())) @ ref[2].t()
    want = torch.nn.functional.cross_entropy(out @ ref[3].t(), y.reshape(-1))
    want.backward()
    assert abs(float(loss.detach()) - float(want.detach())) <= 1e-2
    for p, q in zip(params + [x], ref):
        err = float((p.grad.double() - q.grad).norm() / q.grad.norm())
        assert err <= 3e-2, err  # eight roundings of 2^-8 (h, g, u, dg, du, dL, y and the gradient)
    before = [p.grad.clone() for p in params]
    norm = F.clip_grad_norm_(params, 1e-3)
    total = norm64(before)
    assert abs(float(norm) - total) <= 1e-5 * total
    for p, g in zip(params, before):
        scaled = g.double() * (1e-3 / (total + 1e-6))
        R.assert_within(p.grad, (scaled, R.rounded(scaled, scaled.abs() * 1e-5, BF16)), "clipped")
    no_device_error()


def test_example_trains():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, norms = example.train(tokens=300, hidden=128, features=264, vocab=500, steps=6)
    assert losses[-1] < losses[0] and all(n > 0 for n in norms)
    no_device_error()


def test_autograd_forms_copy_what_the_kernels_cannot_read():
    g = gen(4)
    base = normal(g, 40, 72)
    x = base[:, 3:67].detach().requires_grad_()  # rows off the 16-byte boundaries
    W, b = normal(g, 24, 64).requires_grad_(), normal(g, 24).requires_grad_()
    r = normal(g, 24, 40).t().requires_grad_()
    y = F.fused_linear(x, W, b, r, activation="silu")
    dy = normal(g, 24, 40).t()
    y.backward(dy)
    xc = x.detach().contiguous()
    pre = torch.empty(40, 24, dtype=BF16, device="cuda")
    want = F.flce_linear_forward(xc, W.detach(), b.detach(), r.detach().contiguous(),
                                 activation="silu", pre=pre)
    grads = F.flce_linear_backward(dy.contiguous(), xc, W.detach(), b.detach(), activation="silu",
                                   pre=pre, dW_dtype=BF16, db_dtype=BF16)
    assert torch.equal(y, want) and torch.equal(r.grad, dy)
    for t, w in zip((x, W, b), grads):
        assert torch.equal(t.grad, w)


# ---------------------------------------------------------------- refusals
def test_refusals():
    g = gen(3)
    x, W, b = normal(g, 4, 64), normal(g, 16, 64), normal(g, 16)
    with pytest.raises(TypeError):
        F.flce_linear_forward(x.float(), W)
    with pytest.raises(TypeError):
        F.flce_linear_forward(x, W.half())
    with pytest.raises(ValueError):
        F.flce_linear_forward(x, W[:, :32])
    with pytest.raises(ValueError):
        F.flce_linear_forward(x, W, b[:8])
    with pytest.raises(ValueError):
        F.flce_linear_forward(x, W, activation="tanh")
    with pytest.raises(ValueError):
        F.flce_linear_forward(x, W, residual=normal(g, 4, 15))
    with pytest.raises(ValueError):
        F.flce_linear_forward(x.t().contiguous().t(), W)
    with pytest.raises(F.FlceError):  # K not a multiple of 8
        F.flce_linear_forward(normal(g, 4, 12), normal(g, 16, 12))
    with pytest.raises(F.FlceError):  # rows of x off the 16-byte boundaries
        F.flce_linear_forward(strided(x, 3), W)
    with pytest.raises(F.FlceError):
        F.flce_linear_forward(strided(x, 8, 1), W)
    with pytest.raises(ValueError):
        F.flce_linear_backward(normal(g, 4, 16), x, W, activation="silu")
    with pytest.raises(TypeError):
        F.flce_linear_backward(normal(g, 4, 16), x, W, dW_dtype=FP16)
    with pytest.raises(ValueError):
        F.flce_gated_forward(x, W, W[:8])
    with pytest.raises(F.FlceError):  # F not a multiple of 8
        F.flce_gated_forward(x, normal(g, 12, 64), normal(g, 12, 64))
    with pytest.raises(ValueError):
        F.flce_gated_backward(normal(g, 4, 16), x, W, W, torch.empty(2, 4, 8, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        F.flce_grad_norm([])
    with pytest.raises(TypeError):
        F.flce_grad_norm([torch.zeros(4, dtype=torch.float64, device="cuda")])
    with pytest.raises(TypeError):
        F.flce_grad_norm([torch.zeros(4)])
    with pytest.raises(ValueError):
        F.flce_grad_norm([torch.zeros(4, 6, device="cuda")[:, :5]])
    with pytest.raises(F.FlceError):
        F.flce_clip_grads([torch.zeros(4, device="cuda")], -1.0)
    with pytest.raises(F.FlceError):
        F.flce_clip_grads([torch.zeros(4, device="cuda")], float("nan"))
    with pytest.raises(ValueError):
        F.flce_clip_grads([torch.zeros(4, device="cuda")], 1.0, out=[])
    with pytest.raises(TypeError):
        F.flce_clip_grads([torch.zeros(4, device="cuda")], 1.0,
                          out=[torch.zeros(4, dtype=BF16, device="cuda")])
    with pytest.raises(ValueError):
        F.flce_clip_grads([torch.zeros(4, 2, device="cuda")], 1.0,
                          out=[torch.zeros(2, 4, device="cuda").t()])
    no_device_error()
