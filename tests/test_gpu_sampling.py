"""Sampling from logits against the definition in 64 bits: the same tokens."""
import itertools

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
import stream_reference as R

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def words(g, B, V, sharp=1.0):
    """Logits with a wide bulk and some likely words."""
    z = torch.randn(B, V, generator=g, device="cuda") * 2
    z += torch.rand(B, V, generator=g, device="cuda").pow(60) * 12
    return z * sharp


def check(z, u, **kw):
    """The call's tokens are the reference's, row by row."""
    got = F.flce_sample(z, u, **kw)
    assert got.dtype == torch.int64 and got.shape == (z.shape[0],)
    rows = {k: v.tolist() if torch.is_tensor(v) else [v] * z.shape[0] for k, v in kw.items()
            if k in ("temperature", "top_k", "top_p", "min_p")}
    zs, us = z.float().cpu(), u.tolist()
    want = [R.sample(zs[b], us[b], **{k: v[b] for k, v in rows.items()}) for b in range(z.shape[0])]
    assert got.tolist() == want
    return got


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.3), dict(top_k=1), dict(top_k=40),
            dict(top_k=5000, temperature=1.5), dict(top_p=0.9), dict(top_p=0.1), dict(top_p=0.999, temperature=2.0),
            dict(min_p=0.05), dict(min_p=1.0), dict(top_k=50, top_p=0.8, min_p=0.1, temperature=0.7),
            dict(top_k=3000, top_p=0.99, temperature=3.0)]


@pytest.mark.parametrize("kw", SETTINGS, ids=str)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
@pytest.mark.parametrize("B,V", [(1, 1), (3, 5), (2, 257), (7, 1000), (33, 4099), (2, 50257), (160, 9000)])
def test_sample(B, V, dtype, kw):
    g = gen(B * 1000003 + V)
    z = words(g, B, V).to(dtype)
    check(z, torch.rand(B, generator=g, device="cuda"), **kw)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
def test_large_vocabularies(dtype):
    g = gen(4)
    z = words(g, 3, 1 << 20).to(dtype)
    u = torch.rand(3, generator=g, device="cuda")
    for kw in (dict(), dict(top_k=100, top_p=0.9), dict(top_p=0.97), dict(top_k=30000)):
        check(z, u, **kw)


def test_a_setting_for_each_row():
    g = gen(5)
    B, V = 90, 3001
    z, u = words(g, B, V), torch.rand(B, generator=g, device="cuda")
    rows = list(itertools.product((0.0, 0.6, 1.4), (0, 1, 7, 200, 5000), (1.0, 0.5), (0.0, 0.1, 1.0)))[:B]
    t, k, p, m = (torch.tensor(c, device="cuda") for c in zip(*rows))
    kw = dict(temperature=t.float(), top_k=k.int(), top_p=p.float(), min_p=m.float())
    check(z, u, **kw)
    check(z, u, **{**kw, "top_k": 30})
    # Values out of range in a tensor: as the documentation has it.
    odd = dict(temperature=torch.tensor([-1.0, float("nan"), 1.0, 1.0, 1.0, 1.0, 1.0, 1.0], device="cuda"),
               top_k=torch.tensor([0, 0, -3, 0, 0, 0, 0, 0], dtype=torch.int32, device="cuda"),
               top_p=torch.tensor([1.0, 1, 1, 7, -2, float("nan"), 1, 1], device="cuda"),
               min_p=torch.tensor([0.0, 0, 0, 0, 0, 0, 3, float("nan")], device="cuda"))
    same = dict(temperature=torch.tensor([0.0, 0, 1, 1, 1, 1, 1, 1], device="cuda"),
                top_k=torch.zeros(8, dtype=torch.int32, device="cuda"),
                top_p=torch.tensor([1.0, 1, 1, 1, 0, 0, 1, 1], device="cuda"),
                min_p=torch.tensor([0.0, 0, 0, 0, 0, 0, 1, 0], device="cuda"))
    assert torch.equal(F.flce_sample(z[:8], u[:8], **odd), F.flce_sample(z[:8], u[:8], **same))


def test_ties():
    """Equal logits: the lower index comes first, in more of them than are ever sorted."""
    V = 20000
    z = torch.zeros(5, V, device="cuda")
    z[1, ::2] = 1.0
    z[2] = -0.0
    z[2, ::3] = 0.0  # the zeros are equal
    z[3, 5000:] = -1.0
    z[4] = (torch.arange(V, device="cuda") % 3).float()
    u = torch.tensor([0.999, 0.3, 0.7, 0.9999, 0.5], device="cuda")
    for kw in (dict(), dict(top_k=7), dict(top_k=9000), dict(top_p=0.25), dict(top_p=0.5), dict(min_p=1.0),
               dict(top_k=15000, top_p=0.9), dict(top_k=6667), dict(temperature=0.0)):
        check(z, u, **kw)
        check(z.bfloat16(), u, **kw)


def test_flat_distributions():
    """Nuclei of thousands of different logits."""
    g = gen(6)
    z = torch.randn(4, 60000, generator=g, device="cuda") * torch.tensor([[1e-3], [0.3], [1.0], [30.0]], device="cuda")
    u = torch.rand(4, generator=g, device="cuda")
    for kw in (dict(), dict(top_p=0.5), dict(top_p=0.999), dict(top_k=30000), dict(top_k=30000, top_p=0.7),
               dict(temperature=50.0, top_p=0.3), dict(temperature=INF), dict(temperature=INF, top_p=0.5)):
        check(z, u, **kw)


def test_masked_and_non_finite():
    V = 3000
    g = gen(7)
    z = words(g, 8, V)
    z[0] = -INF                    # nothing left
    z[1, 17] = float("nan")
    z[2] = -INF
    z[2, 1234] = -5.0              # one word left
    z[3, [5, 900, 2000]] = INF
    z[4] = torch.finfo(FP32).min   # the type's lowest value is a logit like another
    z[5, 1:] = torch.finfo(FP32).min
    z[6, :2990] = -INF             # fewer words than top_k
    z[7] = -INF
    z[7, -1] = 0.0                 # the last word alone
    u = torch.rand(8, generator=g, device="cuda")
    for kw in (dict(), dict(top_k=50), dict(top_p=0.9), dict(top_k=100, top_p=0.5, min_p=0.2), dict(temperature=0.0),
               dict(temperature=0.01), dict(temperature=1e-20), dict(temperature=1e20), dict(top_k=2, temperature=0.5)):
        got = check(z, u, **kw)
        assert got.tolist()[:3] == [-1, -1, 1234] and int(got[7]) == V - 1
    low = z.to(BF16)
    low[4] = torch.finfo(BF16).min
    check(low, u, top_p=0.9)


def test_random_numbers_at_the_ends():
    z = torch.tensor([[-INF, 0.0, 1.0, -INF, 2.0, -INF]], device="cuda").repeat(7, 1)
    u = torch.tensor([0.0, -1.0, float("nan"), 1.0 - 2.0 ** -24, 1.0, 2.0, INF], device="cuda")
    assert F.flce_sample(z, u).tolist() == [1, 1, 1, 4, 4, 4, 4]


def test_every_share_is_met():
    """Evenly spread random numbers give each word its share, to one draw."""
    n = 4096
    z = torch.tensor([0.3, -1.0, 2.0, -INF, 1.9, 0.0, -3.0], device="cuda")
    u = (torch.arange(n, device="cuda", dtype=torch.float64) + 0.5).div(n).float()
    for kw, kept in ((dict(), [0, 1, 2, 4, 5, 6]), (dict(top_k=3), [0, 2, 4]), (dict(min_p=0.15), [0, 2, 4])):
        got = torch.bincount(F.flce_sample(z.expand(n, 7).contiguous(), u, temperature=0.9, **kw), minlength=7)
        w = torch.zeros(7, dtype=torch.float64)
        w[kept] = (z[kept].double().cpu() / 0.9).exp()
        share = w / w.sum() * n
        assert bool(((got.cpu() - share).abs() <= 1).all()), (got, share)


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (8, 8), (5, 16)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=str)
def test_pitches_and_alignment(dtype, offset, pad):
    """Rows anywhere, with larger logits outside of them; the call writes its tokens alone."""
    g = gen(8)
    B, V = 5, 1237
    z, u = words(g, B, V).to(dtype), torch.rand(B, generator=g, device="cuda")
    buf = torch.full((offset + B * (V + pad) + 32,), 1e4, dtype=dtype, device="cuda")
    view = buf[offset:offset + B * (V + pad)].view(B, V + pad)[:, :V].copy_(z)
    out = torch.full((B + 2,), -7, dtype=torch.int64, device="cuda")
    for kw in (dict(), dict(top_k=20, top_p=0.9)):
        want = F.flce_sample(z, u, **kw)
        got = F.flce_sample(view, u, out=out[1:-1], **kw)
        assert got.data_ptr() == out[1:].data_ptr() and torch.equal(got, want)
        assert out[[0, -1]].tolist() == [-7, -7]


@pytest.mark.parametrize("kw", [dict(), dict(top_p=0.9), dict(top_k=60, top_p=0.8, temperature=0.7)], ids=str)
def test_tokens_do_not_depend_on_the_batch(kw):
    """A row alone (many blocks), in a batch of 40 and of 600 (few blocks): one token."""
    g = gen(9)
    z, u = words(g, 600, 33000).to(BF16), torch.rand(600, generator=g, device="cuda")
    all_ = F.flce_sample(z, u, **kw)
    assert torch.equal(all_[:40], F.flce_sample(z[:40], u[:40], **kw))
    for b in (0, 7, 599):
        assert torch.equal(all_[b:b + 1], F.flce_sample(z[b:b + 1], u[b:b + 1], **kw))
    assert torch.equal(all_, F.flce_sample(z, u, **kw))


def test_rows_beyond_32_bits():
    """Rows whose offset passes 2^32 elements."""
    B, ld = 5, (1 << 30) + 8
    buf = torch.empty(B * ld, dtype=BF16, device="cuda")
    view = buf.view(B, ld)[:, :5000]
    g = gen(10)
    view.copy_(words(g, B, 5000).to(BF16))
    check(view, torch.rand(B, generator=g, device="cuda"), top_p=0.9)


def test_streams_graphs_and_empty():
    g = gen(11)
    z, u = words(g, 12, 7000), torch.rand(12, generator=g, device="cuda")
    want = F.flce_sample(z, u, top_p=0.8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.flce_sample(z, u, top_p=0.8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens = F.flce_sample(z, u, top_p=0.8)
    u2 = torch.rand(12, generator=g, device="cuda")
    expected = F.flce_sample(z, u2, top_p=0.8)
    u.copy_(u2)
    graph.replay()
    assert torch.equal(tokens, expected)
    assert F.flce_sample(z[:0], u[:0]).shape == (0,)


def test_refusals():
    z, u = torch.zeros(3, 50, device="cuda"), torch.zeros(3, device="cuda")
    for bad, error in ((dict(temperature=-1.0), F.FlceError), (dict(top_k=-1), F.FlceError), (dict(top_p=1.5), F.FlceError),
                       (dict(min_p=-0.1), F.FlceError), (dict(top_k=2.5), ValueError), (dict(top_k=float("nan")), ValueError),
                       (dict(temperature=u[:2]), ValueError), (dict(top_k=u), TypeError), (dict(top_p=u.double()), TypeError),
                       (dict(min_p="0"), TypeError), (dict(temperature=u.cpu()), TypeError)):
        with pytest.raises(error):
            F.flce_sample(z, u, **bad)
    for logits, numbers, error in ((z[0], u, ValueError), (z.double(), u, TypeError), (z, u[:2], ValueError),
                                   (z, u.double(), TypeError), (z.t(), torch.zeros(50, device="cuda"), ValueError)):
        with pytest.raises(error):
            F.flce_sample(logits, numbers)
    with pytest.raises(F.FlceError):
        F.flce_sample(torch.zeros(1, (1 << 20) + 1, device="cuda"), u[:1])


def test_the_heads_serving_side():
    """Norm, the head's product and the draw in a row; the distribution is the loss head's."""
    torch.manual_seed(2)
    B, H, V = 40, 128, 777
    norm = F.FusedRMSNorm(H, device="cuda")
    x, r = torch.randn(B, H, device="cuda").bfloat16(), torch.randn(B, H, device="cuda").bfloat16()
    W, b = torch.randn(V, H, device="cuda").mul_(0.3).bfloat16(), torch.randn(V, device="cuda").bfloat16()
    u = torch.rand(B, device="cuda")
    with torch.no_grad():
        y, _ = norm(x, r)
        tokens = F.fused_linear_sample(y, W, b, u=u, logit_scale=0.5, temperature=0.8, top_k=30)
        logits = F.flce_linear_forward(y, W, b)
    assert tokens.tolist() == [R.sample(logits[i].float(), float(u[i]), temperature=1.6, top_k=30) for i in range(B)]
    torch.manual_seed(9)
    a = F.fused_linear_sample(y, W, b)
    torch.manual_seed(9)
    assert torch.equal(a, F.fused_linear_sample(y, W, b))
    # The greedy word is the one of least loss.
    best = F.fused_linear_sample(y, W, b, temperature=0.0)
    losses = torch.stack([F.flce_forward(y, W, b, torch.full((B,), v, device="cuda"), reduction="none")[0]
                          for v in range(0, V, 97)])
    mine = F.flce_forward(y, W, b, best, reduction="none")[0]
    assert bool((mine <= losses.amin(0) + 2e-2).all())  # the logits are rounded to bf16, of up to 16


def test_tokens_share_no_memory_with_the_inputs():
    z, both = torch.zeros(4, 100, device="cuda"), torch.zeros(8, dtype=torch.int64, device="cuda")
    u = both.view(torch.float32)[6:10]
    with pytest.raises(ValueError, match="overlap"):
        F.flce_sample(z, u, out=both[:4])
    with pytest.raises(ValueError, match="overlap"):
        F.flce_sample(z, torch.zeros(4, device="cuda"), top_p=u, out=both[:4])
    assert F.flce_sample(z, both.view(torch.float32)[8:12], out=both[:4]).data_ptr() == both.data_ptr()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("values", [1, 2, 7, 40])
def test_lists_full_of_equal_logits(dtype, values):
    """A list whose items are of few values, over the signs: the cut lies among equal ones."""
    V = 1 << 17
    g = torch.Generator(device="cuda").manual_seed(values)
    z = torch.full((6, V), -30.0, device="cuda")
    at = torch.randperm(V, generator=g, device="cuda")[:1200]
    z[:, at] = torch.linspace(-0.02, 0.02, values, device="cuda").repeat(1200 // values + 1)[:1200]
    z = z.to(dtype)
    u = torch.tensor([0.0, 0.2, 0.5, 0.7, 0.9, 0.999999], device="cuda")
    for kw in (dict(top_p=0.5), dict(top_p=0.999), dict(top_k=600), dict(top_k=999, top_p=0.3)):
        check(z, u, **kw)
