"""Cases of the operators between the gated block, the loss head and a served token: the root-mean-square norm with
the residual's addition (forward, backward, output in 8 bits), dropout from a counter-based generator, and sampling
from logits.

``run`` computes one pass, either with the library's entry points (``own``) or in the plain form: elementary torch
operations in 32 bits (sampling in 64: its tokens sit between neighbouring sums), rounded once at the end. ``exact``
is the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
MASK32 = 0xFFFFFFFF
MOST_BYTES = 4 * 8192 * 14336 * 2  # of the largest listed case


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding token joins the residual stream and is normed: latency.
        dict(name="norm_1", op="norm", M=1, H=4096, dtype="bf16", stream="bf16", res=True, p=0.0, train=False),
        # Prompt tokens of an odd count and an odd width, without a residual.
        dict(name="norm_1999", op="norm", M=1999, H=1111, dtype="fp16", stream="fp16", res=False, p=0.0, train=False),
        # A training step at the benchmark's head shape, with dropout on the branch that joins the stream.
        dict(name="norm_train_8192", op="norm", M=8192, H=4096, dtype="bf16", stream="bf16", res=True, p=0.1,
             train=True),
        # A training step of a mid-size model whose residual stream is kept in 32 bits.
        dict(name="norm_train_3001", op="norm", M=3001, H=2048, dtype="bf16", stream="fp32", res=True, p=0.0,
             train=True),
        # A ragged decoding batch whose next product takes 8 bits, one scale for each token.
        dict(name="norm8_45", op="norm8", M=45, H=4096, dtype="bf16", stream="bf16", res=True, p=0.0, scales="row"),
        # A long prompt in 8 bits, one scale for each 128 columns.
        dict(name="norm8_8192", op="norm8", M=8192, H=4096, dtype="bf16", stream="bf16", res=True, p=0.0,
             scales="block"),
        # A small batch of a training step: the branch joins the stream through dropout.
        dict(name="dropout_512", op="dropout", M=512, H=2048, dtype="bf16", res=True, p=0.1, train=False),
        # Dropout on the hidden features of a wide feed-forward block, forward and backward.
        dict(name="dropout_train_8192", op="dropout", M=8192, H=14336, dtype="bf16", res=False, p=0.2, train=True),
        # One sequence, the common serving settings: latency.
        dict(name="sample_1", op="sample", B=1, V=128256, dtype="bf16", rows=False, temperature=0.8, top_k=50,
             top_p=0.9, min_p=0.0),
        # A batch in which every request brings settings of its own.
        dict(name="sample_64", op="sample", B=64, V=32000, dtype="fp32", rows=True, temperature=1.0, top_k=50,
             top_p=0.9, min_p=0.05),
        # Rollouts: the whole distribution of an odd vocabulary, no truncation.
        dict(name="sample_37", op="sample", B=37, V=50257, dtype="fp16", rows=False, temperature=1.0, top_k=0,
             top_p=1.0, min_p=0.0),
        # A large batch that samples from the nucleus.
        dict(name="sample_512", op="sample", B=512, V=128256, dtype="bf16", rows=False, temperature=1.0, top_k=0,
             top_p=0.95, min_p=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm8", "dropout", "sample", "sample"))
    if op == "sample":
        c = dict(op=op, B=_log(rng, 1, 512), V=_log(rng, 1000, 262144),
                 dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")), rows=rng.random() < 0.4,
                 temperature=rng.choice((0.6, 0.7, 0.8, 1.0, 1.0, 1.2)), top_k=rng.choice((0, 0, 20, 50, 200, 1000)),
                 top_p=rng.choice((1.0, 1.0, 0.8, 0.9, 0.95, 0.99)), min_p=rng.choice((0.0, 0.0, 0.02, 0.05, 0.1)))
        while c["B"] * c["V"] * TYPES[c["dtype"]].itemsize > 512 * 128256 * 2:
            c["B"] = max(1, c["B"] // 2)
        return c
    while True:
        H = _log(rng, 64, 16384)
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        c = dict(op=op, M=_log(rng, 1, 16384), H=max(8, H // 8 * 8) if rng.random() < 0.8 else H, dtype=dtype,
                 res=rng.random() < 0.75,
                 p=rng.choice((0.05, 0.1, 0.2, 0.5)) if op == "dropout" or rng.random() < 0.3 else 0.0)
        if op != "dropout":
            c["stream"] = rng.choice((dtype, dtype, "fp32")) if c["res"] else dtype
        if op == "norm8":
            c["scales"] = rng.choice(("row", "block"))
        else:
            c["train"] = rng.random() < 0.6
        if work(c)["bytes"] <= MOST_BYTES:
            return c


# ---------------------------------------------------------------- prepare
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 29)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = dict(case=case)
    if case["op"] == "sample":
        return _prepare_sample(s, case, normal, uniform)
    dt, M, H = TYPES[case["dtype"]], case["M"], case["H"]
    # A branch's output, with channels of unequal size, and the stream that it joins.
    s["x"] = normal(M, H).mul_(normal(H, std=0.3).exp_()).to(dt)
    st = TYPES[case.get("stream", case["dtype"])]
    s["r"] = normal(M, H, std=3.0).to(st) if case["res"] else None
    s["seed"] = (int(seed) * 0x9E3779B97F4A7C15 + 12345) % (1 << 62)
    if case["op"] != "dropout":
        s["w"] = normal(H, std=0.2).add_(1.0).to(dt)
    if case.get("train"):
        s["dy"] = normal(M, H, std=1e-2).to(dt)
        s["dh"] = normal(M, H, std=1e-2).to(st) if case["op"] == "norm" and case["res"] else None
    return s


def _prepare_sample(s, case, normal, uniform):
    B, V = case["B"], case["V"]
    # A wide bulk, and some hundreds of words that the context makes likely; rows of unequal certainty.
    z = normal(B, V, std=2.0).add_(uniform(B, V).pow_(60).mul_(12.0)).mul_(uniform(B, 1).add_(0.5))
    s["logits"], s["u"] = z.to(TYPES[case["dtype"]]), uniform(B)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        s[name] = case[name]
    if case["rows"]:
        on = lambda: uniform(B) < 0.6  # noqa: E731
        # Some requests are greedy (temperature 0); each limit is off (0 or 1) in some.
        s["temperature"] = torch.where(uniform(B) < 0.15, 0.0, case["temperature"] * uniform(B).mul_(0.6).add_(0.6))
        s["top_k"] = torch.where(on(), (uniform(B) * (2 * case["top_k"])).floor(), 0.0).to(torch.int32)
        s["top_p"] = torch.where(on(), 1.0 - uniform(B) * 0.4, 1.0)
        s["min_p"] = torch.where(on(), uniform(B) * (2 * case["min_p"]), 0.0)
    return s


# -------------------------------------------------------------------- run
def run(s):
    if own:
        return _OWN[s["case"]["op"]](s, s["case"])
    return _PLAIN[s["case"]["op"]](s, s["case"])


def _own_norm(s, c):
    import linear_cross_entropy_gemm_gb300 as F
    x, w, r = s["x"], s["w"], s["r"]
    if not c["train"]:
        return F.flce_rms_norm_forward(x, w, r, eps=EPS, dropout=c["p"], seed=s["seed"])
    rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    y, h = F.flce_rms_norm_forward(x, w, r, eps=EPS, dropout=c["p"], seed=s["seed"], rstd=rstd)
    dx, dr, dw = F.flce_rms_norm_backward(s["dy"], h, w, rstd, s["dh"], dropout=c["p"], seed=s["seed"],
                                          dW_dtype=x.dtype, needs=(True, r is not None, True))
    return y, h, dx, dr, dw


def _own_norm8(s, c):
    import linear_cross_entropy_gemm_gb300 as F
    return F.flce_rms_norm_quantized(s["x"], s["w"], s["r"], eps=EPS, scales=c["scales"], dropout=c["p"],
                                     seed=s["seed"])


def _own_dropout(s, c):
    import linear_cross_entropy_gemm_gb300 as F
    y = F.flce_dropout(s["x"], c["p"], s["seed"], residual=s["r"])
    return (y, F.flce_dropout(s["dy"], c["p"], s["seed"])) if c["train"] else y


def _own_sample(s, c):
    import linear_cross_entropy_gemm_gb300 as F
    return F.flce_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                         min_p=s["min_p"])


_OWN = {"norm": _own_norm, "norm8": _own_norm8, "dropout": _own_dropout, "sample": _own_sample}


def _factors(M, H, p, seed, device):
    """D(x) = factor x: 0 or 65536 / (65536 - t), by 16 random bits for each element (Philox4x32-10, eight columns of a
    row to a counter), None without dropout."""
    t = int(math.floor(p * 65536 + 0.5))
    if t == 0:
        return None
    groups = -(-H // 8)
    zero = torch.zeros((M, groups), dtype=torch.int64, device=device)
    c0 = zero + torch.arange(groups, dtype=torch.int64, device=device)
    c1 = zero + torch.arange(M, dtype=torch.int64, device=device)[:, None]
    c2, c3, k0, k1 = zero, zero, seed & MASK32, (seed >> 32) & MASK32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & MASK32) ^ c1 ^ k0, b & MASK32, ((a >> 32) & MASK32) ^ c3 ^ k1, a & MASK32
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    words = torch.stack((c0, c1, c2, c3), -1)
    bits = torch.stack((words & 0xFFFF, words >> 16), -1).reshape(M, groups * 8)[:, :H]
    return (bits >= t).to(torch.float32) * (65536.0 / max(1, 65536 - t))


def _plain_sum(s, c):
    """h = r + D(x), and D's factors."""
    x = s["x"].float()
    f = _factors(*x.shape, c["p"], s["seed"], x.device)
    h = x if f is None else x * f
    return (h if s["r"] is None else h + s["r"].float()), f


def _plain_norm(s, c):
    h, f = _plain_sum(s, c)
    w, dt, st = s["w"].float(), s["x"].dtype, TYPES[c["stream"]]
    rstd = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    xhat = h * rstd
    y = (xhat * w).to(dt)
    if not c["train"]:
        return y, h.to(st)
    dy = s["dy"].float()
    g = dy * w
    e = (g - xhat * (g * xhat).mean(-1, keepdim=True)) * rstd
    if s["dh"] is not None:
        e = e + s["dh"].float()
    return y, h.to(st), (e if f is None else e * f).to(dt), e.to(st) if c["res"] else None, (dy * xhat).sum(0).to(dt)


def _plain_norm8(s, c):
    h, _ = _plain_sum(s, c)
    M, H = h.shape
    y = h * (1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)) * s["w"].float()
    if c["scales"] == "row":
        scale = y.abs().amax(-1) / 448.0
        q = y / scale[:, None].clamp(min=1e-38)
    else:
        blocks = -(-H // 128)
        padded = torch.zeros((M, blocks * 128), dtype=torch.float32, device=h.device)
        padded[:, :H] = y
        padded = padded.view(M, blocks, 128)
        scale = padded.abs().amax(-1) / 448.0
        q = (padded / scale[..., None].clamp(min=1e-38)).view(M, -1)[:, :H]
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale, h.to(TYPES[c["stream"]])


def _plain_dropout(s, c):
    x, dt = s["x"].float(), s["x"].dtype
    f = _factors(*x.shape, c["p"], s["seed"], x.device)
    y = x * f
    if s["r"] is not None:
        y = y + s["r"].float()
    return (y.to(dt), (s["dy"].float() * f).to(dt)) if c["train"] else y.to(dt)


def _plain_sample(s, c):
    z = s["logits"].double()
    B, V = z.shape

    def column(v):
        return v.double()[:, None] if torch.is_tensor(v) else torch.full((B, 1), float(v), dtype=torch.float64,
                                                                         device=z.device)

    t, k, p, least = (column(s[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
    greedy = t <= 0
    z, order = torch.sort(z, dim=-1, descending=True, stable=True)
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, t))
    place = torch.arange(V, device=z.device)[None, :]
    w = w * (place < torch.where(greedy, 1.0, torch.where(k <= 0, float(V), k)))
    sums = torch.cumsum(w, -1)
    keep = ((sums - w < p * sums[:, -1:]) | (p >= 1)) & (w >= least)
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, order, w * keep)
    sums = torch.cumsum(kept, -1)
    return (sums > s["u"].double()[:, None] * sums[:, -1:]).to(torch.uint8).argmax(-1)


_PLAIN = {"norm": _plain_norm, "norm8": _plain_norm8, "dropout": _plain_dropout, "sample": _plain_sample}


# ------------------------------------------------------------------- work
def work(case):
    size = TYPES[case["dtype"]].itemsize
    if case["op"] == "sample":
        n = case["B"] * case["V"]
        return {"bytes": n * size + case["B"] * (4 + 8 + (16 if case["rows"] else 0)), "flops": 4 * n}
    M, H = case["M"], case["H"]
    n = M * H
    if case["op"] == "dropout":
        return {"bytes": n * size * ((3 if case["res"] else 2) + (2 if case["train"] else 0)), "flops": 2 * n}
    stream = TYPES[case["stream"]].itemsize if case["res"] else 0
    # x, weight, the residual in and the sum out (without a residual and dropout the sum is x).
    b = n * size + H * size + 2 * n * stream
    if not case["res"] and case["p"] > 0:
        b += n * size
    if case["op"] == "norm8":
        scales = M if case["scales"] == "row" else M * -(-H // 128)
        return {"bytes": b + n + 4 * scales, "flops": 7 * n}
    if not case["train"]:
        return {"bytes": b + n * size, "flops": 5 * n}
    # The backward: dy and the stream's gradient in, the gradients of x and of the stream out (one tensor where they
    # are equal), the weight's.
    b += n * size + n * size + n * stream + H * size
    if case["res"] and (case["p"] > 0 or case["stream"] != case["dtype"]):
        b += n * stream
    return {"bytes": b + n * size, "flops": 18 * n}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s, case)
    x, r = s["x"].double(), s["r"]
    M, H = x.shape
    d = _exact_factors(M, H, case["p"], s["seed"], x.device)
    h = torch.addcmul(torch.zeros_like(x) if r is None else r.double(), x, d)
    if case["op"] == "dropout":
        return (h, s["dy"].double() * d) if case["train"] else h
    w = s["w"].double()
    size = torch.sqrt(torch.einsum("mh,mh->m", h, h) / H + EPS)[:, None]
    y = h / size * w
    if case["op"] == "norm8":
        if case["scales"] == "row":
            scale = torch.linalg.vector_norm(y, math.inf, dim=1) / 448
            each = scale[:, None].expand(M, H)
        else:
            parts = [torch.linalg.vector_norm(b, math.inf, dim=1) / 448 for b in y.split(128, dim=1)]
            scale = torch.stack(parts, 1)
            each = scale.repeat_interleave(128, dim=1)[:, :H]
        return y / each, scale, h
    if not case["train"]:
        return y, h
    # y_c = w_c h_c / size with size^2 = mean h^2 + eps: the derivative of size is h_c / (H size).
    dy = s["dy"].double()
    along = torch.einsum("mh,mh,h->m", dy, h, w)[:, None]
    e = dy * w / size - h * along / (H * size ** 3)
    if s["dh"] is not None:
        e = e + s["dh"].double()
    return y, h, e * d, e if case["res"] else None, torch.einsum("mh,mh->h", dy, h / size)


def _exact_factors(M, H, p, seed, device):
    """Philox4x32-10 in halves of 16 bits, whose products fit 64-bit whole numbers with room to spare."""
    drop = round(p * 65536)
    if drop == 0:
        return torch.ones((), dtype=torch.float64, device=device)

    def product(m, v):
        ml, mh, vl, vh = m & 0xFFFF, m >> 16, v % 65536, v // 65536
        low, mid = ml * vl, ml * vh + mh * vl
        total = low + (mid % 65536) * 65536
        return mh * vh + mid // 65536 + total // 2 ** 32, total % 2 ** 32

    rows, cols = torch.meshgrid(torch.arange(M, device=device), torch.arange(-(-H // 8), device=device), indexing="ij")
    x, key = [cols, rows, torch.zeros_like(rows), torch.zeros_like(rows)], [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        (h0, l0), (h1, l1) = product(0xD2511F53, x[0]), product(0xCD9E8D57, x[2])
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    halves = [part for v in x for part in (v % 65536, v // 65536)]
    stays = torch.stack(halves, 2).flatten(1)[:, :H] >= drop
    return torch.where(stays, 65536.0 / (65536 - drop), 0.0).double()


def _exact_sample(s, case):
    """Row by row: the words by falling logit, cut three times, then the draw in the vocabulary's order."""
    z, u = s["logits"].double(), s["u"].double().tolist()
    of = lambda name, b: float(s[name][b]) if torch.is_tensor(s[name]) else float(s[name])  # noqa: E731
    tokens = []
    for b in range(case["B"]):
        t, k, p, least = (of(n, b) for n in ("temperature", "top_k", "top_p", "min_p"))
        row = z[b]
        if t <= 0 or k == 1:
            tokens.append(int((row == row.max()).nonzero()[0]))
            continue
        words = torch.argsort(row, descending=True, stable=True)
        if 0 < k < case["V"]:
            words = words[:int(k)]
        weights = torch.exp((row[words] - row[words[0]]) / t)
        if p < 1:
            before = torch.cat((weights.new_zeros(1), torch.cumsum(weights, 0)[:-1]))
            count = max(1, int((before < p * weights.sum()).sum()))
            words, weights = words[:count], weights[:count]
        words, weights = words[weights >= least], weights[weights >= least]
        words, at = torch.sort(words)
        sums = torch.cumsum(weights[at], 0)
        tokens.append(int(words[torch.searchsorted(sums, u[b] * sums[-1], right=True)]))
    return torch.tensor(tokens, device=z.device)
