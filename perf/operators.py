"""Cases of the operators around the loss head: the linear layer with its bias, activation and residual in one
pass, the gated feed-forward projection, and the global gradient norm with clipping; forward and backward.

``run`` computes one pass, either with the library's entry points (``own``) or in the plain form: elementary
torch operations in 32 bits, rounded once at the end. ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LINEAR_ACT = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")
GATED_ACT = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One token through a square projection whose result joins the residual stream: a decoding step, where
        # latency counts.
        dict(name="linear_1", op="linear", M=1, K=4096, N=4096, act="none", bias=False, res=True, dtype="bf16",
             train=False),
        # The down projection of a batch of decoding sequences.
        dict(name="linear_32", op="linear", M=32, K=14336, N=4096, act="none", bias=False, res=True, dtype="bf16",
             train=False),
        # The first layer of a plain feed-forward block over an odd count of prompt tokens.
        dict(name="linear_1999", op="linear", M=1999, K=4096, N=16384, act="gelu_tanh", bias=True, res=False,
             dtype="fp16", train=False),
        # A training step of a mid-size layer with bias and activation, an odd count of tokens.
        dict(name="linear_train_3001", op="linear", M=3001, K=2048, N=8192, act="gelu", bias=True, res=False,
             dtype="fp16", train=True),
        # A training step of the down projection into the residual stream at the benchmark's head shape.
        dict(name="linear_train_8192", op="linear", M=8192, K=14336, N=4096, act="none", bias=False, res=True,
             dtype="bf16", train=True),
        # One decoding token through the gated block's two projections.
        dict(name="gated_1", op="gated", M=1, K=4096, F=14336, act="silu", dtype="bf16", train=False),
        # A ragged decoding batch.
        dict(name="gated_45", op="gated", M=45, K=4096, F=14336, act="silu", dtype="bf16", train=False),
        # A prompt of odd length, a narrower block.
        dict(name="gated_777", op="gated", M=777, K=2048, F=5632, act="gelu_tanh", dtype="fp16", train=False),
        # A training step at the benchmark's head shape.
        dict(name="gated_train_8192", op="gated", M=8192, K=4096, F=14336, act="silu", dtype="bf16", train=True),
        # The norm over the gradients of many small tensors (adapters, norms, biases): latency.
        dict(name="norm_small", op="norm", count=96, most=65536, dtype="bf16", shape_seed=11, pad=True),
        # The norm over the head's 32-bit weight gradient and some of its neighbours.
        dict(name="norm_head", op="norm", count=3, most=128256 * 4096, dtype="fp32", shape_seed=5, pad=True),
        # The gradients of a few transformer blocks, clipped into the buffer the optimiser reads.
        dict(name="clip_blocks", op="clip", count=60, most=4096 * 14336, dtype="bf16", shape_seed=3, pad=True,
             ratio=0.3, out=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("linear", "linear", "linear_train", "linear_train", "gated", "gated", "gated_train",
                       "gated_train", "norm", "clip"))
    if kind in ("norm", "clip"):
        c = dict(op=kind, count=_log(rng, 1, 300), most=_log(rng, 100, 1 << 26),
                 dtype=rng.choice(("bf16", "fp16", "fp32", "mixed")), shape_seed=rng.randrange(1 << 30),
                 pad=rng.random() < 0.7)
        if kind == "clip":
            clipped = rng.random() < 0.75
            # Below the limit the gradients stay as they are, and the call works in place.
            c.update(ratio=rng.uniform(0.05, 0.8) if clipped else rng.uniform(1.5, 20.0),
                     out=clipped or rng.random() < 0.5)
        while sum(_sizes(c)) > 60 * 4096 * 14336 // 8:
            c["most"] = max(100, c["most"] // 2)
        return c
    op, train = kind.split("_")[0], kind.endswith("train")
    while True:
        M = _log(rng, 16 if train else 1, 8192)
        K = 8 * _log(rng, 32, 2048)
        N = _log(rng, 8, 16384)
        dtype = rng.choice(("bf16", "bf16", "fp16"))
        if op == "gated":
            c = dict(op=op, M=M, K=K, F=max(8, N // 8 * 8), act=rng.choice(GATED_ACT), dtype=dtype, train=train)
        else:
            if rng.random() < 0.7:
                N = max(8, N // 8 * 8)
            c = dict(op=op, M=M, K=K, N=N, act=rng.choice(LINEAR_ACT), bias=rng.random() < 0.5,
                     res=rng.random() < 0.5, dtype=dtype, train=train)
        if 12 * M * K * N <= 12 * 8192 * 4096 * 14336:
            return c


def _sizes(case):
    """Element counts of a gradient list: spread over their logarithm, one of the largest size."""
    rng = random.Random(case["shape_seed"])
    sizes = [_log(rng, 1, case["most"]) for _ in range(case["count"] - 1)] + [case["most"]]
    rng.shuffle(sizes)
    return sizes


def _kinds(case):
    """Type and spread of each gradient."""
    rng = random.Random(case["shape_seed"] + 1)
    names = ("bf16", "fp32") if case["dtype"] == "mixed" else (case["dtype"],)
    return [(rng.choice(names), 10.0 ** rng.uniform(-4, -2)) for _ in range(case["count"])]


# ---------------------------------------------------------------- prepare
def _gradient_views(case, flats=None):
    """The gradients as views of one flat buffer for each type, 16-byte aligned or packed one after another;
    with `flats`, the same views of other buffers."""
    sizes, kinds = _sizes(case), _kinds(case)
    at, place = {}, []
    for n, (t, _) in zip(sizes, kinds):
        start = at.get(t, 0)
        place.append((t, start, n))
        end = start + n
        at[t] = -(-end // 8) * 8 if case["pad"] else end
    if flats is None:
        flats = {t: torch.zeros(n, dtype=TYPES[t], device="cuda") for t, n in at.items()}
    return flats, [flats[t][s:s + n] for t, s, n in place]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 13)
    if case["op"] in ("norm", "clip"):
        flats, grads = _gradient_views(case)
        square = 0.0
        for g, (_, std) in zip(grads, _kinds(case)):
            g.copy_(torch.randn(g.shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std))
            square += std * std * g.numel()
        s = dict(case=case, grads=grads, flats=flats)
        if case["op"] == "clip":
            s["max_norm"] = case["ratio"] * math.sqrt(square)
            if case["out"]:
                s["out_flats"], s["out"] = _gradient_views(case, {t: torch.zeros_like(f) for t, f in flats.items()})
        return s
    dt, M, K = TYPES[case["dtype"]], case["M"], case["K"]
    N = case["F"] if case["op"] == "gated" else case["N"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dt)

    # Activations as a norm layer leaves them, with channels of unequal size; weights at a trained layer's scale.
    x = torch.randn((M, K), generator=gen, device="cuda", dtype=torch.float32)
    x = x.mul_(torch.randn((K,), generator=gen, device="cuda").mul_(0.3).exp_()).to(dt)
    s = dict(case=case, x=x)
    if case["op"] == "gated":
        s["Wg"], s["Wu"] = normal(N, K, std=K ** -0.5), normal(N, K, std=K ** -0.5)
    else:
        s["W"] = normal(N, K, std=K ** -0.5)
        s["b"] = normal(N, std=0.1) if case["bias"] else None
        s["r"] = normal(M, N) if case["res"] else None
    if case["train"]:
        s["dy"] = normal(M, N, std=1e-2)
    return s


# -------------------------------------------------------------------- run
def run(s):
    op, train = s["case"]["op"], s["case"].get("train")
    if own:
        return _OWN[op](s, train)
    return _PLAIN[op](s, train)


def _own_linear(s, train):
    import linear_cross_entropy_gemm_gb300 as F
    x, W, b, r, act = s["x"], s["W"], s["b"], s["r"], s["case"]["act"]
    if not train:
        return F.flce_linear_forward(x, W, b, r, activation=act)
    pre = torch.empty(x.shape[0], W.shape[0], dtype=x.dtype, device=x.device) if act != "none" else None
    y = F.flce_linear_forward(x, W, b, r, activation=act, pre=pre)
    dx, dW, db = F.flce_linear_backward(s["dy"], x, W, b, activation=act, pre=pre, dW_dtype=x.dtype,
                                        db_dtype=x.dtype)
    return y, dx, dW, db


def _own_gated(s, train):
    import linear_cross_entropy_gemm_gb300 as F
    x, Wg, Wu, act = s["x"], s["Wg"], s["Wu"], s["case"]["act"]
    if not train:
        return F.flce_gated_forward(x, Wg, Wu, activation=act)
    pre = torch.empty(2, x.shape[0], Wg.shape[0], dtype=x.dtype, device=x.device)
    h = F.flce_gated_forward(x, Wg, Wu, activation=act, pre=pre)
    dx, dWg, dWu = F.flce_gated_backward(s["dy"], x, Wg, Wu, pre, activation=act, dW_dtype=x.dtype)
    return h, dx, dWg, dWu


def _own_norm(s, train):
    import linear_cross_entropy_gemm_gb300 as F
    return F.flce_grad_norm(s["grads"])


def _own_clip(s, train):
    import linear_cross_entropy_gemm_gb300 as F
    norm = F.flce_clip_grads(s["grads"], s["max_norm"], out=s.get("out"))
    return norm, s["out_flats"] if "out" in s else s["flats"]


_OWN = {"linear": _own_linear, "gated": _own_gated, "norm": _own_norm, "clip": _own_clip}


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _act(z, name):
    """The activation and its derivative as functions of z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    p = _sigmoid(z)
    if name == "silu":
        return z * p, p * (1.0 + z * (1.0 - p))
    return p, p * (1.0 - p)


def _plain_linear(s, train):
    x, W, act, dt = s["x"].float(), s["W"].float(), s["case"]["act"], s["x"].dtype
    z = x @ W.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y, slope = (z, None) if act == "none" else _act(z, act)
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(dt)
    if not train:
        return y
    dz = s["dy"].float()
    if slope is not None:
        dz = dz * slope
    db = None if s["b"] is None else dz.sum(0).to(dt)
    return y, (dz @ W).to(dt), (dz.t() @ x).to(dt), db


def _plain_gated(s, train):
    x, Wg, Wu, dt = s["x"].float(), s["Wg"].float(), s["Wu"].float(), s["x"].dtype
    u = x @ Wu.t()
    a, slope = _act(x @ Wg.t(), s["case"]["act"])
    h = (a * u).to(dt)
    if not train:
        return h
    dh = s["dy"].float()
    dg, du = dh * u * slope, dh * a
    return h, (dg @ Wg + du @ Wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)


def _plain_norm(s, train):
    return torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()


def _plain_clip(s, train):
    norm = _plain_norm(s, train)
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    [o.copy_(g.float() * scale) for g, o in zip(s["grads"], s["out"] if "out" in s else s["grads"])]
    return norm, s["out_flats"] if "out" in s else s["flats"]


_PLAIN = {"linear": _plain_linear, "gated": _plain_gated, "norm": _plain_norm, "clip": _plain_clip}


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        n = sum(k * TYPES[t].itemsize for k, (t, _) in zip(_sizes(case), _kinds(case)))
        m = sum(_sizes(case))
        if op == "norm":
            return {"bytes": n + 4, "flops": 2 * m}
        # In place and below the limit nothing has to be written.
        return {"bytes": (2 if case["out"] else 1) * n + 4, "flops": 3 * m}
    M, K = case["M"], case["K"]
    if op == "gated":
        F = case["F"]
        if case["train"]:
            return {"bytes": 2 * (2 * M * K + 4 * F * K + 2 * M * F), "flops": 12 * M * K * F}
        return {"bytes": 2 * (M * K + 2 * F * K + M * F), "flops": 4 * M * K * F}
    N, extra = case["N"], (case["M"] * case["N"] if case["res"] else 0) + (case["N"] if case["bias"] else 0)
    if case["train"]:
        return {"bytes": 2 * (2 * M * K + 2 * N * K + 2 * M * N + extra + (N if case["bias"] else 0)),
                "flops": 6 * M * K * N}
    return {"bytes": 2 * (M * K + N * K + M * N + extra), "flops": 2 * M * K * N}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits."""
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        total = 0.0
        for g in s["grads"]:
            for part in g.split(1 << 26):
                d = part.double()
                total += float(torch.dot(d, d))
        norm = torch.tensor(math.sqrt(total), dtype=torch.float64)
        if case["op"] == "norm":
            return norm
        c = min(1.0, s["max_norm"] / (math.sqrt(total) + 1e-6))
        return norm, {t: f.double() * c for t, f in s["flats"].items()}
    x = s["x"].double()

    def curve(z, name):
        if name == "none":
            return z, None
        if name == "relu":
            return z.clamp(min=0), torch.where(z > 0, 1.0, 0.0).to(z)
        if name == "gelu":
            cdf = torch.special.ndtr(z)
            return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":
            # (1 + tanh w) / 2 is the logistic function of 2 w.
            p = torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            return z * p, p + z * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
        p = torch.special.expit(z)
        return (z * p, p + z * p * (1 - p)) if name == "silu" else (p, p * (1 - p))

    if case["op"] == "gated":
        Wg, Wu = s["Wg"].double(), s["Wu"].double()
        a, slope = curve(torch.einsum("mk,fk->mf", x, Wg), case["act"])
        u = torch.einsum("mk,fk->mf", x, Wu)
        if not case["train"]:
            return a * u
        dh = s["dy"].double()
        dg, du = dh * u * slope, dh * a
        return (a * u, torch.einsum("mf,fk->mk", dg, Wg) + torch.einsum("mf,fk->mk", du, Wu),
                torch.einsum("mf,mk->fk", dg, x), torch.einsum("mf,mk->fk", du, x))
    W = s["W"].double()
    z = torch.einsum("mk,nk->mn", x, W)
    if s["b"] is not None:
        z += s["b"].double()
    y, slope = curve(z, case["act"])
    if s["r"] is not None:
        y = y + s["r"].double()
    if not case["train"]:
        return y
    dz = s["dy"].double() if slope is None else s["dy"].double() * slope
    db = None if s["b"] is None else dz.sum(0)
    return y, torch.einsum("mn,nk->mk", dz, W), torch.einsum("mn,mk->nk", dz, x), db
