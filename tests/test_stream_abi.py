"""The operators on the residual stream, and sampling, without a GPU: struct layouts, enums,
workspace sizes, the generator's published vectors, and the refusals before every launch."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
import stream_reference as R
from linear_cross_entropy_gemm_gb300 import _lib
from linear_cross_entropy_gemm_gb300 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "flce.h")
AT = 4096  # an aligned address that is never dereferenced: the calls are refused first
INVALID, ALIGNMENT, SMALL, UNSUPPORTED = 1, 2, 3, 7
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


@pytest.mark.parametrize("struct,name", [(_lib.FlceRmsNormParams, "flce_rms_norm_params_t"),
                                         (_lib.FlceDropoutParams, "flce_dropout_params_t"),
                                         (_lib.FlceSampleParams, "flce_sample_params_t")])
def test_struct_layouts_match_the_header(tmp_path, struct, name):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"flce.h\"\nint main(void) {\n"
                   + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields)
                   + f'  printf("%zu\\n", sizeof({name}));\n  return 0;\n}}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [getattr(struct, f).offset for f in fields] + [ctypes.sizeof(struct)]


def test_scales_match_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    got = {m.group(1).lower(): int(m.group(2)) for m in re.finditer(r"FLCE_SCALES_(\w+)\s*=\s*(\d+)", src)}
    assert got == _lib.SCALES


def test_philox_vectors():
    """Known answers that the generator's authors publish."""
    full = 0xFFFFFFFF
    assert R.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert R.philox([full] * 4, [full] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert R.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


# ------------------------------------------------------------ C refusals
def norm(**kw):
    return _lib.FlceRmsNormParams(**{**dict(M=4, H=64, eps=1e-6), **kw})


def forward(lib, p, x=AT, w=AT, r=AT, seed=None, y=AT, h=AT, rstd=AT, scales=None):
    return lib.flce_rms_norm_forward(ctypes.byref(p), x, w, r, seed, y, h, rstd, scales, None)


def backward(lib, p, dy=AT, h=AT, w=AT, rstd=AT, dh=AT, seed=None, dx=AT, dr=None, dW=AT, ws=AT, n=1 << 40):
    return lib.flce_rms_norm_backward(ctypes.byref(p), dy, h, w, rstd, dh, seed, dx, dr, dW, ws, n, None)


NORM_BAD = [(dict(M=-1), INVALID), (dict(H=0), INVALID), (dict(H=32769), UNSUPPORTED),
            (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
            (dict(dtype=0, stream_dtype=1), INVALID), (dict(dtype=2, stream_dtype=0), INVALID),
            (dict(dtype=1, weight_dtype=0), INVALID), (dict(ld_x=63), INVALID), (dict(ld_res=-64), INVALID),
            (dict(ld_h=8), INVALID), (dict(ld_y=63), INVALID), (dict(eps=-1e-6), INVALID),
            (dict(eps=NAN), INVALID), (dict(eps=float("inf")), INVALID), (dict(dropout=-0.1), INVALID),
            (dict(dropout=1.5), INVALID), (dict(dropout=NAN), INVALID), (dict(dW_fp32=2), INVALID),
            (dict(scales=3), INVALID)]


@pytest.mark.parametrize("kw,status", NORM_BAD, ids=str)
def test_norm_parameters_refused(lib, kw, status):
    p = norm(**kw)
    assert forward(lib, p) == status
    assert backward(lib, p) == status
    assert lib.flce_rms_norm_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("arg", ["x", "w", "r", "y", "h", "rstd"])
def test_norm_forward_alignment(lib, arg):
    for dtype in (0, 2):
        p = norm(dtype=dtype, stream_dtype=dtype, weight_dtype=dtype)
        assert forward(lib, p, **{arg: AT + 1}) == ALIGNMENT


def test_norm_pointers(lib):
    p = norm()
    assert lib.flce_rms_norm_forward(None, AT, AT, AT, None, AT, AT, AT, None, None) == INVALID
    assert forward(lib, p, x=None) == forward(lib, p, y=None) == INVALID
    assert forward(lib, p, seed=AT + 4) == ALIGNMENT
    # Scales are given exactly where the output is quantised.
    assert forward(lib, p, scales=AT) == INVALID and forward(lib, norm(scales=1)) == INVALID
    assert forward(lib, norm(scales=2), scales=AT + 2) == ALIGNMENT
    assert forward(lib, norm(M=0), x=None, y=None) == 0
    for arg in ("dy", "h", "rstd"):
        assert backward(lib, p, **{arg: None}) == INVALID
    for arg in ("dy", "h", "w", "dh", "dx", "dr", "rstd"):
        assert backward(lib, p, **{arg: AT + 1}) == ALIGNMENT
    assert backward(lib, norm(dW_fp32=1), dW=AT + 2) == ALIGNMENT
    assert backward(lib, norm(scales=1)) == INVALID
    assert backward(lib, p, ws=None) == INVALID
    need = lib.flce_rms_norm_workspace_size(ctypes.byref(p))
    assert need >= 64 * 4 and backward(lib, p, n=need - 1) == SMALL
    assert backward(lib, p, dx=None, dr=None, dW=None, ws=None) == 0
    # One buffer for two gradients that differ.
    assert backward(lib, norm(dropout=0.1), dx=AT, dr=AT) == INVALID
    assert backward(lib, norm(stream_dtype=2), dx=AT, dr=AT) == INVALID


DROP_BAD = [(dict(M=-1), INVALID), (dict(H=-1), INVALID), (dict(dtype=3), INVALID), (dict(out_dtype=-1), INVALID),
            (dict(dtype=0, out_dtype=1), INVALID), (dict(ld_x=7), INVALID), (dict(ld_y=-8), INVALID),
            (dict(ld_res=3), INVALID), (dict(dropout=-1e-9), INVALID), (dict(dropout=1.01), INVALID),
            (dict(dropout=NAN), INVALID), (dict(M=(1 << 31) + 1), UNSUPPORTED),
            (dict(H=(1 << 34) + 8, ld_x=0), UNSUPPORTED), (dict(M=1 << 30, H=1 << 20), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", DROP_BAD, ids=str)
def test_dropout_refused(lib, kw, status):
    p = _lib.FlceDropoutParams(**{**dict(M=4, H=8, dropout=0.5), **kw})
    assert lib.flce_dropout(ctypes.byref(p), AT, AT, None, AT, None) == status


def test_dropout_pointers(lib):
    p = ctypes.byref(_lib.FlceDropoutParams(M=4, H=8, dropout=0.5))
    assert lib.flce_dropout(None, AT, AT, None, AT, None) == INVALID
    assert lib.flce_dropout(p, None, AT, None, AT, None) == INVALID
    assert lib.flce_dropout(p, AT, AT, None, None, None) == INVALID
    assert lib.flce_dropout(p, AT + 1, AT, None, AT, None) == ALIGNMENT
    assert lib.flce_dropout(p, AT, AT + 1, None, AT, None) == ALIGNMENT
    assert lib.flce_dropout(p, AT, AT, AT + 4, AT, None) == ALIGNMENT
    empty = ctypes.byref(_lib.FlceDropoutParams(M=0, H=8, dropout=0.5))
    assert lib.flce_dropout(empty, None, None, None, None, None) == 0


SAMPLE_BAD = [(dict(B=-1), INVALID), (dict(V=0), INVALID), (dict(dtype=3), INVALID), (dict(ld=63), INVALID),
              (dict(V=(1 << 20) + 1), UNSUPPORTED), (dict(B=(1 << 28) + 1), UNSUPPORTED),
              (dict(temperature=-0.5), INVALID), (dict(temperature=NAN), INVALID), (dict(top_k=-1), INVALID),
              (dict(top_p=-0.1), INVALID), (dict(top_p=1.1), INVALID), (dict(top_p=NAN), INVALID),
              (dict(min_p=-0.1), INVALID), (dict(min_p=1.1), INVALID), (dict(min_p=NAN), INVALID)]


@pytest.mark.parametrize("kw,status", SAMPLE_BAD, ids=str)
def test_sample_refused(lib, kw, status):
    p = _lib.FlceSampleParams(**{**dict(B=4, V=64, temperature=1.0, top_p=1.0), **kw})
    assert lib.flce_sample(ctypes.byref(p), AT, AT, None, None, None, None, AT, None) == status


def test_sample_pointers(lib):
    p = ctypes.byref(_lib.FlceSampleParams(B=4, V=64, temperature=1.0, top_p=1.0))
    good = [AT, AT, AT, AT, AT, AT, AT]
    assert lib.flce_sample(None, *good, None) == INVALID
    for i, off in enumerate((1, 2, 2, 2, 2, 2, 4)):
        bad = list(good)
        bad[i] = AT + off
        assert lib.flce_sample(p, *bad, None) == ALIGNMENT
    for i in (0, 1, 6):
        bad = list(good)
        bad[i] = None
        assert lib.flce_sample(p, *bad, None) == INVALID
    empty = ctypes.byref(_lib.FlceSampleParams(B=0, V=64, temperature=1.0, top_p=1.0))
    assert lib.flce_sample(empty, None, None, None, None, None, None, None, None) == 0


# ------------------------------------------------------- Python refusals
def test_host_tensors_are_refused():
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    for call in (lambda: F.flce_rms_norm_forward(x, None), lambda: F.flce_rms_norm_quantized(x, None),
                 lambda: F.flce_rms_norm_backward(x, x, None, torch.zeros(2)),
                 lambda: F.flce_dropout(x, 0.1, 3), lambda: F.flce_sample(x, torch.zeros(2))):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_arguments_that_need_no_device():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="scales"):
        F.flce_rms_norm_quantized(x, None, scales="column")
    with pytest.raises(TypeError, match="dW_dtype"):
        F.flce_rms_norm_backward(x, x, None, x, dW_dtype=torch.float16)
    with pytest.raises(ValueError, match="logit_scale"):
        F.fused_linear_sample(x, x, logit_scale=0.0)
    for p in (-0.1, 1.1, NAN):
        with pytest.raises(ValueError, match="probability"):
            F.fused_dropout(x, p)
        with pytest.raises(ValueError, match="probability"):
            F.FusedRMSNorm(8, dropout=p)
        with pytest.raises(ValueError, match="probability"):
            F.GatedFeedForward(8, 8, dropout=p)


def test_a_block_without_the_new_arguments_is_as_before():
    block = F.GatedFeedForward(16, 24)
    assert [n for n, _ in block.named_parameters()] == ["gate", "up", "down"]
    assert block.norm is None and block.dropout == 0.0
    assert [n for n, _ in F.GatedFeedForward(16, 24, norm_eps=1e-5).named_parameters()][-1] == "norm.weight"


# ------------------------------------------------------------- reference
def test_the_norms_gradient_against_differences():
    """The formula that the kernels are held to, against autograd and against differences."""
    torch.manual_seed(0)
    x, r = torch.randn(3, 10, dtype=torch.float64), torch.randn(3, 10, dtype=torch.float64)
    w, dy, dh = torch.randn(10, dtype=torch.float64), torch.randn(3, 10, dtype=torch.float64), \
        torch.randn(3, 10, dtype=torch.float64)
    f, eps = (torch.rand(3, 10) > 0.3).double() / 0.7, 0.1

    def objective(x, r, w):
        h = r + x * f
        y = h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w
        return (y * dy).sum() + (h * dh).sum()

    inputs = [t.clone().requires_grad_() for t in (x, r, w)]
    objective(*inputs).backward()
    h = r + x * f
    rstd = (h.square().mean(-1) + eps).rsqrt()
    dr, _, dx, _, dW, _ = R.norm_grad(dy, h, w, rstd, dh, f)
    for got, want in ((dx, inputs[0].grad), (dr, inputs[1].grad), (dW, inputs[2].grad)):
        assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)
    step = 1e-5
    for k, got in ((0, dx), (1, dr), (2, dW)):
        for at in (0, 7):
            args = [[x, r, w], [x, r, w]]
            for side, sign in ((0, 1), (1, -1)):
                t = args[side][k].clone()
                t.view(-1)[at] += sign * step
                args[side][k] = t
            diff = (objective(*args[0]) - objective(*args[1])) / (2 * step)
            # Central differences are off by a step squared times the third derivative.
            assert abs(float(diff - got.reshape(-1)[at])) < 1e-7


def test_the_sampling_reference_on_cases_by_hand():
    z = [0.0, 2.0, 2.0, 1.0, float("-inf")]
    assert R.sample(z, 0.3, temperature=0.0) == 1
    assert R.sample(z, 0.9, top_k=1) == 1
    assert [R.sample(z, u, top_k=2) for u in (0.0, 0.49, 0.5, 0.99)] == [1, 1, 2, 2]
    assert [R.sample(z, u, min_p=1.0) for u in (0.49, 0.5)] == [1, 2]
    # e^-2, 1, 1, e^-1 in the vocabulary's order: sums .0541, .4540, .8539, 1.
    assert [R.sample(z, u) for u in (0.05, 0.055, 0.453, 0.455, 0.853, 0.855)] == [0, 1, 1, 2, 2, 3]
    # .3995 lies before the second, .799 before the third.
    assert [R.sample(z, 0.99, top_p=p) for p in (0.39, 0.41, 0.79, 0.81)] == [1, 2, 2, 3]
    assert R.sample([float("-inf")] * 3, 0.5) == R.sample([0.0, NAN], 0.5) == -1
    assert R.sample([0.0, float("inf"), float("inf")], 0.6) == 2


# --------------------------------------------------------------- sources
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_cross_entropy_gemm_gb300", "csrc")


@pytest.mark.parametrize("name", ["rms_norm.cu", "rms_norm.cuh", "rms_norm_grad.cuh", "rms_norm_bf16.cu",
                                  "rms_norm_grad_bf16.cu", "dropout.cu", "sample.cu", "stream_ops.cuh"])
def test_dependent_kernels(name):
    """They wait for their predecessor, once in each kernel, and use no read-only loads: what
    they read may still be written while they are resident."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|ldu\.global|__restrict__", text)
    bodies = re.split(r"__global__", text)[1:]
    assert bodies or name not in ("rms_norm.cu", "rms_norm.cuh", "rms_norm_grad.cuh", "dropout.cu", "sample.cu")
    for body in bodies:
        assert body.count("griddep_wait()") == 1
