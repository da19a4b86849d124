"""The layer operators' C ABI without a GPU: struct layouts, enums, workspace
sizes and the refusals that precede every launch."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from linear_cross_entropy_gemm_gb300 import _lib
from linear_cross_entropy_gemm_gb300 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "flce.h")
AT = 4096  # an aligned address that is never dereferenced: the calls are refused first
INVALID, ALIGNMENT, SMALL, UNSUPPORTED = 1, 2, 3, 7


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def linear(**kw):
    v = dict(M=4, K=64, N=16)
    v.update(kw)
    return _lib.FlceLinearParams(**v)


def gated(**kw):
    v = dict(M=4, K=64, F=16, activation=4)
    v.update(kw)
    return _lib.FlceGatedParams(**v)


@pytest.mark.parametrize("struct,name", [(_lib.FlceLinearParams, "flce_linear_params_t"),
                                         (_lib.FlceGatedParams, "flce_gated_params_t")])
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


def test_enums_match_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    acts = {m.group(1).lower(): int(m.group(2)) for m in re.finditer(r"FLCE_ACT_(\w+)\s*=\s*(\d+)", src)}
    types = {m.group(1).lower(): int(m.group(2)) for m in re.finditer(r"FLCE_DTYPE_(\w+)\s*=\s*(\d+)", src)}
    assert acts == _lib.ACTIVATIONS and types == _lib.DTYPES


LINEAR_BAD = [(dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID),
              (dict(K=12), ALIGNMENT), (dict(ld_x=68), ALIGNMENT), (dict(ld_x=32), INVALID),
              (dict(ld_x=-64), INVALID), (dict(ld_y=15), INVALID), (dict(ld_res=8), INVALID),
              (dict(activation=6), INVALID), (dict(activation=-1), INVALID),
              (dict(has_bias=2), INVALID), (dict(input_fp16=2), INVALID), (dict(dW_fp32=-1), INVALID),
              (dict(M=1 << 31), UNSUPPORTED), (dict(N=1 << 25), UNSUPPORTED),
              (dict(M=1 << 30, N=1 << 24), UNSUPPORTED)]
GATED_BAD = [(dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(F=0), INVALID),
             (dict(F=12), ALIGNMENT), (dict(K=12), ALIGNMENT), (dict(ld_h=20), ALIGNMENT),
             (dict(ld_h=8), INVALID), (dict(activation=9), INVALID), (dict(M=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", LINEAR_BAD, ids=str)
def test_linear_parameters_refused(lib, kw, status):
    p = ctypes.byref(linear(**kw))
    assert lib.flce_linear_forward(p, AT, AT, AT, AT, AT, None, None, 0, None, None) == status
    assert lib.flce_linear_backward(p, AT, AT, AT, AT, AT, AT, None, AT, 1 << 40, None, None) == status
    assert lib.flce_linear_workspace_size(p, 1) == 0


@pytest.mark.parametrize("kw,status", GATED_BAD, ids=str)
def test_gated_parameters_refused(lib, kw, status):
    p = ctypes.byref(gated(**kw))
    assert lib.flce_gated_forward(p, AT, AT, AT, AT, None, None, 0, None, None) == status
    assert lib.flce_gated_backward(p, AT, AT, AT, AT, AT, AT, AT, AT, AT, 1 << 40, None, None) == status
    assert lib.flce_gated_workspace_size(p, 1) == 0


def test_pointers_refused(lib):
    p = ctypes.byref(linear())
    fwd = lib.flce_linear_forward
    assert fwd(None, AT, AT, None, None, AT, None, None, 0, None, None) == INVALID
    assert fwd(p, None, AT, None, None, AT, None, None, 0, None, None) == INVALID
    assert fwd(p, AT, None, None, None, AT, None, None, 0, None, None) == INVALID
    assert fwd(p, AT, AT, None, None, None, None, None, 0, None, None) == INVALID
    assert fwd(p, AT + 8, AT, None, None, AT, None, None, 0, None, None) == ALIGNMENT
    assert fwd(p, AT, AT + 2, None, None, AT, None, None, 0, None, None) == ALIGNMENT
    assert fwd(p, AT, AT, None, None, AT + 1, None, None, 0, None, None) == ALIGNMENT
    assert fwd(p, AT, AT, None, None, AT, AT + 4, None, 0, None, None) == ALIGNMENT
    both = ctypes.byref(linear(has_bias=1, has_residual=1))
    assert fwd(both, AT, AT, None, AT, AT, None, None, 0, None, None) == INVALID
    assert fwd(both, AT, AT, AT, None, AT, None, None, 0, None, None) == INVALID
    assert fwd(both, AT, AT, AT + 2, AT, AT, None, None, 0, None, None) == ALIGNMENT
    bwd = lib.flce_linear_backward
    assert bwd(p, AT, AT, AT, None, AT, AT, AT, AT, 1 << 40, None, None) == INVALID  # db, no bias
    assert bwd(p, AT, AT, AT, None, AT, AT, None, None, 0, None, None) == INVALID
    assert bwd(p, AT, AT, AT, None, AT, AT, None, AT, 16, None, None) == SMALL
    assert bwd(p, AT, AT, AT, None, AT + 8, AT, None, AT, 1 << 40, None, None) == ALIGNMENT
    act = ctypes.byref(linear(activation=2))
    assert bwd(act, AT, AT, AT, None, AT, AT, None, AT, 1 << 40, None, None) == INVALID  # no z
    assert bwd(p, None, None, None, None, None, None, None, None, 0, None, None) == 0  # nothing asked
    q = ctypes.byref(gated())
    assert lib.flce_gated_forward(q, AT, AT, AT, AT + 2, None, None, 0, None, None) == ALIGNMENT
    assert lib.flce_gated_forward(q, AT, AT, None, AT, None, None, 0, None, None) == INVALID
    gb = lib.flce_gated_backward
    assert gb(q, AT, AT, AT, AT, AT, AT, AT, None, AT, 1 << 40, None, None) == INVALID
    assert gb(q, AT, AT, AT, AT, None, AT, AT, AT, AT, 1 << 40, None, None) == INVALID
    assert gb(q, AT, AT, AT, AT, AT, AT, AT, AT, AT, 16, None, None) == SMALL


def test_no_tokens_is_a_no_op(lib):
    p, q = ctypes.byref(linear(M=0)), ctypes.byref(gated(M=0))
    assert lib.flce_linear_forward(p, None, None, None, None, None, None, None, 0, None, None) == 0
    assert lib.flce_gated_forward(q, None, None, None, None, None, None, 0, None, None) == 0
    assert lib.flce_linear_workspace_size(p, 1) == 0 and lib.flce_gated_workspace_size(q, 1) == 0


def test_workspace_sizes(lib):
    p = ctypes.byref(linear(M=1000, N=515, has_bias=1))
    assert lib.flce_linear_workspace_size(p, 1) >= 1000 * 520 * 2 + 515 * 4
    q = ctypes.byref(gated(M=1000, F=520))
    assert lib.flce_gated_workspace_size(q, 1) >= 2 * 1000 * 520 * 2
    assert lib.flce_linear_workspace_size(None, 1) == 0
    assert lib.flce_grad_norm_workspace_size(5) > 0 and lib.flce_grad_norm_workspace_size(-1) == 0


def test_gradient_lists_refused(lib):
    def call(ptrs, numel, types, norm=AT, ws=AT, nbytes=1 << 30, out=None, max_norm=1.0, eps=1e-6,
             count=None):
        n = len(ptrs)
        a = (ctypes.c_void_p * n)(*ptrs)
        o = None if out is None else (ctypes.c_void_p * n)(*out)
        args = (n if count is None else count, a)
        rest = ((ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*types))
        st = lib.flce_clip_grads(*args, o, *rest, max_norm, eps, norm, ws, nbytes, None)
        if out is None and max_norm == 1.0 and eps == 1e-6:
            assert lib.flce_grad_norm(*args, *rest, norm, ws, nbytes, None) == st
        return st

    assert call([AT], [-1], [0]) == INVALID
    assert call([AT], [4], [3]) == INVALID
    assert call([None], [4], [0]) == INVALID
    assert call([AT + 1], [4], [0]) == ALIGNMENT
    assert call([AT + 2], [4], [2]) == ALIGNMENT
    assert call([AT], [4], [0], norm=None) == INVALID
    assert call([AT], [4], [0], norm=AT + 2) == ALIGNMENT
    assert call([AT], [4], [0], ws=None) == INVALID
    assert call([AT], [4], [0], nbytes=8) == SMALL
    assert call([AT], [4], [0], count=-1) == INVALID
    assert call([AT], [1 << 49], [0]) == UNSUPPORTED
    assert call([AT], [4], [0], out=[None]) == INVALID
    assert call([AT], [4], [2], out=[AT + 2]) == ALIGNMENT
    assert call([AT], [4], [0], max_norm=-1.0) == INVALID
    assert call([AT], [4], [0], max_norm=float("nan")) == INVALID
    assert call([AT], [4], [0], eps=float("inf")) == INVALID
