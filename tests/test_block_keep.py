"""The forms of the kept values, without a GPU: refusals of unknown ones, and the enum."""
import ctypes
import os
import re

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F
from linear_cross_entropy_gemm_gb300 import _lib
from linear_cross_entropy_gemm_gb300 import build as B

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "flce.h")
AT = 4096  # an aligned address that is never dereferenced: the calls are refused first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def test_enum_matches_the_header():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    keep = {m.group(1).lower(): int(m.group(2)) for m in re.finditer(r"FLCE_KEEP_(\w+)\s*=\s*(\d+)", src)}
    assert keep == _lib.KEEP


@pytest.mark.parametrize("keep", [-1, 2])
def test_linear_form_refused(lib, keep):
    p = ctypes.byref(_lib.FlceLinearParams(M=4, K=64, N=16, activation=4, keep=keep))
    assert lib.flce_linear_forward(p, AT, AT, None, None, AT, AT, None, 0, None, None) == 1
    assert lib.flce_linear_backward(p, AT, AT, AT, AT, AT, AT, None, AT, 1 << 40, None, None) == 1
    assert lib.flce_linear_workspace_size(p, 1) == 0


@pytest.mark.parametrize("keep", [-1, 2])
def test_gated_form_refused(lib, keep):
    p = ctypes.byref(_lib.FlceGatedParams(M=4, K=64, F=16, activation=4, keep=keep))
    assert lib.flce_gated_forward(p, AT, AT, AT, AT, AT, None, 0, None, None) == 1
    assert lib.flce_gated_backward(p, AT, AT, AT, AT, AT, AT, AT, AT, AT, 1 << 40, None, None) == 1
    assert lib.flce_gated_workspace_size(p, 1) == 0


def test_autograd_form_refuses_unknown_names():
    x, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="keep"):
        F.fused_linear(x, W, activation="silu", keep="exact")
    with pytest.raises(ValueError, match="keep"):
        F.gated_linear(x, W, W, keep="exact")
