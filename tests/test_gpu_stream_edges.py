"""Norm and dropout in the calls that depend on what the process did before, and in the forms that
the module and the calls document."""
import os
import subprocess
import sys

import pytest
import torch

import linear_cross_entropy_gemm_gb300 as F

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

WIDE_ODD = """
import sys
sys.path[:0] = [%r, %r]
import torch
import linear_cross_entropy_gemm_gb300 as F
import stream_reference as R
H, pad, p, seed = %d, %d, 0.25, 77
g = torch.Generator(device="cuda").manual_seed(H)
M = 3
rows = lambda: torch.randn(M, H + pad, device="cuda", generator=g)[:, :H]
x, r, dy = rows(), rows(), rows()
f = R.factors(M, H, p, seed)
rstd = torch.empty(M, device="cuda")
y, h = F.flce_rms_norm_forward(x, None, r, dropout=p, seed=seed, rstd=rstd)
dx, dr, _ = F.flce_rms_norm_backward(dy, h, None, rstd, dropout=p, seed=seed)
e, e_err, d, d_err, _, _ = R.norm_grad(dy, h, None, rstd, None, f)
R.assert_near(dr, e, e_err, "dresidual")
R.assert_near(dx, d, d_err, "dx")
"""


@pytest.mark.parametrize("H,pad", [(23553, 0), (24001, 0), (24575, 0), (24576, 1), (24577, 0), (32767, 0)])
def test_wide_odd_rows_as_a_processs_first_call(H, pad):
    """The backward with dropout off the 16-byte boundaries takes 48 KiB of shared memory for the random
    bits at 23553 .. 24576 columns, beside what it always has: the opt-in above 48 KiB counts both. In a
    process of its own: a wider call before would have opted in."""
    run = subprocess.run([sys.executable, "-c", WIDE_ODD % (os.path.dirname(HERE), HERE, H, pad)],
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_h_false_returns_none():
    x = torch.randn(5, 64, device="cuda")
    for kw in (dict(), dict(residual=x.clone()), dict(dropout=0.5, seed=1)):
        want = F.flce_rms_norm_forward(x, None, **kw)
        y, h = F.flce_rms_norm_forward(x, None, h=False, **kw)
        assert h is None and torch.equal(y, want[0])
        want = F.flce_rms_norm_quantized(x, None, **kw)
        y8, scale, h = F.flce_rms_norm_quantized(x, None, h=False, **kw)
        assert h is None and torch.equal(y8.float(), want[0].float()) and torch.equal(scale, want[1])
    assert F.flce_rms_norm_forward(x, None)[1] is x


def test_the_module_without_a_residual_gives_y_alone():
    """In training with dropout as in evaluation: what norm(x) returns is of one kind."""
    norm = F.FusedRMSNorm(64, dropout=0.5, dtype=torch.float32, device="cuda")
    x = torch.randn(6, 64, device="cuda", requires_grad=True)
    torch.manual_seed(3)
    y = norm(x)
    assert torch.is_tensor(y) and y.shape == x.shape
    torch.manual_seed(3)
    want, h = F.fused_rms_norm(x, norm.weight, None, norm.eps, 0.5)
    assert torch.equal(y, want) and bool((h == 0).any())
    dy = torch.randn_like(y)
    (got,) = torch.autograd.grad(y, x, dy)
    assert torch.equal(got, torch.autograd.grad(want, x, dy)[0])
    assert len(norm(x, x)) == 2
    norm.eval()
    assert torch.is_tensor(norm(x)) and torch.equal(norm(x), F.fused_rms_norm(x, norm.weight, eps=norm.eps))
