"""The choice of kernel forms, without a GPU: the shapes of block_plans.py reach every form that a
call can take, so that the tests on the GPU run each of them, and a change of the choice that
leaves one without a test fails here."""
import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

import block_plans as P
from linear_cross_entropy_gemm_gb300 import _lib
from linear_cross_entropy_gemm_gb300 import build as B

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return _lib.load()


def covered(op):
    return {plan for shape in getattr(P, op.upper()) for plan in P.plans(op, *shape)}


@pytest.mark.parametrize("op", ["linear", "gated"])
@pytest.mark.parametrize("seed", [1, 2])
def test_every_form_that_calls_take_has_a_tested_shape(op, seed):
    rng = random.Random(seed)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    have, missing = covered(op), {}
    for _ in range(40000):
        M, K, N = log(1, 16384), 8 * log(1, 2048), log(1, 16384)
        if op == "gated":
            N = -(-N // 8) * 8
        for plan in P.plans(op, M, K, N):
            if plan not in have:
                missing.setdefault(plan, (M, K, N))
    assert not missing


def test_forms_that_must_not_lose_their_test():
    """Those that real shapes take seldom, and the ones of the largest products."""
    linear, gated = covered("linear"), covered("gated")
    for have in (linear, gated):
        for form in [(0, 1, 192, 3), (0, 1, 256, 2), (0, 1, 128, 2), (0, 1, 256, 1), (0, 1, 224, 1),
                     (0, 1, 128, 1), (0, 1, 64, 1), (0, 1, 192, 1), (128, 0, 0, 2), (128, 0, 0, 8)]:
            assert ("forward", *form) in have
        for form in [(0, 1, 256, 2), (0, 1, 128, 2), (0, 2, 256, 1), (0, 2, 192, 1), (0, 1, 256, 1)]:
            assert ("dx", *form) in have and ("dW", *form) in have
        for tokens in (16, 32, 64):
            for slices in (1, 2, 4, 8):
                assert ("forward", tokens, 0, 0, slices) in have
                assert ("dx", tokens, 0, 0, slices) in have or (have is gated and slices == 1)


def test_plan_refusals_and_layout(lib, tmp_path):
    plan, bad = _lib.FlcePlan(), ctypes.byref(_lib.FlceLinearParams(M=4, K=12, N=16))
    good = ctypes.byref(_lib.FlceLinearParams(M=4, K=64, N=16))
    assert lib.flce_linear_plan(bad, 0, ctypes.byref(plan)) == 2
    assert lib.flce_linear_plan(good, 3, ctypes.byref(plan)) == 1
    assert lib.flce_linear_plan(good, -1, ctypes.byref(plan)) == 1
    assert lib.flce_linear_plan(good, 0, None) == 1
    assert lib.flce_linear_plan(None, 0, ctypes.byref(plan)) == 1
    assert lib.flce_linear_plan(ctypes.byref(_lib.FlceLinearParams(M=0, K=64, N=16)), 0,
                                ctypes.byref(plan)) == 1
    assert lib.flce_gated_plan(ctypes.byref(_lib.FlceGatedParams(M=4, K=64, F=16)), 3,
                               ctypes.byref(plan)) == 1
    assert lib.flce_gated_plan(ctypes.byref(_lib.FlceGatedParams(M=4, K=64, F=12)), 0,
                               ctypes.byref(plan)) == 2
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in _lib.FlcePlan._fields_]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"flce.h\"\nint main(void) {\n"
                   + "".join(f'  printf("%zu\\n", offsetof(flce_plan_t, {f}));\n' for f in fields)
                   + '  printf("%zu\\n", sizeof(flce_plan_t));\n  return 0;\n}\n')
    subprocess.run([cc, "-I", INCLUDE, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True, text=True)
    assert [int(v) for v in got.stdout.split()] == \
        [getattr(_lib.FlcePlan, f).offset for f in fields] + [ctypes.sizeof(_lib.FlcePlan)]
