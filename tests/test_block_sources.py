"""Rules that the sources of the layer operators' kernels keep."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_cross_entropy_gemm_gb300", "csrc")
DEPENDENT = ["block_rowwise.cu", "block_small.cu", "block_gemm.cu", "block_epilogues.cuh",
             "pair_engine.cuh", "grad_norm.cu"]


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


@pytest.mark.parametrize("name", DEPENDENT)
def test_dependent_kernels_use_no_read_only_loads(name):
    """A kernel that is launched dependently is resident while its predecessor writes the
    inputs, so they are not read-only for its lifetime: no ld.global.nc, by __ldg, by PTX
    or by pointers that let the compiler choose it."""
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|ldu\.global|__restrict__", code(name))


@pytest.mark.parametrize("name", ["block_rowwise.cu", "block_small.cu", "pair_engine.cuh", "grad_norm.cu"])
def test_dependent_kernels_wait_for_their_predecessor(name):
    """Every kernel holds the wait, once."""
    text = code(name)
    bodies = re.split(r"__global__", text)[1:]
    assert bodies
    for body in bodies:
        assert body.count("griddep_wait()") == 1, body[:200]
