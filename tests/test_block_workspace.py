"""Workspace sizes of the linear layer's backward, without a GPU."""
import ctypes

import pytest

from linear_cross_entropy_gemm_gb300 import _lib
from linear_cross_entropy_gemm_gb300 import build as B

AT = 4096  # an aligned address that is never dereferenced: the calls are refused first


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def sizes(lib, **kw):
    p = ctypes.byref(_lib.FlceLinearParams(**kw))
    return lib.flce_linear_workspace_size(p, 1), lib.flce_linear_workspace_size(p, 2)


def test_dz_takes_scratch_only_where_it_is_not_dy(lib):
    any_dy, aligned = sizes(lib, M=8192, K=1024, N=4096)
    assert any_dy >= 8192 * 4096 * 2 and 0 < aligned <= 4096
    any_dy, aligned = sizes(lib, M=8192, K=1024, N=4096, has_bias=1)
    assert any_dy - aligned == 8192 * 4096 * 2
    # A dy of little extent is copied where enough SMs read it.
    any_dy, aligned = sizes(lib, M=15, K=1024, N=64)
    assert any_dy >= 15 * 64 * 2 and 0 < aligned <= 4096
    for kw in (dict(activation=4), dict(N=4100), dict(ld_y=4099), dict(M=15, N=64, K=16384)):
        any_dy, aligned = sizes(lib, **{**dict(M=8192, K=1024, N=4096), **kw})
        assert any_dy == aligned >= 15 * 64 * 2
    p = ctypes.byref(_lib.FlceLinearParams(M=8192, K=1024, N=4096))
    assert lib.flce_linear_workspace_size(p, 3) == 0
    need = lib.flce_linear_workspace_size(p, 2)
    # dy off the boundary needs the whole; on it, not less than it asks for.
    assert lib.flce_linear_backward(p, AT + 2, AT, AT, None, AT, AT, None, AT, need, None, None) == 3
    assert lib.flce_linear_backward(p, AT, AT, AT, None, AT, AT, None, AT, need - 1, None, None) == 3
