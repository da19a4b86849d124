"""The build without torch: the library for C callers needs the CUDA toolkit alone."""
import os
import types

import pytest

from linear_cross_entropy_gemm_gb300 import build as B


@pytest.mark.parametrize("missing", ["torch", "headers", None])
def test_the_c_library_builds_without_torch(monkeypatch, tmp_path, missing):
    """The commands of a forced build, recorded instead of run."""
    ran, moved = [], []

    class Process:
        returncode = 0

        def __init__(self, cmd, **_):
            ran.append(cmd)

        def communicate(self):
            return b"", None

    def run(cmd, **_):
        ran.append(cmd)
        return types.SimpleNamespace(returncode=0, stdout=b"")

    monkeypatch.setattr(B.subprocess, "Popen", Process)
    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B.os, "replace", lambda a, b: moved.append(os.path.basename(b)))
    monkeypatch.setattr(B, "_nvcc", lambda: "/cuda/bin/nvcc")
    if missing == "torch":
        find = B.importlib.util.find_spec
        monkeypatch.setattr(B.importlib.util, "find_spec",
                            lambda name, *a: None if name == "torch" else find(name, *a))
    elif missing == "headers":
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        (tmp_path / "Python.h").write_text("")
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert B.build(force=True) == B.LIB
    others = [c for c in ran if c[0] != "/cuda/bin/nvcc"]
    if missing is None:
        assert moved == ["libflce_gb300.so", "_flce_torch.so"] and len(others) == 2
    else:
        assert moved == ["libflce_gb300.so"] and not others


def test_up_to_date_without_torch_looks_at_the_library_alone(monkeypatch, tmp_path):
    lib = tmp_path / "lib.so"
    lib.write_text("")
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "none.so"))
    monkeypatch.setattr(B, "_deps", lambda: [])
    assert not B.up_to_date()
    find = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.up_to_date()
