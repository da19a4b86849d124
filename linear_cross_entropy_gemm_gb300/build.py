"""Build the sm_103a shared library ``libflce_gb300.so`` in-tree with nvcc, and
``_flce_torch.so``, the Python calls of the layer operators, with g++.

Each translation unit under ``csrc/`` is compiled in parallel, then linked
with the static CUDA runtime. Rebuilds only when a source or header is newer
than the libraries. No CMake, no torch extension machinery.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libflce_gb300.so")
CALLS = os.path.join(PKG, "_flce_torch.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the FLCE library needs the CUDA 13 toolkit to build")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [CALLS_SRC, __file__]


def _calls_wanted() -> bool:
    """Whether the Python calls can be built: torch and Python's headers are here. The
    library for C callers needs neither."""
    headers = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return importlib.util.find_spec("torch") is not None and os.path.exists(headers)


def _calls_commands(obj: str):
    """g++ commands that compile and link the Python calls against the installed torch."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found: the FLCE library needs a C++ compiler to build")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=1", "-I", INCLUDE,
                "-I", os.path.join(torch, "include"), "-I", sysconfig.get_paths()["include"],
                "-I", os.path.join(cuda, "include"), "-c", CALLS_SRC, "-o", obj]
    link = [cxx, "-shared", "-o", CALLS + ".tmp", obj, "-L", os.path.join(torch, "lib"), "-L", PKG,
            "-l:libflce_gb300.so", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def up_to_date() -> bool:
    made = [LIB, CALLS] if _calls_wanted() else [LIB]
    if not all(os.path.exists(m) for m in made):
        return False
    t = min(os.path.getmtime(m) for m in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link; returns the library path. Raises on a compile error."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    calls_link = None
    if _calls_wanted():
        calls_compile, calls_link = _calls_commands(os.path.join(BUILD, "torch_calls.o"))
        if verbose:
            print(" ".join(calls_compile), flush=True)
        procs.append((CALLS_SRC, subprocess.Popen(calls_compile, stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    else:
        print("torch or Python.h is missing: building the C library alone", flush=True)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stdout.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError("compilation failed on: " + ", ".join(os.path.basename(f) for f in failed))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        sys.stdout.write(r.stdout.decode(errors="replace"))
        raise RuntimeError("link of libflce_gb300.so failed")
    os.replace(tmp, LIB)
    if calls_link is None:
        return LIB
    r = subprocess.run(calls_link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        sys.stdout.write(r.stdout.decode(errors="replace"))
        raise RuntimeError("link of _flce_torch.so failed")
    os.replace(CALLS + ".tmp", CALLS)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
