"""Build libsdm.so (the C-ABI CUDA library) and _layers.so (the Python binding of its
layer entry points) in-tree for sm_103a.

Each translation unit under csrc/ is compiled by its own process (in parallel:
nvcc for the library's, the host compiler for the binding's, against torch's
headers), then linked into ``sparse_state_linear_sdm_gb300/libsdm.so`` and
``_layers.so``.  The CUDA runtime is linked statically into the library, so it
builds and loads on its own; the binding needs it and torch, and is rebuilt when
torch or Python is another than the one it was compiled for.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import platform
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsdm.so")
BINDING = os.path.join(PKG, "_layers.so")
BINDING_SRC = os.path.join(CSRC, "sdm_binding.cpp")
BINDING_TAG = BINDING + ".tag"  # what the binding was compiled for
HEADER = os.path.join(os.path.dirname(PKG), "include", "sdm.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the SDM CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer_than(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def up_to_date() -> bool:
    """Whether the library is newer than its sources."""
    return _newer_than(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER])


def _binding_tag() -> str:
    import torch

    return f"torch {torch.__version__}, python {sys.version}, {platform.machine()}"


def binding_up_to_date() -> bool:
    """Whether the binding is newer than its sources and was compiled for this torch and Python."""
    if not _newer_than(BINDING, [BINDING_SRC, HEADER]) or not os.path.exists(BINDING_TAG):
        return False
    with open(BINDING_TAG) as f:
        return f.read() == _binding_tag()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _compile_binding(cc: str) -> str:
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")]
    obj = os.path.join(BUILD, "sdm_binding.o")
    _run([shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-Wall",
          *[a for d in dirs for a in ("-isystem", d)], "-c", BINDING_SRC, "-o", obj], "compiling the binding")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    _run([shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libsdm.so", "-L", libs,
          "-ltorch_python", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], "linking the binding")
    if os.path.exists(BINDING_TAG):
        os.remove(BINDING_TAG)  # until the new one is in place
    os.replace(tmp, BINDING)
    with open(BINDING_TAG, "w") as f:
        f.write(_binding_tag())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Builds the library where it is absent or stale; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False, **library) -> str:
    """Builds the library (with the arguments of build()) and, beside it, the binding where they are absent or
    stale; returns the binding's path."""
    if not force and binding_up_to_date():
        build(**library)
        return BINDING
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_binding, nvcc())
        build(force=force, **library)
        _link_binding(obj.result())
    return BINDING


if __name__ == "__main__":
    build_binding(force="--force" in sys.argv, verbose=True,
                  extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
