"""Build libep.so in-tree: each .cu compiled for sm_103a in parallel, then linked.
Beside it _layer_bind.so, the compiled part of layer.py (g++, against torch's headers): where it cannot be
built, a warning says why and the library stands without the layer operators' Python calls.

Usage: python -m combine_get_dispatch_layout_gb300.build [--force]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(PKG, "libep.so")
BIND = os.path.join(PKG, "_layer_bind.so")
BIND_SOURCE = os.path.join(CSRC, "layer_bind.cpp")
OBJ = os.path.join(PKG, "_build")
BIND_STAMP = os.path.join(OBJ, "layer_bind.stamp")   # what _layer_bind.so was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(built: str, deps: list[str]) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(d) > os.path.getmtime(built) for d in deps)


def _lib_stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _bind_against() -> str:
    import torch

    return f"torch {torch.__version__}, python {sys.version.split()[0]}"


def _bind_stale() -> bool:
    """The binding loads only into the Python and the torch whose headers it was built with."""
    if _older(BIND, [BIND_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h"))) or not os.path.exists(BIND_STAMP):
        return True
    with open(BIND_STAMP) as f:
        return f.read() != _bind_against()


def _build_bind() -> None:
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.abspath(_nvcc()))) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"), BIND_SOURCE, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BIND_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(BIND_STAMP, "w") as f:
        f.write(_bind_against())


def _build_lib(verbose: bool) -> None:
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(len(sources())) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(1) as ex:
        bind = ex.submit(_build_bind) if force or _bind_stale() else None
        if force or _lib_stale():
            _build_lib(verbose)
        try:
            if bind:
                bind.result()
        except Exception as e:   # (the library does not need it; layer.py raises where it is missing)
            warnings.warn(f"the layer operators' Python binding was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
