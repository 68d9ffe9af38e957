"""Build libsmlp.so in-tree with hipcc for gfx950, and the Python module of the short calls.

    python -m moe_shared_expert_amd.build

Every call recompiles all sources (object files go to ``_build/`` next to this file,
the library to ``libsmlp.so`` and the module to ``_calls.so`` next to this file).
"""
from __future__ import annotations

import concurrent.futures as cf
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsmlp.so")
CALLS = os.path.join(PKG, "_calls.so")

SOURCES = ["api.cpp", "layout.cpp", "skinny.hip", "gemm.hip", "aux.hip", "latent.hip", "ceilings.hip",
           "noalloc.hip", "moe.cpp", "route.hip", "fp8.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found (need ROCm in /opt/rocm)")
    return exe


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), "-c", os.path.join(CSRC, src), "-o", obj, "-O3", "-fPIC", "-std=c++17",
           "-I", INCLUDE, "-I", CSRC, "-Wall", "-Wno-unused-function"]
    if src.endswith(".hip"):
        # Packed fp32 vector ops are disabled in device code.
        cmd += ["--offload-arch=" + ARCH, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-munsafe-fp-atomics"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_calls() -> str:
    """torch_calls.cpp against torch's headers (host code only)."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, "torch_calls.o")
    cmd = [shutil.which("g++") or "g++", "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj, "-O2", "-fPIC",
           "-std=c++17", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"], "-Wall"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, LIB, "-L" + lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def build(verbose: bool = False) -> str:
    """The library first: it needs hipcc alone.  The module needs g++ and torch's headers, and
    is left out where torch is not installed (only the binding uses it)."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        calls = ex.submit(_compile_calls) if _has_torch() else None
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", "-o", tmp, *objs, "--offload-arch=" + ARCH, "-Wl,-soname,libsmlp.so"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if calls:
        _link_calls(calls.result())
    if verbose:
        print("built", LIB, *(("and", CALLS) if calls else ("(torch is not installed: no _calls.so)",)))
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
