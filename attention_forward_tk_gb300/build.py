"""Compile in-tree: the CUDA library ``_build/libtk_attn.so`` for sm_103a, and
``_build/_tk_torch.so``, the compiled torch helpers of the serving calls.

Four translation units compiled side by side (attention, Based and GEMM; per-head
norm with rotation; the 8-bit paged cache; the host-buffer pipeline),
one ``-gencode``; no cmake.
The same commands work on x86_64 and aarch64 hosts.
"""
from __future__ import annotations

import os
import subprocess
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
CSRC = os.path.join(_HERE, "csrc")
INCLUDE = os.path.join(_ROOT, "include")
BUILD_DIR = os.path.join(_HERE, "_build")
LIB = os.path.join(BUILD_DIR, "libtk_attn.so")
BINDING = os.path.join(BUILD_DIR, "_tk_torch.so")
BINDING_SOURCE = os.path.join(CSRC, "tk_torch.cpp")
SOURCES = [os.path.join(CSRC, f) for f in ("tk_attn.cu", "tk_norm_rope.cu", "tk_kv8.cu",
                                            "tk_attn_host.cpp")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
    os.path.join(INCLUDE, "tk_attn.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared", "--threads", "4",
    "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build libtk_attn.so if it is missing or older than its sources."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(p) for p in DEPS if os.path.exists(p))
        if os.path.getmtime(LIB) >= newest:
            return LIB
    tmp = f"{LIB}.tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp, *SOURCES]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libtk_attn.so")
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False) -> str:
    """Build _tk_torch.so (after libtk_attn.so, which it links) if it is missing
    or older than its sources."""
    import sysconfig

    import torch

    os.makedirs(BUILD_DIR, exist_ok=True)
    deps = [BINDING_SOURCE, os.path.join(INCLUDE, "tk_attn.h")]
    if not force and os.path.exists(BINDING) and \
            os.path.getmtime(BINDING) >= max(os.path.getmtime(p) for p in deps):
        return BINDING
    tmp = f"{BINDING}.tmp{os.getpid()}"
    torch_dir = os.path.dirname(torch.__file__)
    headers = os.path.join(torch_dir, "include")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-I", cuda, "-I", sysconfig.get_paths()["include"],
           "-isystem", headers, "-isystem", os.path.join(headers, "torch", "csrc", "api", "include"),
           BINDING_SOURCE, "-o", tmp, "-L", BUILD_DIR, "-l:libtk_attn.so", "-L",
           os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("the compiler failed building _tk_torch.so")
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_binding(force="--force" in sys.argv))
