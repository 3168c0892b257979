"""Builds the CUDA library libllama_attn.so for sm_100a (nvcc) and the Python
module _binding.so that calls its paged-cache entry points (g++), in-tree."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "llama_attn.cu")
LIB = os.path.join(PKG, "libllama_attn.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING_SRC = os.path.join(PKG, "csrc", "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_STAMP = os.path.join(PKG, "_binding.torch")


def sources():
    csrc = os.path.join(PKG, "csrc")
    files = [os.path.join(csrc, f) for f in os.listdir(csrc) if f.endswith((".cu", ".cuh"))]
    return files + [os.path.join(INCLUDE, "llama_attn.h")]


def nvcc_command(out: str = LIB, extra=()):
    return ["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
            "-shared", "-Xcompiler", "-fPIC", "-I" + INCLUDE, *extra, "-o", out, SRC]


def binding_command(out: str = BINDING):
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
            "-I" + os.path.join(base, "include"), "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), BINDING_SRC, "-o", out,
            "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _stale(target: str, files) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(f) > os.path.getmtime(target) for f in files)


def _torch_version() -> str:
    import torch
    return torch.__version__


def build_binding(force: bool = False) -> str:
    """The Python module. It holds torch's C++ interface, so another torch makes it stale too
    (its stamp names the version that it was built against)."""
    version = _torch_version()
    built_for = None
    if os.path.exists(BINDING_STAMP):
        with open(BINDING_STAMP) as f:
            built_for = f.read()
    if force or built_for != version or _stale(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "llama_attn.h")]):
        tmp = BINDING + f".tmp{os.getpid()}"
        subprocess.check_call(binding_command(tmp))
        os.replace(tmp, BINDING)
        with open(BINDING_STAMP, "w") as f:
            f.write(version)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    # The library first: it needs nvcc only, and a C program needs nothing else.
    if force or _stale(LIB, sources()):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = nvcc_command(tmp, ["-Xptxas", "-v"] if verbose else [])
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
