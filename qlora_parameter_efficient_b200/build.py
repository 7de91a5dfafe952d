"""Builds libqlora.so in-tree with nvcc for sm_100a (B200).

    python -m qlora_parameter_efficient_b200.build            # release: libqlora.so, _mx_bind-*.so
    python -m qlora_parameter_efficient_b200.build --debug    # libqlora_debug.so, QLORA_DEBUG=1

libqlora.so needs the CUDA toolkit alone.  _mx_bind-*.so, the short way from Python into the microscaled
calls, is built where torch and its headers are found; without it the same calls go through ctypes.

The debug library checks the kernels' index invariants on the device (a failed check is
reported as QLORA_ERR_DEVICE by qlora_get_device_error); load it with QLORA_LIB=<path>.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libqlora.so")
DEBUG_LIB = os.path.join(HERE, "libqlora_debug.so")
SOURCES = ["qlora_api.cu", "noalloc.cu"]
DEPS = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))
BINDING_SOURCE = os.path.join(CSRC, "mx_bind.cpp")
HEADER = os.path.join(os.path.dirname(HERE), "include", "qlora.h")

NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-shared", "-Xcompiler", "-fPIC",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, d) for d in DEPS] + [HEADER]
    return all(os.path.getmtime(d) <= t for d in deps if os.path.exists(d))


def build_library(force: bool = False, verbose: bool = False, debug: bool = False, out: str = None) -> str:
    lib = out or (DEBUG_LIB if debug else LIB)
    if not force and up_to_date(lib):
        return lib
    flags = NVCC_FLAGS + (["-DQLORA_DEBUG=1"] if debug else [])
    cmd = [nvcc(), *flags, "-o", lib + ".tmp", *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libqlora.so")
    os.replace(lib + ".tmp", lib)
    return lib


def build_binding(force: bool = False, verbose: bool = False) -> str | None:
    """The CPython module csrc/mx_bind.cpp (host code only: g++ against torch's headers), for the torch and the
    Python that run this.  None, with a line that says so, where there is no torch to build it against."""
    try:
        import torch
    except ImportError:
        print("no torch: the Python binding of the microscaled calls is not built", flush=True)
        return None
    root = os.path.dirname(torch.__file__)
    if not os.path.exists(os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h")):
        print(f"no headers in {root}: the Python binding of the microscaled calls is not built", flush=True)
        return None
    from . import _mx_bind_path
    binding = _mx_bind_path()
    if not force and os.path.exists(binding) and all(
            os.path.getmtime(d) <= os.path.getmtime(binding) for d in (BINDING_SOURCE, HEADER)):
        return binding
    import sysconfig
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = os.path.join(root, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in includes],
           "-o", binding + ".tmp", BINDING_SOURCE, f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building the binding")
    os.replace(binding + ".tmp", binding)
    return binding


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
    print(build_binding(force="--force" in sys.argv, verbose=True))
