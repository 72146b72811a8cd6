"""Build libmoe.so (the CUDA library behind include/moe.h) in-tree for sm_100a, and
_binding.so (csrc/binding.cpp, the tensor arguments of the row operators).

    python -m expert_routing_grouped_layer_b200.build [--force] [--verbose]

nvcc cross-compiles without a GPU. The shared object lands next to this file
so that it travels with the source tree and is the one the binding loads.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmoe.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_STAMP = os.path.join(HERE, "_binding.torch")  # the torch version it was compiled for

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr", "--threads", "0",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _binding_stale(torch_version: str) -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_STAMP):
        return True
    with open(BINDING_STAMP) as f:
        if f.read() != torch_version:
            return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(d) > t for d in (BINDING_SRC, os.path.join(INCLUDE, "moe.h")))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile the native module against the installed torch's headers (no nvcc). It is
    compiled again when its sources or torch's version change."""
    import sysconfig

    import torch
    if not force and not _binding_stale(torch.__version__):
        return BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(torch.__version__)
    return BINDING


def build_library(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-I", INCLUDE, "-I", CSRC, "-o", tmp] + sources()
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The library, which needs no torch, then the native module, which is left out where
    torch is not installed (the calls that need it say so)."""
    build_library(force, verbose, extra)
    try:
        build_binding(force, verbose)
    except ImportError as e:
        print("%s is not built: %s" % (os.path.basename(BINDING), e), file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ())
    print(LIB)
