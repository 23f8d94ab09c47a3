"""Build libgale.so (all CUDA sources under csrc/) for sm_100a with nvcc, and the
compiled part of the Python binding (binding.cpp) with g++.

Run ``python -m bit_expert_gemv_b200.build`` (or call ``build()``); both are
written next to this file so that they travel with the package.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgale.so")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SOURCE = os.path.join(HERE, "binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-O3", "-shared",
    "--expt-relaxed-constexpr", "--threads", "0",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps + glob.glob(os.path.join(ROOT, "include", "*.h")) +
               [os.path.abspath(__file__)])


def _stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile binding.cpp against torch and the built libgale.so; returns the module's path."""
    if not force and not _older(BINDING, [BINDING_SOURCE]):
        return BINDING
    from torch.utils import cpp_extension as ext
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
           *[a for p in ext.include_paths() for a in ("-isystem", p)], "-isystem", "/usr/local/cuda/include",
           BINDING_SOURCE, "-o", tmp, "-L" + HERE, "-l:libgale.so", "-Wl,-rpath,$ORIGIN",
           *["-L" + p for p in ext.library_paths()], "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile every csrc/*.cu into libgale.so, and the binding; returns the library path."""
    if not force and not _stale():
        build_binding(verbose=verbose)
        return LIB
    tmp = LIB + ".tmp"
    cmd = [NVCC, *FLAGS, *extra, *sources(), "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(force=force, verbose=verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
