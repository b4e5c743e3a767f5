"""Build step of the CUDA library: nvcc for sm_100a into ``libgg.so`` next to this file, and of
the Python module ``_native_...`` (``csrc/binding.cpp``, the quick way into the layer's calls).

Run ``python -m moe_grouped_gemm_ragged_b200._build`` (or call :func:`build`). Each is rebuilt
when a source of its own under ``csrc/`` or ``include/`` is newer than it. The module reads torch's
tensors through what it was compiled against, so its name tells that torch: another torch finds
none, makes its own, or goes without.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings

try:
    from ._native_name import native_name
except ImportError:  # run as a file
    from _native_name import native_name

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgg.so")
BINDING = os.path.join(CSRC, "binding.cpp")
# for this interpreter and this torch only: others do not find it
NATIVE = os.path.join(PKG, native_name() + sysconfig.get_config_var("EXT_SUFFIX"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(INCLUDE, "*.h"))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False, out: str = None, defines=()) -> str:
    """Compile ``csrc/*.cu`` into ``libgg.so`` (sm_100a) unless it is up to date, then the Python
    module; where that cannot be compiled, a warning says so.

    ``out`` and ``defines`` (``NAME=VALUE`` strings) build another copy with other tuning
    macros; such a copy is always rebuilt."""
    target = out or LIB
    if out is not None or force or stale():
        _build_library(target, verbose, defines)
    if out is None:
        try:
            build_binding(force, verbose)
        except (subprocess.CalledProcessError, OSError, ImportError) as e:
            if os.path.exists(NATIVE):  # of older sources
                os.remove(NATIVE)
            warnings.warn(f"csrc/binding.cpp could not be built ({e}); the layer's calls go "
                          "through ctypes, some microseconds slower", RuntimeWarning)
    return target


def _build_library(target: str, verbose: bool, defines) -> None:
    tmp = target + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *NVCC_FLAGS, *[f"-D{d}" for d in defines], "-I", INCLUDE, "-I", CSRC,
           *sources(), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, target)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile ``csrc/binding.cpp`` against this interpreter's torch unless it is up to date."""
    inputs = [BINDING, os.path.join(INCLUDE, "gg.h")]
    if (not force and os.path.exists(NATIVE)
            and all(os.path.getmtime(f) <= os.path.getmtime(NATIVE) for f in inputs)):
        return NATIVE
    import torch
    from torch.utils import cpp_extension

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-DGG_MODULE={native_name()}",
           *[f"-I{d}" for d in cpp_extension.include_paths()],
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-I", INCLUDE, BINDING, "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, NATIVE)
    return NATIVE


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
