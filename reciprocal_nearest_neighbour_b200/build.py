"""Build ``librnn.so`` and ``_fast.*.so`` in-tree, the first with nvcc for sm_100a.

``python -m reciprocal_nearest_neighbour_b200.build`` (or ``build()``) compiles
``csrc/*.cu`` into ``reciprocal_nearest_neighbour_b200/librnn.so`` next to this
file.  The CUDA runtime is linked statically and the driver's tensor-map
encoder is looked up at run time, so the library loads on a machine without
a GPU (its entry points then fail with RNN_ECUDA).  ``csrc/fast.cpp`` becomes
the extension module ``_fast`` (g++, against torch's headers): the short way from
tensors to some of the library's calls.  Its file is named by the Python and the
torch that it was built for (``fast_path()``), and no other is loaded.  The library
needs neither, and is built also where the module cannot be: its calls then take
their Python forms.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "librnn.so")
FAST_SOURCE = os.path.join(CSRC, "fast.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "rnn.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def _older(path: str, deps) -> bool:
    return not os.path.exists(path) or \
        any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def fast_path() -> str:
    """The extension module's file for this Python and this torch."""
    import torch

    kind = re.sub(r"[^0-9A-Za-z.-]", "_", f"{sysconfig.get_config_var('SOABI')}.torch{torch.__version__}")
    return os.path.join(PKG, f"_fast.{kind}.so")


def _fast_stale() -> bool:
    return _older(fast_path(), [FAST_SOURCE, os.path.join(INCLUDE, "rnn.h")])


def build_fast(force: bool = False) -> str:
    """The extension module of csrc/fast.cpp."""
    fast = fast_path()
    if not force and not _fast_stale():
        return fast
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    nvcc = shutil.which(os.environ.get("NVCC", "nvcc")) or "/usr/local/cuda/bin/nvcc"
    cuda = os.path.join(os.environ.get("CUDA_HOME") or os.path.dirname(os.path.dirname(nvcc)), "include")
    system = [os.path.join(torch_dir, "include"),
              os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], cuda, "/usr/local/cuda/include"]
    tmp = fast + f".tmp{os.getpid()}"
    subprocess.check_call(
        [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE,
         *(f"-isystem{p}" for p in system), FAST_SOURCE, "-L", os.path.join(torch_dir, "lib"),
         "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", tmp])
    os.replace(tmp, fast)
    return fast


def build_library(force: bool = False, verbose: bool = False) -> str:
    """The CUDA library."""
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, *sources(), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and the extension module where it can be built."""
    build_library(force, verbose)
    try:
        build_fast(force)
    except (OSError, subprocess.CalledProcessError) as e:
        if _fast_stale() and os.path.exists(fast_path()):
            os.remove(fast_path())      # of other sources: it may not fit the library
        print(f"{LIB}: without the extension module ({e})", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
