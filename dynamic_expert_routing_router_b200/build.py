"""Build libbeam_moe.so in-tree from csrc/*.cu for sm_100a (B200), and the compiled
half of the Python binding, _marshal-<torch and Python>.so, from csrc/marshal.cpp.

    python -m dynamic_expert_routing_router_b200.build [--force] [--verbose]

nvcc cross-compiles without a GPU.  The CUDA runtime is linked statically, so
the library does not depend on which libcudart the host process loaded.  The
library needs nvcc alone; where torch or g++ is missing it is all that is built.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbeam_moe.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def marshal_path() -> str:
    """Where the binding's compiled half is for this torch and this Python: it
    reads torch's C++ objects inline, so one built against another is never
    loaded, and its name says which it belongs to."""
    import torch
    return os.path.join(PKG, f"_marshal-torch{torch.__version__}-{sys.implementation.cache_tag}.so")


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """g++ against torch's own headers and libraries."""
    src, path = os.path.join(CSRC, "marshal.cpp"), marshal_path()
    if not force and os.path.exists(path) and os.path.getmtime(path) >= os.path.getmtime(src):
        return path
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    includes = [os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           *[f"-I{i}" for i in includes], "-o", path, src, f"-L{os.path.join(root, 'lib')}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    for other in glob.glob(os.path.join(PKG, "_marshal*.so")):
        if other != path:  # of another torch or Python
            os.remove(other)
    return path


def build_library(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not _stale():
        return LIB
    cmd = [nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-shared",
           "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC, *extra,
           "-o", LIB, *sources()]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return LIB


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The library, then the binding's compiled half where it can be built."""
    build_library(force, verbose, extra)
    for what, there in (("torch", importlib.util.find_spec("torch")), ("g++", shutil.which("g++"))):
        if not there:
            print(f"{what} not found: the Python binding's compiled half is not built",
                  file=sys.stderr)
            return LIB
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ())
    print(LIB)
