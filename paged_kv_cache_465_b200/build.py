"""Builds libpagedattn.so in-tree with nvcc for sm_100a (no JIT cache; torch is not needed).

    python paged_kv_cache_465_b200/build.py [-v]

The CUDA sources are compiled as one translation unit (library.cu includes pagedattn.cu and
the kernel headers), the host allocator separately; the CUDA runtime is linked statically so the
library has no dependency on the process's libcudart.

Where torch and its headers are installed, the helper of the drafted step's binding (checks of
tensors, csrc/tensors.cpp) is compiled against them as well. Its file name says which torch and
which Python it fits, so that another one never loads it. Only the calls of a drafted step need it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libpagedattn.so")
HELPER_SOURCE = os.path.join(CSRC, "tensors.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def helper_path(torch) -> str:
    """The binding's helper for this torch and this Python."""
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(HERE, f"_tensors-torch{torch.__version__}-abi{abi}"
                              + sysconfig.get_config_var("EXT_SUFFIX"))


def _helper_command(torch, out):
    root = os.path.dirname(torch.__file__)
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *(x for i in inc for x in ("-I", i)),
            HELPER_SOURCE, "-L", os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-o", out]


def _sources():
    return sorted(p for p in (os.path.join(CSRC, f) for f in os.listdir(CSRC)) if p != HELPER_SOURCE)


def _stale(built, deps) -> bool:
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    return any(os.path.getmtime(p) > t for p in deps)


def _run(cmds, verbose) -> None:
    for c in cmds:
        r = subprocess.run(c, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("build failed: " + " ".join(c))


def build_helper(force: bool = False, verbose: bool = False) -> str | None:
    """The helper's path, or None where torch or its headers are not installed."""
    try:
        import torch
    except ImportError:
        return None
    if not os.path.exists(os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "Dtype.h")):
        return None
    path = helper_path(torch)
    if force or _stale(path, [HELPER_SOURCE, __file__]):
        _run([_helper_command(torch, path + ".tmp")], verbose)
        os.replace(path + ".tmp", path)
    return path


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    if force or _stale(LIB, _sources() + [os.path.join(INCLUDE, "pagedattn.h"), __file__]):
        nvcc = _nvcc()
        os.makedirs(BUILD, exist_ok=True)
        common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC, "-Xcompiler", "-fPIC"]
        cu_obj = os.path.join(BUILD, "pagedattn.o")
        cpp_obj = os.path.join(BUILD, "allocator.o")
        _run([
            [nvcc, *ARCH, "-lineinfo", *common, "-Xptxas", "-v" if verbose else "-O3",
             "-c", os.path.join(CSRC, "library.cu"), "-o", cu_obj] + list(extra or []),
            [nvcc, *common, "-Wno-deprecated-gpu-targets", "-x", "c++", "-c", os.path.join(CSRC, "allocator.cpp"), "-o", cpp_obj],
            [nvcc, *ARCH, "-shared", "-cudart", "static", cu_obj, cpp_obj, "-o", LIB + ".tmp"],
        ], verbose)
        os.replace(LIB + ".tmp", LIB)
    if build_helper(force, verbose) is None:
        sys.stderr.write("torch or its headers are not installed: the drafted step's calls will have "
                         "no binding until this is run with them\n")
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    print(LIB)
