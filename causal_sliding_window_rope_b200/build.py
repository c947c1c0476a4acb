"""Builds libcswattn.so in-tree with nvcc for sm_100a.

    python -m causal_sliding_window_rope_b200.build

The CUDA runtime is linked statically and the driver is reached through the
runtime's entry-point query, so the library also loads (without computing) on
a machine that has no GPU driver.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcswattn.so")
LIB_CHECK = os.path.join(PKG, "libcswattn_check.so")  # CSWATTN_CHECK=1: device-side bounds checks
LIB_BINDING = os.path.join(PKG, "_paged_binding.so")  # Python module: checks and makes the paged cache's calls
SOURCES = ["cswattn.cu"]
BINDING_SOURCE = os.path.join(CSRC, "paged_binding.cpp")
HEADER = os.path.join(ROOT, "include", "cswattn.h")


def deps() -> list[str]:
    """Every file the library is compiled from: the translation unit, every
    kernel header next to it and the public header."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [HEADER, os.path.abspath(__file__)])


NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def stale(lib: str | None = None) -> bool:
    lib = lib or LIB
    if not os.path.exists(lib):
        return True
    if lib == LIB_BINDING and binding_id().encode() not in open(lib, "rb").read():
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in (binding_deps() if lib == LIB_BINDING else deps()))


def binding_deps() -> list[str]:
    return [BINDING_SOURCE, HEADER, os.path.abspath(__file__)]


def torch_dir() -> str | None:
    """Where PyTorch is installed, without importing it."""
    try:
        spec = importlib.util.find_spec("torch")
    except ValueError:
        return None
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def torch_version() -> str | None:
    base = torch_dir()
    if base is None:
        return None
    with open(os.path.join(base, "version.py")) as f:
        found = re.search(r"""__version__ = ['"]([^'"]+)""", f.read())
    return found.group(1) if found else None


def binding_id(version: str | None = None) -> str:
    """The PyTorch and the Python that the module is compiled for, which it
    holds as a text."""
    return f"_paged_binding for PyTorch {version or torch_version()} and Python {sys.version_info[0]}.{sys.version_info[1]}"


def binding_lacks() -> str | None:
    """What this machine lacks to compile the Python module, or None."""
    base = torch_dir()
    if base is None:
        return "PyTorch"
    if not os.path.exists(os.path.join(base, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return "PyTorch's headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None


def build_binding(force: bool = False) -> str:
    """Compile the Python module _paged_binding (host code only, against the
    installed Python's and PyTorch's headers)."""
    if not force and not stale(LIB_BINDING):
        return LIB_BINDING
    if binding_lacks():
        raise RuntimeError(f"_paged_binding cannot be built without {binding_lacks()}")
    import torch
    base = torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    tmp = LIB_BINDING + f".tmp{os.getpid()}"
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        f'-DBUILT_FOR="{binding_id()}"',
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
        "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
        "-isystem", os.path.join(cuda, "include"), BINDING_SOURCE, "-o", tmp,
        "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, LIB_BINDING)
    return LIB_BINDING


def build_library(force: bool = False, verbose: bool = False, check: bool = False) -> str:
    """Compile libcswattn.so (or, with check, libcswattn_check.so): nvcc alone."""
    lib = LIB_CHECK if check else LIB
    if not force and not stale(lib):
        return lib
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"),
           *(["-DCSWATTN_CHECK=1"] if check else []),
           *(os.path.join(CSRC, s) for s in SOURCES), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.check_call(cmd)
    os.replace(tmp, lib)
    return lib


def build(force: bool = False, verbose: bool = False, check: bool = False) -> str:
    """Compile libcswattn.so (or, with check, libcswattn_check.so: the same
    library with CSWATTN_CHECK=1 device-side bounds checks), and the Python
    module that makes the paged cache's calls where it can be compiled: the
    library is a C library, which needs neither Python nor PyTorch."""
    lib = build_library(force, verbose, check)
    if binding_lacks():
        print(f"_paged_binding is not built, and the paged calls from Python are missing: no {binding_lacks()} here",
              file=sys.stderr)
    else:
        build_binding(force)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv, check="--check" in sys.argv))
