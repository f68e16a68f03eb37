"""Build libgdn.so in place with nvcc for sm_100a (B200), and _layer.so, the quick
binding of its decode-layer operators, with the host compiler.

Usage: python -m chunked_gated_delta_14_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgdn.so")
BINDING = os.path.join(HERE, "_layer.so")
BINDING_SOURCE = os.path.join(CSRC, "layer_binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def binding_for() -> str:
    """What _layer.so is built for: torch's C++ tensors change from one release to the next."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}, C++ ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def binding_is_current() -> bool:
    """Whether _layer.so is there and was built for this torch and this Python (it says so itself
    too, as ``built_for``, but only to who has loaded it)."""
    try:
        with open(BINDING + ".for") as f:
            return os.path.exists(BINDING) and f.read() == binding_for()
    except OSError:
        return False


def build_binding(force: bool = False) -> str:
    """_layer.so: a Python extension over torch's C++ tensors (no kernels, not linked to libgdn.so)."""
    deps = [BINDING_SOURCE, os.path.join(INCLUDE, "gdn.h")]
    if not force and binding_is_current() and os.path.getmtime(BINDING) > max(map(os.path.getmtime, deps)):
        return BINDING
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = BINDING + f".tmp{os.getpid()}"
    flags = [f"-I{p}" for p in [INCLUDE, *cpp_extension.include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]]
    subprocess.check_call([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DGDN_BUILT_FOR="{binding_for()}"', *flags, BINDING_SOURCE,
                           "-o", tmp, *[f"-L{p}" for p in cpp_extension.library_paths()], "-lc10", "-lc10_cuda", "-ltorch_cpu",
                           "-ltorch", "-ltorch_python"])
    if os.path.exists(BINDING + ".for"):
        os.remove(BINDING + ".for")      # never the new mark beside the old binding
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(binding_for())
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """libgdn.so, and _layer.so where a host compiler and torch's and Python's headers are there:
    without it every call works, with three times the host's time for the small ones."""
    lib = build_library(force, verbose)
    try:
        build_binding(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        print(f"{BINDING} not built ({e}): decode-layer calls go through layer.py alone", file=sys.stderr)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC,
           "--expt-relaxed-constexpr", *sources(), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
