"""Build libhstu.so in-tree with nvcc for sm_100a, and _serving.so, the Python
binding of the serving calls, with g++.

    python -m jagged_pointwise_attention_b200.build [--force] [--verbose]

The library is one translation unit (csrc/hstu_api.cu includes every kernel)
linked against the static CUDA runtime; it resolves the driver's tensor-map
encoder at run time, so loading it needs no GPU.
"""

from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libhstu.so")
BINDING = os.path.join(PKG, "_serving.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build(out: str = LIB) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in _sources())


def binding_tag() -> str:
    """What _serving.so fits, written into it: torch and its C++ ABI, CPython."""
    import torch

    return "built for torch %s, C++11 ABI %d, CPython %d.%d" % (
        torch.__version__, int(torch._C._GLIBCXX_USE_CXX11_ABI), *sys.version_info[:2])


def binding_needs_build(out: str = BINDING) -> bool:
    if not os.path.exists(out):
        return True
    newest = max(os.path.getmtime(BINDING_SRC), os.path.getmtime(os.path.join(INCLUDE, "hstu.h")))
    if os.path.getmtime(out) < newest:
        return True
    with open(out, "rb") as f:
        return binding_tag().encode() + b"\0" not in f.read()


def build_binding(force: bool = False) -> str:
    """_serving.so against the installed torch (its headers, its C++ ABI)."""
    if not force and not binding_needs_build(BINDING):
        return BINDING
    import torch

    tdir = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
        "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
        '-DHSTU_BINDING_TAG="%s"' % binding_tag(),
        "-I", INCLUDE, "-isystem", os.path.join(tdir, "include"),
        "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
        "-o", tmp, BINDING_SRC, "-L", os.path.join(tdir, "lib"),
        "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"])
    os.replace(tmp, BINDING)
    return BINDING


def build_library(force: bool, verbose: bool, out: str, extra) -> str:
    if not force and not needs_build(out):
        return out
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = out + ".tmp.%d" % os.getpid()
    cmd = [nvcc] + NVCC_FLAGS + list(extra) + (["-Xptxas", "-v"] if verbose else []) + [
        "-I", INCLUDE, "-I", CSRC, "-o", tmp, os.path.join(CSRC, "hstu_api.cu")]
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, out: str = LIB, extra=()) -> str:
    """The library, which needs no torch, then the binding."""
    build_library(force, verbose, out, extra)
    if out == LIB:
        build_binding(force)
    return out


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
