"""Builds libfqa.so in-tree with nvcc for sm_100a (B200), and the native part of
the Python binding, _binding.so, with the host compiler.

Usage: python -m quantized_fp8_attention_b200.build [--force] [--verbose]
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfqa.so")
BINDING = os.path.join(PKG, "_binding.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-shared", "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfqa.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "fqa.h")])


def binding_sources():
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "fqa.h")]


def stale(lib: str = LIB, srcs=None) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in (sources() if srcs is None else srcs))


def build_binding(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale(BINDING, binding_sources()):
        return BINDING
    import sysconfig

    from torch.utils import cpp_extension
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = cpp_extension.library_paths()[0]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           *[f"-I{d}" for d in cpp_extension.include_paths()], f"-I{os.path.dirname(os.path.dirname(nvcc()))}/include",
           f"-I{sysconfig.get_paths()['include']}", os.path.join(CSRC, "binding.cpp"), f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl", "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    build_binding(force, verbose)
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"),
           os.path.join(CSRC, "fqa.cu"), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
