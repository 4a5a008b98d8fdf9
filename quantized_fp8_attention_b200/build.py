"""Builds libfqa.so in-tree with nvcc for sm_100a (B200), and the native part of
the Python binding, _binding.so, with the host compiler.

Usage: python -m quantized_fp8_attention_b200.build [--force] [--verbose]
"""

from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

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


def binding_built_for() -> bytes:
    """What the binding's machine code depends on besides its sources."""
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}".encode()


def _trailer(body: bytes) -> bytes:
    return b"\n%s %s" % (binding_built_for(), hashlib.sha256(body).hexdigest().encode())


def binding_fits() -> bool:
    """Whether _binding.so is there, whole, and built for this torch and Python: the
    line that build_binding() puts after the linker's output says so."""
    try:
        with open(BINDING, "rb") as f:
            data = f.read()
    except OSError:
        return False
    at = data.rfind(b"\n")
    return at >= 0 and data[at:] == _trailer(data[:at])


def build_binding(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale(BINDING, binding_sources()) and binding_fits():
        return BINDING
    from torch.utils import cpp_extension
    tmp = BINDING + f".tmp{os.getpid()}"
    libs = cpp_extension.library_paths()[0]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           *[f"-I{d}" for d in cpp_extension.include_paths()], f"-I{os.path.dirname(os.path.dirname(nvcc()))}/include",
           f"-I{sysconfig.get_paths()['include']}", os.path.join(CSRC, "binding.cpp"), f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl", "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        subprocess.run(cmd, check=True)
        with open(tmp, "rb") as f:
            trailer = _trailer(f.read())
        with open(tmp, "ab") as f:
            f.write(trailer)
        os.replace(tmp, BINDING)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, which every call needs, then the binding, without which calls
    are only slower: where it cannot be compiled the library is built all the
    same."""
    lib = build_lib(force, verbose)
    try:
        build_binding(force, verbose)
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the native part of the binding was not built: {e}", RuntimeWarning, stacklevel=2)
    return lib


def build_lib(force: bool = False, verbose: bool = False) -> str:
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
