"""Build libskinny.so in-tree with nvcc for sm_100a, and the Python binding of
the calls for any number of tokens (_binding.so) with g++.

    python -m fp8_weight_only_w4a16_b200.build [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("skinny.cu", "stream_read.cu", "tile_gemm.cu", "quantize.cu", "verify.cu",
                                           "pack.cpp")]
HEADERS = [os.path.join(CSRC, "layout.h"), os.path.join(CSRC, "ptx.cuh"), os.path.join(CSRC, "tcgen05.cuh"),
           os.path.join(ROOT, "include", "skinny.h")]
LIBRARY = os.path.join(PKG, "libskinny.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def needs_build() -> bool:
    if not os.path.exists(LIBRARY):
        return True
    t = os.path.getmtime(LIBRARY)
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIBRARY
    tmp = LIBRARY + ".tmp%d" % os.getpid()
    cmd = [nvcc_path(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC,-O3", "-shared",
           "-I", os.path.join(ROOT, "include"), *SOURCES, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(tmp, LIBRARY)
    return LIBRARY


def build_binding(force: bool = False) -> str:
    """Compile _binding.so against the installed torch (its headers and libraries)."""
    import sysconfig

    import torch

    newest = max(os.path.getmtime(f) for f in (BINDING_SOURCE, os.path.join(ROOT, "include", "skinny.h")))
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest:
        return BINDING
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    for d in (os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-I", d]
    cmd += [BINDING_SOURCE, "-o", tmp, "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    build_binding(force=True)
    print(LIBRARY)
