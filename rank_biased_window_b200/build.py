"""Builds the in-tree CUDA library ``librfb_attn.so`` for sm_100a with nvcc, and
the serving calls' Python extension ``_serving_bind.so`` with the host compiler.

    python -m rank_biased_window_b200.build [--verbose-ptxas] [--force]

The library is a plain C-ABI shared object (see include/rfb_attn.h); the
Python binding loads it with ctypes.  The CUDA runtime is linked statically and
the driver's tensor-map encoder is fetched at run time, so the .so depends on
nothing but the NVIDIA driver, and nvcc is all that building it takes.  The
extension holds host code only and belongs to the Python and torch that it was
built with (which its stamp file names); it needs their headers.  Where it
cannot be built the library is there all the same, and the serving calls say
that they are not.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "librfb_attn.so")
BIND = os.path.join(PKG, "_serving_bind.so")
BIND_STAMP = os.path.join(PKG, "_serving_bind.stamp")
BIND_SOURCE = os.path.join(CSRC, "serve", "bind.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "**", "*.cu"), recursive=True)
                  + glob.glob(os.path.join(CSRC, "**", "*.cuh"), recursive=True)
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(target, inputs) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in inputs)


def up_to_date() -> bool:
    return _newer(LIB, sources())


def _bind_of_these_sources() -> bool:
    return _newer(BIND, [BIND_SOURCE, os.path.abspath(__file__), *glob.glob(os.path.join(INCLUDE, "*.h"))])


def _bind_stamp() -> str:
    import torch
    return f"torch {torch.__version__} {sys.implementation.cache_tag}"


def bind_up_to_date() -> bool:
    """Built from these sources, for this Python and torch."""
    if not (_bind_of_these_sources() and os.path.exists(BIND_STAMP)):
        return False
    with open(BIND_STAMP) as f:
        return f.read() == _bind_stamp()


def build_bind(force: bool = False) -> str:
    if not force and bind_up_to_date():
        return BIND
    import torch
    where = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = BIND + f".tmp{os.getpid()}"
    cxx = os.environ.get("CXX", "g++")
    # torch's C++ runtime, by name: a compiler that finds no libstdc++.so links its archive
    # instead, without a word, and a second runtime in the process crashes where its streams
    # meet the first one's locales (a number put into one) and in exceptions across the two.
    runtime = subprocess.run([cxx, "-print-file-name=libstdc++.so.6"], capture_output=True,
                             text=True).stdout.strip()
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", f'-DRFB_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(where, "include"),
           "-isystem", os.path.join(where, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-L", os.path.join(where, "lib"),
           "-o", tmp, BIND_SOURCE, *([runtime] if os.path.isabs(runtime) else []),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("building _serving_bind.so failed")
    os.replace(tmp, BIND)
    with open(tmp, "w") as f:
        f.write(_bind_stamp())
    os.replace(tmp, BIND_STAMP)
    return BIND


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    """The library, and the extension where it can be built."""
    build_library(force, ptxas_verbose, quiet)
    try:
        build_bind(force)
    except (RuntimeError, ImportError, OSError) as e:
        if os.path.exists(BIND) and not _bind_of_these_sources():
            os.remove(BIND)  # it would call this library by another's signatures
        sys.stderr.write(f"{LIB} is built; the serving calls' extension is not: {e}\n")
    return LIB


def build_library(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-O3", "-std=c++17", "-lineinfo", "-shared",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC,
           "-o", tmp, os.path.join(CSRC, "serve", "rfb_library.cu")]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building librfb_attn.so")
    if not quiet or ptxas_verbose:
        sys.stdout.write(res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas, quiet=False))
