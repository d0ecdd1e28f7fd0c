"""Builds libmx.so (the CUDA kernels + C ABI) in-tree for sm_100a with nvcc, and _mxcall.so, the binding's compiled
call path (csrc/binding.cpp), with g++ against the installed torch.

    python -m mxfp8_block_scaled_07_b200.build [--verbose]

nvcc cross-compiles on hosts without a GPU. The library is written next to this file, so it
travels with the source tree; nothing is installed elsewhere.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmx.so")
SOURCES = [os.path.join(CSRC, f) for f in ("libmx.cu",)]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("ptx.cuh", "quantize.cuh", "quantize_tma.cuh", "swizzle.cuh",
                                                       "grid_equal.cuh", "gemm.cuh", "gemm_few.cuh", "blockwise.cuh", "fastdiv.cuh", "fp4.cuh",
                                                       "route.cuh", "experts.cuh", "rope.cuh", "cache.cuh", "attend.cuh",
                                                       "attend_many.cuh")] + [
    os.path.join(ROOT, "include", "mx.h")
]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    # No fast-math / flush-to-zero: BF16 subnormal inputs must stay subnormal in the quantizer.
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
]


CALL_LIB = os.path.join(HERE, "_mxcall.so")
CALL_SOURCE = os.path.join(CSRC, "binding.cpp")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def needs_build(lib: str = LIB, deps=None) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in (DEPS if deps is None else deps))


def _run(cmd, verbose: bool):
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    if verbose:
        sys.stdout.write(res.stdout + res.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or needs_build():
        tmp = LIB + f".tmp{os.getpid()}"
        _run([nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp, *SOURCES], verbose)
        os.replace(tmp, LIB)
    build_call(force, verbose)
    return LIB


def call_tag() -> str:
    """What _mxcall.so depends on beside its source: the torch whose C++ library it is linked against, and the Python."""
    import torch

    return f"torch {torch.__version__} {torch.version.git_version} {sysconfig.get_config_var('SOABI')}"


def built_for(lib: str = CALL_LIB):
    """The call_tag() that a built _mxcall.so carries (read from the file: one of another torch must not be loaded);
    None if it carries none."""
    with open(lib, "rb") as f:
        found = re.search(rb"mx-call-tag:([^;\0]*);", f.read())
    return found.group(1).decode() if found else None


def call_needs_build() -> bool:
    return needs_build(CALL_LIB, [CALL_SOURCE, os.path.join(ROOT, "include", "mx.h")]) or built_for() != call_tag()


def build_call(force: bool = False, verbose: bool = False) -> str:
    """_mxcall.so, linked against the libmx.so beside it."""
    if not force and not call_needs_build():
        return CALL_LIB
    import torch

    site = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    includes = [os.path.join(site, "include"), os.path.join(site, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = CALL_LIB + f".tmp{os.getpid()}"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f'-DMX_CALL_TAG="{call_tag()}"',
          *(x for p in includes for x in ("-isystem", p)), "-o", tmp, CALL_SOURCE, "-L" + HERE, "-l:libmx.so",
          "-L" + os.path.join(site, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, CALL_LIB)
    return CALL_LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
