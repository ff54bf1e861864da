"""Builds libw4.so in-tree with nvcc for sm_100a (no GPU needed to compile),
and the _tensors extension (the tensor front end of the per-layer operators)
with the C++ compiler against torch's headers.  Without torch the library is
built alone: the C ABI needs nothing else.

    python -m weight_only_int4_quantize_b200.build [--verbose]

Each .cu file compiles separately (objects under _build/), then one shared
library links them with the static CUDA runtime.  Rebuilds only what changed.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libw4.so")
TENSORS = os.path.join(PKG, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))

SOURCES = ["abi.cu", "quantize.cu", "gemv.cu", "gemv_stream.cu", "act_int8.cu", "gemm_tc.cu", "awq.cu", "block.cu", "noalloc.cu",
           "fp4_quant.cu", "fp4_gemm.cu", "kv8_append.cu", "kv8_attn.cu", "kv8_attn_tc.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC)")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "tensors.cpp"]
    files.append(os.path.join(INCLUDE, "w4.h"))
    return max(os.path.getmtime(f) for f in files)


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    hdr_time = _deps_mtime()
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if os.path.exists(o) and os.path.getmtime(o) >= hdr_time and not extra_flags:
            continue
        cmd = [nvcc, *ARCH, *FLAGS, *(extra_flags or []), "-c", s, "-o", o]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    if (not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs)):
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", *objs, "-o", LIB]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    try:
        import torch  # noqa: F401
    except ImportError:
        print("torch cannot be imported: the _tensors extension is not built", file=sys.stderr)
    else:
        build_tensors(verbose)
    return LIB


def build_tensors(verbose: bool = False) -> str:
    """Compiles csrc/tensors.cpp into the package's _tensors module."""
    import torch
    from torch.utils import cpp_extension
    src = os.path.join(CSRC, "tensors.cpp")
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(INCLUDE, "w4.h"), torch.__file__))
    if os.path.exists(TENSORS) and os.path.getmtime(TENSORS) >= newest:
        return TENSORS
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           f"-isystem{sysconfig.get_paths()['include']}", f"-isystem{cuda}/include",
           *[f"-isystem{p}" for p in cpp_extension.include_paths()], src,
           *[f"-L{p}" for p in cpp_extension.library_paths()], "-ltorch_python", "-ltorch_cuda",
           "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-o", TENSORS]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return TENSORS


if __name__ == "__main__":
    v = "--verbose" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None
    print(build(verbose=v, extra_flags=extra))
