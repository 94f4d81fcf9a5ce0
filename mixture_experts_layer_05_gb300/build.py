"""Build libgbmoe.so (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc, and ``_block``,
the compiled argument marshalling of the decoder-block entry points (torch tensors to C ABI).

Each translation unit compiles in parallel to ``_build/*.o`` at the repository root;
the objects link into ``mixture_experts_layer_05_gb300/libgbmoe.so`` next to this file.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgbmoe.so")
EXT = os.path.join(PKG, "_block.so")
EXT_SOURCE = os.path.join(CSRC, "block_py.cpp")
SOURCES = ["api.cu", "topk.cu", "align.cu", "gemm.cu", "gemm_tn.cu", "gemm_fp8.cu", "fp8.cu", "gemm_fp4.cu", "fp4.cu",
           "combine.cu",
           "align_static.cu", "block_api.cu", "norm.cu", "kvappend.cu", "attn.cu",
           "attn_decode.cu", "attn_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libgbmoe.so")
    return path


def flags(verbose_ptxas: bool = False) -> list:
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                "-I", os.path.join(ROOT, "include")]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _compile(src: str, verbose_ptxas: bool, defines=(), build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
    cmd = ([nvcc()] + flags(verbose_ptxas) + [f"-D{d}" for d in defines]
           + ["-c", os.path.join(CSRC, src), "-o", obj])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _build_ext() -> None:
    """_block.so from block_py.cpp with the host compiler and torch's headers and libraries."""
    newest = max(os.path.getmtime(p) for p in (EXT_SOURCE, os.path.join(ROOT, "include", "gbmoe.h")))
    if os.path.exists(EXT) and os.path.getmtime(EXT) > newest:
        return
    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(at, "include"), os.path.join(os.path.dirname(nvcc()), "..", "include"),
               sysconfig.get_paths()["include"]]
    tmp = f"{EXT}.{os.getpid()}.tmp"
    cmd = ([os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC",
            "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
           + [f"-I{p}" for p in include]
           + [EXT_SOURCE, "-o", tmp, f"-L{os.path.join(at, 'lib')}", "-ltorch_python",
              "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"])
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on block_py.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def build(force: bool = False, verbose_ptxas: bool = False, defines=(), lib: str = LIB,
          build_dir: str = BUILD) -> str:
    """Compile every CUDA source and link libgbmoe.so; returns the library path.

    ``defines`` (NAME=VALUE strings) override compile-time tunables of csrc/kernels.h;
    with ``lib`` / ``build_dir`` such a variant builds next to the default library.
    """
    with ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(_build_ext)
        _build_lib(force, verbose_ptxas, defines, lib, build_dir)
        ext.result()
    return lib


def _build_lib(force, verbose_ptxas, defines, lib, build_dir) -> None:
    os.makedirs(build_dir, exist_ok=True)
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    hdrs = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    hdrs.append(os.path.join(ROOT, "include", "gbmoe.h"))
    if (not force and os.path.exists(lib)
            and os.path.getmtime(lib) > max(os.path.getmtime(p) for p in srcs + hdrs)):
        return
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas, defines, build_dir), SOURCES))
    tmp = lib + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
