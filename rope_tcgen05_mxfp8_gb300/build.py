"""Build libqkvcte.so in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into one shared library
with the CUDA runtime linked statically (the library needs libcuda.so only when it
first talks to a GPU). Output: rope_tcgen05_mxfp8_gb300/_lib/libqkvcte.so.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libqkvcte.so")

SOURCES = ["qkv_cte_api.cu", "qkv_gemm_mxf8.cu", "qkv_gemm_mxf8_head.cu", "qkv_gemm_mxf8_stats.cu", "qkv_gemm_mxf8_fused.cu", "qk_norm_rope.cu", "row_quant.cu", "rope_permute.cu",
           "layer_norm.cu", "rope_axes.cu", "linear_api.cu", "qkv_gemm_mxf8_linear.cu",
           "qkv_gemm_mxf8_linear_f32.cu", "linear_few.cu", "block_ops_api.cu", "kv_cache_copy.cu", "cache_attention_few.cu", "cache_attention.cu", "kv_cache_api.cu"]
HEADERS = ["ptx.cuh", "internal.h", "qkv_gemm_mxf8.cuh", "qk_norm_rope.cuh", "fp32x2.cuh", "kernel_kinds.cuh", "api_common.h",
           "block_ops.h", "vec_io.cuh", "linear_epilogue.cuh", "heads_tensor.h", "kv_cache.h", "kv_cache.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", "-Xcompiler", "-Wformat", "-Xcompiler", "-Werror=format",
                     "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    paths = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    paths.append(os.path.join(INCLUDE, "qkv_cte.h"))
    paths.append(os.path.abspath(__file__))
    return paths


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + ["-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if v else None
    print(build(force=True, verbose=v, extra_flags=extra))
