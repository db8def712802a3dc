"""Build libwst.so (the C-ABI CUDA library) in-tree for sm_103a.

Each CUDA translation unit is compiled by nvcc in parallel into
``_build/*.o`` and linked into ``warp_specialized_tensor_gb300/libwst.so``.
The CUDA runtime is linked statically and the driver entry point for tensor
maps is fetched at run time, so the library loads on a machine without a GPU
driver (the C ABI then reports WST_ERR_CUDA on use).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import time
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwst.so")

SOURCES = ["gemm_dense.cu", "grouped_ws.cu", "ikbo_ws.cu", "ikbo_attn.cu", "wst_api.cu", "expert_parallel.cu",
           "moe_route.cu", "moe_plan.cu", "moe_combine.cu", "fp8_quant.cu", "fp8_gemm.cu", "wgrad_ws.cu",
           "cache_append.cu", "tree_attn.cu", "w4_gemm.cu"]
HEADERS = ["sm103.cuh", "wst_common.cuh", "gemm_ws.cuh", "grouped_ws.cuh", "ikbo_ws.cuh", "ikbo_attn_ws.cuh",
           "fp8_gemm.cuh", "wgrad_ws.cuh", "work_split.cuh", "tree_attn.cuh", "w4_gemm.cuh", "wst_host.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "wst.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs() if os.path.exists(f))


def _flags(verbose_ptxas: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    """Compile (if stale) and return the path of libwst.so."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    t0 = time.time()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + _flags(verbose_ptxas) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for src, obj, r in results:
        if r.returncode != 0 or (verbose_ptxas and r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s" % src)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + [o for _, o, _ in results] + \
        ["-cudart", "static", "-Xlinker", "--no-undefined", "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libwst.so failed")
    os.replace(tmp, LIB)
    if not quiet:
        print("built %s in %.1fs" % (LIB, time.time() - t0))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, quiet=False)
