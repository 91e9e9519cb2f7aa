"""Build libdsaidx.so in-tree with nvcc for sm_103a (no CMake, no torch).

Each translation unit compiles in parallel, then one link step. The library
statically links the CUDA runtime and reaches the driver's tensor-map encoder
through cudaGetDriverEntryPointByVersion, so it needs no -lcuda.
"""
from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build", platform.machine())
STAMP = os.path.join(BUILD, "lib.stamp")
LIB = os.path.join(HERE, "libdsaidx.so")
SOURCES = ["api.cu", "store.cu", "topk.cu", "topk_fp8.cu", "topk_fp4.cu", "topk_static.cu",
           "api_attn.cu", "rope.cu", "kv.cu", "attn.cu", "attn_fp8.cu", "attn_fp4.cu",
           "attn_span.cu", "span_bf16.cu", "span_fp8.cu", "span_fp4.cu", "span_cap_bf16.cu", "span_cap_fp8.cu",
           "span_cap_fp4.cu", "span_bias_bf16.cu", "span_bias_fp8.cu", "span_bias_fp4.cu", "span_wide_bf16.cu",
           "span_wide_fp8.cu", "span_wide_fp4.cu", "batch.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    p = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(p):
        return p
    raise RuntimeError("nvcc not found")


def _newer(src_paths, out) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in src_paths)


def build(verbose: bool = False, force: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(HERE, "..", "include", "dsaidx.h"))
    cc = nvcc()

    def one(src):
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        if force or _newer([s] + headers, o):
            cmd = [cc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr, flush=True)
        return o

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(one, SOURCES))
    if force or _newer(objs, LIB) or not os.path.exists(STAMP) or _newer([LIB], STAMP):
        cmd = [cc, *ARCH, "-shared", "-o", LIB, *objs, "-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        with open(STAMP, "w") as f:
            f.write(platform.machine())
    return LIB


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv)
