"""Builds libmoeroute.so (the C ABI and its CUDA kernels) for sm_103a with nvcc.

Each translation unit is compiled in parallel, then linked into one shared
library next to this file (`_build/libmoeroute.so`).  No torch extension
machinery is involved: the library exports plain C symbols.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmoeroute.so")
SOURCES = ["api.cu", "topk_signature.cu", "topk_signature_tpr.cu", "block_counts.cu", "stitch.cu",
           "affinity_load.cu", "route.cu", "noalloc.cu", "gate_topk.cu", "kmeans.cu",
           "replicate.cu", "mask_select.cu", "spectral.cu", "selftest.cu",
           "score_topk.cu", "score_fast_f32.cu", "score_fast_bf16.cu", "score_fast_f16.cu",
           "score_fast16_f32.cu", "score_fast16_bf16.cu", "score_fast16_f16.cu",
           "score_grad.cu", "score_grad_f32.cu", "score_grad_bf16.cu", "score_grad_f16.cu", "block_plan.cu", "expert_order.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(os.path.dirname(HERE), "include")]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    cmd = [nvcc(), *ARCH, "-shared", "-o", LIB, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
