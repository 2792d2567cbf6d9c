"""Builds libmuse_moe.so in-tree with nvcc for sm_100a (no JIT, no torch extension).

    python -m latent_mixture_experts_moe_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "muse_moe.cu")
LIB = os.path.join(PKG, "libmuse_moe.so")
KERNEL_SOURCES = ("muse_moe.cu", "few_tokens.cuh", "gemm_umma.cuh", "gemm_umma_2sm.cuh", "gemm_umma_fp4.cuh", "gemm_umma_w4a4.cuh",
                  "gemv_fp4.cuh", "int8_rows.cuh", "int8_splitk.cuh", "nvfp4_act.cuh", "route_kernels.cuh", "ptx.cuh")
DEPS = [os.path.join(PKG, "csrc", f) for f in KERNEL_SOURCES] + [os.path.join(ROOT, "include", "muse_moe.h")]

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and not verbose_ptxas and up_to_date():
        return LIB
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), SRC, "-o", LIB + ".tmp"]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libmuse_moe.so")
    if verbose_ptxas:
        sys.stdout.write(res.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv)
    print(LIB)
