"""Build the HIP library in-tree: hipcc for gfx950, one object per source,
linked into ``dense_gemm_tuning_amd/lib/libdgt_gemm.so``.

Usage: ``python -m dense_gemm_tuning_amd.build`` (or ``build()``).  Objects go
to ``dense_gemm_tuning_amd/_build/``; nothing is cached outside the tree.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJDIR = os.path.join(HERE, "_build")
LIBDIR = os.path.join(HERE, "lib")
LIBPATH = os.path.join(LIBDIR, "libdgt_gemm.so")

SOURCES = ["gemm_api.cpp", "k_naive.hip", "k_lds.hip", "k_mfma_f32.hip", "k_mfma_f32_dma.hip",
           "k_mfma_bf16.hip", "k_mfma_bf16_dma.hip", "k_skinny16.hip", "k_skinny_dma.hip",
           "k_skinny_f32.hip",
           "k_splitk.hip", "mx4_api.cpp", "k_mx4_quant.hip", "k_mx4_tile.hip", "k_mx4_skinny.hip",
           "k_mx4_rows.hip", "orth_api.cpp",
           "k_orth.hip", "k_orth_small.hip", "gated_api.cpp", "k_gated_regs.hip", "k_gated_tile.hip", "k_gated_strip.hip",
           "k_w4_quant.hip", "k_w4_strip.hip", "k_w4_rows.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
# Packed fp32 VALU instructions are switched off for every device pass.
CFLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-Wno-unused-function"]


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *CFLAGS, *lang, "-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(jobs: int = 8) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(jobs, len(SOURCES)))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIBPATH + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBPATH)
    return LIBPATH


if __name__ == "__main__":
    print(build())
    sys.exit(0)
