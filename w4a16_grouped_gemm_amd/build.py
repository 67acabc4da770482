"""Build the gfx950 HIP library libmoe_w4a16.so in-tree with hipcc.

Flags: gfx950 only; -O3; no FP contraction (the combine must be exactly the
IEEE multiply / FMA it names); fp32 denormals preserved (no flush-to-zero);
packed-fp32 instructions disabled; MFMA accumulators in ordinary VGPRs
(the epilogue reads them with plain VALU instructions, no AGPR copies), but
for the W8A8 products, whose largest tile holds 256 of them per lane.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "libmoe_w4a16.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "route.hip", "permute.hip", "gemm_w4a16.hip", "decode.hip", "gemm_mxfp4.hip", "finalize.hip", "pack.hip",
           "route_scored.hip", "norm_int8.hip", "gemm_w8a8.hip", "api_w8a8.hip", "norm_fp8.hip", "gemm_fp8.hip",
           "api_fp8.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
         "-fno-gpu-flush-denormals-to-zero", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I" + INCLUDE, "-I" + CSRC]
# Accumulators in ordinary VGPRs, except where a wave holds more of them than there are (256)
VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
AGPR_SOURCES = {"gemm_w8a8.hip"}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    flags = FLAGS if src in AGPR_SOURCES else FLAGS + VGPR_FORM
    cmd = [HIPCC, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
