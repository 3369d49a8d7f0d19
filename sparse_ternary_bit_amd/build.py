"""Build libstq.so (all HIP kernels + the C ABI) for gfx950 with hipcc.

Usage: python -m sparse_ternary_bit_amd.build   (or build() from Python).
The library is written next to this file so it ships with the source tree.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libstq.so")

SOURCES = ["stq_api.hip", "k_codec.hip", "k_gemv.hip", "k_gemm.hip", "k_moe.hip", "k_sens.hip", "k_gated.hip",
           "k_swiglu.hip", "k_q8.hip", "k_logprobs.hip", "k_norm.hip",
           "k_route.hip", "k_combine.hip", "k_head.hip", "k_probe.hip"]
# per-file extra flags: the encoders must not contract fp64 arithmetic; the
# matrix-core probe keeps its accumulators in VGPRs (in the AGPR form the
# compiler moves them between the two files every round)
EXTRA = {"k_codec.hip": ["-ffp-contract=off"], "k_sens.hip": ["-ffp-contract=off"],
         "k_probe.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}

COMMON = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    # packed fp32 VALU ops are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the STQ1_0 library needs ROCm's hipcc")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src.replace(".hip", ".o"))
    cmd = [_hipcc(), *COMMON, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
