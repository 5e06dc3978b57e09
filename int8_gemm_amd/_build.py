"""Build libconvrot.so in-tree with hipcc for gfx950 (no GPU needed)."""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libconvrot.so")
SOURCES = ("api.hip", "rotate.hip", "dequant.hip", "gemm.hip", "check.hip",
           "api_mx4.hip", "mx4.hip", "gemm_mx4.hip", "norm.hip",
           "api_attention.hip", "rope.hip", "attention.hip")

# -ffp-contract=off: the numerics contract spells out every fp32 rounding; a
# fused multiply-add would skip one. The packed-fp32 feature is turned off for
# the device pass (the host pass warns that it does not know it).
HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the convrot library)")


# the GEMMs keep their MFMA accumulators in VGPRs (their waves are sized so
# that they fit); otherwise the allocator shuffles accumulator blocks between
# AGPR ranges every K-step
_VGPR_FORM = ["-mllvm", "--amdgpu-mfma-vgpr-form"]
EXTRA_FLAGS = {"gemm.hip": _VGPR_FORM, "gemm_mx4.hip": _VGPR_FORM, "attention.hip": _VGPR_FORM}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, *EXTRA_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link libconvrot.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
