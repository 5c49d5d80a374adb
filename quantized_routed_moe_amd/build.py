"""Build the gfx950 HIP library libqrmoe.so in place (hipcc, no JIT cache)."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libqrmoe.so")
BUILD = os.path.join(ROOT, "_build")

SOURCES = ["api.cpp", "pack.hip", "route.hip", "expert_vec.hip", "decode.hip", "expert_mfma.hip",
           "expert_ops.cpp", "grouped_mm.hip", "grouped_vec.hip", "mxfp4.hip", "swiglu.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# -ffp-contract=off: floating-point operations round exactly as written (fused
# multiply-adds only where the source asks for one), so every kernel that
# shares a computation produces the same bits.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", "-I", os.path.join(ROOT, "include"),
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-Wno-unused-result"]
# MFMA results in ordinary VGPRs: the epilogues read every result, and from
# AGPRs each read would be one more VALU instruction.
VGPR_MFMA = ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]
# Except where a wave's 256 accumulators leave no ordinary VGPRs to work with.
AGPR_MFMA = {"grouped_mm.hip"}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    form = [] if src in AGPR_MFMA else VGPR_MFMA
    cmd = [HIPCC, *FLAGS, *form, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source for gfx950 and link libqrmoe.so (always rebuilds)."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libqrmoe.so failed")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
