"""Build libgemm355.so from csrc/ with hipcc for gfx950, in-tree.

Usage: python -m dense_tiled_gemm_fp8_amd.build  (or call build()).
Every call recompiles.  Objects go to _build/, the library next to this file.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libgemm355.so")
SOURCES = ["kernels.hip", "quant.hip", "plan.hip", "api.hip", "w4.hip", "kvcache.hip", "norm.hip",
           "block.hip"]
ARCH = "gfx950"

HIPCC_FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++20", "-fPIC",
    "-fvisibility=hidden",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]

# flags of single files
FILE_FLAGS = {
    # sums of matrix instructions go through vector instructions, which cannot
    # read accumulation registers
    "block.hip": ["-mllvm", "--amdgpu-mfma-vgpr-form=1"],
}


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + HIPCC_FLAGS + FILE_FLAGS.get(src, []) + ["-I", os.path.join(ROOT, "include"), "-c",
                                                              os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


def device_asm(src: str = "kernels.hip") -> str:
    """AMD GCN assembly of our own device code (for instruction-mix checks)."""
    os.makedirs(BUILD, exist_ok=True)
    out = os.path.join(BUILD, os.path.splitext(src)[0] + ".s")
    cmd = [hipcc()] + HIPCC_FLAGS + FILE_FLAGS.get(src, []) + ["-I", os.path.join(ROOT, "include"), "--cuda-device-only",
                                                              "-S", os.path.join(CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc -S failed:\n%s%s" % (r.stdout, r.stderr))
    return out


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
