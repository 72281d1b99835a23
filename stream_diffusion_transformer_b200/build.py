"""Builds libzimage_dit.so in place with nvcc for sm_100a.

    python -m stream_diffusion_transformer_b200.build [--verbose]

The library is one translation unit (csrc/zimage_dit.cu includes the kernel
headers); it links the CUDA runtime statically and reaches the driver's
tensor-map encoder through the runtime's entry-point query, so the only
run-time dependency is the NVIDIA driver.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libzimage_dit.so")
SOURCES = [os.path.join(PKG, "csrc", "zimage_dit.cu")]
DEPS = SOURCES + [os.path.join(PKG, "csrc", f) for f in
                  ("zi_common.cuh", "zi_gemm.cuh", "zi_attention.cuh", "zi_rows.cuh",
                   "zi_cluster.cuh", "zi_fp4.cuh", "zi_attention_masked.cuh")] + \
       [os.path.join(ROOT, "include", "zimage_dit.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-shared",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libzimage_dit.so")


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include")]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    tmp = LIB + ".tmp"
    cmd += ["-o", tmp, *SOURCES]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
