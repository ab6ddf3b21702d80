"""Build the HIP library ``_build/libmamba_ssd_hip.so`` for gfx950 with hipcc.

Every source is compiled to an object in parallel, then linked into one shared
library that exports the C ABI of ``include/ssd.h``.  Run as
``python -m mamba_ssd_chunked_amd.build``.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libmamba_ssd_hip.so")
SOURCES = ["ssd_abi.cpp", "k_scan.hip", "k_chunk_fwd.hip", "k_chunk_bwd.hip", "k_chunk_wide.hip",
           "k_moments.hip", "k_pr.hip", "k_diag.hip", "k_quat.hip", "k_step.hip",
           "noalloc_scratch.hip", "k_stream.hip", "k_delta.hip", "k_delta_bwd.hip",
           "k_delta_step.hip", "k_norm.hip", "k_linear.hip", "k_linear_bwd.hip", "k_linear_step.hip",
           "k_group_norm.hip"]
ARCH = "gfx950"

# Packed fp32 instructions are switched off for all device code.  Inline assembly that the compiler
# warns of (registers it does not give away) fails the build.
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Wall", "-Werror=inline-asm",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _hipcc() -> str:
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")
    return p


def _compile(src: str) -> str:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(jobs: int | None = None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 4)
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(int(sys.argv[1]) if len(sys.argv) > 1 else None))
