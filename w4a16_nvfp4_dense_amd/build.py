"""Builds libffn_nvfp4.so (the HIP kernels and the C ABI) for gfx950, in-tree.

Run ``python -m w4a16_nvfp4_dense_amd.build``; ``__graft_entry__.build()``
calls :func:`build`. Each source is compiled to an object under ``_build/``
(in parallel), then linked into ``w4a16_nvfp4_dense_amd/lib/``.
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
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libffn_nvfp4.so")

# longest compiles first (they start first in the pool)
SOURCES = ["wave_dual.hip", "fp8_dual.hip", "fp8_dual_silu.hip", "fp8_dual_gelu.hip", "wave_down.hip",
           "fp8_down_silu.hip", "fp8_down_gelu.hip", "fp8_down.hip", "mfma_launch.hip", "smallm_launch.hip",
           "int8_tile.hip", "moe_gemm.hip", "int8_rows.hip", "moe_route.hip", "moe_plan.hip", "moe_combine.hip",
           "gemv.hip", "quantize.hip", "w4a4.hip", "noalloc.hip", "stream_read.hip",
           "abi.cpp", "abi_fp8.cpp", "abi_w4a4.cpp", "abi_int8.cpp", "abi_moe.cpp"]

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")

CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    # keep the compiler from emitting packed fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC] + CFLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = [l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l]
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n" + "\n".join(msgs))
    if msgs:
        sys.stderr.write("\n".join(msgs) + "\n")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
