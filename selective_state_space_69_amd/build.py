"""Build libssscan.so (the HIP selective-scan library) in-tree for gfx950.

    python -m selective_state_space_69_amd.build

Each translation unit is compiled by hipcc in parallel, then linked into
selective_state_space_69_amd/libssscan.so.  Packed-fp32 instructions are
disabled for all device code.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libssscan.so")
BUILD = os.path.join(PKG, "_build")

# slowest translation units first, so that the parallel build finishes sooner
SOURCES = ["ss_fwd_bf16_f32.hip", "ss_fwd_bf16_bf16.hip", "ss_fwd_f32_f32.hip",
           "ss_fwd_f32_bf16.hip", "ss_fwd_hw.hip", "ss_fwd_hw1.hip", "ss_bwd.hip", "ss_ssd.hip", "ss_conv.hip",
           "ss_complex.hip", "ss_step.hip", "ss_carry.hip", "ss_fwd.hip", "ss_runtime.hip",
           "ss_norm.hip", "ss_linear.hip", "ss_linear_mm.hip",
           "ss_linear_rows.hip", "ss_ckpt.hip",
           "ss_api.cpp", "ss_block_api.cpp"]
ARCH = os.environ.get("SS_SCAN_ARCH", "gfx950")
FLAGS = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=" + ARCH, "-I" + INCLUDE, "-I" + CSRC,
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function"]


def _hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    p = os.path.join(rocm, "bin", "hipcc")
    return p if os.path.exists(p) else "hipcc"


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr))
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp%d" % os.getpid()
    cmd = [_hipcc(), "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    return OUT


if __name__ == "__main__":
    build()
    sys.exit(0)
