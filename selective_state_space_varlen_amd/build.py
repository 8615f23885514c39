"""Build libssmpack.so (HIP, gfx950) in-tree with hipcc.

Usage: python -m selective_state_space_varlen_amd.build
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
LIB = os.path.join(HERE, "libssmpack.so")
BUILD = os.path.join(ROOT, "_build")

SOURCES = ["pack_indices.hip", "conv1d_pack.hip", "scan_fwd.hip", "scan_bwd.hip", "qk_norm.hip",
           "delta_fwd.hip", "delta_bwd.hip", "delta_step.hip", "decay_fwd.hip", "decay_dq.hip", "decay_dkv.hip",
           "decay_bwd.hip", "decay_step.hip", "layer_norm_fwd.hip", "layer_norm_bwd.hip", "dropout.hip", "pack_plan.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # keep hipcc from emitting packed-FP32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
    "-Wno-unused-command-line-argument",
]


HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE]


def _compile(src: str) -> str:
    """.hip sources go through hipcc for gfx950; .cpp sources are host-only
    code and go through the host compiler."""
    stem, ext = os.path.splitext(src)
    obj = os.path.join(BUILD, stem + ".o")
    if ext == ".hip":
        cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    else:
        cmd = [CXX, *HOST_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    return obj


def build(verbose: bool = True) -> str:
    """Compile every kernel source for gfx950 (and the host sources) and link
    libssmpack.so."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
