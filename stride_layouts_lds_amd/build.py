"""Build libstride_layouts_lds.so in-tree with hipcc for gfx950.

    python -m stride_layouts_lds_amd.build        # or build() from Python

Every HIP translation unit is compiled for gfx950 only, with packed-fp32
instruction generation disabled, then linked into one shared library next
to this file.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libstride_layouts_lds.so")
SOURCES = ["api.cpp", "api_ops.cpp", "api_gated.cpp", "describe.cpp", "layout_algebra.cpp", "gemm_f16.hip", "gemm_mx.hip",
           "gemm_block.hip", "quantize.hip", "orthogonalize.hip",
           "ortho_gram.hip", "quantize_rows.hip", "gemm_i8.hip", "gated.hip", "gated_prepare.hip", "gated_backward.hip", "probes.hip", "scratch.hip"]
HEADERS = ["sl_maps.hpp", "sl_kernels.hpp", "sl_ops.hpp", "sl_device.hpp", "layout_algebra.hpp", "describe.hpp",
           "api_common.hpp", "api_ops.hpp", "ortho_device.hpp", "dense.hpp", "activation.hpp"]
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc"), shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")


def _flags():
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
            # no packed-fp32 instruction generation
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(HERE, "..", "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + _flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = True, jobs: int | None = None) -> str:
    """Compile every source (always) and link the shared library."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, int(os.environ.get("MAX_JOBS", os.cpu_count() or 4))))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
