"""Build the MI355X MoE library (libmoe_mi355x.so) in-tree with hipcc for gfx950.

Usage: python -m expert_grouped_gemm_amd.build  (or import and call build()).
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_mi355x.so")
SOURCES = ["gemm_bf16.hip", "gemm_fp8.hip", "api.hip", "router.hip", "dispatch.hip", "gemm.hip", "combine.hip",
           "burst.hip", "owner_return.hip", "noalloc.hip", "gemm_w4a8.hip", "backward.hip", "mxfp4.hip",
           "gemm_w4a4.hip", "expert_backward.hip", "expert_backward_weights.hip", "expert_backward_checkpoint.hip",
           "int8.hip", "gemm_int8.hip", "gemm_int8_rows.hip", "gemm_checkpoint.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -packed-fp32-ops off: hipcc -O3 would otherwise emit packed fp32 adds/muls/fmas.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function"]

# The SDWA peephole pass takes 100 of 160 seconds on the byte conversions in this file's 80 unrolled epilogues; without
# it the same kernels compile in 60.
FILE_FLAGS = {"expert_backward_checkpoint.hip": ["-mllvm", "-amdgpu-sdwa-peephole=0"]}


def build(verbose: bool = False, jobs: int = 8) -> str:
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(obj_dir, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [HIPCC, *FLAGS, *FILE_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l)
        if out.strip() and (verbose or pr.returncode):
            print(out, file=sys.stderr)
        if pr.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
