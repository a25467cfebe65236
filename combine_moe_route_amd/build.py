"""Build libmoeroute.so in-tree with hipcc for gfx950.

    python -m combine_moe_route_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoeroute.so")
SOURCES = ["api.hip", "route_topk.hip", "route_scored.hip", "dispatch.hip", "combine.hip",
           "combine_sender.hip", "grouped_gemm.hip", "grouped_gemm_bf16.hip", "gated_act.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # fp32 math stays IEEE: no fast-math, correctly rounded division
    "-fno-fast-math",
    # never let the compiler form packed-fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wl,-rpath,/opt/rocm/lib",
]


def command(out: str = LIB, extra=()):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    return [hipcc, *HIPCC_FLAGS, *extra, "-o", out, *[os.path.join(CSRC, s) for s in SOURCES]]


def build(out: str = LIB, extra=()) -> str:
    tmp = out + ".tmp"
    cmd = command(tmp, extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass warns about the device-only target feature; drop that line
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + " ".join(cmd) + "\n" + err)
    if err.strip():
        sys.stderr.write(err + "\n")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build())
