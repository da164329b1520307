"""Build the HIP library libkda.so (gfx950) in-tree with hipcc.

Usage: python -m gated_delta_rule_amd.build [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkda.so")
SOURCES = ["kda_abi.hip", "kda_noalloc.hip", "kda_prefill.hip", "kda_prefill_pipe.hip", "kda_segment.hip", "kda_recurrent.hip",
           "kda_layer.hip", "kda_backward.hip", "kda_ssm_abi.hip", "kda_ssm_conv.hip", "kda_ssm_scan.hip",
           "kda_ssm_bwd.hip", "kda_ssm_recurrent.hip", "kda_spec.hip",
           "kda_attn_abi.hip", "kda_attn_f32.hip", "kda_attn_fwd.hip", "kda_attn_step.hip", "kda_attn_bwd_f32.hip", "kda_attn_bwd.hip", "kda_pages.hip"]
HEADERS = ["kda_device.h", "kda_launch.h", "kda_chunk.h", "kda_ssm_launch.h", "kda_ssm_tile.h",
           "kda_host.h", "kda_attn_launch.h", "kda_attn_tile.h", "kda_attn_mma.h"]
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # packed fp32 VALU instructions are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


def build(verbose: bool = False, resource_usage: bool = False) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *FLAGS, f"-I{os.path.join(ROOT, 'include')}", "-o", tmp, *srcs]
    if resource_usage:
        cmd.insert(1, "-Rpass-analysis=kernel-resource-usage")
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                    if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{out}")
    if verbose or resource_usage:
        print(out, flush=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, resource_usage="--resources" in sys.argv)
    print(LIB)
