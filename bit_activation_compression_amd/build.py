"""Build the codec's C-ABI library (libfc.so) for gfx950 with hipcc, in-tree.

Each .hip translation unit is compiled on its own (in parallel), then linked.
Device code: -O3, no floating-point contraction (the codec's rounding steps
are specified one by one), no packed-FP32 instructions, NaN handling off
(non-finite input is outside the contract) so min/max fold into DPP forms.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfc.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["fc_api.hip", "fc_quantize.hip", "fc_dequant_sum_requant.hip", "fc_dequantize.hip",
           "fc_sum.hip", "fc_linear_quantize.hip", "fc_allreduce_small.hip", "fc_stream.hip",
           "fc_generic.hip", "fc_residual_norm.hip", "fc_dequantize_residual_norm.hip",
           "fc_mxfp4.hip", "fc_matmul_mxfp4.hip",
           "fc_matmul_mxfp4_few.hip",
           "fc_train_api.hip", "fc_layer_norm.hip", "fc_layer_norm_backward.hip",
           "fc_activation_backward.hip", "fc_linear_act.hip", "fc_linear_input_grad.hip",
           "fc_linear_weight_grad.hip"]
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-honor-nans", "-mno-amdgpu-ieee",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    # --no-undefined: a kernel whose host-side launch stub was not emitted
    # fails here rather than when the library is loaded
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,--no-undefined", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose="-q" not in sys.argv)
