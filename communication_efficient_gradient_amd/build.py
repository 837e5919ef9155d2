"""Build libgq.so (hand-written HIP for gfx950) in-tree.

    python -m communication_efficient_gradient_amd.build

Each .hip translation unit is compiled in parallel with hipcc, then linked
into ``communication_efficient_gradient_amd/libgq.so``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "libgq")
LIB = os.path.join(HERE, "libgq.so")
SOURCES = ["api.hip", "stream_quant.hip", "sort_quant.hip", "deq.hip",
           "layer_quant.hip", "topk_quant.hip", "elias.hip",
           "alloc_quant.hip", "binopt_quant.hip", "act_api.hip",
           "act_pack.hip", "layer_norm.hip", "act_linear.hip",
           "act_wgrad.hip", "step_api.hip", "fp8_pack.hip", "fp8_linear.hip",
           "fp8_wgrad.hip", "adamw.hip"]
ARCH = os.environ.get("GQ_OFFLOAD_ARCH", "gfx950")

# -ffp-contract=off: the rounding decisions must see exactly the fp32
# operation sequence the method defines (no fused multiply-add).
# -packed-fp32-ops off: no v_pk_*_f32 instructions.
HIPFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def hipcc() -> str:
    return shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, src.replace(".hip", ".o"))
    cmd = [hipcc(), *HIPFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs,
           "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="-q" not in sys.argv)
