"""Build libblockq.so (HIP for gfx950) in-tree with hipcc.

Usage: python -m block_quantized_wire_amd.build   (or call build()).
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libblockq.so")
SOURCES = ["bq_abi.cpp", "bq_i8.hip", "bq_mx.hip", "bq_mxc.hip", "bq_mm.hip", "bq_noalloc.hip",
           "bq_i4.hip", "bq_mmi4.hip", "bq_moe.hip", "bq_kv.hip", "bq_attn.hip", "bq_attn_64.hip",
           "bq_attn_256.hip"]
HEADERS = ["bq_device.h", "bq_launch.h", "bq_ranges.h", "bq_attn.h"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # the codec definitions round every product and sum separately, in IEEE binary32
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def sources() -> list[str]:
    return [os.path.join(CSRC, s) for s in SOURCES]


def build(verbose: bool = False) -> str:
    """Compile every HIP source for gfx950 into block_quantized_wire_amd/libblockq.so."""
    tmp = LIB + ".tmp"
    include = ["-I", os.path.join(ROOT, "include")]
    with tempfile.TemporaryDirectory() as d:
        # the sources side by side: the attention's alone take a minute each
        cmds = [[HIPCC, *FLAGS, *include, "-c", s, "-o", os.path.join(d, os.path.basename(s) + ".o")]
                for s in sources()]
        if verbose:
            print("\n".join(" ".join(c) for c in cmds), flush=True)
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda c: subprocess.run(c, check=True), cmds))
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *(c[-1] for c in cmds), "-o", tmp],
                       check=True)
    os.replace(tmp, LIB)
    return LIB


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [os.path.join(CSRC, h) for h in HEADERS] + [
        os.path.join(ROOT, "include", h) for h in ("blockq.h", "blockq_moe.h", "blockq_kv.h")]
    return any(os.path.getmtime(d) > t for d in deps)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
