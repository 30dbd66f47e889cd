"""Build the gfx950 libraries in-tree with hipcc.

  libdcr.so        the delta encode / apply library, its 4-bit weight calls and
                   those of a training turn (C-ABI in include/dcr.h)
  libdcr_synth.so  the seeded synthetic input generator (test / bench inputs)

Run ``python -m bit_exact_xor_amd.build`` (or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")

LIB_DCR = os.path.join(HERE, "libdcr.so")
LIB_SYNTH = os.path.join(HERE, "libdcr_synth.so")

ARCH = os.environ.get("DCR_OFFLOAD_ARCH", "gfx950")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# packed fp32 instructions stay off in all HIP code built here
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-I", INCLUDE, "-I", CSRC]

DCR_SOURCES = ["dcr_plan.cpp", "dcr_kernels.hip", "dcr_transcode.hip", "dcr_pack.hip", "dcr_fp4.hip",
               "dcr_fp4_matmul.hip", "dcr_fp4_rows.hip", "dcr_fp4_tile.hip", "dcr_fp4_tile4.hip", "dcr_fp4_grad.hip",
               "dcr_experts.hip", "dcr_rows.hip", "dcr_logprobs.hip", "dcr_adamw.hip"]


def _compile(out: str, sources: list[str], extra: list[str] | None = None) -> None:
    """Compile each source (some at a time), then link the objects."""
    with tempfile.TemporaryDirectory(prefix="dcr_build_") as tmp:
        def one(src):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            subprocess.run([HIPCC, *COMMON, *(extra or []), "-c", "-x", "hip", src, "-o", obj], check=True)
            return obj
        with ThreadPoolExecutor(max_workers=min(4, os.cpu_count() or 1)) as pool:
            objs = list(pool.map(one, [os.path.join(CSRC, s) for s in sources]))
        subprocess.run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", out + ".tmp", *objs], check=True)
    os.replace(out + ".tmp", out)


def build(verbose: bool = True) -> None:
    _compile(LIB_DCR, DCR_SOURCES)
    _compile(LIB_SYNTH, ["synth.hip"])
    if verbose:
        print(f"built {LIB_DCR} and {LIB_SYNTH} for {ARCH}")


if __name__ == "__main__":
    build()
    sys.exit(0)
