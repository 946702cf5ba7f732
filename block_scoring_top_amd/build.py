"""Compiles the HIP sources into ``block_scoring_top_amd/libblockscore.so``
for gfx950 (MI355X).  Run as a module or call :func:`build`."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libblockscore.so")
SOURCES = ["api.hip", "score_decode.hip", "score_prefill.hip", "topk.hip", "expand.hip", "compress.hip", "kv4.hip",
           "attn.hip", "attn_gather_bf16_kv4.hip", "attn_gather_bf16_kv16.hip", "attn_gather_f16_kv4.hip",
           "attn_gather_f16_kv16.hip", "attn_prefill_bf16_kv4.hip", "attn_prefill_bf16_kv16.hip",
           "attn_prefill_f16_kv4.hip", "attn_prefill_f16_kv16.hip"]
ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-fvisibility=hidden",
    # packed FP32 VALU forms are kept out of every code object
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"),
]


# Per-source extras.  The prefill scorer keeps its MFMA accumulators in
# architectural VGPRs (gfx950 allows either file): its epilogue then reads them
# without v_accvgpr moves, at the same occupancy.
# The top-k kernels issue their device atomics from one lane and use the
# result later: the atomic optimizer's wave-level rewrite reads the result at
# once (a wait on every atomic), so it is turned off there.
EXTRA = {"score_prefill.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
         "topk.hip": ["-mllvm", "-amdgpu-atomic-optimizer-strategy=None"]}


def _compile(src: str, objdir: str, verbose: bool) -> str:
    obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)
    return obj


def build(verbose: bool = False) -> str:
    objdir = os.path.join(ROOT, "_build", "hip")
    os.makedirs(objdir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, objdir, verbose), SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
