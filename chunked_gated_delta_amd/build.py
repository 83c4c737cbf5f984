"""Build libkda.so (all HIP sources, gfx950 only) in-tree with hipcc."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkda.so")
STAMPS_LIB = os.path.join(PKG, "libkda_stamps.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    # packed fp32 arithmetic stays off on this hardware (hand-written or compiler-generated)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # matrix-core accumulators stay in ordinary VGPRs (the scan reads them on the vector ALUs every step)
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall", "-Wno-unused-function",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _compile(src: str, obj: str, defines=()) -> list:
    return [HIPCC, *FLAGS, *defines, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src]


def build(verbose: bool = False) -> str:
    """Compile every source under csrc/ into chunked_gated_delta_amd/libkda.so, and beside it
    libkda_stamps.so, the same library with the segment pass's phase stamps compiled in (a
    measurement build that bench.py --phase-stamps loads; the product never does).  Always recompiles
    every source, a few at a time."""
    noise = "is not a recognized feature for this target"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        msgs = "\n".join(ln for ln in r.stdout.splitlines() if noise not in ln)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {os.path.basename(cmd[-1])}:\n{msgs}")
        if verbose and msgs:
            print(msgs, file=sys.stderr)

    workers = max(1, min(8, int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(workers) as pool:
        jobs = []
        for out, defines in ((LIB, ()), (STAMPS_LIB, ("-DKDA_PHASE_STAMPS=1",))):
            objs = [os.path.join(tmp, os.path.basename(out) + "." + os.path.basename(src) + ".o") for src in sources()]
            jobs.append((out, objs, [pool.submit(run, _compile(src, obj, defines)) for src, obj in zip(sources(), objs)]))
        for out, objs, done in jobs:
            for f in done:
                f.result()
            run([HIPCC, *FLAGS, "-shared", "-o", out + ".tmp", *objs])
    for out, _, _ in jobs:
        os.replace(out + ".tmp", out)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
