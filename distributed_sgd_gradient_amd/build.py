"""Build the gfx950 HIP library ``libadasum.so`` in-tree.

    python distributed_sgd_gradient_amd/build.py

(Run it by path: importing the package would load the library it builds.)

Compiles every source under ``csrc/`` with hipcc for gfx950, up to four at a
time, and links one shared library next to this file.  Always recompiles (the
build takes about a minute).
"""

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libadasum.so")

SOURCES = ["adasum.hip", "kernels.hip", "noalloc.hip", "plan.cpp", "layer_ops.hip", "embedding.hip", "layer_norm.hip",
           "checkpoint.hip", "linear_grad.hip", "rms.hip", "relative_bias.hip", "orthogonal.hip",
           "orthogonal_narrow.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # keep the compiler from forming packed-fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # no implicit fused multiply-add: products and sums that the kernels
    # write separately stay separately rounded (explicit fma() is kept)
    "-ffp-contract=off",
    "-fvisibility=hidden",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def build(verbose=False):
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work:
        objects = [os.path.join(work, s + ".o") for s in SOURCES]
        compiles = [[hipcc()] + HIPCC_FLAGS + ["-I", INCLUDE, "-I", CSRC, "-c", "-o", o, os.path.join(CSRC, s)]
                    for s, o in zip(SOURCES, objects)]
        with ThreadPoolExecutor(max_workers=4) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), compiles))
        _run([hipcc(), "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp] + objects, verbose)
    os.replace(tmp, LIB)
    return LIB


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed building libadasum.so")


if __name__ == "__main__":
    print(build(verbose=True))
