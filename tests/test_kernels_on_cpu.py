"""Kernels of the layer operators on the CPU, from their own sources.

The sources are compiled as ordinary C++ against tests/on_cpu/hip, which runs
every lane as a fiber; launches become calls.  Buffers end at pages that must
not be touched, LDS and outputs start as garbage, waves run in random order
and signed overflow ends the program.
"""

import os
import platform
import re
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "distributed_sgd_gradient_amd", "csrc")
HERE = os.path.join(ROOT, "tests", "on_cpu")
CLANG = shutil.which("clang++") or "/opt/rocm/llvm/bin/clang++"

pytestmark = pytest.mark.skipif(platform.machine() != "x86_64" or not os.path.exists(CLANG),
                                reason="needs clang++ on x86-64")


def as_cpp(name):
    """The kernel source with every launch written as a call."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text, n = re.subn(r"(\b\w+(?:<[^<>;(){}]*>)?)<<<(.*?)>>>\(", r"on_cpu::launch(\1, \2)(", text, flags=re.S)
    assert n > 0 and "<<<" not in text
    return text


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    work = tmp_path_factory.mktemp("on_cpu")

    def build(name):
        exe = work / name
        if not exe.exists():
            (work / f"{name}.inc").write_text(as_cpp(f"{name}.hip"))
            res = subprocess.run([CLANG, "-std=c++17", "-O1", "-ftrapv", "-ffp-contract=off", "-w", "-I", HERE, "-I",
                                  CSRC, "-I", str(work), "-o", str(exe), os.path.join(HERE, f"{name}.cpp")],
                                 capture_output=True, text=True)
            assert res.returncode == 0, res.stderr[:4000]
        return str(exe)
    return build


def run(exe, *args):
    res = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and res.stdout.endswith("done\n"), (res.returncode, res.stdout[-500:], res.stderr[-500:])
    return res.stdout


def test_checkpoint(program):
    """Packing and reading back, and the pieces of a row of 2^31 - 1 values."""
    run(program("checkpoint"))


UNIFORM, HALF, ONE, NONE, OUTSIDE, FALLING = range(6)
F32, F16, BF16 = range(3)


@pytest.mark.parametrize("n,vocab,hidden,kind,dtype,grad,token_bytes,accumulate", [
    (1, 1, 1, UNIFORM, F32, F32, 8, 0),
    (700, 40, 33, OUTSIDE, BF16, F32, 4, 0),
    (700, 40, 33, HALF, F16, F16, 8, 1),
    (3000, 3, 8, UNIFORM, F32, BF16, 8, 0),
    (9000, 1, 16, ONE, BF16, BF16, 4, 0),
    (9000, 5, 7, FALLING, F32, F32, 8, 1),
    (2000, 60, 20, NONE, F32, F32, 8, 0),
    (2000, 140000, 5, UNIFORM, BF16, F32, 8, 0),
    (25000, 5000, 1031, UNIFORM, F32, F32, 8, 0),
    (25000, 5000, 1031, HALF, BF16, F32, 4, 1),
    (65536, 30522, 1024, FALLING, BF16, F32, 8, 0),
])
def test_embedding_grad(program, n, vocab, hidden, kind, dtype, grad, token_bytes, accumulate):
    """The grouped list is right at every position and the sums are exact."""
    run(program("embedding"), n, vocab, hidden, kind, dtype, grad, token_bytes, accumulate)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (37, 7), (70, 100), (33, 250), (9, 513), (6, 1001), (5, 2050),
                                         (3, 4097), (2, 16384), (2, 16383)])
def test_layer_norm(program, rows, hidden, dtype):
    """Forward and backward, from x and from kept rows, rows with gaps."""
    for kept in (0, 1):
        run(program("layer_norm"), rows, hidden, dtype, kept, (rows + kept) % 2)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,out,width", [(1, 1, 1), (33, 7, 15), (31, 8, 16), (70, 130, 5), (65, 3, 300),
                                            (100, 140, 270), (300, 40, 33), (129, 259, 257)])
def test_linear_grad(program, rows, out, width, dtype):
    """Exact sums of narrow and ragged operands, rows with gaps."""
    for grad in {F32, dtype}:
        run(program("linear_grad"), rows, out, width, dtype, grad, rows % 2)
