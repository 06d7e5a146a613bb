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
