"""The relative bias's gradient on the CPU, from its own source (see
test_kernels_on_cpu.py): sums of the groups of a workgroup."""

import subprocess

import pytest

from test_kernels_on_cpu import BF16, CLANG, CSRC, F16, F32, HERE, as_cpp, pytestmark, run  # noqa: F401


@pytest.fixture(scope="module")
def sums(tmp_path_factory):
    work = tmp_path_factory.mktemp("relative_bias_sums")
    (work / "relative_bias.inc").write_text(as_cpp("relative_bias.hip"))
    exe = work / "relative_bias_sums"
    res = subprocess.run([CLANG, "-std=c++17", "-O1", "-ftrapv", "-ffp-contract=off", "-w", "-I", HERE, "-I", CSRC, "-I",
                          str(work), "-o", str(exe), f"{HERE}/relative_bias_sums.cpp"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[:4000]
    return str(exe)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("queries,keys", [(64, 300), (64, 64), (80, 400), (100, 100)])
def test_groups_are_joined_in_fp64(sums, queries, keys, dtype):
    """An fp32 sum is of one group's rows, 4096 at most: what small groups hold is
    not lost beside a large one's."""
    run(sums, queries, keys, dtype)
