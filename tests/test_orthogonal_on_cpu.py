"""Orthogonal updates on the CPU, from their own sources (see
test_kernels_on_cpu.py), against the definition in long double where it is
hard: matrices of low rank over many steps, and values far below 1."""

import math
import subprocess

import pytest

from test_kernels_on_cpu import BF16, CLANG, CSRC, F16, F32, HERE, as_cpp, pytestmark, run  # noqa: F401

DEFAULT = (3.4445, -4.7750, 2.0315)
STEEP = (4.5, -5.88, 1.54)
HALF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}  # half a step, relative


@pytest.fixture(scope="module")
def orthogonal(tmp_path_factory):
    work = tmp_path_factory.mktemp("orthogonal")
    for name in ("orthogonal", "orthogonal_narrow"):
        (work / f"{name}.inc").write_text(as_cpp(f"{name}.hip"))
    exe = work / "orthogonal_cases"
    res = subprocess.run([CLANG, "-std=c++17", "-O1", "-ftrapv", "-ffp-contract=off", "-w", "-I", HERE, "-I", CSRC, "-I",
                          str(work), "-o", str(exe), f"{HERE}/orthogonal_cases.cpp"], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[:4000]
    return str(exe)


def narrow_limit(out, steps, coefficients, rounded):
    """The result's rounding; what fp64 leaves where the update has no direction,
    2^-53 of sums of 64 terms, raised by a in every step; and, where a rounded
    update has directions of any size, 5e-6 of those that steps of one G bring to
    1 (2^30 times 2^-50 of rounding beside a square of 0.1, and half of it)."""
    raised = math.prod(abs(k[0]) for k in (coefficients * steps)[:steps])
    return HALF[out] + 64 * 2.0 ** -53 * raised + (5 * 2.0 ** -20 if rounded else 0)


@pytest.mark.parametrize("rows,cols,rank,rounded,steps,coefficients", [
    (32, 300, 4, 0, 8, [DEFAULT]),
    (32, 300, 4, 0, 9, [DEFAULT]),
    (32, 300, 4, 0, 12, [DEFAULT]),
    (32, 300, 4, 0, 16, [DEFAULT]),
    (32, 300, 4, 1, 10, [DEFAULT]),
    (32, 300, 4, 1, 16, [DEFAULT]),
    (500, 61, 8, 0, 14, [DEFAULT]),
    (64, 64, 8, 0, 16, [STEEP]),
    (16, 90, 2, 0, 16, [DEFAULT]),
    (7, 5, 1, 0, 16, [DEFAULT]),
    (48, 70, 3, 1, 13, [DEFAULT, STEEP, (1.5, -0.5, 0.0)]),
    (20, 40, 0, 0, 16, [DEFAULT]),
    (1, 9, 0, 0, 16, [DEFAULT]),
])
@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_narrow_low_rank_over_many_steps(orthogonal, rows, cols, rank, rounded, steps, coefficients, out):
    limit = narrow_limit(out, steps, coefficients, rounded)
    run(orthogonal, rows, cols, F32, out, steps, rank, rounded, 1e-7, limit, *[c for k in coefficients for c in k])


@pytest.mark.parametrize("rows,cols,steps,eps,coefficients,value", [
    (65, 66, 5, 1e2, [DEFAULT], 1),  # beside a norm of some 40
    (65, 66, 5, 1e4, [DEFAULT], 1),
    (65, 66, 5, 1e8, [DEFAULT], 1),
    (65, 66, 5, 1e10, [DEFAULT], 1),
    (65, 66, 5, 1e25, [DEFAULT], 1),
    (140, 70, 12, 1e6, [DEFAULT], 1),
    # steps that shrink every value, or take cubes only; B far below its largest
    (65, 66, 3, 1e-7, [(0.01, 0.2, 0.3)], 1),
    (65, 66, 3, 1e5, [(0.01, 0.2, 0.3)], 1),
    (65, 66, 2, 1e5, [(0.0, 1.0, 0.0)], 3),
    (65, 66, 3, 1e4, [(0.001, 25.0, -25.0), (0.5, 0.0, 0.0), DEFAULT], 25),
    (65, 66, 2, 1e4, [(1.0, -31.5, 31.5)], 31.5),
])
def test_wide_values_far_below_one(orthogonal, rows, cols, steps, eps, coefficients, value):
    """A step's operands lose 2^-22 of themselves in two parts, and sums of k
    terms sqrt(k) roundings, which the coefficients scale; relative to the result
    whatever its scale is.  (Cubes take three times what X is off by; `value`
    bounds b and c where they are larger.)"""
    part = 2.0 ** -22 + math.sqrt(max(rows, cols)) * 2.0 ** -24
    limit = max(6.81, value) * part * math.sqrt(steps)
    k = [c for three in coefficients for c in three]
    run(orthogonal, rows, cols, F32, F32, steps, 0, 0, eps, limit, *k)
    if value == 1 and eps < 1e5:
        run(orthogonal, rows, cols, BF16, BF16, steps, 0, 0, eps, math.hypot(limit, 2.0 ** -8 / math.sqrt(3)), *k)
