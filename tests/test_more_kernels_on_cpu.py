"""Kernels of the residual norm, the relative bias and the orthogonal updates
on the CPU, from their own sources (see test_kernels_on_cpu.py)."""

import pytest

from test_kernels_on_cpu import BF16, F16, F32, as_cpp, program, pytestmark, run  # noqa: F401


@pytest.fixture(scope="module")
def orthogonal(program, tmp_path_factory):  # noqa: F811
    """The program of both sources of the orthogonal updates."""
    work = tmp_path_factory.getbasetemp()
    for folder in work.glob("on_cpu*"):
        (folder / "orthogonal_narrow.inc").write_text(as_cpp("orthogonal_narrow.hip"))
    return program("orthogonal")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (37, 7), (70, 100), (33, 250), (9, 513), (6, 1001), (5, 2050),
                                         (3, 4097), (2, 16384), (2, 16383)])
def test_rms(program, rows, hidden, dtype):  # noqa: F811
    """Forward and backward, rows with gaps, with all operands and the fewest."""
    for wide in {0, int(dtype != F32)}:
        for more in (0, 1):
            run(program("rms"), rows, hidden, dtype, wide, more)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("batch,heads,queries,keys,offset,buckets,reach,both", [
    (1, 1, 1, 1, 0, 2, 2, 0),
    (2, 3, 1, 70, 69, 32, 128, 0),
    (2, 1, 7, 5, 0, 4, 9, 1),
    (3, 2, 40, 33, 0, 20, 60, 1),
    (1, 2, 70, 150, 80, 32, 128, 0),
    (2, 1, 130, 141, 0, 32, 128, 1),
    (1, 1, 18, 1100, -30, 64, 300, 1),
    (1, 1, 300, 3, 1000000000, 32, 128, 1),
    # buckets joined in pieces: of few splits, and of eight or more
    (1, 2, 3, 17001, 40, 32, 128, 1),
    (1, 1, 600, 2001, -3, 8, 20, 0),
])
def test_relative_bias(program, batch, heads, queries, keys, offset, buckets, reach, both, dtype):  # noqa: F811
    run(program("relative_bias"), batch, heads, queries, keys, offset, buckets, reach, both, dtype)


@pytest.mark.parametrize("count,rows,cols,dtype,out_dtype,steps", [
    (1, 1, 1, F32, F32, 5),
    (2, 5, 9, BF16, BF16, 5),
    (1, 30, 130, F16, F16, 5),
    (2, 200, 64, F32, F16, 4),
    (1, 48, 50, BF16, F32, 5),
    (1, 17, 300, F32, F32, 1),
    (1, 65, 66, F32, F32, 5),
    (1, 140, 20, F32, F32, 2),
    (1, 140, 131, F32, BF16, 1),
    (1, 258, 260, BF16, BF16, 1),
])
def test_orthogonal(orthogonal, count, rows, cols, dtype, out_dtype, steps):
    run(orthogonal, count, rows, cols, dtype, out_dtype, steps)
