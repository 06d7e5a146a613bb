"""Orthogonal updates, host side: workspace sizes.  No call here reaches a kernel."""

import random

import pytest

from distributed_sgd_gradient_amd import _native
from test_layers_host import BF16, F16, F32

CAP = 4 << 30


def need(count, rows, cols, dtype):
    return _native.check(_native.lib().adasum_orthogonalize_workspace_bytes(count, rows, cols, dtype))


@pytest.mark.parametrize("count,rows,cols,dtype", [(64, 3038, 25571, F32), (64, 1250, 19083, F32),
                                                   (65536, 4080, 19521, BF16), (65536, 4096, 4096, BF16),
                                                   (33, 19083, 1250, F16)])
def test_workspace_of_many_is_capped(count, rows, cols, dtype):
    assert need(1, rows, cols, dtype) <= need(count, rows, cols, dtype) <= CAP


def test_workspace_of_two_or_more_is_capped():
    """Whatever the shape: two or more share no more than 4 GiB."""
    rng = random.Random(1)
    for _ in range(3000):
        rows, cols = (int(2 ** rng.uniform(6.1, 14.5)) for _ in range(2))
        dtype = rng.choice([F32, F16, BF16])
        if need(1, rows, cols, dtype) <= CAP:
            assert need(rng.choice([2, 3, 5, 11, 32, 64, 65536]), rows, cols, dtype) <= CAP, (rows, cols, dtype)


@pytest.mark.parametrize("rows,cols,dtype", [(775, 4283, F32), (1024, 4096, F32), (137, 1164, F32), (1024, 1024, BF16),
                                             (4080, 19521, BF16), (64, 500, F32), (300, 50, F16)])
def test_a_workspace_for_many_is_for_fewer_too(rows, cols, dtype):
    many = [need(count, rows, cols, dtype) for count in (*range(1, 131), 1000, 65536)]
    assert many == sorted(many)
    # asked for in any order, and of the transpose
    other = [need(count, cols, rows, dtype) for count in (65536, 1000, *range(130, 0, -1))]
    assert other == many[::-1]


def refusal(*coefficients):
    """What an otherwise good call without a workspace, which is looked at last, is refused for."""
    from test_more_layers_host import CALLS, coefficients as array
    args = {**CALLS["adasum_orthogonalize"], "steps": len(coefficients), "workspace": None,
            "coefficients": array(*[c for three in coefficients for c in three])}
    lib = _native.lib()
    assert lib.adasum_orthogonalize(*args.values()) == _native.EINVAL
    return lib.adasum_last_error().decode()


# Steep first steps: the largest singular value reaches 1.992, 1.966, 1.866, 1.560, .. at most.
STEEP = [(8.2051604139, -22.9015997, 16.4606545), (4.0663961, -2.8611614, 0.5183957), (3.9095949, -2.8233675, 0.5250336)]


def test_coefficients_below_two_are_allowed():
    """Values up to 2 are what is stated; 0.1 % of room at the start and 1 % at each
    step are for rounding."""
    for k in ([STEEP[0]], STEEP, [(1.99, 0.0, 0.0), (0.95, 0.0, 0.0)], [(-1.99, 0.0, 0.0)]):
        assert "workspace" in refusal(*k)
    for k in ([(2.0, 0.0, 0.0)], [(1.99, 0.0, 0.0), (1.0, 0.0, 0.0)], [(1.4, 0.0, 0.0), (1.4, 0.0, 0.0), (1.1, 0.0, 0.0)],
              [(8.3, -23.3, 17.0)]):
        assert "below 2" in refusal(*k)


def byte_set(p, rows, cols, stride, size):
    return {p + r * stride * size + c for r in range(rows) for c in range(cols * size)}


def test_matrices_between_each_others_rows():
    """Random places in one buffer: a call is refused for an overlap exactly where
    bytes are shared, or where strides in bytes differ and the spans do.  (What is
    let through is refused later: nothing lies there.)"""
    from test_more_layers_host import CALLS, at, pointers
    lib, rng, let, refused = _native.lib(), random.Random(2), 0, 0
    for _ in range(4000):
        rows, cols, count = rng.randint(1, 4), rng.randint(1, 5), rng.randint(1, 4)
        stride = cols + rng.choice([0, 1, cols, 2 * cols, 3 * cols])
        out_stride = rng.choice([stride, stride, cols + rng.randint(0, 9)])
        dtype, out_dtype = rng.choice([(F32, F32), (F32, F32), (F32, BF16), (F16, F32)])
        size, out_size = (4 if t == F32 else 2 for t in (dtype, out_dtype))
        x = [at(0) + 4 * rng.randint(0, 60) for _ in range(count)]
        out = [rng.choice([p, at(0) + 4 * rng.randint(0, 60), at(3) + 4 * rng.randint(0, 40)]) for p in x]
        if rng.random() < 0.4:  # side by side
            out = [at(3) + i * cols * out_size for i in range(count)]
        named = []
        for p, q in zip(x, out):
            if p != q or stride != out_stride or dtype != out_dtype:
                named.append((p, stride, size, False))
            named.append((q, out_stride, out_size, True))
        want = False
        for i, (p, s, n, w) in enumerate(named):
            for q, t, m, v in named[:i]:
                if not (w or v):
                    continue
                if rows == 1 or s * n == t * m:
                    want |= bool(byte_set(p, rows, cols, s, n) & byte_set(q, rows, cols, t, m))
                else:
                    want |= p < q + ((rows - 1) * t + cols) * m and q < p + ((rows - 1) * s + cols) * n
        args = {**CALLS["adasum_orthogonalize"], "x": pointers(*x), "out": pointers(*out), "count": count, "rows": rows,
                "cols": cols, "x_stride": stride, "out_stride": out_stride, "dtype": dtype, "out_dtype": out_dtype}
        assert lib.adasum_orthogonalize(*args.values()) < 0
        assert ("overlaps" in lib.adasum_last_error().decode()) == want
        let, refused = let + (not want), refused + want
    assert let > 500 and refused > 500


def test_matrices_of_other_shapes_between_each_others_rows():
    from distributed_sgd_gradient_amd.updates import _apart
    rng, let, refused = random.Random(3), 0, 0
    for _ in range(4000):
        rows, stride, size = rng.randint(1, 4), rng.randint(8, 14), rng.choice([2, 4])
        calls, named = {}, []
        for cols in rng.sample(range(1, 8), 2):
            a, b = (size * rng.randint(0, 70) for _ in range(2))
            if rng.random() < 0.5:
                b = a
            r = rng.choice([rows, rows + 1])
            calls[r, cols, stride if r > 1 else cols, stride if r > 1 else cols] = ([a], [b])
            if a != b:
                named.append((byte_set(a, r, cols, stride, size), False))
            named.append((byte_set(b, r, cols, stride, size), True))
        want = any((w or v) and bool(p & q) for i, (p, w) in enumerate(named) for q, v in named[:i])
        try:
            _apart(calls, size, size, None)
            assert not want
            let += 1
        except ValueError as e:
            assert want and "overlaps" in str(e)
            refused += 1
    assert let > 500 and refused > 500
