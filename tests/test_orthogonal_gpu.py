"""Orthogonal updates on the GPU where they are hard: low rank over many steps, and values far below 1.
Against the formula in 64 bits; tolerances are counted in roundings."""

import math
import random

import pytest
import torch

import distributed_sgd_gradient_amd as A
from conftest import flush_print
from test_layers_gpu import BF16, DTYPES, F16, F32, gen, ids
from test_more_layers_gpu import plain_orthogonal, spectrum, tolerance

pytestmark = pytest.mark.gpu

DEFAULT = (3.4445, -4.7750, 2.0315)
STEEP = (4.5, -5.88, 1.54)
HALF = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}


def whole(seed, *shape):
    return torch.randint(-7, 8, shape, generator=gen(seed)).double()


def low_rank(seed, count, n, m, rank, rounded, dtype=F32):
    """Of exactly that rank, or rounded to it from a product that does not fit."""
    x = whole(seed, count, n, rank) @ whole(seed + 1, count, rank, m)
    return (x * (math.pi if rounded else 1.0)).to(dtype).cuda()


def off(got, want):
    got, want = got.double(), want.double()
    return float(((got - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)).max())


@pytest.mark.parametrize("out", DTYPES, ids=ids)
@pytest.mark.parametrize("n,m,rank,rounded,steps,coefficients", [
    (32, 300, 4, False, 8, [DEFAULT]),
    (32, 300, 4, False, 9, [DEFAULT]),
    (32, 300, 4, False, 12, [DEFAULT]),
    (300, 32, 4, False, 16, [DEFAULT]),
    (32, 300, 4, True, 10, [DEFAULT]),
    (61, 769, 8, False, 14, [DEFAULT]),
    (64, 64, 8, False, 16, [STEEP]),
    (16, 2000, 2, False, 16, [DEFAULT]),
    (48, 5000, 3, True, 9, [DEFAULT, STEEP, (1.5, -0.5, 0.0)]),
    (1, 5, 1, True, 16, [DEFAULT]),
])
def test_narrow_low_rank_over_many_steps(gpu, n, m, rank, rounded, steps, coefficients, out):
    """Off by the result's rounding, by what fp64 leaves where the update has no
    direction (2^-53 of sums of 64 terms, here and in the reference, raised by a
    in every step) and, of a rounded update, by 5e-6 of the directions that the
    steps of one G bring to 1."""
    flush_print(f"low rank {n}x{m} rank {rank} {steps} steps to {out}")
    ks = (coefficients * steps)[:steps]
    x = low_rank(600, 3, n, m, rank, rounded)
    got = A.orthogonalize(x, steps=steps, coefficients=ks, dtype=out)
    limit = HALF[out] + 128 * 2.0 ** -53 * math.prod(abs(k[0]) for k in ks) + (5 * 2.0 ** -20 if rounded else 0)
    far = off(got, plain_orthogonal(x, ks))
    flush_print(f"  off by {far:.3g} of the norm, limit {limit:.3g}")
    assert far <= limit
    # alone, in place, and as a captured graph: the same bits
    assert torch.equal(A.orthogonalize(x[1], steps=steps, coefficients=ks, dtype=out), got[1])
    if out == F32:
        y, z = x.clone(), torch.empty_like(x)
        assert torch.equal(A.orthogonalize(y, steps=steps, coefficients=ks, out=y), got)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            A.orthogonalize(x, steps=steps, coefficients=ks, out=z)
        for _ in range(3):
            z.zero_()
            g.replay()
            assert torch.equal(A.orthogonalize(x, steps=steps, coefficients=ks), got)
            torch.cuda.synchronize()
            assert torch.equal(z, got)


def test_narrow_special_matrices_over_many_steps(gpu):
    x = low_rank(610, 5, 20, 90, 3, True)
    want = A.orthogonalize(x, steps=16)
    x[1] = 0
    x[2, 3, 4] = float("nan")
    x[3, 19, 89] = float("inf")
    got = A.orthogonalize(x, steps=16)
    assert torch.equal(got[[0, 4]], want[[0, 4]]) and not bool(got[1].any()) and bool(got[2:4].isnan().all())


@pytest.mark.parametrize("out", DTYPES, ids=ids)
@pytest.mark.parametrize("n,m", [(65, 66), (300, 400), (512, 512), (130, 900)])
def test_wide_updates_far_below_eps(gpu, n, m, out):
    """X keeps its digits however small the update is beside eps; matrices of one
    call may differ in that.  scale brings the results into out's range."""
    x = spectrum(620, n, m, F32, "strong", 3)
    norm = float(x[0].double().norm())
    x[1] *= 2.0 ** -20
    for ratio in (0.3, 3.0, 1e2, 1e4, 1e8):
        eps = norm * ratio
        got = A.orthogonalize(x, dtype=out, eps=eps, scale=ratio)
        want = plain_orthogonal(x, eps=eps, scale=ratio)
        for i in (0, 1, 2):
            if i == 1 and out == F16:
                continue  # below fp16's normal numbers
            far = off(got[i], want[i])
            flush_print(f"  {n}x{m} to {out}, eps {ratio:g} of the norm, matrix {i}: off by {far:.3g}")
            assert far <= tolerance(out, max(n, m), 5)
        assert torch.equal(A.orthogonalize(x[2], dtype=out, eps=eps, scale=ratio),
                           A.orthogonalize(x[2:], dtype=out, eps=eps, scale=ratio)[0])


def test_wide_steps_that_shrink(gpu):
    x = spectrum(630, 200, 300, F32)
    for ks in ([(0.01, 0.2, 0.3)] * 3, [(1e-3, 0.0, 0.0)] * 5, [(0.02, 0.0, 0.0), (3.0, -3.2, 1.2)]):
        got = A.orthogonalize(x, steps=len(ks), coefficients=ks)
        far = off(got, plain_orthogonal(x, ks))
        flush_print(f"  shrinking: off by {far:.3g}")
        assert far <= tolerance(F32, 300, len(ks))
    assert not bool(A.orthogonalize(x, coefficients=(0.0, 0.0, 0.0)).any())


@pytest.mark.parametrize("out", DTYPES, ids=ids)
@pytest.mark.parametrize("n,m", [(40, 90), (120, 200), (300, 500)])
def test_values_just_below_two(gpu, n, m, out):
    """The steepest steps that are allowed, on singular values that they take to
    their peaks.  A step's operands lose a part of themselves, which b and c scale,
    and the next one scales that by a at most."""
    ks = [(8.2051604139, -22.9015997, 16.4606545), (4.0663961, -2.8611614, 0.5183957)]
    s = torch.zeros(n, dtype=torch.float64)
    s[:12] = torch.tensor([0.86, 0.3, 0.25, 0.2, 0.15, 0.12, 0.1, 0.08, 0.05, 0.03, 0.02, 0.01])
    left = torch.linalg.qr(torch.randn(n, n, generator=gen(640), dtype=torch.float64))[0]
    right = torch.linalg.qr(torch.randn(m, n, generator=gen(641), dtype=torch.float64))[0]
    x = ((left * s) @ right.t().contiguous()).float().cuda()
    for steps in (1, 2):
        got = A.orthogonalize(x, steps=steps, coefficients=ks[:steps], dtype=out)
        want = plain_orthogonal(x, ks[:steps])
        assert float(torch.linalg.matrix_norm(want, 2)) > 1.8
        part = 2.0 ** -12 if out == BF16 and n > 256 else 2.0 ** -22 + math.sqrt(m) * 2.0 ** -24
        limit = 39.4 * part * (1 if steps == 1 else 4.1) + 3.4 * part * (steps - 1) + HALF[out]
        far = off(got, want)
        flush_print(f"  {n}x{m} to {out}, {steps} steps: off by {far:.3g}, limit {limit:.3g}")
        assert far <= limit


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("rows,widths", [(96, (70, 70, 70)), (30, (70, 70, 70)), (200, (131, 33, 33)), (300, (64, 300, 7)),
                                         (1, (5, 9, 5))])
def test_column_slices_of_one_buffer(gpu, rows, widths, dtype):
    """A fused weight's parts, in place and as outputs: the bits of matrices that lie
    apart, and every other column as it was."""
    flush_print(f"slices {rows} x {widths} {dtype}")
    wide = spectrum(650, rows, sum(widths) + 6, dtype)
    firsts = [3 + sum(widths[:i]) for i in range(len(widths))]
    parts = [wide[:, a:a + w] for a, w in zip(firsts, widths)]
    want = [A.orthogonalize(p.contiguous()) for p in parts]
    buffer = torch.full_like(wide, 7.0)
    outs = [buffer[:, a:a + w] for a, w in zip(firsts, widths)]
    before = wide.clone()
    for _ in range(3):
        got = A.orthogonalize(parts, out=outs)
        assert all(torch.equal(g, w) for g, w in zip(got, want)) and torch.equal(wide, before)
        assert bool((buffer[:, :3] == 7).all()) and bool((buffer[:, -3:] == 7).all())
        wide.copy_(before)
        A.orthogonalize(parts, out=parts)
        assert all(torch.equal(p, w) for p, w in zip(parts, want))
        assert torch.equal(wide[:, :3], before[:, :3]) and torch.equal(wide[:, -3:], before[:, -3:])
        wide.copy_(before)
    with pytest.raises((ValueError, A.AdasumError), match="overlaps"):
        A.orthogonalize(parts, out=[outs[0], outs[1], buffer[:, firsts[2] - 1:firsts[2] - 1 + widths[2]]])


def test_many_column_slices(gpu):
    """One view of all heads: [heads, rows, columns] of a [rows, heads * columns]."""
    wide = spectrum(651, 128, 64 * 40, BF16)
    heads = wide.view(128, 40, 64).transpose(0, 1)
    want = A.orthogonalize(heads.contiguous())
    assert torch.equal(A.orthogonalize(heads), want)
    assert A.orthogonalize(heads, out=heads) is heads and torch.equal(heads, want)


@pytest.mark.parametrize("n,m,dtype,kind", [
    (8192, 300, F32, "strong"), (300, 8192, F32, "rank"), (300, 8192, BF16, "strong"), (32768, 70, F32, "strong"),
    (32768, 64, F32, "strong"), (7, 32768, BF16, "normal"), (4500, 4300, F32, "strong"), (4300, 4500, F16, "normal"),
    (6000, 5000, BF16, "strong"), (1025, 9000, F32, "normal"),
])
def test_great_sides(gpu, n, m, dtype, kind):
    """Sides above 4096.  Of a matrix of rank 3, rounded to fp32, what that rounding
    adds, 2^-24 of the norm, is raised by 3.4445^5 = 485 here and in the reference;
    the parts' 2^-22 likewise."""
    flush_print(f"great sides {n}x{m} {dtype} {kind}")
    x = spectrum(660, n, m, dtype, kind)
    got = A.orthogonalize(x)
    far = off(got, plain_orthogonal(x))
    limit = tolerance(dtype, max(n, m), 5)
    if kind == "rank":
        limit += 485 * 2.0 ** -22
    flush_print(f"  off by {far:.3g}, limit {limit:.3g}")
    assert far <= limit
    assert torch.equal(A.orthogonalize(x), got)


@pytest.mark.parametrize("seed", range(24))
def test_anything_allowed(gpu, seed):
    """Random sides, counts, types, strides, steps, eps and places against the formula."""
    rng = random.Random(seed)
    n, m = (int(2 ** rng.uniform(0, 9)) for _ in range(2))
    if seed % 3 == 0:
        n = rng.choice([1, 15, 16, 17, 33, 48, 63, 64, 65, 127, 128, 129, 257])
    count, steps = rng.choice([1, 2, 5, 33, 130]) if n * m < 20000 else rng.choice([1, 3]), rng.randint(1, 8)
    dtype, out = rng.choice(DTYPES), rng.choice(DTYPES)
    x = spectrum(700 + seed, n, m, F32, "strong" if min(n, m) > 3 else "normal", count) * 1000
    ratio = rng.choice([1e-8, 0.2, 1.0, 30.0, 3e3])  # eps beside the norm
    eps, scale = ratio * float(x[0].double().norm()), max(1.0, ratio) * rng.uniform(0.5, 2.0)
    scale = float(torch.tensor(scale).float())
    x = x.to(dtype)
    flush_print(f"{count}x{n}x{m} {dtype} to {out}, {steps} steps, eps {ratio:g} of the norm")
    wide = torch.full((count, n + 2, m + rng.randint(0, 5)), float("nan"), dtype=dtype, device="cuda")
    view = wide[:, 1:n + 1, :m]
    view.copy_(x)
    got = A.orthogonalize(view, steps=steps, eps=eps, scale=scale, dtype=out)
    want = plain_orthogonal(x, [DEFAULT] * steps, eps, scale)
    limit = tolerance(out, max(n, m), steps)
    far = off(got, want)
    flush_print(f"  off by {far:.3g}, limit {limit:.3g}")
    assert far <= limit
    if out == dtype:
        assert A.orthogonalize(view, steps=steps, eps=eps, scale=scale, out=view) is view and torch.equal(view, got)
        assert bool(wide[:, 0].isnan().all()) and bool(wide[:, -1].isnan().all()) and bool(wide[:, :, m:].isnan().all())
