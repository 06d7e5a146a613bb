"""Residual norm, relative bias and orthogonal updates on the GPU against their
formulas in 64 bits.  Tolerances are counted in roundings as in
test_layers_gpu.py."""

import math

import numpy as np
import pytest
import torch

import distributed_sgd_gradient_amd as A
import oracle
from conftest import flush_print
from distributed_sgd_gradient_amd import _native
from test_layers_gpu import BF16, DTYPES, E, F16, F32, TINY, U, gen, ids, randn, strided, tokens_of, unaligned, within

pytestmark = pytest.mark.gpu

STREAMS = [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


# ---------------------------------------------------------------- residual norm

# The sum of a row's squares: 16 terms in a lane, 6 steps across a wave, 16
# waves; the mean, eps and the root add 3 and half of them count.
SUM = 38
RSTD = (SUM + 2) / 2 + 2


def plain_rms(h, w, eps):
    h = h.double()
    r = 1.0 / torch.sqrt(h.square().mean(-1) + eps)
    y = h * r[..., None]
    return (y if w is None else y * w.double()), r


def plain_rms_grad(dy, h, rstd, w, dh):
    """dx, dweight, and the magnitudes that their errors are counted in."""
    dy, r = dy.double(), rstd.double()[..., None]
    n = h.double() * r
    g = dy if w is None else dy * w.double()
    m = (g * n).mean(-1, keepdim=True)
    dx = r * (g - n * m)
    mx = r * (4 * (g.abs() + (n * m).abs()) + n.abs() * (SUM + 8) * (g * n).abs().mean(-1, keepdim=True)) * E
    if dh is not None:
        dx = dx + dh.double()
    lead = tuple(range(dy.dim() - 1))
    return dx, (dy * n).sum(lead), mx, (dy * n).abs().sum(lead)


def check_rms(rows, hidden, dtype, stream, param, seed, put=lambda t: t):
    x, res = randn(seed, rows, hidden, dtype=dtype), randn(seed + 1, rows, hidden, dtype=stream, std=2.0)
    w = randn(seed + 2, hidden, mean=1.0, std=0.3, dtype=param)
    want_h = (x.float() + res.float()).to(stream)
    for weight in (w, None):
        for residual in (res, None):
            y, h, rstd = A.rms_norm(put(x), weight, residual=None if residual is None else put(residual), eps=1e-6)
            assert torch.equal(h, x if residual is None else want_h)
            ry, rr = plain_rms(h, weight, 1e-6)
            within(rstd, rr, RSTD * E * rr, "rstd")
            within(y, ry, ((RSTD + 3) * E + U[dtype]) * ry.abs() * 1.001 + TINY[dtype], "y")
            got = A.rms_norm_pack(put(x), weight, residual=None if residual is None else put(residual), eps=1e-6)
            assert same([got[0], got[3], got[4]], [y, h, rstd]) and same(got[1:3], A.checkpoint_pack(y))
            only = A.rms_norm_pack(put(x), weight, residual=residual, values=False, eps=1e-6)
            assert only[0] is None and same(only[1:], got[1:])
    return y, h, rstd


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=ids)
@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 1024), (3, 7), (129, 8), (65, 31), (40, 250), (9, 513),
                                         (7, 1001), (5, 2050), (3, 4097), (2, 8200), (2, 16384)])
def test_rms(gpu, rows, hidden, dtype, stream):
    flush_print(f"rms rows={rows} hidden={hidden} {dtype} stream {stream}")
    check_rms(rows, hidden, dtype, stream, F32, 300)


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=ids)
@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 1024), (3, 7), (2001, 8), (65, 31), (4000, 250), (900, 513),
                                         (1031, 1001), (500, 2050), (300, 4097), (301, 8200), (280, 16384)])
def test_rms_grad(gpu, rows, hidden, dtype, stream):
    flush_print(f"rms_grad rows={rows} hidden={hidden} {dtype} stream {stream}")
    dy, h = randn(310, rows, hidden, dtype=dtype), randn(311, rows, hidden, dtype=stream, std=2.0)
    dh = randn(312, rows, hidden, dtype=stream)
    for param in {F32, dtype}:
        w = randn(313, hidden, mean=1.0, std=0.3, dtype=param)
        rstd = plain_rms(h, None, 1e-6)[1].float()
        for along in (dh, None):
            dx, dw = A.rms_norm_grad(dy, h, rstd, w, dh=along)
            rx, rw, mx, mw = plain_rms_grad(dy, h, rstd, w, along)
            within(dx, rx, mx + (U[stream] + 2 * E) * rx.abs() + TINY[stream], "dx")
            # a lane's rows, the wave's and the workgroup's, and the products'
            within(dw, rw, (min(rows, 1024) + 10) * E * mw + (U[param] + E) * rw.abs() + TINY[param], "dweight")
    dx, dw = A.rms_norm_grad(dy, h, rstd)
    rx, _, mx, _ = plain_rms_grad(dy, h, rstd, None, None)
    assert dw is None
    within(dx, rx, mx + (U[stream] + 2 * E) * rx.abs() + TINY[stream], "dx without weight")


def test_rms_grad_against_differences(gpu):
    """The formula's gradients against central differences of the 64-bit norm."""
    rows, hidden, eps, d = 3, 40, 1e-3, 1e-6
    x, res, w = randn(320, rows, hidden), randn(321, rows, hidden), randn(322, hidden, mean=1.0, std=0.2)
    dy, dh = randn(323, rows, hidden), randn(324, rows, hidden)
    _, h, rstd = A.rms_norm(x, w, residual=res, eps=eps)
    dx, dw = A.rms_norm_grad(dy, h, rstd, w, dh=dh)

    def loss(hh, ww):
        return float((plain_rms(hh, ww, eps)[0] * dy.double()).sum() + (hh * dh.double()).sum())
    hd, wd = h.double(), w.double()
    for r, c in ((0, 0), (1, 7), (2, 39)):
        step = torch.zeros_like(hd)
        step[r, c] = d
        diff = (loss(hd + step, wd) - loss(hd - step, wd)) / (2 * d)
        assert abs(diff - float(dx[r, c])) <= 1e-5 * (1 + abs(diff))
    for c in (0, 13):
        step = torch.zeros_like(wd)
        step[c] = d
        diff = (loss(hd, wd + step) - loss(hd, wd - step)) / (2 * d)
        assert abs(diff - float(dw[c])) <= 1e-5 * (1 + abs(diff))


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=ids)
def test_rms_strides_places_and_segments(gpu, dtype, stream):
    rows, hidden = 77, 301
    check_rms(rows, hidden, dtype, stream, dtype, 330, strided)
    check_rms(rows, hidden, dtype, stream, dtype, 330, unaligned)
    x, res = randn(331, rows, hidden, dtype=dtype), randn(332, rows, hidden, dtype=stream)
    dy, w = randn(333, rows, hidden, dtype=dtype), randn(334, hidden, dtype=dtype)
    y, h, rstd = A.rms_norm(x, w, residual=res)
    # the stream in place, and outputs with gaps that stay as they were
    place, out = strided(res), strided(torch.zeros_like(x))
    got = A.rms_norm(strided(x), w, residual=place, h=place, out=out)
    assert got[1] is place and got[0] is out and same(got, (y, h, rstd))
    for t in (place, out):
        assert bool(t._base[:, :2].isnan().all()) and bool(t._base[:, 2 + hidden:].isnan().all())
    # leading dimensions
    many = A.rms_norm(x.view(7, 11, hidden), w, residual=res.view(7, 11, hidden))
    assert many[0].shape == (7, 11, hidden) and many[2].shape == (7, 11)
    assert same([t.reshape(s.shape) for t, s in zip(many, (y, h, rstd))], (y, h, rstd))
    # the gradient along the stream in place, dweight added to a segment
    dh = randn(335, rows, hidden, dtype=stream)
    dx, dw = A.rms_norm_grad(dy, h, rstd, w, dh=dh)
    seg = torch.full((hidden + 6,), 1.5, dtype=F32, device="cuda")
    along = strided(dh)
    a, b = A.rms_norm_grad(strided(dy), strided(h), rstd, w, dh=along, dx=along, dweight=seg[3:3 + hidden])
    assert a is along and torch.equal(a, dx) and b.data_ptr() == seg[3:].data_ptr()
    assert torch.equal(b.to(dtype), dw)
    first = b.double().clone()
    A.rms_norm_grad(dy, h, rstd, w, dweight=b, accumulate=True)
    _, rw, _, mw = plain_rms_grad(dy, h, rstd, w, None)
    within(b, first + rw, (rows + 10) * E * mw + 2 * E * (first + rw).abs(), "dweight added")
    assert bool((seg[:3] == 1.5).all()) and bool((seg[-3:] == 1.5).all())


def test_rms_of_special_rows(gpu):
    """Zeros, NaN, infinities and squares out of fp32's range stay in their
    rows; no rows are no work."""
    for dtype, stream in STREAMS:
        x, res, w = randn(340, 6, 90, dtype=dtype), randn(341, 6, 90, dtype=stream), randn(342, 90)
        y, h, rstd = A.rms_norm(x, w, residual=res)
        x2, res2 = x.clone(), res.clone()
        x2[1], res2[1] = 0, 0
        x2[2, 5] = float("nan")
        res2[3, 7] = float("inf")
        got = A.rms_norm_pack(x2, w, residual=res2)
        assert same([t[[0, 4, 5]] for t in (got[0], got[3], got[4])], [t[[0, 4, 5]] for t in (y, h, rstd)])
        assert not bool(got[0][1].any()) and abs(float(got[4][1]) - 1000) <= 1e-3
        assert bool(got[0][2].isnan().all()) and bool(got[4][2].isnan())
        assert float(got[4][3]) == 0 and bool(got[0][3, 7].isnan()) and not bool(got[0][3, :7].any())
        if stream == F32 or dtype == BF16:
            res2[4] = 1e25
            assert float(A.rms_norm(x2, w, residual=res2)[2][4]) == 0
        none = A.rms_norm_pack(x[:0], w, residual=res[:0])
        assert none[0].shape == (0, 90) and none[2].shape == (0, 3)
        dx, dw = A.rms_norm_grad(x[:0], res[:0], rstd[:0], w)
        assert dx.shape == (0, 90) and not bool(dw.any())


@pytest.mark.parametrize("hidden", (7, 256, 1000, 4096, 16383))
def test_rms_rounds_once(gpu, hidden):
    """rstd and an fp32 y are off by half a step, 2^-24 of the value, and what
    terms of 2^-24 of 2^-24 leave: below 2^-44."""
    x, w = randn(350, 37, hidden, dtype=F32) * 3, randn(351, hidden, dtype=F32)
    y, _, rstd = A.rms_norm(x, w)
    eps = float(torch.tensor(1e-6))
    r = (x.double().square().mean(1) + eps).rsqrt()
    bound = 2.0 ** -24 + 2.0 ** -44
    within(rstd, r, bound * r, "rstd")
    want = x.double() * r[:, None] * w.double()
    within(y, want, bound * want.abs(), "y")


def test_rms_of_infinite_weights(gpu):
    x = randn(352, 4, 100, dtype=F32)
    w = torch.ones(100, device="cuda")
    w[3], w[4] = float("inf"), float("-inf")
    y = A.rms_norm(x, w)[0]
    assert torch.equal(y[:, 3], x[:, 3].sign() * w[3]) and torch.equal(y[:, 4], x[:, 4].sign() * w[4])
    assert bool(y[:, 5:].isfinite().all())


def test_rms_grad_sums_are_bounded(gpu):
    """As for the layer norm: a sum takes 1024 terms, 2 steps across the wave
    and 3 other waves at most, whatever the number of rows."""
    rows, d = 1 << 27, 1 + 2.0 ** -11 - 2.0 ** -23
    dy, one = torch.full((rows, 2), d, device="cuda"), torch.ones(rows, device="cuda")
    h, w = torch.ones(rows, 2, device="cuda"), torch.ones(2, device="cuda")
    dw = A.rms_norm_grad(dy, h, one, w)[1]
    within(dw, torch.full((2,), rows * d, dtype=torch.float64), 1030 * E * rows * d, "dweight")


# ---------------------------------------------------------------- relative bias


def bucket(d, buckets, reach, both):
    """From the definition, in whole numbers."""
    m = buckets // 2 if both else buckets
    e, n = m // 2, abs(d) if both else max(-d, 0)
    b = n
    if n >= e:
        b = e
        while b < m - 1 and n ** (m - e) * e ** (b + 1 - e) >= reach ** (b + 1 - e) * e ** (m - e):
            b += 1
    return b + m if both and d > 0 else b


def bucket_matrix(queries, keys, offset, buckets, reach, both):
    first = 1 - queries - offset
    of = torch.tensor([bucket(first + k, buckets, reach, both) for k in range(queries + keys - 1)])
    return torch.stack([of[queries - 1 - i:queries - 1 - i + keys] for i in range(queries)]).cuda()


SHAPES = [  # batch, heads, queries, keys, offset, buckets, reach, both
    (1, 1, 1, 1, 0, 2, 2, False),
    (2, 3, 1, 515, 514, 32, 128, False),
    (2, 1, 7, 5, 0, 4, 9, True),
    (3, 12, 33, 40, 7, 32, 128, True),
    (2, 2, 512, 512, 0, 32, 128, True),
    (5, 2, 200, 130, -11, 20, 60, False),
    (1, 2, 70, 2100, 2030, 64, 256, True),
    (70, 1, 17, 9, 0, 32, 100, True),
    (1, 300, 3, 2, 0, 256, 1000, True),
    (2, 1, 65, 33, 1000000000, 32, 128, True),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("batch,heads,queries,keys,offset,buckets,reach,both", SHAPES)
def test_relative_bias(gpu, batch, heads, queries, keys, offset, buckets, reach, both, dtype):
    flush_print(f"relative_bias {batch}x{heads}x{queries}x{keys} offset {offset} {buckets} {reach} {both} {dtype}")
    of = bucket_matrix(queries, keys, offset, buckets, reach, both)
    kind = dict(offset=offset, bidirectional=both, max_distance=reach)
    scores = randn(351, batch, heads, queries, keys, dtype=dtype, std=3.0)
    if keys > 1:
        scores[:, :, :, -1] = float("-inf")  # masked
    for param in {F32, dtype}:
        table = randn(350, buckets, heads, dtype=param)
        want = table.double().t()[:, of]
        got = A.relative_bias(table, queries, keys, dtype=dtype, **kind)
        within(got, want, U[dtype] * want.abs() + TINY[dtype] if dtype != param else 0.0 * want, "bias")
        want = want + scores.double()
        got = A.relative_bias(table, scores=scores, **kind)
        within(got, want, (U[dtype] + E) * want.abs() * 1.001 + TINY[dtype], "scores")
    # rows with gaps, a table with gaps, in place
    place = strided(scores.view(-1, keys))
    view = place._base.view(batch, heads, queries, -1)[..., 2:2 + keys]
    assert A.relative_bias(strided(table), scores=view, out=view, **kind) is view
    assert torch.equal(view, got)
    assert bool(place._base[:, :2].isnan().all()) and bool(place._base[:, 2 + keys:].isnan().all())


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
@pytest.mark.parametrize("batch,heads,queries,keys,offset,buckets,reach,both", SHAPES)
def test_relative_bias_grad(gpu, batch, heads, queries, keys, offset, buckets, reach, both, dtype):
    flush_print(f"relative_bias_grad {batch}x{heads}x{queries}x{keys} {offset} {buckets} {reach} {both} {dtype}")
    of = bucket_matrix(queries, keys, offset, buckets, reach, both).reshape(-1)
    kind = dict(offset=offset, bidirectional=both, max_distance=reach)
    ds = randn(352, batch, heads, queries, keys, dtype=dtype)
    flat = ds.double().reshape(batch, heads, -1)

    def sums(t):
        return torch.zeros(heads, buckets, dtype=torch.float64, device="cuda").index_add_(1, of, t.sum(0)).t()
    want, mag = sums(flat), sums(flat.abs())
    chain = min(batch * queries, 4096) + 17  # rows, groups of a workgroup, and the join's roundings
    for out in {F32, dtype}:
        got = A.relative_bias_grad(ds, buckets, dtype=out, **kind)
        within(got, want, chain * E * mag + (U[out] + E) * want.abs() + TINY[out], f"dtable {out}")
    # rows with gaps of NaN, added to a segment
    view = strided(ds.view(-1, keys))._base.view(batch, heads, queries, -1)[..., 2:2 + keys]
    seg = torch.zeros(buckets * heads + 6, dtype=dtype, device="cuda")
    out = seg[3:3 + buckets * heads]
    got = A.relative_bias_grad(ds, buckets, **kind)
    assert A.relative_bias_grad(view, buckets, out=out, accumulate=True, **kind) is out
    assert torch.equal(out.view(buckets, heads), got)
    assert not bool(seg[:3].any()) and not bool(seg[-3:].any())
    A.relative_bias_grad(ds, buckets, out=out, accumulate=True, **kind)
    twice = want + got.double()
    within(out.view(buckets, heads), twice, chain * E * mag + (U[dtype] + E) * twice.abs() + TINY[dtype], "added")


@pytest.mark.parametrize("buckets,reach,both", [(32, 128, True), (32, 128, False), (64, 4096, True), (6, 81, True),
                                                (256, 1 << 20, True), (255, 129, False), (4, 2, True), (3, 2, False),
                                                (12, 7, False), (16, 1 << 16, True)])
def test_borders_are_exact(gpu, buckets, reach, both):
    """Every border, many of them whole powers, at the distance itself and one
    before it: the table is its own index."""
    m = buckets // 2 if both else buckets
    e = m // 2
    at = {1, 2, reach - 1, reach, reach + 1}
    for k in range(e, m):
        x = e * (reach / e) ** ((k - e) / (m - e))
        at |= {max(1, round(x) + i) for i in (-1, 0, 1)}
    table = torch.arange(buckets, dtype=F32, device="cuda")[:, None]
    for n in sorted(at):
        want = [float(bucket(d, buckets, reach, both)) for d in (-n, -n + 1)]
        got = A.relative_bias(table, 1, 2, offset=n, bidirectional=both, max_distance=reach).view(-1).tolist()
        assert got == want, n
        if both:
            assert A.relative_bias(table, 1, 1, offset=-n, max_distance=reach).item() == bucket(n, buckets, reach, both)


def test_relative_bias_far_and_empty(gpu):
    table = randn(360, 32, 2)
    assert A.relative_bias(table, 0, 5).shape == (2, 0, 5)
    none = torch.empty(0, 2, 7, 5, device="cuda")
    assert A.relative_bias(table, scores=none).shape == none.shape
    grad = A.relative_bias_grad(none, 32)
    assert grad.shape == (32, 2) and not bool(grad.any())
    kept = torch.full((32, 2), 2.5, device="cuda")
    A.relative_bias_grad(none[..., :0, :], 32, out=kept, accumulate=True)
    assert bool((kept == 2.5).all())
    # a cache of more than 2^31 keys' offset: the far bucket on either side
    far = 2 ** 31 - 1
    got = A.relative_bias(table, 3, 4, offset=far)
    assert torch.equal(got, table[15][:, None, None].expand(2, 3, 4))
    assert torch.equal(A.relative_bias(table, 3, 4, offset=-far), table[31][:, None, None].expand(2, 3, 4))


@pytest.mark.parametrize("batch,heads,queries,keys,offset,buckets,reach,both", [
    (1, 3, 1, 70001, 70000, 32, 128, True),
    (1, 3, 1, 70001, -300, 32, 128, True),
    (2, 2, 5, 33000, 20000, 32, 128, True),
    (1, 1, 700, 2003, 0, 8, 20, False),
    (3, 1, 1025, 2047, 900, 256, 1000, True),
    (40, 2, 200, 700, 3, 32, 128, False),
])
def test_relative_bias_of_long_rows(gpu, batch, heads, queries, keys, offset, buckets, reach, both):
    """Tiles in one bucket, and buckets joined in pieces."""
    flush_print(f"long rows {batch}x{heads}x{queries}x{keys} {offset} {buckets} {reach} {both}")
    of = bucket_matrix(queries, keys, offset, buckets, reach, both)
    kind = dict(offset=offset, bidirectional=both, max_distance=reach)
    table = randn(363, buckets, heads)
    assert torch.equal(A.relative_bias(table, queries, keys, **kind), table.t()[:, of])
    ds = randn(364, batch, heads, queries, keys)
    flat = ds.double().reshape(batch, heads, -1)

    def sums(t):
        return torch.zeros(heads, buckets, dtype=torch.float64, device="cuda").index_add_(1, of.reshape(-1), t.sum(0)).t()
    want, mag = sums(flat), sums(flat.abs())
    got = A.relative_bias_grad(ds, buckets, **kind)
    within(got, want, (min(batch * queries, 4096) + 17) * E * mag + 2 * E * want.abs(), "dtable")
    assert torch.equal(A.relative_bias_grad(ds, buckets, **kind), got)
    seg = torch.full((buckets, heads), 1.5, device="cuda")
    A.relative_bias_grad(ds, buckets, out=seg, accumulate=True, **kind)
    within(seg, want + 1.5, (min(batch * queries, 4096) + 17) * E * mag + 2 * E * (want + 1.5).abs(), "added")


def test_relative_bias_grad_keeps_nan_in_its_bucket(gpu):
    ds = randn(361, 2, 3, 50, 60)
    want = A.relative_bias_grad(ds, 32)
    ds[1, 2, 49, 0] = float("nan")  # distance 49
    got = A.relative_bias_grad(ds, 32)
    bad = torch.zeros(32, 3, dtype=torch.bool, device="cuda")
    bad[bucket(-49, 32, 128, True), 2] = True
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])


def test_relative_bias_offsets_beyond_2_pow_31(gpu):
    """Scores whose elements lie behind the 2^31st."""
    batch, heads, queries, keys = 17, 16, 1024, 8200
    table = randn(362, 32, heads)
    scores = torch.empty(batch, heads, queries, keys, dtype=BF16, device="cuda").normal_()
    assert scores.numel() > 2 ** 31
    last = scores[-1].clone()
    of = bucket_matrix(8, keys, queries - 8, 32, 128, True)
    want = last[:, -8:].float() + table.t()[:, of]
    out = A.relative_bias(table, scores=scores, out=scores)
    assert torch.equal(out[-1, :, -8:], want.to(BF16))
    grad = A.relative_bias_grad(out, 32, dtype=F32)
    ref = torch.zeros(heads, 32, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    whole = bucket_matrix(queries, keys, 0, 32, 128, True)
    for n in range(batch):
        v = out[n].double()
        for b in range(32):
            there = v * (whole == b)
            ref[:, b] += there.sum((1, 2))
            mag[:, b] += there.abs_().sum((1, 2))
    within(grad, ref.t(), (4096 + 17) * E * mag.t() + 2 * E * ref.t().abs(), "dtable")


# ---------------------------------------------------------------- orthogonal updates

K = (3.4445, -4.7750, 2.0315)


def plain_orthogonal(x, coefficients=[K] * 5, eps=1e-7, scale=1.0):
    """In 64 bits, on the CPU's or the GPU's float64 products."""
    x = x.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.size(-2) > x.size(-1)
    if tall:
        x = x.transpose(-2, -1).contiguous()
    for a, b, c in coefficients:
        p = x @ x.transpose(-2, -1).contiguous()
        x = a * x + (b * p + c * (p @ p)) @ x
    return scale * (x.transpose(-2, -1) if tall else x)


def tolerance(out, k, steps):
    """Relative to the norm, with roundings taken as independent: a step's
    operands lose 2^-12 of themselves (two parts: 2^-22, and the sums sqrt(k)
    roundings), which the coefficients of the products, 4.775 + 2.0315, scale;
    the steps' errors add in squares; and the result is rounded."""
    part = 2.0 ** -12 if out == BF16 else 2.0 ** -22 + math.sqrt(k) * E
    return math.sqrt((6.81 * part) ** 2 * steps + U[out] ** 2 / 3)


def check_orthogonal(got, want, out, k, steps=5, what="orthogonal"):
    got, want = got.double(), want.double()
    far = float(((got - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)).max())
    limit = tolerance(out, k, steps)
    flush_print(f"  {what}: off by {far:.3g} of the norm, limit {limit:.3g}")
    assert far <= limit


def spectrum(seed, n, m, dtype, kind="normal", count=None):
    g = torch.randn(*(() if count is None else (count,)), n, m, generator=gen(seed), dtype=torch.float64)
    if kind == "strong":
        g = g + 3 * torch.randn(n, 2, generator=gen(seed + 1), dtype=torch.float64) @ torch.randn(
            2, m, generator=gen(seed + 2), dtype=torch.float64)
    if kind == "rank":
        g = torch.randn(n, 3, generator=gen(seed + 1), dtype=torch.float64) @ torch.randn(
            3, m, generator=gen(seed + 2), dtype=torch.float64)
    return (1e-3 * g).to(dtype).cuda()


@pytest.mark.parametrize("out", DTYPES, ids=ids)
@pytest.mark.parametrize("n,m", [(1, 1), (1, 300), (5, 3), (64, 64), (63, 65), (128, 128), (129, 130), (61, 769),
                                 (700, 33), (256, 500), (400, 257), (1000, 520)])
def test_orthogonalize(gpu, n, m, out):
    flush_print(f"orthogonalize {n}x{m} to {out}")
    for dtype in {F32, out}:
        for kind in ("normal", "strong") if min(n, m) > 3 else ("normal",):
            x = spectrum(400, n, m, dtype, kind)
            got = A.orthogonalize(x, dtype=out, scale=0.7)
            assert got.shape == x.shape and got.dtype == out
            check_orthogonal(got, plain_orthogonal(x, scale=float(np.float32(0.7))), out, max(n, m), what=f"{dtype} {kind}")


@pytest.mark.parametrize("out", DTYPES, ids=ids)
def test_orthogonalize_low_rank(gpu, out):
    """Directions that are not there stay away: rounding X to 16 bits alone
    would raise noise to 4e-2 of the norm.  (What fp32 itself does to X0 is
    raised by 3.4445^5 = 485: 485 * 2^-24 more.)"""
    x = spectrum(410, 300, 420, F32, "rank")
    got, want = A.orthogonalize(x, dtype=out).double(), plain_orthogonal(x)
    far = float((got - want).norm() / want.norm())
    flush_print(f"  rank 3 to {out}: off by {far:.3g}")
    assert far <= tolerance(out, 420, 5) + 485 * E


def test_orthogonalize_one_step_and_own_coefficients(gpu):
    """A step is the formula itself; coefficients may differ from step to step."""
    x = spectrum(420, 90, 140, F32)
    ks = [(3.0, -3.2, 1.2), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)]
    for steps in (1, 2, 3):
        got = A.orthogonalize(x, steps=steps, coefficients=ks[:steps])
        check_orthogonal(got, plain_orthogonal(x, ks[:steps]), F32, 140, steps)
    got = A.orthogonalize(x, steps=2, coefficients=ks[1])
    check_orthogonal(got, plain_orthogonal(x, [ks[1]] * 2), F32, 140, 2)
    # the cubic steps converge to the orthogonal factor
    got = A.orthogonalize(x, steps=16, coefficients=(1.5, -0.5, 0.0)).double()
    eye = got @ got.t().contiguous()
    within(eye, torch.eye(90, dtype=torch.float64), 1e-4, "orthogonal")


def test_orthogonalize_more_than_a_launch_takes(gpu):
    flush_print("131 matrices of 16 x 30")
    x = spectrum(429, 16, 30, F32, count=131)
    got = A.orthogonalize(x)
    for i in (0, 127, 128, 130):
        assert torch.equal(A.orthogonalize(x[i]), got[i])


def test_orthogonalize_many_and_lists(gpu):
    """Matrices do not notice each other: more than one launch takes, strided,
    in lists of shapes, in place, as segments of one buffer; bitwise."""
    for dtype in (F32, BF16):
        x = spectrum(430, 40, 70, dtype, count=37)
        got = A.orthogonalize(x)
        for i in (0, 31, 32, 36):
            assert torch.equal(A.orthogonalize(x[i]), got[i])
        wide = torch.full((37, 50, 90), float("nan"), dtype=dtype, device="cuda")
        view = wide[:, 3:43, 5:75]
        view.copy_(x)
        assert torch.equal(A.orthogonalize(view), got)
        assert A.orthogonalize(view, out=view) is view and torch.equal(view, got)
        mask = torch.ones_like(wide, dtype=torch.bool)
        mask[:, 3:43, 5:75] = False
        assert bool(wide[mask].isnan().all())
        shapes = [(40, 70), (70, 40), (40, 70), (9, 200), (1, 5)]
        flat = torch.zeros(sum(a * b for a, b in shapes) + 3, dtype=dtype, device="cuda")
        segs, at = [], 3  # segments start at any element
        for i, (a, b) in enumerate(shapes):
            segs.append(flat[at:at + a * b].view(a, b))
            segs[-1].copy_(spectrum(440 + i, a, b, dtype))
            at += a * b
        want = [A.orthogonalize(s.clone()) for s in segs]
        assert same(A.orthogonalize(segs), want)
        assert same(A.orthogonalize(segs, out=segs), want) and same(segs, want)
    assert A.orthogonalize([]) == []
    assert A.orthogonalize(x[:0]).shape == (0, 40, 70)
    assert A.orthogonalize(torch.empty(0, 5, device="cuda")).shape == (0, 5)


def test_orthogonalize_special_matrices(gpu):
    """Zeros stay zeros; an infinity or NaN fills its matrix only; scales that
    squares in fp32 would not survive; the transpose gives the transpose."""
    for out in DTYPES:
        x = spectrum(450, 70, 90, F32, count=6)
        want = A.orthogonalize(x, dtype=out)
        y = x.clone()
        y[1] = 0
        y[2, 3, 4] = float("nan")
        y[3, 69, 89] = float("inf")
        got = A.orthogonalize(y, dtype=out)
        assert same(got[[0, 4, 5]], want[[0, 4, 5]])
        assert not bool(got[1].any()) and bool(got[2:4].isnan().all())
        # eps = 2^-120 is 2^-26 of the smaller norm, which some roundings notice
        for f in (2.0 ** 100, 2.0 ** -90):
            a = A.orthogonalize(x * f, dtype=out, eps=2.0 ** -120)
            check_orthogonal(a, plain_orthogonal(x * f, eps=2.0 ** -120), out, 90)
        assert torch.equal(A.orthogonalize(x * 2.0 ** 100, dtype=out), A.orthogonalize(x * 2.0 ** 90, dtype=out))
        t = A.orthogonalize(x.transpose(1, 2).contiguous(), dtype=out)
        check_orthogonal(t.transpose(1, 2), plain_orthogonal(x), out, 90)
    # the narrow path
    x = spectrum(452, 20, 90, F32, count=5)
    for steps, k in ((5, K), (1, (1.5, -0.5, 0.0))):
        want = A.orthogonalize(x, steps=steps, coefficients=k)
        y = x.clone()
        y[1] = 0
        y[2, 3, 4] = float("nan")
        y[3, 19, 89] = float("inf")
        got = A.orthogonalize(y, steps=steps, coefficients=k)
        assert same(got[[0, 4]], want[[0, 4]]) and not bool(got[1].any()) and bool(got[2:4].isnan().all())
    # eps counts where the update is as small
    x = spectrum(451, 30, 40, F32) * 1e-6
    check_orthogonal(A.orthogonalize(x, eps=1e-6), plain_orthogonal(x, eps=1e-6), F32, 40)


def test_orthogonalize_large(gpu):
    """BERT-Large's matrices, one and as many as fill the card, against 64-bit
    products on the GPU: every tile that the kernels take."""
    for count, (n, m), dtype in ((1, (1024, 1024), BF16), (1, (4096, 1024), F32), (1, (1024, 4096), BF16),
                                 (24, (1024, 1024), BF16), (9, (1024, 1024), BF16), (8, (4096, 1024), BF16),
                                 (16, (1024, 1024), F16), (6, (4000, 1000), F32), (20, (300, 500), BF16),
                                 (33, (700, 260), BF16), (40, (64, 64), BF16), (33, (3, 2000), F32)):
        flush_print(f"orthogonalize {count}x{n}x{m} {dtype}")
        x = spectrum(460, n, m, dtype, "strong" if min(n, m) > 3 else "normal", count)
        got = A.orthogonalize(x)
        for i in {0, count // 2, count - 1}:
            check_orthogonal(got[i], plain_orthogonal(x[i]), dtype, max(n, m))
        if count > 1:  # bitwise the same for the same matrix
            x[0] = x[count - 1]
            got = A.orthogonalize(x)
            assert torch.equal(got[0], got[count - 1])


def test_orthogonalize_two_at_once(gpu):
    """Two calls on two streams, each with a workspace of its own."""
    x, y = spectrum(470, 300, 400, BF16, count=5), spectrum(471, 50, 900, F32, count=3)
    want = A.orthogonalize(x), A.orthogonalize(y)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (one, two):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        a = A.orthogonalize(x, stream=one)
        b = A.orthogonalize(y, stream=two)
        c = A.orthogonalize(x, stream=two)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[0])


# ---------------------------------------------------------------- together


def all_calls(seed, dtype):
    """Every new entry point on fixed inputs, with workspaces of their own."""
    rows, hidden = 300, 264
    x, res, dy = (randn(seed + i, rows, hidden, dtype=dtype) for i in range(3))
    w, table = randn(seed + 3, hidden), randn(seed + 4, 32, 4)
    scores = randn(seed + 5, 3, 4, 90, 101, dtype=dtype)
    update = spectrum(seed + 6, 140, 90, dtype, count=3)

    def run():
        y, codes, scales, h, rstd = A.rms_norm_pack(x, w, residual=res)
        dx, dw = A.rms_norm_grad(dy, h, rstd, w, dh=res)
        out = A.relative_bias(table, scores=scores, offset=11)
        dt = A.relative_bias_grad(scores, 32, offset=11)
        return [y, codes, scales, h, rstd, dx, dw, out, dt, A.orthogonalize(update)]
    return run


@pytest.mark.parametrize("dtype", DTYPES, ids=ids)
def test_captured_and_replayed(gpu, dtype):
    """Captured from the first call on; replays with eager work between them."""
    g = torch.cuda.CUDAGraph()
    run = all_calls(500, dtype)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = run()
    want = [t.clone() for t in run()]
    for _ in range(4):
        for t in captured:
            t.zero_()
        g.replay()
        assert same(run(), want)
        torch.cuda.synchronize()
        assert same(captured, want)


def test_streams_and_repeats(gpu):
    """Bitwise the same on repeats, on another stream, given and current."""
    run = all_calls(510, BF16)
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            got = run()
        side.synchronize()
        assert same(got, want) and same(run(), want)
    x, w = randn(520, 50, 70), randn(521, 70)
    y = A.rms_norm(x, w)
    up = spectrum(522, 60, 70, F32)
    o = A.orthogonalize(up)
    side.wait_stream(torch.cuda.current_stream())
    got, there = A.rms_norm(x, w, stream=side), A.orthogonalize(up, stream=side)
    side.synchronize()
    assert same(got, y) and torch.equal(there, o)


def test_given_workspaces(gpu):
    """A workspace that holds anything, larger than needed, used again."""
    L = _native.lib()
    dirty = torch.full((1 << 26,), 0xff, dtype=torch.uint8, device="cuda")
    x, dy, w = randn(530, 70, 100), randn(531, 70, 100), randn(532, 100)
    _, h, rstd = A.rms_norm(x, w)
    ds, up = randn(533, 2, 3, 40, 50), spectrum(534, 90, 61, F32, count=2)
    calls = [lambda ws: A.rms_norm_grad(dy, h, rstd, w, workspace=ws), lambda ws: [A.relative_bias_grad(ds, 8, workspace=ws)],
             lambda ws: [A.orthogonalize(up, workspace=ws)], lambda ws: [A.orthogonalize(up, dtype=BF16, workspace=ws)]]
    needs = [L.adasum_rms_grad_workspace_bytes(70, 100, 0), L.adasum_relative_bias_grad_workspace_bytes(2, 3, 40, 50, 0),
             L.adasum_orthogonalize_workspace_bytes(2, 90, 61, 0), L.adasum_orthogonalize_workspace_bytes(2, 90, 61, 2)]
    for call, need in zip(calls, needs):
        assert same(call(dirty), call(None))
        dirty.fill_(0xff)
        exact = torch.full((need + 16,), 0xff, dtype=torch.uint8, device="cuda")
        assert same(call(exact[:need]), call(None))
        assert bool((exact[need:] == 0xff).all())
        with pytest.raises(A.AdasumError, match="workspace"):
            call(dirty[:need - 1])
        with pytest.raises(A.AdasumError, match="aligned"):
            call(dirty[8:])


def test_a_training_step(gpu):
    """Workers' microbatches through a residual norm, attention scores with a
    learned bias and a linear layer whose gradient reads the packed rows; every
    gradient into its segment, the combine over the workers, and the combined
    matrices made orthogonal in place.  Against the same step in 64 bits."""
    workers, rows, hidden, out, heads, length, buckets = 4, 96, 72, 40, 3, 24, 8
    lengths = [hidden, buckets * heads, out * hidden, out]
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    w, lin = randn(540, hidden, mean=1.0, std=0.1), randn(541, out, hidden, std=0.1)
    table = randn(542, buckets, heads)
    of = bucket_matrix(length, length, 0, buckets, 16, True)
    kind = dict(max_distance=16)
    flats, exact = [], []
    for k in range(workers):
        x, res = randn(550 + k, rows, hidden), randn(560 + k, rows, hidden)
        dz = randn(570 + k, rows, out, std=1e-2)
        scores = randn(580 + k, 4, heads, length, length)
        flat = torch.empty(int(off[-1]), device="cuda")
        segs = [flat[off[i]:off[i + 1]] for i in range(4)]
        ref = [torch.zeros(n, dtype=torch.float64, device="cuda") for n in lengths]
        for half in range(2):
            acc, part = half == 1, slice(half * 48, half * 48 + 48)
            y, codes, scales, h, rstd = A.rms_norm_pack(x[part], w, residual=res[part])
            A.linear_grad(dz[part], codes, scales, dweight=segs[2], dbias=segs[3], accumulate=acc)
            dx, _ = A.rms_norm_grad(dz[part] @ lin, h, rstd, w, dweight=segs[0], accumulate=acc)
            s = A.relative_bias(table, scores=scores[2 * half:2 * half + 2], **kind)
            p = torch.softmax(s, -1)
            ds = p * (1 - p)  # some gradient of the scores
            A.relative_bias_grad(ds, buckets, out=segs[1], accumulate=acc, **kind)
            _, dw, _, _ = plain_rms_grad(dz[part].double() @ lin.double(), h, rstd, w, None)
            ref[0] += dw
            ref[1] += torch.zeros(heads, buckets, dtype=torch.float64, device="cuda").index_add_(
                1, of.view(-1), ds.double().sum(0).view(heads, -1)).t().reshape(-1)
            ref[2] += (dz[part].double().t() @ A.checkpoint_unpack(codes, scales).double()).reshape(-1)
            ref[3] += dz[part].double().sum(0)
        flats.append(flat)
        exact.append(torch.cat(ref).cpu().numpy())
    combined = A.combine(flats, off)
    want = oracle.combine(exact, off, out_format="f32")["out"]
    got = combined.double().cpu().numpy()
    for i in range(4):
        a, c = got[off[i]:off[i + 1]], want[off[i]:off[i + 1]]
        err = float(np.linalg.norm(a - c) / np.linalg.norm(c))
        flush_print(f"  segment {i}: relative L2 {err:.3g}")
        assert err <= 1e-5  # the combine's own tolerance; fp32 gradients are off by about 1e-6
    others = combined.clone()
    seg = combined[off[2]:off[3]].view(out, hidden)
    A.orthogonalize(seg, out=seg, scale=0.5)
    # the formula on what was combined
    check_orthogonal(seg, plain_orthogonal(others[off[2]:off[3]].view(out, hidden), scale=0.5), F32, hidden)
    assert torch.equal(combined[:off[2]], others[:off[2]]) and torch.equal(combined[off[3]:], others[off[3]:])


def test_overlaps_are_refused(gpu):
    raw = torch.zeros(1 << 16, device="cuda")
    a, b = raw[:600].view(6, 100), raw[500:1100].view(6, 100)
    w, stat = raw[2000:2100], raw[3000:3006]
    with pytest.raises(A.AdasumError, match="overlaps"):
        A.rms_norm(a, w, out=b)
    with pytest.raises(A.AdasumError, match="overlaps"):
        A.rms_norm(a, w, residual=raw[4000:4600].view(6, 100), h=raw[4100:4700].view(6, 100))
    with pytest.raises(A.AdasumError, match="overlaps"):
        A.rms_norm_grad(raw[4000:4600].view(6, 100), a, stat, w, dx=b)
    with pytest.raises(A.AdasumError, match="overlaps"):
        A.rms_norm_grad(raw[4000:4600].view(6, 100), a, stat, w, dweight=raw[550:650])
    with pytest.raises(A.AdasumError, match="overlaps"):
        A.relative_bias(raw[:64].view(32, 2), scores=raw[1000:1200].view(2, 10, 10), out=raw[1100:1300].view(2, 10, 10))
    with pytest.raises(A.AdasumError, match="overlaps"):
        A.relative_bias_grad(raw[:200].view(2, 10, 10), 32, out=raw[190:254])
    with pytest.raises(A.AdasumError, match=r"out\[0\] overlaps x\[0\]"):
        A.orthogonalize(raw[:200].view(2, 10, 10), out=raw[50:250].view(2, 10, 10))
    with pytest.raises(A.AdasumError, match="overlaps"):  # in place, and read as another matrix too
        A.orthogonalize([a, a], out=[a, raw[5000:5600].view(6, 100)])


def test_python_refusals(gpu):
    x, w = torch.zeros(6, 40, device="cuda"), torch.zeros(40, device="cuda")
    stat, table, s = torch.ones(6, device="cuda"), torch.zeros(32, 2, device="cuda"), torch.zeros(1, 2, 5, 7, device="cuda")
    bad = [lambda: A.rms_norm(x, w[:39]), lambda: A.rms_norm(x, residual=x[:5]), lambda: A.rms_norm(x, h=x),
           lambda: A.rms_norm(x, residual=x.to(F16)), lambda: A.rms_norm(x.double()), lambda: A.rms_norm(x.t()),
           lambda: A.rms_norm(x[:1].expand(6, 40)), lambda: A.rms_norm_pack(x, values=False, out=x.clone()),
           lambda: A.rms_norm(x, residual=x, h=x.to(F16)), lambda: A.rms_norm(x, out=x.to(F16)),
           lambda: A.rms_norm_grad(x, x, stat[:5]), lambda: A.rms_norm_grad(x, x[:5], stat),
           lambda: A.rms_norm_grad(x, x, stat, dweight=w), lambda: A.rms_norm_grad(x, x, stat, w, accumulate=True),
           lambda: A.rms_norm_grad(x, x, stat, w, dh=x.to(F16)), lambda: A.rms_norm_grad(x, x, stat, w, dx=x[:5]),
           lambda: A.relative_bias(table), lambda: A.relative_bias(table, 5, 0), lambda: A.relative_bias(table, -1, 5),
           lambda: A.relative_bias(table, 5, 7, scores=s), lambda: A.relative_bias(table, scores=s, dtype=F16),
           lambda: A.relative_bias(table[:, :1].contiguous(), scores=s), lambda: A.relative_bias(table, scores=s[0, 0]),
           lambda: A.relative_bias(w, 2, 3), lambda: A.relative_bias(table, 5, 7, out=s),
           lambda: A.relative_bias_grad(s, 32, accumulate=True), lambda: A.relative_bias_grad(s, 32, out=w),
           lambda: A.relative_bias_grad(s.transpose(2, 3), 32), lambda: A.relative_bias_grad(s[0, 0], 32),
           lambda: A.orthogonalize(w), lambda: A.orthogonalize(x.t()), lambda: A.orthogonalize(x[:1].expand(6, 40)),
           lambda: A.orthogonalize([x, x.to(F16)]), lambda: A.orthogonalize(x, steps=0),
           lambda: A.orthogonalize(x, coefficients=(1, 2)), lambda: A.orthogonalize(x, coefficients=[K] * 4),
           lambda: A.orthogonalize([x, x], out=[x]), lambda: A.orthogonalize(x, out=x[:5]),
           lambda: A.orthogonalize(x.double()), lambda: A.orthogonalize(x, dtype=torch.float64)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            flush_print(f"case {i} was not refused")
    for call in (lambda: A.orthogonalize(x, coefficients=(3.0, 0, 0)), lambda: A.relative_bias(table, 5, 7, max_distance=3),
                 lambda: A.relative_bias_grad(s, 1)):
        with pytest.raises(A.AdasumError):
            call()


def test_timed(gpu):
    run = all_calls(590, F32)
    run()
    torch.cuda.synchronize()
    _native.profile_begin()
    run()
    times = _native.profile_end()
    assert {k: v["launches"] for k, v in times.items()} == {"norm": 2, "bias": 2, "orthogonal": 1}


def test_lists_whose_calls_would_overwrite_each_other_are_refused(gpu):
    flush_print("outputs over another shape's matrices")
    raw = torch.randn(4096, device="cuda")
    a, b = raw[:60].view(6, 10), raw[64:164].view(10, 10)
    free = raw[1024:1124].view(10, 10)
    before = raw.clone()
    with pytest.raises(ValueError, match="overlaps"):
        A.orthogonalize([a, b], out=[raw[100:160].view(6, 10), free])
    with pytest.raises(ValueError, match="overlaps"):
        A.orthogonalize([a, b], out=[raw[2000:2060].view(6, 10), raw[2050:2150].view(10, 10)])
    assert torch.equal(raw, before)
    want = A.orthogonalize([a, b])
    got = A.orthogonalize([a, b], out=[a, b])
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
