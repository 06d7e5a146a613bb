"""Residual norm, relative bias and orthogonal updates, host side: every entry
point refuses invalid arguments before any HIP call (no call here reaches a
kernel), and the workspace sizes and the Python front end's checks."""

import ctypes

import pytest
import torch

import distributed_sgd_gradient_amd as A
from distributed_sgd_gradient_amd import _native
from test_layers_host import BF16, F16, F32, INF, NAN, at

GOOD = (3.4445, -4.7750, 2.0315)


def coefficients(*k):
    return (ctypes.c_double * len(k))(*k)


def pointers(*p):
    return (ctypes.c_void_p * len(p))(*p)


# Valid calls, as name -> value in the order of the C signature; every case
# below breaks one thing.
CALLS = {
    "adasum_rms": dict(x=at(0), rows=10, hidden=64, x_stride=64, dtype=BF16, residual=at(1), residual_stride=64,
                       stream_dtype=F32, weight=at(2), param_dtype=F32, eps=1e-6, y=at(3), y_stride=64, h=at(4),
                       h_stride=64, rstd=at(5), codes=at(6), scales=at(7), stream=None),
    "adasum_rms_grad": dict(dy=at(0), rows=10, hidden=64, dy_stride=64, dtype=BF16, h=at(1), h_stride=64,
                            stream_dtype=F32, dh=at(2), dh_stride=64, rstd=at(3), weight=at(4), param_dtype=F32,
                            dx=at(5), dx_stride=64, dweight=at(6), grad_dtype=F32, accumulate=0, workspace=at(7),
                            workspace_bytes=1 << 30, stream=None),
    "adasum_relative_bias": dict(table=at(0), buckets=32, heads=4, table_stride=4, table_dtype=F32, max_distance=128,
                                 bidirectional=1, batch=2, queries=10, keys=20, offset=3, scores=at(1),
                                 scores_stride=20, out=at(2), out_stride=20, dtype=F32, stream=None),
    "adasum_relative_bias_grad": dict(dscores=at(0), batch=2, heads=4, queries=10, keys=20, stride=20, dtype=F32,
                                      offset=3, buckets=32, max_distance=128, bidirectional=1, dtable=at(1),
                                      grad_dtype=F32, accumulate=0, workspace=at(2), workspace_bytes=1 << 30,
                                      stream=None),
    "adasum_orthogonalize": dict(x=pointers(at(0), at(1)), count=2, rows=30, cols=40, x_stride=40, dtype=F32, steps=2,
                                 coefficients=coefficients(*GOOD, *GOOD), eps=1e-7, scale=1.0,
                                 out=pointers(at(2), at(3)), out_stride=40, out_dtype=F32, workspace=at(4),
                                 workspace_bytes=1 << 30, stream=None),
}

BAD = [
    ("adasum_rms", dict(x=None), "x is NULL"),
    ("adasum_rms", dict(y=None, codes=None, scales=None), "y is NULL"),
    ("adasum_rms", dict(rstd=None), "rstd is NULL"),
    ("adasum_rms", dict(hidden=16385, x_stride=1 << 15, residual_stride=1 << 15, y_stride=1 << 15, h_stride=1 << 15),
     "16384"),
    ("adasum_rms", dict(hidden=0), "width"),
    ("adasum_rms", dict(rows=-1), "rows"),
    ("adasum_rms", dict(rows=1 << 31), "rows"),
    ("adasum_rms", dict(rows=1 << 30, x_stride=1 << 20), "2^40"),
    ("adasum_rms", dict(x_stride=63), "stride"),
    ("adasum_rms", dict(residual_stride=63), "stride"),
    ("adasum_rms", dict(y_stride=63), "stride"),
    ("adasum_rms", dict(h_stride=63), "stride"),
    ("adasum_rms", dict(eps=0.0), "eps"),
    ("adasum_rms", dict(eps=1e-40), "eps"),
    ("adasum_rms", dict(eps=NAN), "eps"),
    ("adasum_rms", dict(eps=INF), "eps"),
    ("adasum_rms", dict(dtype=3), "dtype"),
    ("adasum_rms", dict(stream_dtype=F16), "stream_dtype"),
    ("adasum_rms", dict(param_dtype=3), "param_dtype"),
    ("adasum_rms", dict(codes=None), "belong together"),
    ("adasum_rms", dict(scales=None), "belong together"),
    ("adasum_rms", dict(residual=None), "without a residual"),
    ("adasum_rms", dict(residual=None, h=None), "without a residual"),
    ("adasum_rms", dict(h=at(1), h_stride=65), "overlaps"),
    ("adasum_rms", dict(h=at(1) + 4), "overlaps"),
    ("adasum_rms", dict(y=at(0)), "overlaps"),
    ("adasum_rms", dict(rstd=at(6) + 600), "overlaps"),
    ("adasum_rms", dict(rstd=at(5) + 2), "aligned"),
    ("adasum_rms", dict(weight=at(2) + 2), "aligned"),
    ("adasum_rms_grad", dict(dy=None), "dy is NULL"),
    ("adasum_rms_grad", dict(h=None), "h is NULL"),
    ("adasum_rms_grad", dict(rstd=None), "rstd is NULL"),
    ("adasum_rms_grad", dict(dx=None), "dx is NULL"),
    ("adasum_rms_grad", dict(dx=at(1)), "overlaps"),
    ("adasum_rms_grad", dict(dx=at(2), dx_stride=65), "overlaps"),
    ("adasum_rms_grad", dict(dweight=at(5)), "overlaps"),
    ("adasum_rms_grad", dict(stream_dtype=F16), "stream_dtype"),
    ("adasum_rms_grad", dict(param_dtype=-1), "param_dtype"),
    ("adasum_rms_grad", dict(grad_dtype=4), "grad_dtype"),
    ("adasum_rms_grad", dict(dh_stride=1), "stride"),
    ("adasum_rms_grad", dict(dx_stride=1), "stride"),
    ("adasum_rms_grad", dict(hidden=20000, dy_stride=20000, h_stride=20000, dh_stride=20000, dx_stride=20000), "16384"),
    ("adasum_rms_grad", dict(workspace=None), "workspace"),
    ("adasum_rms_grad", dict(workspace_bytes=8), "workspace"),
    ("adasum_rms_grad", dict(workspace=at(7) + 8), "aligned"),
    ("adasum_relative_bias", dict(table=None), "table is NULL"),
    ("adasum_relative_bias", dict(out=None), "out is NULL"),
    ("adasum_relative_bias", dict(buckets=1, bidirectional=0), "buckets"),
    ("adasum_relative_bias", dict(buckets=2), "buckets"),
    ("adasum_relative_bias", dict(buckets=33), "buckets"),
    ("adasum_relative_bias", dict(buckets=258), "buckets"),
    ("adasum_relative_bias", dict(max_distance=8), "max_distance"),
    ("adasum_relative_bias", dict(max_distance=16, bidirectional=0), "max_distance"),
    ("adasum_relative_bias", dict(max_distance=(1 << 30) + 1), "max_distance"),
    ("adasum_relative_bias", dict(heads=0), "heads"),
    ("adasum_relative_bias", dict(batch=-1), "batch"),
    ("adasum_relative_bias", dict(queries=-1), "queries"),
    ("adasum_relative_bias", dict(keys=0), "keys"),
    ("adasum_relative_bias", dict(offset=1 << 31), "offset"),
    ("adasum_relative_bias", dict(offset=-(1 << 31)), "offset"),
    ("adasum_relative_bias", dict(table_stride=3), "stride"),
    ("adasum_relative_bias", dict(scores_stride=19), "stride"),
    ("adasum_relative_bias", dict(out_stride=19), "stride"),
    ("adasum_relative_bias", dict(batch=1 << 20, queries=1 << 10), "2^31"),
    ("adasum_relative_bias", dict(heads=1 << 27, table_stride=1 << 27, queries=1, keys=1), "too large"),
    ("adasum_relative_bias", dict(table_dtype=5), "dtype"),
    ("adasum_relative_bias", dict(dtype=5), "dtype"),
    ("adasum_relative_bias", dict(out=at(1) + 4), "overlaps"),
    ("adasum_relative_bias", dict(out=at(1), out_stride=21), "overlaps"),
    ("adasum_relative_bias", dict(out=at(0)), "overlaps"),
    ("adasum_relative_bias", dict(scores=at(1) + 1), "aligned"),
    ("adasum_relative_bias_grad", dict(dscores=None), "dscores is NULL"),
    ("adasum_relative_bias_grad", dict(dtable=None), "dtable is NULL"),
    ("adasum_relative_bias_grad", dict(dtable=at(0)), "overlaps"),
    ("adasum_relative_bias_grad", dict(stride=19), "stride"),
    ("adasum_relative_bias_grad", dict(grad_dtype=3), "dtype"),
    ("adasum_relative_bias_grad", dict(buckets=0), "buckets"),
    ("adasum_relative_bias_grad", dict(max_distance=0), "max_distance"),
    ("adasum_relative_bias_grad", dict(heads=1 << 17, queries=1, keys=1), "too large"),
    ("adasum_relative_bias_grad", dict(workspace=None), "workspace"),
    ("adasum_relative_bias_grad", dict(workspace_bytes=64), "workspace"),
    ("adasum_orthogonalize", dict(x=None), "x is NULL"),
    ("adasum_orthogonalize", dict(out=None), "out is NULL"),
    ("adasum_orthogonalize", dict(x=pointers(at(0), None)), "x[1] is NULL"),
    ("adasum_orthogonalize", dict(out=pointers(None, at(2))), "out[0] is NULL"),
    ("adasum_orthogonalize", dict(x=pointers(at(0), at(1) + 2)), "x[1] is not aligned"),
    ("adasum_orthogonalize", dict(out=pointers(at(2), at(2))), "overlaps"),
    ("adasum_orthogonalize", dict(out=pointers(at(2), at(0) + 4)), "overlaps"),
    ("adasum_orthogonalize", dict(out=pointers(at(0), at(1)), out_stride=41), "overlaps"),
    ("adasum_orthogonalize", dict(out=pointers(at(1), at(0))), "overlaps"),
    ("adasum_orthogonalize", dict(out=pointers(at(2), at(4))), "overlaps"),
    ("adasum_orthogonalize", dict(count=-1), "count"),
    ("adasum_orthogonalize", dict(count=(1 << 16) + 1), "count"),
    ("adasum_orthogonalize", dict(rows=-1), "rows"),
    ("adasum_orthogonalize", dict(rows=(1 << 15) + 1), "rows"),
    ("adasum_orthogonalize", dict(cols=0), "cols"),
    ("adasum_orthogonalize", dict(cols=(1 << 15) + 1), "cols"),
    ("adasum_orthogonalize", dict(x_stride=39), "stride"),
    ("adasum_orthogonalize", dict(out_stride=39), "stride"),
    ("adasum_orthogonalize", dict(dtype=3), "dtype"),
    ("adasum_orthogonalize", dict(out_dtype=3), "dtype"),
    ("adasum_orthogonalize", dict(steps=0), "steps"),
    ("adasum_orthogonalize", dict(steps=17), "steps"),
    ("adasum_orthogonalize", dict(coefficients=None), "coefficients"),
    ("adasum_orthogonalize", dict(coefficients=coefficients(*GOOD, NAN, 0, 0)), "finite"),
    ("adasum_orthogonalize", dict(coefficients=coefficients(2.0, 0, 0, 1, 0, 0)), "below 2"),
    ("adasum_orthogonalize", dict(coefficients=coefficients(*GOOD, 3.4445, 0.0, 2.0315)), "below 2"),
    ("adasum_orthogonalize", dict(coefficients=coefficients(1.0, -32.0, 31.0, 1, 0, 0)), "below"),
    ("adasum_orthogonalize", dict(coefficients=coefficients(1.5, -0.5, 0, 3.4445, -4.7750, 12.0)), "below 2"),
    ("adasum_orthogonalize", dict(eps=0.0), "eps"),
    ("adasum_orthogonalize", dict(eps=NAN), "eps"),
    ("adasum_orthogonalize", dict(scale=INF), "scale"),
    ("adasum_orthogonalize", dict(workspace=None), "workspace"),
    ("adasum_orthogonalize", dict(workspace_bytes=1), "workspace"),
    ("adasum_orthogonalize", dict(workspace=at(4) + 8), "aligned"),
]


@pytest.mark.parametrize("case", range(len(BAD)), ids=lambda i: f"{BAD[i][0][7:]}-{next(iter(BAD[i][1]))}-{i}")
def test_refusals(case):
    name, change, text = BAD[case]
    lib = _native.lib()
    args = {**CALLS[name], **change}
    assert set(args) == set(CALLS[name])
    assert getattr(lib, name)(*args.values()) == _native.EINVAL
    assert text in lib.adasum_last_error().decode()


def test_every_entry_point_is_covered():
    new = {n for n in _native.SIGNATURES if any(w in n for w in ("rms", "relative", "orthogonal")) and
           not n.endswith("bytes")}
    assert new == set(CALLS)
    for name in CALLS:
        assert len(CALLS[name]) == len(_native.SIGNATURES[name][1])


def test_nothing_is_no_work():
    lib = _native.lib()
    for name, empty in (("adasum_rms", dict(rows=0)), ("adasum_rms_grad", dict(rows=0, accumulate=1)),
                        ("adasum_relative_bias", dict(batch=0)), ("adasum_relative_bias", dict(queries=0)),
                        ("adasum_relative_bias_grad", dict(queries=0, accumulate=1)),
                        ("adasum_orthogonalize", dict(count=0)), ("adasum_orthogonalize", dict(rows=0))):
        assert getattr(lib, name)(*{**CALLS[name], **empty}.values()) == _native.OK


def test_coefficients_that_are_allowed():
    """All of these keep singular values below 2: refused for the workspace
    only, which is checked after them."""
    for k in (GOOD, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (1.0, 0.0, 0.0), (0.0, 0.0, 0.0), (-1.0, 0.0, 0.0)):
        args = {**CALLS["adasum_orthogonalize"], "steps": 16, "coefficients": coefficients(*(k * 16)), "workspace": None}
        assert _native.lib().adasum_orthogonalize(*args.values()) == _native.EINVAL
        assert "workspace" in _native.lib().adasum_last_error().decode()


def test_workspace_sizes():
    lib = _native.lib()
    assert lib.adasum_rms_grad_workspace_bytes(0, 64, F32) == 0
    assert lib.adasum_rms_grad_workspace_bytes(5, 64, F32) >= 64 * 4
    assert lib.adasum_rms_grad_workspace_bytes(5, 20000, F32) == _native.EINVAL
    for rows, hidden, together in ((1 << 27, 2, 16), (1 << 24, 1000, 4), (1 << 20, 16384, 1)):
        parts = -(-rows // (1024 * together))  # a partial sum for every 1024 rows that a workgroup takes at a time
        assert lib.adasum_rms_grad_workspace_bytes(rows, hidden, BF16) >= parts * hidden * 4
    assert lib.adasum_relative_bias_grad_workspace_bytes(2, 3, 10, 20, F32) >= 3 * 29 * 4
    assert lib.adasum_relative_bias_grad_workspace_bytes(0, 3, 10, 20, F32) >= 3 * 29 * 4
    assert lib.adasum_relative_bias_grad_workspace_bytes(2, 0, 10, 20, F32) == _native.EINVAL
    # an fp32 sum for every 4096 rows that a group of lanes takes
    assert lib.adasum_relative_bias_grad_workspace_bytes(1 << 18, 1, 64, 64, F32) >= (1 << 18) // 64 // 16 * 127 * 4
    assert lib.adasum_orthogonalize_workspace_bytes(0, 30, 40, F32) == 0
    assert lib.adasum_orthogonalize_workspace_bytes(1, 0, 40, F32) == 0
    one = lib.adasum_orthogonalize_workspace_bytes(1, 1000, 600, F32)
    assert one >= 2 * (4 * 1000 * 600 + 2 * 600 * 600)
    assert lib.adasum_orthogonalize_workspace_bytes(1, 600, 1000, F32) == one
    # the widest: 16 bytes of X's parts and, in two parts, 8 of A and 8 of B for each element; one at a time
    side = 1 << 15
    most = lib.adasum_orthogonalize_workspace_bytes(1 << 16, side, side, F32)
    assert 16 * side * side <= most <= 20 * side * side
    assert lib.adasum_orthogonalize_workspace_bytes(1 << 16, 4096, 4096, BF16) <= 4 << 30
    # matrices of one call take turns
    assert lib.adasum_orthogonalize_workspace_bytes(1 << 16, 1000, 600, F32) <= 64 * one
    assert lib.adasum_orthogonalize_workspace_bytes(1, 30, 1 << 16, F32) == _native.EINVAL
    assert lib.adasum_orthogonalize_workspace_bytes(1, 30, 40, 9) == _native.EINVAL


def test_python_refuses():
    x, s = torch.zeros(4, 8), torch.zeros(2, 3, 8)
    for call in (lambda: A.rms_norm(x), lambda: A.rms_norm_pack(x), lambda: A.rms_norm_grad(x, x, x[:, 0]),
                 lambda: A.relative_bias(x, 2, 3), lambda: A.relative_bias(x, scores=s),
                 lambda: A.relative_bias_grad(s, 32), lambda: A.orthogonalize(x), lambda: A.orthogonalize([x, x])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_matrices_of_other_shapes_stay_apart():
    from distributed_sgd_gradient_amd.updates import _apart

    small, large = (4, 8, 8, 8), (8, 8, 8, 8)  # 128 and 256 bytes of fp32
    _apart({small: ([0], [0]), large: ([128], [128])}, 4, 4, None)  # in place, one behind the other
    _apart({small: ([0], [1024]), large: ([0], [2048])}, 4, 4, None)  # one input read twice
    for x, y in (([0, 128], [128, 1024]), ([0, 128], [1024, 124]), ([0, 512], [1024, 1148])):
        with pytest.raises(ValueError, match="overlaps"):
            _apart({small: (x[:1], y[:1]), large: (x[1:], y[1:])}, 4, 4, None)
    space = torch.empty(64, dtype=torch.uint8)
    at = space.data_ptr()
    _apart({small: ([at - 128], [at - 128]), large: ([at + 64], [at + 64])}, 4, 4, space)
    with pytest.raises(ValueError, match="overlaps"):
        _apart({small: ([at - 128], [at - 128]), large: ([at + 60], [at + 60])}, 4, 4, space)
