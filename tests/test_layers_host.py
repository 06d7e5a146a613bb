"""Layer operators, host side: every entry point refuses invalid arguments
before any HIP call (no call here reaches a kernel), and the workspace sizes
and the Python front end's checks."""

import ctypes

import pytest
import torch

import distributed_sgd_gradient_amd as A
from distributed_sgd_gradient_amd import _native

BASE = 0x7F0000000000  # never dereferenced: validation fails first
F32, F16, BF16 = 0, 1, 2


def at(i):
    return BASE + (i << 32)


# Valid calls, as name -> value in the order of the C signature; every case
# below breaks one thing.
CALLS = {
    "adasum_embedding": dict(table=at(0), vocab=100, hidden=64, table_stride=64, table_dtype=F32, tokens=at(1),
                             token_bytes=8, n=10, scale=1.0, out=at(2), out_stride=64, out_dtype=F32, stream=None),
    "adasum_embedding_grad": dict(dy=at(0), n=10, hidden=64, dy_stride=64, dtype=F32, tokens=at(1), token_bytes=8,
                                  vocab=100, scale=1.0, grad=at(2), grad_dtype=F32, accumulate=0, workspace=at(3),
                                  workspace_bytes=1 << 30, stream=None),
    "adasum_layer_norm": dict(x=at(0), rows=10, hidden=64, x_stride=64, dtype=F32, weight=at(1), bias=at(2),
                              param_dtype=F32, eps=1e-5, y=at(3), y_stride=64, mean=at(4), rstd=at(5), codes=None,
                              scales=None, stream=None),
    "adasum_layer_norm_grad": dict(dy=at(0), rows=10, hidden=64, dy_stride=64, dtype=F32, x=at(1), x_stride=64,
                                   mean=at(2), codes=None, scales=None, rstd=at(3), weight=at(4), param_dtype=F32,
                                   dx=at(5), dx_stride=64, dweight=at(6), dbias=at(7), grad_dtype=F32, accumulate=0,
                                   workspace=at(8), workspace_bytes=1 << 30, stream=None),
    "adasum_checkpoint_pack": dict(x=at(0), rows=10, hidden=64, x_stride=64, dtype=F32, codes=at(1), scales=at(2),
                                   stream=None),
    "adasum_checkpoint_unpack": dict(codes=at(0), scales=at(1), rows=10, hidden=64, out=at(2), out_stride=64,
                                     dtype=F32, stream=None),
    "adasum_linear_grad": dict(dy=at(0), rows=10, out=64, dy_stride=64, dtype=F32, codes=at(1), scales=at(2), in_=64,
                               dweight=at(3), dbias=at(4), grad_dtype=F32, accumulate=0, workspace=at(5),
                               workspace_bytes=1 << 30, stream=None),
}

NAN, INF = float("nan"), float("inf")
BAD = [
    ("adasum_embedding", dict(table=None), "table is NULL"),
    ("adasum_embedding", dict(tokens=None), "tokens is NULL"),
    ("adasum_embedding", dict(out=None), "out is NULL"),
    ("adasum_embedding", dict(vocab=0), "vocab"),
    ("adasum_embedding", dict(vocab=(1 << 24) + 1), "vocab"),
    ("adasum_embedding", dict(hidden=0), "width"),
    ("adasum_embedding", dict(hidden=-1), "width"),
    ("adasum_embedding", dict(table_stride=63), "stride"),
    ("adasum_embedding", dict(hidden=(1 << 23) + 1, table_stride=1 << 24, out_stride=1 << 24), "2^23"),
    ("adasum_embedding_grad", dict(hidden=(1 << 23) + 1, dy_stride=1 << 24), "2^23"),
    ("adasum_embedding", dict(out_stride=63), "stride"),
    ("adasum_embedding", dict(n=-1), "rows"),
    ("adasum_embedding", dict(n=1 << 31), "rows"),
    ("adasum_embedding", dict(n=1 << 30, out_stride=1 << 20), "2^40"),
    ("adasum_embedding", dict(token_bytes=2), "token_bytes"),
    ("adasum_embedding", dict(table_dtype=3), "dtype"),
    ("adasum_embedding", dict(out_dtype=-1), "dtype"),
    ("adasum_embedding", dict(scale=INF), "scale"),
    ("adasum_embedding", dict(scale=1e39), "scale"),
    ("adasum_embedding", dict(table=at(0) + 2), "aligned"),
    ("adasum_embedding", dict(tokens=at(1) + 4), "aligned"),
    ("adasum_embedding", dict(out=at(0) + 100 * 64 * 4 - 4), "overlaps"),
    ("adasum_embedding", dict(out=at(1) + 8), "overlaps"),
    ("adasum_embedding_grad", dict(dy=None), "dy is NULL"),
    ("adasum_embedding_grad", dict(grad=None), "grad is NULL"),
    ("adasum_embedding_grad", dict(workspace=None), "workspace"),
    ("adasum_embedding_grad", dict(workspace_bytes=16), "workspace"),
    ("adasum_embedding_grad", dict(workspace=at(3) + 8), "aligned"),
    ("adasum_embedding_grad", dict(workspace=at(2)), "overlaps"),
    ("adasum_embedding_grad", dict(grad=at(0)), "overlaps"),
    ("adasum_embedding_grad", dict(scale=NAN), "scale"),
    ("adasum_embedding_grad", dict(vocab=0), "vocab"),
    ("adasum_embedding_grad", dict(vocab=0, n=0), "vocab"),
    ("adasum_embedding_grad", dict(dtype=7), "dtype"),
    ("adasum_embedding_grad", dict(grad_dtype=7), "dtype"),
    ("adasum_embedding_grad", dict(dy_stride=0), "stride"),
    ("adasum_embedding_grad", dict(token_bytes=0), "token_bytes"),
    ("adasum_layer_norm", dict(x=None), "x is NULL"),
    ("adasum_layer_norm", dict(y=None), "y is NULL"),
    ("adasum_layer_norm", dict(rstd=None), "rstd is NULL"),
    ("adasum_layer_norm", dict(hidden=16385, x_stride=16385, y_stride=16385), "16384"),
    ("adasum_layer_norm", dict(eps=0.0), "eps"),
    ("adasum_layer_norm", dict(eps=-1e-5), "eps"),
    ("adasum_layer_norm", dict(eps=1e-40), "eps"),
    ("adasum_layer_norm", dict(eps=NAN), "eps"),
    ("adasum_layer_norm", dict(codes=at(6)), "belong together"),
    ("adasum_layer_norm", dict(scales=at(6)), "belong together"),
    ("adasum_layer_norm", dict(y=at(0)), "overlaps"),
    ("adasum_layer_norm", dict(mean=at(5)), "overlaps"),
    ("adasum_layer_norm", dict(codes=at(6), scales=at(6) + 639), "overlaps"),
    ("adasum_layer_norm", dict(param_dtype=3), "param_dtype"),
    ("adasum_layer_norm", dict(rstd=at(5) + 2), "aligned"),
    ("adasum_layer_norm_grad", dict(dy=None), "dy is NULL"),
    ("adasum_layer_norm_grad", dict(mean=None), "mean is NULL"),
    ("adasum_layer_norm_grad", dict(x=None), "mean belongs to x"),
    ("adasum_layer_norm_grad", dict(x=None, mean=None), "codes is NULL"),
    ("adasum_layer_norm_grad", dict(codes=at(9)), "not both"),
    ("adasum_layer_norm_grad", dict(rstd=None), "rstd is NULL"),
    ("adasum_layer_norm_grad", dict(dx=None), "dx is NULL"),
    ("adasum_layer_norm_grad", dict(dx=at(0)), "overlaps"),
    ("adasum_layer_norm_grad", dict(dbias=at(6)), "overlaps"),
    ("adasum_layer_norm_grad", dict(workspace=None), "workspace"),
    ("adasum_layer_norm_grad", dict(workspace_bytes=0), "workspace"),
    ("adasum_layer_norm_grad", dict(grad_dtype=5), "grad_dtype"),
    ("adasum_layer_norm_grad", dict(param_dtype=5), "param_dtype"),
    ("adasum_layer_norm_grad", dict(dx_stride=10), "stride"),
    ("adasum_layer_norm_grad", dict(x_stride=10), "stride"),
    ("adasum_checkpoint_pack", dict(x=None), "x is NULL"),
    ("adasum_checkpoint_pack", dict(codes=None), "codes is NULL"),
    ("adasum_checkpoint_pack", dict(scales=None), "scales is NULL"),
    ("adasum_checkpoint_pack", dict(codes=at(0) + 1), "overlaps"),
    ("adasum_checkpoint_pack", dict(x_stride=1), "stride"),
    ("adasum_checkpoint_pack", dict(rows=-5), "rows"),
    ("adasum_checkpoint_unpack", dict(out=None), "out is NULL"),
    ("adasum_checkpoint_unpack", dict(out=at(1) - 4), "overlaps"),
    ("adasum_checkpoint_unpack", dict(dtype=9), "dtype"),
    ("adasum_linear_grad", dict(dy_stride=(1 << 28) + 1), "2^28"),
    ("adasum_linear_grad", dict(dy=None), "dy is NULL"),
    ("adasum_linear_grad", dict(dweight=None), "dweight is NULL"),
    ("adasum_linear_grad", dict(in_=0), "in_features"),
    ("adasum_linear_grad", dict(out=0), "width"),
    ("adasum_linear_grad", dict(dbias=at(3) + 4), "overlaps"),
    ("adasum_linear_grad", dict(rows=1 << 20, workspace=None), "workspace"),
    ("adasum_linear_grad", dict(rows=1 << 20, workspace_bytes=1), "workspace"),
    ("adasum_linear_grad", dict(out=1 << 20, dy_stride=1 << 20, in_=1 << 20), "too large"),
    ("adasum_linear_grad", dict(out=1 << 24, dy_stride=1 << 24, in_=1 << 24), "2^40"),
    ("adasum_linear_grad", dict(grad_dtype=3), "grad_dtype"),
]


@pytest.mark.parametrize("case", range(len(BAD)), ids=lambda i: f"{BAD[i][0][7:]}-{next(iter(BAD[i][1]))}-{i}")
def test_refusals(case):
    name, change, text = BAD[case]
    lib = _native.lib()
    args = {**CALLS[name], **change}
    assert set(args) == set(CALLS[name])
    rc = getattr(lib, name)(*args.values())
    assert rc == _native.EINVAL
    assert text in lib.adasum_last_error().decode()


@pytest.mark.parametrize("name", ["adasum_embedding", "adasum_layer_norm", "adasum_checkpoint_pack",
                                  "adasum_checkpoint_unpack"])
def test_no_rows_is_no_work(name):
    args = {k: (None if isinstance(v, int) and v >= BASE else v) for k, v in CALLS[name].items()}
    args["n" if "n" in args else "rows"] = 0
    assert getattr(_native.lib(), name)(*args.values()) == _native.OK


@pytest.mark.parametrize("name", ["adasum_embedding_grad", "adasum_layer_norm_grad", "adasum_linear_grad"])
def test_no_rows_added_is_no_work(name):
    args = {**CALLS[name], "accumulate": 1}
    args["n" if "n" in args else "rows"] = 0
    assert getattr(_native.lib(), name)(*args.values()) == _native.OK


def test_workspace_sizes():
    lib = _native.lib()
    assert lib.adasum_layer_norm_grad_workspace_bytes(0, 64, F32) == 0
    assert lib.adasum_layer_norm_grad_workspace_bytes(5, 64, F32) >= 2 * 64 * 4
    assert lib.adasum_layer_norm_grad_workspace_bytes(5, 20000, F32) == _native.EINVAL
    assert lib.adasum_linear_grad_workspace_bytes(1, 8, 8, BF16) >= 8 * 8 * 4
    assert lib.adasum_linear_grad_workspace_bytes(1 << 16, 1024, 1024, BF16) >= 2 * 1024 * 1024 * 4
    assert lib.adasum_linear_grad_workspace_bytes(1, 8, 8, 5) == _native.EINVAL
    # two int32 lists of n, and partial sums
    assert lib.adasum_embedding_grad_workspace_bytes(1000, 64, F32) >= 8 * 1000
    assert lib.adasum_embedding_grad_workspace_bytes(-1, 64, F32) == _native.EINVAL
    small = [lib.adasum_embedding_grad_workspace_bytes(n, h, d) for n in (0, 1, 7, 4096) for h in (1, 63, 1024)
             for d in (F32, F16, BF16)]
    assert all(b > 0 for b in small)


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 8)
    c, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8)
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: A.embedding(x, t), lambda: A.embedding_grad(x, t, 5), lambda: A.layer_norm(x),
                 lambda: A.layer_norm_keep(x), lambda: A.layer_norm_grad(x, x, x[:, 0], x[:, 0]),
                 lambda: A.layer_norm_keep_grad(x, c, s, x[:, 0]), lambda: A.checkpoint_pack(x),
                 lambda: A.checkpoint_unpack(c, s), lambda: A.linear_grad(x, c, s)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_every_layer_entry_point_is_covered():
    skip = {"adasum_embedding_grad_workspace_bytes", "adasum_layer_norm_grad_workspace_bytes",
            "adasum_linear_grad_workspace_bytes"}
    layer = {n for n in _native.SIGNATURES if any(w in n for w in ("embedding", "norm", "checkpoint", "linear"))}
    assert layer - skip == set(CALLS)
    for name in CALLS:
        assert len(CALLS[name]) == len(_native.SIGNATURES[name][1])
        assert _native.SIGNATURES[name][0] is ctypes.c_int


@pytest.mark.parametrize("rows,hidden,together", [(1 << 27, 2, 16), (1 << 24, 256, 16), (1 << 24, 1000, 4),
                                                  (1 << 22, 4000, 1), (1 << 20, 16384, 1)])
def test_layer_norm_grad_sums_are_bounded(rows, hidden, together):
    """A partial sum of dweight and dbias for every 1024 rows of each of the
    `together` rows that a workgroup takes at a time."""
    parts = -(-rows // (1024 * together))
    assert _native.lib().adasum_layer_norm_grad_workspace_bytes(rows, hidden, F32) >= parts * 2 * hidden * 4


@pytest.mark.parametrize("rows,out,width,dtype", [(1 << 20, 30522, 1024, BF16), (65537, 32768, 1024, F16),
                                                  (1 << 18, 1024, 16384, F32)])
def test_linear_grad_sums_are_bounded(rows, out, width, dtype):
    """A partial sum of dweight for every 65536 rows."""
    parts = -(-rows // 65536)
    assert parts > 1
    assert _native.lib().adasum_linear_grad_workspace_bytes(rows, out, width, dtype) >= parts * out * width * 4
