"""Python front end of what becomes of a combined gradient: updates whose
matrices are made orthogonal.  Conventions as for the layer operators."""

import ctypes

import torch

from . import _native
from .layers import _call, _code, _like, _on, _ptr, _size, _workspace

STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(t, name, dev):
    """([address], rows, cols, row stride) of [..., rows, cols]."""
    _on(t, name, dev)
    if t.dim() < 2 or t.size(-1) < 1:
        raise ValueError(f"{name} must be [..., rows, cols] with a column at least")
    rows, cols = t.size(-2), t.size(-1)
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be consecutive")
    stride = t.stride(-2) if rows > 1 else cols
    if stride < cols:
        raise ValueError(f"{name}: rows overlap (an expanded tensor: make it contiguous)")
    if t.numel() == 0:
        return [], rows, cols, cols
    at = [t.data_ptr()]
    for n, s in zip(t.shape[:-2], t.stride()[:-2]):
        at = [a + i * s * t.element_size() for a in at for i in range(n)]
    return at, rows, cols, stride


def _coefficients(coefficients, steps):
    """3 * steps numbers, from one triple for all steps or one for each."""
    k = [c for c in coefficients]
    if k and not hasattr(k[0], "__len__"):
        k = [k] * steps
    if len(k) != steps or any(len(c) != 3 for c in k):
        raise ValueError("coefficients must be (a, b, c), or one such triple for each step")
    return (ctypes.c_double * (3 * steps))(*[float(v) for c in k for v in c])


def _apart(calls, x_size, out_size, workspace):
    """Refuses what only the calls of different shapes together overwrite: a
    matrix that another call writes before it is read, or an output twice.  (A
    call of its own looks at its own matrices.)  Rows of one pitch may lie between
    each other's, as column slices of one matrix do."""
    spans = []  # begin, end, written, bytes of a row, of a row and the gap behind it, name
    for (rows, cols, stride, out_stride), (x, y) in calls.items():
        sizes = [(((rows - 1) * s + cols) * n, cols * n, s * n) for s, n in ((stride, x_size), (out_stride, out_size))]
        for a, b in zip(x, y):
            if a != b or stride != out_stride or x_size != out_size:  # not in place
                spans.append((a, a + sizes[0][0], False, *sizes[0][1:], "update"))
            spans.append((b, b + sizes[1][0], True, *sizes[1][1:], "out"))
    if workspace is not None and _size(workspace):
        at, size = workspace.data_ptr(), _size(workspace)
        spans.append((at, at + size, True, size, size, "workspace"))
    reaching = ([], [])  # up to here, of what is read, of what is written
    for span in sorted(spans):
        begin, end, written, width, pitch, name = span
        for kind in (0, 1) if written else (1,):
            reaching[kind][:] = [s for s in reaching[kind] if s[1] > begin]
            for other in reaching[kind]:
                at, last, _, row, gap, other_name = other
                one_row = last - at == row or (end - begin != width and gap != pitch)
                d = (begin - at) % gap
                if one_row or d < row or d + width > gap:
                    raise ValueError(f"{name} overlaps {other_name} of another matrix")
        if not reaching[written] or reaching[written][-1] != span:  # read many times: once
            reaching[written].append(span)


def orthogonalize(update, *, steps=STEPS, coefficients=COEFFICIENTS, eps=1e-7, scale=1.0, dtype=None, out=None,
                  workspace=None, stream=None):
    """Matrices brought near the closest orthogonal ones by Newton-Schulz steps,
    for an update whose directions all count alike: X = update / (its Frobenius
    norm + eps), then ``steps`` times X = a X + (b A + c A^2) X with A = X X^T (of
    a matrix with more rows than columns, of its transpose); the result is
    scale * X.

    update: [..., rows, cols], every leading index a matrix of its own, or a list
    of such tensors (segments of a combined gradient, of any shapes, one dtype),
    for which a list is returned.  Sides are at most 32768.  coefficients:
    (a, b, c), or one triple for each step (16 at most); they must keep singular
    values of up to 1 below 2.  A matrix that holds an infinity or NaN becomes
    NaN, one of zeros stays zero.

    dtype: of the result (default: update's); out: tensors like the result, which
    may be the update itself.  Matrices may be column slices of one buffer, also
    where they are written.  Products are formed from fp16 operands: from one part
    each for bfloat16 results (in 5 steps off by some 0.15 % of the norm, as much as
    their rounding, in 12 by 0.35 %; for less, ask for float32 and round that), from
    two for float32 and float16 results (off by less than products of fp32 values).
    Matrices with a side of at most 64 take fp64 throughout.

    workspace: as for the layer operators; of a list, what its largest call needs
    (matrices of one shape and spacing are one call).  What many matrices need is
    enough for fewer of the same sides.
    """
    single = isinstance(update, torch.Tensor)
    given = [update] if single else list(update)
    if not given:
        return []
    for t in given:
        _on(t, "update")
    dev = given[0].device
    kind = given[0].dtype
    if any(t.dtype != kind for t in given):
        raise ValueError("the matrices of an update must have one dtype")
    outs = None
    if out is not None:
        outs = [out] if single else list(out)
        if len(outs) != len(given):
            raise ValueError(f"{len(outs)} outputs for {len(given)} matrices")
        dtype = outs[0].dtype if dtype is None else dtype
    dtype = kind if dtype is None else dtype
    code, out_code = _code(kind, "update"), _code(dtype, "out")
    if not isinstance(steps, int) or not 1 <= steps <= 16:
        raise ValueError("steps must be in [1, 16]")
    k = _coefficients(coefficients, steps)
    sides = [_matrices(t, "update", dev) for t in given]
    if outs is not None:
        for t, o in zip(given, outs):
            _like(o, "out", dev, t.shape, dtype)
    L = _native.lib()

    def body(st):
        results = outs
        if results is None:
            results = [torch.empty(t.shape, dtype=dtype, device=dev) for t in given]
        calls = {}  # matrices of one shape and spacing go together
        for (at, rows, cols, stride), o in zip(sides, results):
            to, _, _, out_stride = _matrices(o, "out", dev)
            x, y = calls.setdefault((rows, cols, stride, out_stride), ([], []))
            x += at
            y += to
        if len(calls) > 1 and (outs is not None or workspace is not None):
            _apart(calls, given[0].element_size(), results[0].element_size(), workspace)
        needs = [_native.check(L.adasum_orthogonalize_workspace_bytes(len(x), rows, cols, out_code))
                 for (rows, cols, _, _), (x, _) in calls.items()]
        ws = _workspace(workspace, max(needs), dev)
        for (rows, cols, stride, out_stride), (x, y) in calls.items():
            _native.check(L.adasum_orthogonalize(
                (ctypes.c_void_p * len(x))(*x), len(x), rows, cols, stride, code, steps, k, eps, scale,
                (ctypes.c_void_p * len(y))(*y), out_stride, out_code, _ptr(ws), _size(ws), st))
        return results[0] if single else results
    return _call(dev, stream, body)
