"""Python front end of the layer operators: what a worker computes from its
microbatch before its gradient is combined with the others'.

Embedding lookup, layer norm, the norm of a residual stream, relative position
biases, activations kept in 8 bits, and the gradients of the tables and
weights, which may be written straight into (or added to) the
segments of a flat gradient buffer that :func:`combine` reads.  As there, only
argument marshalling happens here; torch provides device memory and streams.

Tensors are matrices of rows: the last dimension is a row, whose elements are
consecutive, and the leading dimensions must collapse into evenly spaced rows
(a slice of columns is fine, an expanded tensor is not).  ``out`` and the like
must not overlap another argument.  The functions work on plain tensors and
record no autograd graph.  ``stream=None`` is the current stream of the
tensors' device; with a stream given, outputs and workspace are allocated on
it, and inputs must stay alive until it has passed the call.

``workspace``: a contiguous tensor of at least the bytes that the library's
``adasum_..._workspace_bytes`` names, aligned to 16 bytes, for callers that
keep one; calls that share it must follow each other on one stream, and graphs
that share it must not run at the same time.  By default each call allocates
its own.
"""

import torch

from . import _native
from .combine import DTYPE_CODES, _current_raw_stream

SCALE_BLOCK = 32  # values of a row that share a scale


def _code(dtype, name):
    code = DTYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"{name}: unsupported dtype {dtype}")
    return code


def _on(t, name, dev=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if dev is not None and t.get_device() != dev.index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    return t


def _rows(t, name):
    """(rows, width, row stride) of a tensor whose last dimension is a row."""
    if t.dim() < 1 or t.size(-1) < 1:
        raise ValueError(f"{name} needs a last dimension of at least one element")
    width = t.size(-1)
    if t.is_contiguous():
        return t.numel() // width, width, width
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be consecutive")
    try:
        m = t.view(-1, width)
    except RuntimeError:
        raise ValueError(f"{name}: the rows must be evenly spaced (make it contiguous)") from None
    rows = m.size(0)
    if rows <= 1:
        return rows, width, width
    if m.stride(0) < width:
        raise ValueError(f"{name}: rows overlap (an expanded tensor: make it contiguous)")
    return rows, width, m.stride(0)


def _param(t, name, dev, width):
    _on(t, name, dev)
    if t.dim() != 1 or t.numel() != width or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {width} elements")
    return _code(t.dtype, name)


def _dense(t, name, dev, shape, dtype=None):
    """A caller's output: contiguous, with the elements of ``shape`` (a flat
    segment of a gradient buffer counts)."""
    _on(t, name, dev)
    count = 1
    for n in shape:
        count *= n
    if not t.is_contiguous() or t.numel() != count:
        raise ValueError(f"{name} must be a contiguous tensor of {count} elements")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    return t


def _like(t, name, dev, shape, dtype):
    """A caller's output matrix: shape and dtype fixed, rows may be strided."""
    _on(t, name, dev)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} of {dtype}")
    return t


def _tokens(t, dev):
    _on(t, "tokens", dev)
    if t.dtype not in (torch.int32, torch.int64):
        raise ValueError("tokens must be int32 or int64")
    if not t.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return t.element_size()


def _packed(codes, scales, dev, rows, shape_name):
    """(width) of kept activations; ``rows`` is what they must have."""
    _on(codes, "codes", dev)
    _on(scales, "scales", dev)
    if codes.dtype != torch.int8 or scales.dtype != torch.uint8:
        raise ValueError("codes must be int8 and scales uint8")
    if codes.dim() < 1 or codes.size(-1) < 1 or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("codes and scales must be contiguous, with rows of at least one element")
    width = codes.size(-1)
    have = codes.numel() // width
    if rows is not None and have != rows:
        raise ValueError(f"codes have {have} rows, {shape_name} has {rows}")
    if scales.numel() != have * _blocks(width):
        raise ValueError(f"scales must have {_blocks(width)} elements per row")
    return have, width


def _blocks(width):
    return -(-width // SCALE_BLOCK)


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
    return workspace


def _lead(t, rows):
    """t's shape without the last dimension (slicing a torch.Size is slow)."""
    return (rows,) if t.dim() == 2 else t.shape[:-1]


def _fresh(t, dtype):
    """A dense tensor of t's shape; empty_like is the cheapest way to one."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _size(t):
    return 0 if t is None else t.numel() * t.element_size()


def _call(dev, stream, body):
    """body(stream handle) with dev and the stream current, so that what it
    allocates belongs to that stream."""
    if stream is None:
        if torch.cuda.current_device() == dev.index:
            return body(_current_raw_stream(dev.index))
        with torch.cuda.device(dev):
            return body(_current_raw_stream(dev.index))
    if stream.device != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {dev}")
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def embedding(table, tokens, *, scale=1.0, dtype=None, out=None, stream=None):
    """scale * table[tokens]: [..., hidden] for tokens of any shape.

    table: [vocab, hidden], vocab at most 2^24.  tokens: int32 or int64; one
    outside [0, vocab) is no token and reads as zeros.  dtype: of the result
    (default: the table's).
    """
    dev = _on(table, "table").device
    if table.dim() != 2:
        raise ValueError("table must be [vocab, hidden]")
    vocab, hidden, stride = _rows(table, "table")
    token_bytes = _tokens(tokens, dev)
    shape = (*tokens.shape, hidden)
    out_stride = hidden
    if out is not None:
        dtype = out.dtype if dtype is None else dtype
        _like(out, "out", dev, shape, dtype)
        out_stride = _rows(out, "out")[2]
    dtype = table.dtype if dtype is None else dtype
    codes = _code(table.dtype, "table"), _code(dtype, "out")

    def body(st):
        y = torch.empty(shape, dtype=dtype, device=dev) if out is None else out
        _native.check(_native.lib().adasum_embedding(
            table.data_ptr(), vocab, hidden, stride, codes[0], tokens.data_ptr(), token_bytes, tokens.numel(),
            scale, y.data_ptr(), out_stride, codes[1], st))
        return y
    return _call(dev, stream, body)


def embedding_grad(dy, tokens, vocab, *, scale=1.0, dtype=None, out=None, accumulate=False, workspace=None,
                   stream=None):
    """The table's gradient [vocab, hidden]: per token, scale times the sum of
    the rows of dy that have it; rows of a token outside [0, vocab) are left
    out.

    dy: [..., hidden] with the leading shape of tokens.  dtype: of the
    gradient (default: dy's).  out: a contiguous tensor of vocab * hidden
    elements, for instance a segment of a gradient buffer; with accumulate the
    gradient is added to it.
    """
    dev = _on(dy, "dy").device
    n, hidden, stride = _rows(dy, "dy")
    token_bytes = _tokens(tokens, dev)
    if tokens.numel() != n:
        raise ValueError(f"{tokens.numel()} tokens for {n} rows of dy")
    code = _code(dy.dtype, "dy")
    if out is not None:
        _dense(out, "out", dev, (vocab, hidden), dtype)
        dtype = out.dtype
    elif accumulate:
        raise ValueError("accumulate needs out")
    dtype = dy.dtype if dtype is None else dtype
    grad_code = _code(dtype, "out")
    L = _native.lib()
    need = _native.check(L.adasum_embedding_grad_workspace_bytes(n, hidden, code))

    def body(st):
        ws = _workspace(workspace, need, dev)
        grad = torch.empty((vocab, hidden), dtype=dtype, device=dev) if out is None else out
        _native.check(L.adasum_embedding_grad(
            dy.data_ptr(), n, hidden, stride, code, tokens.data_ptr(), token_bytes, vocab, scale, grad.data_ptr(),
            grad_code, int(accumulate), _ptr(ws), _size(ws), st))
        return grad
    return _call(dev, stream, body)


def _norm(x, weight, bias, eps, out, stream, keep):
    dev = _on(x, "x").device
    rows, hidden, stride = _rows(x, "x")
    out_stride = hidden
    code = _code(x.dtype, "x")
    param_code = 0
    if weight is not None:
        param_code = _param(weight, "weight", dev, hidden)
    if bias is not None:
        bias_code = _param(bias, "bias", dev, hidden)
        if weight is not None and bias_code != param_code:
            raise ValueError("weight and bias must have one dtype")
        param_code = bias_code
    if out is not None:
        _like(out, "out", dev, x.shape, x.dtype)
        out_stride = _rows(out, "out")[2]

    def body(st):
        y = _fresh(x, x.dtype) if out is None else out
        lead = _lead(x, rows)
        rstd = torch.empty(lead, dtype=torch.float32, device=dev)
        mean = codes = scales = None
        if keep:
            codes = _fresh(x, torch.int8)
            scales = torch.empty((*lead, _blocks(hidden)), dtype=torch.uint8, device=dev)
        else:
            mean = torch.empty_like(rstd)
        _native.check(_native.lib().adasum_layer_norm(
            x.data_ptr(), rows, hidden, stride, code, _ptr(weight), _ptr(bias), param_code, eps, y.data_ptr(),
            out_stride, _ptr(mean), rstd.data_ptr(), _ptr(codes), _ptr(scales), st))
        return (y, rstd, codes, scales) if keep else (y, mean, rstd)
    return _call(dev, stream, body)


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, out=None, stream=None):
    """Layer norm over the last dimension (at most 16384 wide): (y, mean,
    rstd), the row statistics in fp32 for :func:`layer_norm_grad`.

    weight and bias: [hidden] each, of one dtype, or None (1 and 0).
    """
    return _norm(x, weight, bias, eps, out, stream, False)


def layer_norm_keep(x, weight=None, bias=None, *, eps=1e-5, out=None, stream=None):
    """Layer norm that keeps the normalised rows in 8 bits (the format of
    :func:`checkpoint_pack`): (y, rstd, codes, scales), all that
    :func:`layer_norm_keep_grad` needs besides dy; x can be freed."""
    return _norm(x, weight, bias, eps, out, stream, True)


def _norm_grad(dy, x, mean, codes, scales, rstd, weight, dx, dweight, dbias, bias, accumulate, workspace, stream):
    dev = _on(dy, "dy").device
    rows, hidden, stride = _rows(dy, "dy")
    code = _code(dy.dtype, "dy")
    x_stride = hidden
    if x is not None:
        _on(x, "x", dev)
        if x.shape != dy.shape or x.dtype != dy.dtype:
            raise ValueError("x must have the shape and dtype of dy")
        x_stride = _rows(x, "x")[2]
        _dense(mean, "mean", dev, (rows,), torch.float32)
    elif _packed(codes, scales, dev, rows, "dy")[1] != hidden:
        raise ValueError("codes must have the width of dy")
    _dense(rstd, "rstd", dev, (rows,), torch.float32)
    param_code = _param(weight, "weight", dev, hidden) if weight is not None else 0
    dx_stride = hidden
    if dx is not None:
        _like(dx, "dx", dev, dy.shape, dy.dtype)
        dx_stride = _rows(dx, "dx")[2]
    if weight is None and dweight is not None:
        raise ValueError("a norm without weight has no dweight")
    want_weight = weight is not None
    want_bias = dbias is not None or (want_weight if bias is None else bool(bias))
    if accumulate and (not (want_weight or want_bias) or (want_weight and dweight is None) or
                       (want_bias and dbias is None)):
        raise ValueError("accumulate needs dweight for a weight, and dbias unless bias is False")
    given = [t.dtype for t in (dweight, dbias) if t is not None]
    grad_dtype = given[0] if given else weight.dtype if want_weight else torch.float32
    for t, name in ((dweight, "dweight"), (dbias, "dbias")):
        if t is not None:
            _dense(t, name, dev, (hidden,), grad_dtype)
    grad_code = _code(grad_dtype, "dweight")
    L = _native.lib()
    need = 0
    if want_weight or want_bias:
        need = _native.check(L.adasum_layer_norm_grad_workspace_bytes(rows, hidden, code))

    def body(st):
        ws = _workspace(workspace, need, dev)
        d = _fresh(dy, dy.dtype) if dx is None else dx
        dw, db = dweight, dbias
        if want_weight and dw is None:
            dw = torch.empty(hidden, dtype=grad_dtype, device=dev)
        if want_bias and db is None:
            db = torch.empty(hidden, dtype=grad_dtype, device=dev)
        _native.check(L.adasum_layer_norm_grad(
            dy.data_ptr(), rows, hidden, stride, code, _ptr(x), x_stride, _ptr(mean), _ptr(codes), _ptr(scales),
            rstd.data_ptr(), _ptr(weight), param_code, d.data_ptr(), dx_stride, _ptr(dw), _ptr(db), grad_code,
            int(accumulate), _ptr(ws), _size(ws), st))
        return d, dw, db
    return _call(dev, stream, body)


def layer_norm_grad(dy, x, mean, rstd, weight=None, *, dx=None, dweight=None, dbias=None, bias=None,
                    accumulate=False, workspace=None, stream=None):
    """Backward pass of :func:`layer_norm`: (dx, dweight, dbias); dweight None
    for a norm without weight.

    bias: whether dbias is wanted (else None); by default with a weight, or
    where a tensor is given for it.  dx has the dtype of dy and x; dweight and
    dbias that of weight (fp32 without one), or of the tensors given for them
    (segments of a gradient buffer), to which they are added with accumulate.
    """
    if x is None or mean is None:
        raise ValueError("x and mean are needed; with kept rows use layer_norm_keep_grad")
    return _norm_grad(dy, x, mean, None, None, rstd, weight, dx, dweight, dbias, bias, accumulate, workspace, stream)


def layer_norm_keep_grad(dy, codes, scales, rstd, weight=None, *, dx=None, dweight=None, dbias=None, bias=None,
                         accumulate=False, workspace=None, stream=None):
    """Backward pass of :func:`layer_norm_keep`, from the rows kept in 8 bits;
    arguments and results as for :func:`layer_norm_grad`."""
    return _norm_grad(dy, None, None, codes, scales, rstd, weight, dx, dweight, dbias, bias, accumulate, workspace,
                      stream)


def _rms(x, weight, residual, eps, out, h, stream, pack, values):
    dev = _on(x, "x").device
    rows, hidden, stride = _rows(x, "x")
    code = _code(x.dtype, "x")
    param_code = _param(weight, "weight", dev, hidden) if weight is not None else 0
    stream_code, res_stride, h_stride = code, hidden, hidden
    if residual is not None:
        _on(residual, "residual", dev)
        if residual.shape != x.shape or residual.dtype not in (x.dtype, torch.float32):
            raise ValueError("residual must have the shape of x, and its dtype or float32")
        stream_code = _code(residual.dtype, "residual")
        res_stride = _rows(residual, "residual")[2]
        if h is not None:
            _like(h, "h", dev, x.shape, residual.dtype)
            h_stride = _rows(h, "h")[2]
    elif h is not None:
        raise ValueError("without a residual there is no h: it is x")
    out_stride = hidden
    if out is not None:
        if not values:
            raise ValueError("out is for y, which values=False leaves out")
        _like(out, "out", dev, x.shape, x.dtype)
        out_stride = _rows(out, "out")[2]

    def body(st):
        y = out
        if values and y is None:
            y = _fresh(x, x.dtype)
        total = h
        if residual is not None and total is None:
            total = _fresh(x, residual.dtype)
        lead = _lead(x, rows)
        rstd = torch.empty(lead, dtype=torch.float32, device=dev)
        codes = scales = None
        if pack:
            codes = _fresh(x, torch.int8)
            scales = torch.empty((*lead, _blocks(hidden)), dtype=torch.uint8, device=dev)
        _native.check(_native.lib().adasum_rms(
            x.data_ptr(), rows, hidden, stride, code, _ptr(residual), res_stride, stream_code, _ptr(weight), param_code,
            eps, _ptr(y), out_stride, _ptr(total), h_stride, rstd.data_ptr(), _ptr(codes), _ptr(scales), st))
        total = x if residual is None else total
        return (y, codes, scales, total, rstd) if pack else (y, total, rstd)
    return _call(dev, stream, body)


def rms_norm(x, weight=None, *, residual=None, eps=1e-6, out=None, h=None, stream=None):
    """Root-mean-square norm of h = x + residual over the last dimension (at
    most 16384 wide): (y, h, rstd) with y = h * rstd * weight, of x's dtype, and
    rstd = 1 / sqrt(mean(h^2) + eps) in fp32 for :func:`rms_norm_grad`.

    residual: like x, or float32 beside a 16-bit x; h has its dtype and is what
    y is formed from, as it is stored.  h may be the residual itself: the stream
    is then updated in place.  Without a residual h is x.  weight: [hidden], or
    None (1).
    """
    return _rms(x, weight, residual, eps, out, h, stream, False, True)


def rms_norm_pack(x, weight=None, *, residual=None, eps=1e-6, values=True, out=None, h=None, stream=None):
    """:func:`rms_norm` that gives y in 8 bits too: (y, codes, scales, h, rstd),
    codes and scales being those of ``checkpoint_pack(y)``, which
    :func:`linear_grad` takes.  With values=False y is given in 8 bits only (and
    None in its place)."""
    return _rms(x, weight, residual, eps, out, h, stream, True, values)


def rms_norm_grad(dy, h, rstd, weight=None, *, dh=None, dx=None, dweight=None, accumulate=False, workspace=None,
                  stream=None):
    """Backward pass of :func:`rms_norm`: (dx, dweight), dx being the gradient
    of x and of the residual alike, of h's dtype; dweight None without weight.

    dh: the gradient that reaches h past the norm, along the residual stream (of
    h's shape and dtype), added to dx; dx may be dh itself.  dweight has the
    dtype of weight, or of the tensor given for it (a segment of a gradient
    buffer), to which it is added with accumulate.
    """
    dev = _on(dy, "dy").device
    rows, hidden, stride = _rows(dy, "dy")
    code = _code(dy.dtype, "dy")
    _on(h, "h", dev)
    if h.shape != dy.shape or h.dtype not in (dy.dtype, torch.float32):
        raise ValueError("h must have the shape of dy, and its dtype or float32")
    stream_code = _code(h.dtype, "h")
    h_stride = _rows(h, "h")[2]
    _dense(rstd, "rstd", dev, (rows,), torch.float32)
    param_code = _param(weight, "weight", dev, hidden) if weight is not None else 0
    dh_stride = dx_stride = hidden
    if dh is not None:
        _like(dh, "dh", dev, h.shape, h.dtype)
        dh_stride = _rows(dh, "dh")[2]
    if dx is not None:
        _like(dx, "dx", dev, h.shape, h.dtype)
        dx_stride = _rows(dx, "dx")[2]
    if weight is None and dweight is not None:
        raise ValueError("a norm without weight has no dweight")
    if accumulate and dweight is None:
        raise ValueError("accumulate needs dweight")
    grad_dtype = torch.float32
    if weight is not None:
        grad_dtype = weight.dtype if dweight is None else dweight.dtype
    if dweight is not None:
        _dense(dweight, "dweight", dev, (hidden,))
    grad_code = _code(grad_dtype, "dweight")
    L = _native.lib()
    need = _native.check(L.adasum_rms_grad_workspace_bytes(rows, hidden, code)) if weight is not None else 0

    def body(st):
        ws = _workspace(workspace, need, dev)
        d = _fresh(h, h.dtype) if dx is None else dx
        dw = dweight
        if weight is not None and dw is None:
            dw = torch.empty(hidden, dtype=grad_dtype, device=dev)
        _native.check(L.adasum_rms_grad(
            dy.data_ptr(), rows, hidden, stride, code, h.data_ptr(), h_stride, stream_code, _ptr(dh), dh_stride,
            rstd.data_ptr(), _ptr(weight), param_code, d.data_ptr(), dx_stride, _ptr(dw), grad_code, int(accumulate),
            _ptr(ws), _size(ws), st))
        return d, dw
    return _call(dev, stream, body)


def _scores(t, name):
    """(batch, heads, queries, keys, row stride) of [..., heads, queries, keys]."""
    if t.dim() < 3:
        raise ValueError(f"{name} must be [..., heads, queries, keys]")
    heads, queries = t.size(-3), t.size(-2)
    if heads < 1:
        raise ValueError(f"{name} needs a head at least")
    batch = 1
    for n in t.shape[:-3]:
        batch *= n
    _, keys, stride = _rows(t, name)
    return batch, heads, queries, keys, stride


def relative_bias(table, queries=None, keys=None, *, scores=None, offset=0, bidirectional=True, max_distance=128,
                  dtype=None, out=None, stream=None):
    """A learned bias of attention scores by the distance d = j - i - offset
    between key j and query i: table[bucket(d), h] for head h.

    table: [buckets, heads], at most 256 buckets.  Without scores the result is
    [heads, queries, keys] of ``dtype`` (default: the table's); with scores
    [..., heads, queries, keys] it is scores plus the bias, of the scores' dtype,
    and out may be the scores themselves.  offset: the position of the first
    query among the keys (for one new token, the number of keys before it).

    bidirectional: half of the buckets are for keys behind the query (d > 0);
    otherwise those count as distance 0.  With m buckets on a side and e = m // 2,
    distances n below e have one bucket each, those from e on bucket
    e + floor(log(n / e) / log(max_distance / e) * (m - e)), at most m - 1; borders
    that are whole numbers are met exactly.
    """
    dev = _on(table, "table").device
    if table.dim() != 2:
        raise ValueError("table must be [buckets, heads]")
    buckets, heads, stride = _rows(table, "table")
    scores_stride = 0
    if scores is not None:
        _on(scores, "scores", dev)
        if queries is not None or keys is not None:
            raise ValueError("scores have their own queries and keys")
        if dtype is not None and dtype != scores.dtype:
            raise ValueError("the result has the dtype of scores")
        dtype, shape = scores.dtype, tuple(scores.shape)
        batch, have, queries, keys, scores_stride = _scores(scores, "scores")
        if have != heads:
            raise ValueError(f"scores have {have} heads, table has {heads}")
    else:
        if queries is None or keys is None or queries < 0 or keys < 1:
            raise ValueError("without scores, queries and keys (at least one) are needed")
        if dtype is None:
            dtype = table.dtype if out is None else out.dtype
        batch, shape = 1, (heads, queries, keys)
    out_stride = keys
    if out is not None:
        _like(out, "out", dev, shape, dtype)
        out_stride = _rows(out, "out")[2]
    codes = _code(table.dtype, "table"), _code(dtype, "out")

    def body(st):
        y = torch.empty(shape, dtype=dtype, device=dev) if out is None else out
        _native.check(_native.lib().adasum_relative_bias(
            table.data_ptr(), buckets, heads, stride, codes[0], max_distance, int(bidirectional), batch, queries, keys,
            offset, _ptr(scores), scores_stride, y.data_ptr(), out_stride, codes[1], st))
        return y
    return _call(dev, stream, body)


def relative_bias_grad(dscores, buckets, *, offset=0, bidirectional=True, max_distance=128, dtype=None, out=None,
                       accumulate=False, workspace=None, stream=None):
    """The gradient [buckets, heads] of :func:`relative_bias`'s table: per
    bucket and head the sum of dscores [..., heads, queries, keys] over all
    leading dimensions, queries and keys.

    dtype: of the gradient (default: dscores').  out: a contiguous tensor of
    buckets * heads elements, for instance a segment of a gradient buffer; with
    accumulate the gradient is added to it.
    """
    dev = _on(dscores, "dscores").device
    batch, heads, queries, keys, stride = _scores(dscores, "dscores")
    code = _code(dscores.dtype, "dscores")
    if out is not None:
        _dense(out, "out", dev, (buckets, heads), dtype)
        dtype = out.dtype
    elif accumulate:
        raise ValueError("accumulate needs out")
    dtype = dscores.dtype if dtype is None else dtype
    grad_code = _code(dtype, "out")
    L = _native.lib()
    need = _native.check(L.adasum_relative_bias_grad_workspace_bytes(batch, heads, queries, keys, code))

    def body(st):
        ws = _workspace(workspace, need, dev)
        grad = torch.empty((buckets, heads), dtype=dtype, device=dev) if out is None else out
        _native.check(L.adasum_relative_bias_grad(
            dscores.data_ptr(), batch, heads, queries, keys, stride, code, offset, buckets, max_distance,
            int(bidirectional), grad.data_ptr(), grad_code, int(accumulate), _ptr(ws), _size(ws), st))
        return grad
    return _call(dev, stream, body)


def checkpoint_pack(x, *, codes=None, scales=None, stream=None):
    """Activations in 8 bits: (codes, scales), int8 like x and uint8
    [..., ceil(width / 32)].

    32 consecutive values of a row share a power of two: value = code *
    2^(scale - 127).  A value is off by at most 1/127 of its block's largest
    magnitude (or 2^-128); a block that holds an infinity or NaN reads back as
    NaNs.  Gradients formed from kept rows are off accordingly: for normally
    distributed rows 0.8 % of the norm of a dweight.
    """
    dev = _on(x, "x").device
    rows, width, stride = _rows(x, "x")
    code = _code(x.dtype, "x")
    shape = (*_lead(x, rows), _blocks(width))
    if codes is not None:
        _dense(codes, "codes", dev, x.shape, torch.int8)
    if scales is not None:
        _dense(scales, "scales", dev, shape, torch.uint8)

    def body(st):
        c = _fresh(x, torch.int8) if codes is None else codes
        s = torch.empty(shape, dtype=torch.uint8, device=dev) if scales is None else scales
        _native.check(_native.lib().adasum_checkpoint_pack(x.data_ptr(), rows, width, stride, code, c.data_ptr(),
                                                           s.data_ptr(), st))
        return c, s
    return _call(dev, stream, body)


def checkpoint_unpack(codes, scales, dtype=torch.float32, *, out=None, stream=None):
    """The values that :func:`checkpoint_pack`'s codes and scales stand for."""
    dev = _on(codes, "codes").device
    rows, width = _packed(codes, scales, dev, None, "")
    code = _code(dtype, "dtype")
    out_stride = width
    if out is not None:
        _like(out, "out", dev, codes.shape, dtype)
        out_stride = _rows(out, "out")[2]

    def body(st):
        y = _fresh(codes, dtype) if out is None else out
        _native.check(_native.lib().adasum_checkpoint_unpack(codes.data_ptr(), scales.data_ptr(), rows, width,
                                                             y.data_ptr(), out_stride, code, st))
        return y
    return _call(dev, stream, body)


def linear_grad(dy, codes, scales, *, dtype=None, dweight=None, dbias=None, bias=True, accumulate=False,
                workspace=None, stream=None):
    """Gradient of y = x weight^T + bias from activations x kept in 8 bits:
    (dweight [out, in], dbias [out]); dbias None without bias.

    dy: [..., out]; codes, scales: x as :func:`checkpoint_pack` gives it, of
    dy's dtype and leading shape.  Codes carry no type: with an fp16 dy, values
    packed from another type (:func:`layer_norm_keep`'s are fp32 values) become
    infinities above 65504 and are off by up to 2^-25 if they have bits below
    2^-24.  dtype: of the gradients (default: dy's).
    dweight, dbias: contiguous tensors of out * in and out elements, for
    instance segments of a gradient buffer; with accumulate the gradients are
    added to them.
    """
    dev = _on(dy, "dy").device
    rows, out, stride = _rows(dy, "dy")
    code = _code(dy.dtype, "dy")
    width = _packed(codes, scales, dev, rows, "dy")[1]
    bias = bias or dbias is not None
    if accumulate and (dweight is None or (bias and dbias is None)):
        raise ValueError("accumulate needs dweight, and dbias unless bias is False")
    given = [t.dtype for t in (dweight, dbias) if t is not None]
    if dtype is None:
        dtype = given[0] if given else dy.dtype
    if dweight is not None:
        _dense(dweight, "dweight", dev, (out, width), dtype)
    if dbias is not None:
        _dense(dbias, "dbias", dev, (out,), dtype)
    grad_code = _code(dtype, "dweight")
    L = _native.lib()
    need = _native.check(L.adasum_linear_grad_workspace_bytes(rows, out, width, code))

    def body(st):
        ws = _workspace(workspace, need, dev)
        dw = torch.empty((out, width), dtype=dtype, device=dev) if dweight is None else dweight
        db = dbias
        if bias and db is None:
            db = torch.empty(out, dtype=dtype, device=dev)
        _native.check(L.adasum_linear_grad(
            dy.data_ptr(), rows, out, stride, code, codes.data_ptr(), scales.data_ptr(), width, dw.data_ptr(),
            _ptr(db), grad_code, int(accumulate), _ptr(ws), _size(ws), st))
        return dw, db
    return _call(dev, stream, body)
