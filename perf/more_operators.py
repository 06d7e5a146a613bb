"""Workloads of further operators around the combine, and each in its plain form.

What a worker's residual stream and attention scores pass through, and what
becomes of a combined gradient: a root-mean-square norm that adds the residual
and gives its rows in 8 bits too, a learned bias by the distance between query
and key, and an update whose matrices are made orthogonal.  Sizes follow this
repository's BERT-Large and BERT-Base shapes (hidden 1024 and 768, feed-forward
4096, 16 and 12 heads, 512 positions), from one token to 512 sequences of 128
tokens, and odd sizes around them.

A case is a dict: "op" and that operator's sizes and types.

  rms        h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * weight;
             with "pack", y is given in 8 bits too (blocks of 32 values of a
             row that share a power of two)
  rms_grad   with g = dy * weight and n = h * rstd: dx = dh + rstd * (g - n * mean(g * n))
             and dweight = sum over rows of dy * n
  bias       out[h, i, j] = table[bucket(j - i - offset), h], added to scores where
             "batch" is not 0
  bias_grad  dtable[b, h] = sum of dscores[n, h, i, j] where bucket(j - i - offset) = b
  orthogonal X / |X|, then five times X = a X + (b A + c A^2) X with A = X X^T
             (the shorter side's products), times a scale

Buckets: with m = buckets / 2 on each side ("both") or m = buckets on the past's
side alone, distances below e = m / 2 have one each, and those from there on
e + floor(log(distance / e) / log(reach / e) * (m - e)), at most m - 1.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
EPS = 1e-6
STEPS, COEFFICIENTS, FLOOR = 5, (3.4445, -4.7750, 2.0315), 1e-7


def listed():
    return [
        # the largest microbatch's residual additions and norms, 512 sequences of 128 tokens; the next linear layer's
        # gradient takes the rows in 8 bits
        {"name": "rms_pack_block", "op": "rms", "rows": 65536, "hidden": 1024, "dtype": "bf16", "stream": "bf16",
         "pack": True},
        # feed-forward width in fp16 beside an fp32 residual stream, an odd number of rows
        {"name": "rms_wide_stream", "op": "rms", "rows": 8191, "hidden": 4096, "dtype": "f16", "stream": "f32",
         "pack": False},
        # one token of an answer
        {"name": "rms_one_token", "op": "rms", "rows": 1, "hidden": 1024, "dtype": "bf16", "stream": "bf16",
         "pack": False},
        # the backward pass of the largest microbatch, with the gradient that comes along the residual stream
        {"name": "rms_grad_block", "op": "rms_grad", "rows": 65536, "hidden": 1024, "dtype": "bf16", "stream": "bf16",
         "dh": True},
        # an odd width whose rows start at any address
        {"name": "rms_grad_ragged", "op": "rms_grad", "rows": 4095, "hidden": 1001, "dtype": "f32", "stream": "f32",
         "dh": False},
        # the bias on the attention scores of 32 sequences of 512 tokens
        {"name": "bias_scores", "op": "bias", "batch": 32, "heads": 16, "queries": 512, "keys": 512, "offset": 0,
         "buckets": 32, "reach": 128, "both": True, "dtype": "bf16"},
        # one new token against the keys before it
        {"name": "bias_one_token", "op": "bias", "batch": 0, "heads": 12, "queries": 1, "keys": 509, "offset": 508,
         "buckets": 32, "reach": 128, "both": False, "dtype": "f32"},
        # the table's gradient from the scores of 32 sequences
        {"name": "bias_grad_scores", "op": "bias_grad", "batch": 32, "heads": 16, "queries": 512, "keys": 512,
         "offset": 0, "buckets": 32, "reach": 128, "both": True, "dtype": "bf16"},
        # few short sequences of odd lengths, past side only
        {"name": "bias_grad_ragged", "op": "bias_grad", "batch": 3, "heads": 12, "queries": 127, "keys": 131,
         "offset": 4, "buckets": 32, "reach": 128, "both": False, "dtype": "f32"},
        # the update of 24 layers' query projections
        {"name": "orthogonal_attention", "op": "orthogonal", "count": 24, "rows": 1024, "cols": 1024, "dtype": "bf16"},
        # one layer's feed-forward matrix in fp32
        {"name": "orthogonal_feed_forward", "op": "orthogonal", "count": 1, "rows": 4096, "cols": 1024,
         "dtype": "f32"},
        # a small adapter's matrix of odd sizes, where the launches count
        {"name": "orthogonal_adapter", "op": "orthogonal", "count": 1, "rows": 61, "cols": 769, "dtype": "f32"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["rms", "rms_grad", "bias", "bias_grad", "orthogonal"])
    case = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if op in ("rms", "rms_grad"):
        case["rows"] = _spread(rng, 1, 65536)
        case["stream"] = rng.choice(["f32", case["dtype"]])
        most = 65536 * 1024 * 4 // (SIZES[case["dtype"]] + SIZES[case["stream"]])
        case["hidden"] = _spread(rng, 8, min(8192, most // case["rows"]))
        case["pack" if op == "rms" else "dh"] = rng.random() < 0.5
    elif op in ("bias", "bias_grad"):
        case["heads"] = _spread(rng, 1, 16)
        case["keys"] = _spread(rng, 1, 2048)
        case["queries"] = rng.choice([1, _spread(rng, 1, case["keys"]), case["keys"]])
        most = 32 * 16 * 512 * 512 // (case["heads"] * case["keys"] * case["queries"])
        case["batch"] = _spread(rng, 1, max(1, min(64, most // (2 if case["dtype"] == "f32" else 1))))
        if op == "bias" and rng.random() < 0.3:
            case["batch"] = 0
        case["offset"] = rng.choice([0, case["keys"] - case["queries"]])
        case["both"] = rng.random() < 0.5
        case["buckets"] = rng.choice([32, 64, 20])
        case["reach"] = rng.choice([128, 256, 60])
    else:
        case["rows"] = _spread(rng, 8, 4096)
        case["cols"] = _spread(rng, 8, min(4096, 2 ** 22 // case["rows"]))
        one = work({**case, "count": 1})["flops"]
        case["count"] = _spread(rng, 1, max(1, min(24, 5 * 10 ** 11 // one)))
    return case


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0, mean=0.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g)
    return x.to(DTYPES[dtype])


def _stream(g, rows, hidden, dtype):
    """Rows of a residual stream: sizes that differ by row, and a few columns much larger than the others."""
    x = torch.empty((rows, hidden), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
    x *= torch.exp(torch.empty((rows, 1), dtype=torch.float32, device="cuda").normal_(0.0, 0.3, generator=g))
    x *= torch.exp(torch.empty((1, hidden), dtype=torch.float32, device="cuda").normal_(0.0, 0.5, generator=g))
    return x.to(DTYPES[dtype])


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], case["dtype"]
    s = {"case": dict(case)}
    if op == "rms":
        s["x"] = _normal(g, (case["rows"], case["hidden"]), dt, 0.5)
        s["residual"] = _stream(g, case["rows"], case["hidden"], case["stream"])
        s["weight"] = _normal(g, (case["hidden"],), "f32", 0.1, 1.0)
    elif op == "rms_grad":
        s["h"] = _stream(g, case["rows"], case["hidden"], case["stream"])
        s["rstd"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = _normal(g, (case["rows"], case["hidden"]), dt, 1e-2)
        s["dh"] = _normal(g, (case["rows"], case["hidden"]), case["stream"], 1e-2) if case["dh"] else None
        s["weight"] = _normal(g, (case["hidden"],), "f32", 0.1, 1.0)
    elif op == "bias":
        s["table"] = _normal(g, (case["buckets"], case["heads"]), "f32", 1.0)
        s["scores"] = None
        if case["batch"]:
            s["scores"] = _normal(g, (case["batch"], case["heads"], case["queries"], case["keys"]), dt, 3.0)
    elif op == "bias_grad":
        # gradients of scores: large at a few keys of a row, of both signs
        shape = (case["batch"], case["heads"], case["queries"], case["keys"])
        d = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, 1e-2, generator=g)
        d *= torch.exp(torch.empty((1, 1, 1, case["keys"]), dtype=torch.float32, device="cuda").normal_(
            0.0, 1.0, generator=g))
        s["dscores"] = d.to(DTYPES[dt])
    else:
        # a gradient: noise, and a few directions that are much stronger
        n, r, c = case["count"], case["rows"], case["cols"]
        x = torch.empty((n, r, c), dtype=torch.float32, device="cuda").normal_(0.0, 1e-3, generator=g)
        u = torch.empty((n, r, 4), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
        v = torch.empty((n, 4, c), dtype=torch.float32, device="cuda").normal_(0.0, 2e-3, generator=g)
        s["update"] = (x + torch.matmul(u, v)).to(DTYPES[dt])
        s["scale"] = math.sqrt(max(1.0, r / c))
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import distributed_sgd_gradient_amd as A
    case = s["case"]
    op = case["op"]
    if op == "rms":
        if case["pack"]:
            y, codes, scales, h, rstd = A.rms_norm_pack(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return y, A.checkpoint_unpack(codes, scales, torch.bfloat16), h, rstd
        return A.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
    if op == "rms_grad":
        return A.rms_norm_grad(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"])
    shape = {} if op == "orthogonal" else dict(offset=case["offset"], bidirectional=case["both"],
                                               max_distance=case["reach"])
    if op == "bias":
        if case["batch"]:
            return A.relative_bias(s["table"], scores=s["scores"], **shape)
        return A.relative_bias(s["table"], case["queries"], case["keys"], dtype=DTYPES[case["dtype"]], **shape)
    if op == "bias_grad":
        return A.relative_bias_grad(s["dscores"], case["buckets"], dtype=torch.float32, **shape)
    return A.orthogonalize(s["update"], steps=STEPS, coefficients=COEFFICIENTS, eps=FLOOR, scale=s["scale"])


def _pow2(e):
    """2^e for whole numbers e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _eight_bits(x, top):
    """Rows x (fp32) after rounding to 8 bits: 32 values share the least power of two 2^e of which 127 reach the block's
    largest magnitude, e at least -127 and at most `top`."""
    rows, hidden = x.shape
    nb = -(-hidden // BLOCK)
    b = torch.zeros((rows, nb * BLOCK), dtype=x.dtype, device=x.device)
    b[:, :hidden] = x
    b = b.reshape(rows, nb, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    m, e = torch.frexp(amax)
    e = torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp(-127, top)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    # in two factors: 2^-e itself can be out of range
    half = e // 2
    q = (b * _pow2(-half) * _pow2(half - e)).round().clamp(-127, 127)
    return (q * _pow2(half) * _pow2(e - half)).reshape(rows, nb * BLOCK)[:, :hidden]


def _buckets(case):
    """bucket(j - i - offset) for every query i and key j."""
    i = torch.arange(case["queries"], device="cuda")[:, None] + case["offset"]
    d = torch.arange(case["keys"], device="cuda")[None, :] - i
    m = case["buckets"] // 2 if case["both"] else case["buckets"]
    e = m // 2
    n = d.abs() if case["both"] else (-d).clamp(min=0)
    # 64 bits, and a margin for whole numbers that the quotient of logarithms just misses
    far = torch.log(n.clamp(min=1).double() / e) / math.log(case["reach"] / e) * (m - e)
    far = (e + torch.floor(far + 1e-9).long()).clamp(max=m - 1)
    b = torch.where(n < e, n, far)
    return torch.where(d > 0, b + m, b) if case["both"] else b


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "rms":
        h = (s["x"].float() + s["residual"].float()).to(DTYPES[case["stream"]])
        wide = h.float()
        rstd = 1.0 / torch.sqrt(wide.square().mean(1, keepdim=True) + EPS)
        y = (wide * rstd * s["weight"]).to(dt)
        if case["pack"]:
            return y, _eight_bits(y.float(), 9 if case["dtype"] == "f16" else 121).to(torch.bfloat16), h, rstd[:, 0]
        return y, h, rstd[:, 0]
    if op == "rms_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        n = s["h"].float() * rstd
        g = dy * s["weight"]
        dx = (g - n * (g * n).mean(1, keepdim=True)) * rstd
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return dx.to(DTYPES[case["stream"]]), (dy * n).sum(0)
    if op == "bias":
        bias = s["table"].t()[:, _buckets(case)]
        return (bias if s["scores"] is None else s["scores"].float() + bias).to(dt)
    if op == "bias_grad":
        over = s["dscores"].float().sum(0).reshape(case["heads"], -1)
        grad = torch.zeros((case["heads"], case["buckets"]), dtype=torch.float32, device="cuda")
        return grad.index_add_(1, _buckets(case).reshape(-1), over).t().contiguous()
    a, b, c = COEFFICIENTS
    x = s["update"].float()
    tall = case["rows"] > case["cols"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + FLOOR)
    for _ in range(STEPS):
        p = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    x = x * s["scale"]
    return (x.transpose(1, 2).contiguous() if tall else x).to(dt)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, b = case["op"], SIZES[case["dtype"]]
    if op in ("rms", "rms_grad"):
        r, h, st = case["rows"], case["hidden"], SIZES[case["stream"]]
        if op == "rms":
            # with "pack" the 8-bit rows are written, read back and given as bf16 values
            more = 2 * (r * h + r * -(-h // BLOCK)) + 2 * r * h if case["pack"] else 0
            return {"bytes": 2 * (b + st) * r * h + 4 * r + 4 * h + more, "flops": 5 * r * h}
        return {"bytes": (b + (3 if case["dh"] else 2) * st) * r * h + 4 * r + 8 * h, "flops": 9 * r * h}
    if op in ("bias", "bias_grad"):
        n = max(1, case["batch"]) * case["heads"] * case["queries"] * case["keys"]
        table = 4 * case["heads"] * case["buckets"]
        passes = 2 if op == "bias" and case["batch"] else 1
        return {"bytes": passes * b * n + table, "flops": n}
    n, m = sorted((case["rows"], case["cols"]))
    # a step: A and its square, of which one half determines the other, and a product with X
    return {"bytes": 2 * b * case["count"] * n * m, "flops": case["count"] * STEPS * (n * n * m + n * n * n + 2 * n * n * m)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _levels(x, top):
    """Each element of rows x (64 bits) after its block's 8-bit rounding, from the definition."""
    rows, hidden = x.shape
    where = torch.arange(hidden, device=x.device) // BLOCK
    largest = torch.zeros((rows, -(-hidden // BLOCK)), dtype=torch.float64, device=x.device)
    largest.scatter_reduce_(1, where.expand(rows, hidden), x.abs(), "amax")
    step = torch.exp2(torch.ceil(torch.log2(largest / 127.0)).clamp(-127, top))
    # log2 is rounded: take the step on its right side
    step = torch.where((step / 2 >= 2.0 ** -127) & (step / 2 * 127.0 >= largest), step / 2, step)
    step = torch.where((step * 127.0 < largest) & (step < 2.0 ** top), step * 2, step)
    step = torch.where(largest == 0, torch.full_like(step, 2.0 ** -127), step)[:, where]
    return torch.clamp(torch.round(x / step), -127, 127) * step


def _bucket_of(case, d):
    """The bucket of the whole number d = j - i - offset, in whole numbers: the k-th border behind e is the least n with
    (n / e)^(m - e) >= (reach / e)^k."""
    m = case["buckets"] // 2 if case["both"] else case["buckets"]
    e, past = m // 2, -d
    n = abs(d) if case["both"] else max(past, 0)
    if n < e:
        k = n
    elif n >= case["reach"]:
        k = m - 1
    else:
        k = e
        while k < m - 1 and n ** (m - e) * e ** (k + 1 - e) >= case["reach"] ** (k + 1 - e) * e ** (m - e):
            k += 1
    return k + m if case["both"] and d > 0 else k


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rms":
        h = s["x"].double() + s["residual"].double()
        # the norm is that of the rows as they are stored
        kept = h.float().to(DTYPES[case["stream"]]).double()
        rstd = (kept.pow(2).sum(1) / case["hidden"] + EPS).pow(-0.5)
        y = kept * (rstd[:, None] * s["weight"].double())
        if case["pack"]:
            given = y.float().to(DTYPES[case["dtype"]]).double()
            return y, _levels(given, 9 if case["dtype"] == "f16" else 121), h, rstd
        return y, h, rstd
    if op == "rms_grad":
        dy, r, h = s["dy"].double(), s["rstd"].double()[:, None], s["h"].double()
        g = dy * s["weight"].double()
        along = (g * h).sum(1, keepdim=True) * r.pow(3) / case["hidden"]
        dx = g * r - h * along
        if s["dh"] is not None:
            dx += s["dh"].double()
        return dx, torch.ones(case["rows"], dtype=torch.float64, device="cuda") @ (dy * h * r)
    if op in ("bias", "bias_grad"):
        first = 1 - case["queries"] - case["offset"]  # j - i - offset at j = 0 and the last query
        of = torch.tensor([_bucket_of(case, first + k) for k in range(case["queries"] + case["keys"] - 1)],
                          device="cuda")
    if op == "bias":
        # row i is the line of all distances from its place on
        line = s["table"].double().t()[:, of]
        out = line.unfold(1, case["keys"], 1).flip(1)
        return out.clone() if s["scores"] is None else s["scores"].double() + out
    if op == "bias_grad":
        over = torch.zeros((case["heads"], of.numel()), dtype=torch.float64, device="cuda")
        total = s["dscores"].sum(0, dtype=torch.float64)
        for i in range(case["queries"]):
            over[:, case["queries"] - 1 - i:][:, :case["keys"]] += total[:, i]
        hot = (of[:, None] == torch.arange(case["buckets"], device="cuda")[None, :]).double()
        return (over @ hot).t().contiguous()
    a, b, c = COEFFICIENTS
    out = torch.empty(s["update"].shape, dtype=torch.float64, device="cuda")
    for k in range(case["count"]):
        x = s["update"][k].double()
        x = x.t().contiguous() if case["rows"] > case["cols"] else x
        x = x / (torch.linalg.vector_norm(x) + FLOOR)
        for _ in range(STEPS):
            p = x @ x.t()
            q = p @ x
            x = a * x + b * q + c * (p @ q)
        out[k] = s["scale"] * (x.t() if case["rows"] > case["cols"] else x)
    return out
