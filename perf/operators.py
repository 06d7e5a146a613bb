"""The layer operators' workloads, and each operator in its plain form.

What a worker does with its share of a batch before its gradient is combined
with the others': look tokens up in an embedding table, normalise rows, keep
activations in 8 bits for the backward pass, and form the gradients of the
tables and weights from them.  Sizes follow this repository's BERT-Large and
BERT-Base shapes (hidden 1024 and 768, feed-forward 4096, vocabulary 30522,
512 positions, 2 token types) at microbatches from one token to 512 sequences
of 128 tokens, and odd sizes around them.

A case is a dict: "op" and that operator's sizes and types.

  embedding       y[i] = scale * table[token_i]
  embedding_grad  grad[t] = scale * sum over the rows i with token_i = t of dy[i]
  norm            y = (x - mean) * rstd * weight + bias, and the row statistics;
                  with "keep", the normalised rows are also kept in 8 bits
  norm_grad       dx, dweight and dbias from x or from the kept 8-bit rows
  checkpoint      activations into 8 bits, and back
  linear_grad     dweight = dy^T x and dbias = sum of dy's rows, x from 8 bits

A token outside [0, vocab) is no token: its row reads as zeros and adds to no
gradient.  8-bit activations are blocks of 32 consecutive values of a row that
share a power of two: value = code * 2^(scale - 127), code in [-127, 127].
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
EPS = 1e-12  # BERT's layer norm


def listed():
    return [
        # the forward pass over the word table: 512 sequences of 128 tokens
        {"name": "embedding_bert_large", "op": "embedding", "n": 65536, "vocab": 30522, "hidden": 1024, "dtype": "bf16",
         "absent": 0.1},
        # one short sequence, where the launch counts
        {"name": "embedding_one_sequence", "op": "embedding", "n": 128, "vocab": 30522, "hidden": 768, "dtype": "f32",
         "absent": 0.0},
        # the word table's gradient: a long tail of rare tokens, a few very frequent ones, a tenth padding
        {"name": "embedding_grad_words", "op": "embedding_grad", "n": 65536, "vocab": 30522, "hidden": 1024,
         "dtype": "bf16", "grad": "f32", "absent": 0.1},
        # the token-type table's gradient: two rows that take every token, an odd count
        {"name": "embedding_grad_types", "op": "embedding_grad", "n": 8191, "vocab": 2, "hidden": 768, "dtype": "f16",
         "grad": "f16", "absent": 0.0},
        # the forward norm of the largest microbatch, its normalised rows kept in 8 bits
        {"name": "norm_keep_bert_large", "op": "norm", "rows": 65536, "hidden": 1024, "dtype": "bf16", "keep": True},
        # the norm of one row
        {"name": "norm_one_row", "op": "norm", "rows": 1, "hidden": 1024, "dtype": "f32", "keep": False},
        # the backward pass of the largest microbatch, from the activations themselves
        {"name": "norm_grad_bert_large", "op": "norm_grad", "rows": 65536, "hidden": 1024, "dtype": "bf16", "kept": False},
        # an odd width whose rows start at any address, from the kept rows
        {"name": "norm_grad_kept_ragged", "op": "norm_grad", "rows": 4095, "hidden": 1001, "dtype": "f32", "kept": True},
        # feed-forward activations of 128 sequences kept and given back
        {"name": "checkpoint_feed_forward", "op": "checkpoint", "rows": 16384, "hidden": 4096, "dtype": "bf16"},
        # few rows of an odd width: blocks that end inside a row's last vector
        {"name": "checkpoint_ragged", "op": "checkpoint", "rows": 333, "hidden": 1001, "dtype": "f32"},
        # the feed-forward matrix's gradient over the largest microbatch
        {"name": "linear_grad_feed_forward", "op": "linear_grad", "rows": 65536, "out": 4096, "in": 1024, "dtype": "bf16",
         "grad": "f32"},
        # a small head of odd sizes over one microbatch, in fp32
        {"name": "linear_grad_ragged", "op": "linear_grad", "rows": 2047, "out": 769, "in": 1001, "dtype": "f32",
         "grad": "f32"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "norm", "norm_grad", "checkpoint", "linear_grad"])
    case = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"])}
    if op in ("embedding", "embedding_grad"):
        case["n"] = _spread(rng, 1, 65536)
        case["vocab"] = _spread(rng, 2, 30522)
        case["hidden"] = _spread(rng, 8, 1024)
        case["absent"] = rng.choice([0.0, 0.1, 0.5])
        if op == "embedding_grad":
            case["grad"] = rng.choice(["f32", case["dtype"]])
    elif op in ("norm", "norm_grad", "checkpoint"):
        case["rows"] = _spread(rng, 1, 65536)
        case["hidden"] = _spread(rng, 8, min(8192, 65536 * 1024 // case["rows"]))
        if op == "norm":
            case["keep"] = rng.random() < 0.5
        elif op == "norm_grad":
            case["kept"] = rng.random() < 0.5
    else:
        case["rows"] = _spread(rng, 1, 65536)
        case["out"] = _spread(rng, 8, 4096)
        case["in"] = _spread(rng, 8, 2048)
        case["grad"] = rng.choice(["f32", case["dtype"]])
    return case


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0, mean=0.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g)
    return x.to(DTYPES[dtype])


def _tokens(g, case):
    """Frequencies fall with the rank (rank r about as often as 1 / r), the ranks spread over the vocabulary; a share of
    the places are padding."""
    n, vocab = case["n"], case["vocab"]
    u = torch.rand(n, dtype=torch.float64, device="cuda", generator=g)
    rank = torch.exp(u * math.log(vocab + 1)).to(torch.int64).clamp_(1, vocab) - 1
    t = torch.randperm(vocab, device="cuda", generator=g)[rank]
    pad = torch.rand(n, device="cuda", generator=g) < case["absent"]
    return torch.where(pad, torch.full_like(t, -1), t)


def _activations(g, rows, hidden, dtype):
    """Rows with a mean of their own and a few columns that are much larger than the others."""
    x = torch.empty((rows, hidden), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
    x += torch.empty((rows, 1), dtype=torch.float32, device="cuda").normal_(0.0, 0.5, generator=g)
    x *= torch.exp(torch.empty((1, hidden), dtype=torch.float32, device="cuda").normal_(0.0, 0.5, generator=g))
    return x.to(DTYPES[dtype])


def _pow2(e):
    """2^e for whole numbers e in [-126, 127], exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _pack(x, top=121):
    """Codes and scales of rows x: the least power of two 2^e with 127 * 2^e not below the block's largest magnitude
    (e at most `top`), codes rounded to nearest even; a block with a value that is not finite has scale 255."""
    rows, hidden = x.shape
    nb = -(-hidden // BLOCK)
    b = torch.zeros((rows, nb * BLOCK), dtype=x.dtype, device=x.device)
    b[:, :hidden] = x
    b = b.reshape(rows, nb, BLOCK)
    amax = b.abs().amax(2)
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad, torch.ones_like(amax), amax))
    e = torch.where(m > 127.0 / 128.0, e - 6, e - 7).clamp(-127, top)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    # in two factors: 2^-e itself can be out of range
    half = e // 2
    q = b * _pow2(-half)[..., None] * _pow2(half - e)[..., None]
    q = torch.where(bad[..., None], torch.zeros_like(q), q).round().clamp(-127, 127)
    codes = q.reshape(rows, nb * BLOCK)[:, :hidden].to(torch.int8).contiguous()
    scales = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return codes, scales


def _unpack(codes, scales):
    """The values that codes and scales stand for."""
    e = scales.to(torch.int32)
    half = (e - 127) // 2
    nan = torch.full((), float("nan"), device=e.device)
    wide = [torch.where(e == 255, nan, _pow2(k)).repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
            for k in (half, e - 127 - half)]
    return codes.float() * wide[0] * wide[1]


def _top(dtype):
    """The largest block exponent: 127 * 2^e is finite in the activations' type."""
    return 9 if dtype == "f16" else 121


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], case["dtype"]
    s = {"case": dict(case)}
    if op == "embedding":
        s["table"] = _normal(g, (case["vocab"], case["hidden"]), dt, 0.02)
        s["tokens"] = _tokens(g, case)
        s["scale"] = math.sqrt(case["hidden"])
    elif op == "embedding_grad":
        s["dy"] = _normal(g, (case["n"], case["hidden"]), dt, 1e-2)
        s["tokens"] = _tokens(g, case)
        s["scale"] = math.sqrt(case["hidden"])
    elif op == "norm":
        s["x"] = _activations(g, case["rows"], case["hidden"], dt)
        s["weight"] = _normal(g, (case["hidden"],), "f32", 0.1, 1.0)
        s["bias"] = _normal(g, (case["hidden"],), "f32", 0.1)
    elif op == "norm_grad":
        x = _activations(g, case["rows"], case["hidden"], dt)
        xd = x.double()
        mean = xd.mean(1)
        rstd = 1.0 / torch.sqrt((xd - mean[:, None]).square().mean(1) + EPS)
        s["dy"] = _normal(g, (case["rows"], case["hidden"]), dt, 1e-2)
        s["weight"] = _normal(g, (case["hidden"],), "f32", 0.1, 1.0)
        s["rstd"] = rstd.float()
        if case["kept"]:
            s["codes"], s["scales"] = _pack(((xd - mean[:, None]) * rstd[:, None]).float())
        else:
            s["x"], s["mean"] = x, mean.float()
    elif op == "checkpoint":
        s["x"] = _activations(g, case["rows"], case["hidden"], dt)
    else:
        s["dy"] = _normal(g, (case["rows"], case["out"]), dt, 1e-2)
        s["codes"], s["scales"] = _pack(_activations(g, case["rows"], case["in"], dt).float(), _top(dt))
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import distributed_sgd_gradient_amd as A
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "embedding":
        return A.embedding(s["table"], s["tokens"], scale=s["scale"])
    if op == "embedding_grad":
        return A.embedding_grad(s["dy"], s["tokens"], case["vocab"], scale=s["scale"], dtype=DTYPES[case["grad"]])
    if op == "norm":
        if case["keep"]:
            y, rstd, codes, scales = A.layer_norm_keep(s["x"], s["weight"], s["bias"], eps=EPS)
            return y, rstd, A.checkpoint_unpack(codes, scales, torch.bfloat16)
        return A.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "norm_grad":
        if case["kept"]:
            return A.layer_norm_keep_grad(s["dy"], s["codes"], s["scales"], s["rstd"], s["weight"])
        return A.layer_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "checkpoint":
        codes, scales = A.checkpoint_pack(s["x"])
        return A.checkpoint_unpack(codes, scales, dt)
    return A.linear_grad(s["dy"], s["codes"], s["scales"], dtype=DTYPES[case["grad"]])


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "embedding":
        there = (s["tokens"] >= 0) & (s["tokens"] < case["vocab"])
        rows = s["table"][s["tokens"].clamp(0, case["vocab"] - 1)].float() * s["scale"]
        return torch.where(there[:, None], rows, torch.zeros_like(rows)).to(dt)
    if op == "embedding_grad":
        there = (s["tokens"] >= 0) & (s["tokens"] < case["vocab"])
        rows = torch.where(there[:, None], s["dy"].float(), torch.zeros((), device="cuda"))
        grad = torch.zeros((case["vocab"], case["hidden"]), dtype=torch.float32, device="cuda")
        grad.index_add_(0, s["tokens"].clamp(0, case["vocab"] - 1), rows)
        return (grad * s["scale"]).to(DTYPES[case["grad"]])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
        normal = d * rstd
        y = (normal * s["weight"] + s["bias"]).to(dt)
        if case["keep"]:
            return y, rstd[:, 0], _unpack(*_pack(normal)).to(torch.bfloat16)
        return y, mean[:, 0], rstd[:, 0]
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        normal = _unpack(s["codes"], s["scales"]) if case["kept"] else (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["weight"]
        dx = (g - g.mean(1, keepdim=True) - normal * (g * normal).mean(1, keepdim=True)) * rstd
        return dx.to(dt), (dy * normal).sum(0), dy.sum(0)
    if op == "checkpoint":
        return _unpack(*_pack(s["x"].float(), _top(case["dtype"]))).to(dt)
    dy = s["dy"].float()
    grad = DTYPES[case["grad"]]
    return (dy.t() @ _unpack(s["codes"], s["scales"])).to(grad), dy.sum(0).to(grad)


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    op, b = case["op"], SIZES[case["dtype"]]
    if op == "embedding":
        n, h = case["n"], case["hidden"]
        # a table row that several tokens name is read once: about as many rows as there are distinct tokens
        return {"bytes": 8 * n + b * h * (n + min(n, case["vocab"])), "flops": n * h}
    if op == "embedding_grad":
        n, h = case["n"], case["hidden"]
        return {"bytes": 8 * n + b * h * n + SIZES[case["grad"]] * h * case["vocab"], "flops": n * h + h * case["vocab"]}
    if op == "linear_grad":
        r, o, i = case["rows"], case["out"], case["in"]
        return {"bytes": b * r * o + r * i + r * -(-i // BLOCK) + SIZES[case["grad"]] * o * (i + 1),
                "flops": 2 * r * o * i + r * o}
    r, h = case["rows"], case["hidden"]
    kept = r * h + r * -(-h // BLOCK)
    if op == "norm":
        # with "keep": the 8-bit rows are written, read back and given as bf16 values
        more = 4 * r + 2 * kept + 2 * r * h if case["keep"] else 8 * r
        return {"bytes": 2 * b * r * h + 8 * h + more, "flops": 8 * r * h}
    if op == "norm_grad":
        x = kept + 4 * r if case["kept"] else b * r * h + 8 * r
        return {"bytes": 2 * b * r * h + x + 12 * h, "flops": 14 * r * h}
    return {"bytes": 2 * b * r * h + 2 * kept, "flops": 4 * r * h}


# ---------------------------------------------------------------- the definitions in 64 bits


def _levels(x, top):
    """The value of each element of rows x (64 bits) after its block's 8-bit rounding, from the definition: the step is
    the least power of two of which 127 reach the block's largest magnitude."""
    rows, hidden = x.shape
    nb = -(-hidden // BLOCK)
    largest = torch.zeros((rows, nb), dtype=torch.float64, device=x.device)
    largest.scatter_reduce_(1, (torch.arange(hidden, device=x.device) // BLOCK).expand(rows, hidden), x.abs(), "amax")
    step = torch.exp2(torch.ceil(torch.log2(largest / 127.0)).clamp(-127, top))
    # log2 is rounded: take the step on its right side
    step = torch.where((step / 2 >= 2.0 ** -127) & (step / 2 * 127.0 >= largest), step / 2, step)
    step = torch.where((step * 127.0 < largest) & (step < 2.0 ** top), step * 2, step)
    step = torch.where(largest == 0, torch.full_like(step, 2.0 ** -127), step)
    step = step[:, torch.arange(hidden, device=x.device) // BLOCK]
    return torch.clamp(torch.round(x / step), -127, 127) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embedding":
        table = torch.cat([s["table"].double() * s["scale"],
                           torch.zeros((1, case["hidden"]), dtype=torch.float64, device="cuda")])
        t = s["tokens"]
        return table[torch.where((t < 0) | (t >= case["vocab"]), torch.full_like(t, case["vocab"]), t)]
    if op == "embedding_grad":
        # rows in the order of their tokens, summed run by run; the tokens that are none sort to either end
        t, order = torch.sort(s["tokens"])
        bounds = torch.searchsorted(t, torch.arange(case["vocab"] + 1, device="cuda"))
        out = torch.empty((case["vocab"], case["hidden"]), dtype=torch.float64, device="cuda")
        for c in range(0, case["hidden"], 128):
            run_ = torch.zeros((case["n"] + 1, min(128, case["hidden"] - c)), dtype=torch.float64, device="cuda")
            run_[1:] = torch.cumsum(s["dy"][order, c:c + 128].double(), 0)
            out[:, c:c + 128] = (run_[bounds[1:]] - run_[bounds[:-1]]) * s["scale"]
        return out
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS).pow(-0.5)
        normal = (x - mean) * rstd
        y = torch.addcmul(s["bias"].double(), normal, s["weight"].double())
        return (y, rstd[:, 0], _levels(normal, 121)) if case["keep"] else (y, mean[:, 0], rstd[:, 0])
    if op == "norm_grad":
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        if case["kept"]:
            scale = torch.exp2(s["scales"].double() - 127.0)
            normal = s["codes"].double() * scale[:, torch.arange(case["hidden"], device="cuda") // BLOCK]
        else:
            normal = (s["x"].double() - s["mean"].double()[:, None]) * rstd
        h = case["hidden"]
        a, w = dy @ s["weight"].double() / h, s["weight"].double()
        b = ((dy * normal) @ w) / h
        dx = rstd * (dy * w - a[:, None] - normal * b[:, None])
        ones = torch.ones(case["rows"], dtype=torch.float64, device="cuda")
        return dx, ones @ (dy * normal), ones @ dy
    if op == "checkpoint":
        return _levels(s["x"].double(), _top(case["dtype"]))
    scale = torch.exp2(s["scales"].double() - 127.0)
    x = s["codes"].double() * scale[:, torch.arange(case["in"], device="cuda") // BLOCK]
    dy = s["dy"].double()
    return dy.t() @ x, dy.t() @ torch.ones(case["rows"], dtype=torch.float64, device="cuda")
