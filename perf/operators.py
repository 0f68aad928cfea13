"""The gradient-list and embedding operators as measured cases.

Four operators, each with its plain form in elementary torch operations and the
call a user makes of the library:

  norm    the norm of all gradients of a model, over many tensors
  clip    the same, then every gradient scaled by min(1, max_norm / (norm + 1e-6)),
          in place or into another buffer (the optimizer's copy)
  lookup  rows of an embedding table for a batch of tokens, scaled
  grad    the embedding table's gradient from the rows' gradients, added to what
          the gradient buffer holds or written over it

`own` selects the side `run` takes; it is set from outside.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6   # added to the norm before the division, as gradient clipping usually does

# sizes of the eight-tensor list: weights and biases of a few small layers
PATTERN = (4096, 64, 16384, 128, 8192, 256, 2048, 32)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small network or one layer's adapters: latency of one call
        {"name": "norm_small", "op": "norm", "layout": "pattern", "tensors": 8, "unit": 1, "odd": 0, "flat": True,
         "dtype": "f32", "kind": 2, "sigma": 0.577},
        # bf16 weight gradients of a 1B decoder, one allocation per tensor
        {"name": "norm_decoder", "op": "norm", "layout": "decoder", "layers": 16, "hidden": 2048, "ffn": 5632,
         "vocab": 32000, "flat": False, "dtype": "bf16", "kind": 2, "sigma": 1e-3},
        # the small list, norm above the bound, clipped into a second buffer
        {"name": "clip_small", "op": "clip", "layout": "pattern", "tensors": 8, "unit": 1, "odd": 0, "flat": True,
         "dtype": "f32", "out": "f32", "copies": 1, "kind": 2, "sigma": 0.577, "max_norm": 1.0},
        # the encoder's flat fp32 buffer after the reduction, in place, in a step whose
        # norm is below the bound: most steps of a settled run
        {"name": "clip_encoder_below", "op": "clip", "layout": "encoder", "layers": 24, "hidden": 1024, "ffn": 4096,
         "vocab": 30522, "flat": True, "dtype": "f32", "out": "", "copies": 1, "kind": 2, "sigma": 1e-5,
         "max_norm": 1.0},
        # flat buffers of odd tensors on four replicas, each clipped into its optimizer's buffer
        {"name": "clip_replicas_odd", "op": "clip", "layout": "pattern", "tensors": 161, "unit": 40, "odd": 1,
         "flat": True, "dtype": "f32", "out": "f32", "copies": 4, "kind": 2, "sigma": 1e-2, "max_norm": 1.0},
        # bf16 weight gradients of the 1B decoder clipped into the optimizer's fp32 gradients
        {"name": "clip_decoder", "op": "clip", "layout": "decoder", "layers": 16, "hidden": 2048, "ffn": 5632,
         "vocab": 32000, "flat": False, "dtype": "bf16", "out": "f32", "copies": 1, "kind": 2, "sigma": 1e-3,
         "max_norm": 1.0},
        # one new token of each of eight sequences
        {"name": "lookup_step", "op": "lookup", "rows": 32000, "width": 2048, "tokens": 8, "table": "bf16",
         "act": "bf16", "index": "i64", "scaled": True, "first": 0, "pad": 0.0},
        # a batch of encoder sequences, fp32 throughout, a third of it padding
        {"name": "lookup_encoder", "op": "lookup", "rows": 30522, "width": 1024, "tokens": 16384, "table": "f32",
         "act": "f32", "index": "i64", "scaled": False, "first": 0, "pad": 0.3},
        # a training batch on one of two vocabulary shards: tokens of the other shard give zero rows
        {"name": "lookup_shard", "op": "lookup", "rows": 16000, "width": 2048, "tokens": 32767, "table": "f32",
         "act": "bf16", "index": "i32", "scaled": True, "first": 8000, "pad": 0.0},
        # a small encoder batch into the fp32 flat buffer
        {"name": "grad_encoder", "op": "grad", "rows": 30522, "width": 1024, "tokens": 2048, "grad": "f32",
         "act": "f32", "index": "i64", "scaled": False, "first": 0, "pad": 0.3, "accumulate": True},
        # a training batch of the 1B decoder accumulated into the fp32 main gradient
        {"name": "grad_decoder", "op": "grad", "rows": 32000, "width": 2048, "tokens": 32768, "grad": "f32",
         "act": "bf16", "index": "i64", "scaled": True, "first": 0, "pad": 0.0, "accumulate": True},
        # a whole bf16 weight gradient for the reducer, rows without a token written as zero
        {"name": "grad_whole_bf16", "op": "grad", "rows": 32000, "width": 2047, "tokens": 8191, "grad": "bf16",
         "act": "bf16", "index": "i32", "scaled": False, "first": 0, "pad": 0.1, "accumulate": False},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm evenly spread, odd ones among them."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v + rng.choice((0, 0, 1))))


def _draw_list(rng):
    kind = rng.choice(("pattern", "pattern", "decoder", "encoder"))
    if kind == "pattern":
        c = {"layout": "pattern", "tensors": _log(rng, 1, 400), "unit": _log(rng, 1, 200), "odd": rng.choice((0, 1))}
    elif kind == "decoder":
        hidden = 64 * rng.randint(4, 32)
        c = {"layout": "decoder", "layers": rng.randint(1, 16), "hidden": hidden, "ffn": 11 * hidden // 4,
             "vocab": _log(rng, 1000, 32000)}
    else:
        hidden = 64 * rng.randint(2, 16)
        c = {"layout": "encoder", "layers": rng.randint(1, 24), "hidden": hidden, "ffn": 4 * hidden,
             "vocab": _log(rng, 1000, 30522)}
    c["flat"] = rng.random() < 0.5
    c["dtype"] = rng.choice(("f32", "f32", "bf16", "f16"))
    c["kind"] = rng.choice((2, 2, 2, 1, 0))
    c["sigma"] = rng.choice((1e-3, 1e-2, 0.1))
    return c


def draw(rng):
    op = rng.choice(("norm", "clip", "lookup", "grad"))
    if op == "norm":
        return {"op": op, **_draw_list(rng)}
    if op == "clip":
        c = {"op": op, **_draw_list(rng)}
        if rng.random() < 0.25:   # in place, below the bound
            c.update(out="", copies=rng.randint(1, 2), max_norm=1e9)
        else:
            c.update(out=rng.choice(("f32", c["dtype"])), copies=rng.randint(1, 2), max_norm=rng.choice((0.1, 1.0)))
        return c
    width = rng.choice((_log(rng, 64, 4096), 64 * _log(rng, 1, 64), 8 * _log(rng, 8, 512)))
    rows = _log(rng, 2, 131072)
    tokens = _log(rng, 1, 65536)
    while tokens * width > 32768 * 2048 or rows * width > 32000 * 2048:
        tokens, rows = max(1, tokens * 2 // 3), max(2, rows * 2 // 3)
    first = rng.choice((0, 0, rows // 3))
    c = {"op": op, "rows": rows, "width": width, "tokens": tokens, "act": rng.choice(("f32", "bf16", "bf16", "f16")),
         "index": rng.choice(("i32", "i64")), "scaled": rng.random() < 0.5, "first": first,
         "pad": rng.choice((0.0, 0.0, 0.2, 0.6))}
    if op == "lookup":
        c["table"] = rng.choice(("f32", c["act"]))
    else:
        c["accumulate"] = rng.random() < 0.7
        c["grad"] = "f32" if c["accumulate"] else rng.choice(("f32", c["act"]))
    return c


# ------------------------------------------------------------------ the inputs
def _sizes(c):
    if c["layout"] == "pattern":
        return [PATTERN[i % 8] * c["unit"] + (i % 61 if c["odd"] else 0) for i in range(c["tensors"])]
    h, f, v = c["hidden"], c["ffn"], c["vocab"]
    if c["layout"] == "decoder":   # embedding; per layer two norms, four projections, a gated block; norm, head
        return [v * h] + [h, h * h, h * h, h * h, h * h, h, f * h, f * h, h * f] * c["layers"] + [h, v * h]
    return ([v * h, 512 * h, 2 * h, h, h] + ([h * h, h] * 4 + [h, h, f * h, f, h * f, h, h, h]) * c["layers"]
            + [h * h, h])


def _offsets(c):
    """Element offsets of the tensors in their buffer (back to back, or each on a boundary of 128) and its length."""
    at, offs = 0, []
    for n in _sizes(c):
        offs.append(at)
        at += n if c["flat"] else -(-n // 128) * 128
    return offs, at


def _views(c, buf):
    return [buf[o:o + n] for o, n in zip(_offsets(c)[0], _sizes(c))]


def _cdf(c):
    """Frequencies of a vocabulary's tokens, falling as the inverse of their rank; over the whole vocabulary
    (a shard's rows and, where it does not begin at zero, as many others)."""
    v = c["rows"] + (c["rows"] if c["first"] else 0)
    p = 1.0 / (torch.arange(v, dtype=torch.float64) + 2.7)
    return torch.cumsum(p / p.sum(), 0), v


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62) + 97)
    return g


def _normal(n, dtype, sigma, g):
    t = torch.empty(n, dtype=dtype, device="cuda")
    t.normal_(0.0, sigma, generator=g)
    return t


def _prepare_list(c, seed):
    g = _generator(seed)
    n = _offsets(c)[1]
    copies = c.get("copies", 1)
    dtype = TYPES[c["dtype"]]
    first = torch.zeros(n, dtype=dtype, device="cuda")
    if c["flat"]:
        first.normal_(0.0, c["sigma"], generator=g)
    else:
        for v in _views(c, first):
            v.normal_(0.0, c["sigma"], generator=g)
    bufs = [first] + [first.clone() for _ in range(copies - 1)]
    s = {"case": c, "in": bufs, "norm": torch.zeros((), dtype=torch.float32, device="cuda")}
    s["out"] = [torch.zeros(n, dtype=TYPES[c["out"]], device="cuda") for _ in bufs] if c.get("out") else bufs
    # a flat buffer is one tensor to the plain form; separate tensors are taken one by one
    s["pieces"] = [[b] if c["flat"] else _views(c, b) for b in bufs]
    s["out_pieces"] = [[b] if c["flat"] else _views(c, b) for b in s["out"]]
    if own:
        import bucketed_gradient_all_amd as ddp
        names = {"f32": ddp.DDP_F32, "bf16": ddp.DDP_BF16, "f16": ddp.DDP_F16}
        sizes = _sizes(c)
        ptrs = [[v.data_ptr() for v in _views(c, b)] for b in bufs]
        out = [[v.data_ptr() for v in _views(c, b)] for b in s["out"]] if c.get("out") else None
        s["grads"] = ddp.make_grads(sizes, ptrs, [names[c["dtype"]]] * len(sizes), out_ptrs=out,
                                    out_dtype=[names[c["out"]]] * len(sizes) if out else None)
        s["kind"] = {0: ddp.DDP_NORM_INF, 1: ddp.DDP_NORM_L1, 2: ddp.DDP_NORM_L2}[c["kind"]]
    return s


def _prepare_embedding(c, seed):
    g = _generator(seed)
    cdf, v = _cdf(c)
    n, width, rows = c["tokens"], c["width"], c["rows"]
    index = torch.int32 if c["index"] == "i32" else torch.int64
    rank = torch.searchsorted(cdf.cuda(), torch.rand(n, dtype=torch.float64, device="cuda", generator=g))
    step = next(k for k in (7919, 104729, 1299709) if math.gcd(k, v) == 1)
    tokens = (rank.clamp(max=v - 1) * step + 11) % v          # frequent tokens lie all over the vocabulary
    padding = c["first"] + 1 if c["pad"] else -1
    if c["pad"]:   # each run of 128 positions ends in padding
        length = 128 - int(128 * c["pad"])
        tail = torch.arange(n, device="cuda") % 128 >= length
        tokens = torch.where(tail, torch.full_like(tokens, padding), tokens)
    s = {"case": c, "tokens": tokens.to(index), "scale": math.sqrt(width) if c["scaled"] else 1.0, "padding": padding}
    act = TYPES[c["act"]]
    if c["op"] == "lookup":
        s["table"] = _normal(rows * width, TYPES[c["table"]], 0.02, g).view(rows, width)
        s["out"] = torch.empty(n, width, dtype=act, device="cuda")
    else:
        s["dout"] = _normal(n * width, act, 1e-3, g).view(n, width)
        s["grad"] = _normal(rows * width, TYPES[c["grad"]], 1e-3, g).view(rows, width)
    if own:
        import bucketed_gradient_all_amd as ddp
        names = {"f32": ddp.DDP_F32, "bf16": ddp.DDP_BF16, "f16": ddp.DDP_F16}
        s["desc"] = ddp.EmbeddingDesc(rows, width, table_dtype=names[c.get("table", "f32")],
                                      grad_dtype=names[c.get("grad", "f32")], act_dtype=names[c["act"]],
                                      index_dtype=ddp.DDP_I32 if c["index"] == "i32" else ddp.DDP_I64,
                                      scale=s["scale"], first_row=c["first"], padding_idx=padding)
        if c["op"] == "grad":
            s["work"] = torch.empty(ddp.ddp_embedding_grad_workspace_bytes(s["desc"], n), dtype=torch.uint8,
                                    device="cuda")
    return s


def prepare(case, seed):
    return (_prepare_list if case["op"] in ("norm", "clip") else _prepare_embedding)(case, seed)


# ------------------------------------------------------------------ one pass
def _plain_norm(pieces, kind):
    """Sums in 64 bits: they run over up to a billion values."""
    x = [p.float().abs() for p in pieces]
    if kind == 0:
        return torch.stack([p.max() for p in x]).max()
    if kind == 1:
        return torch.stack([p.sum(dtype=torch.float64) for p in x]).sum().float()
    return torch.stack([(p * p).sum(dtype=torch.float64) for p in x]).sum().sqrt().float()


def _inside(s):
    """Rows of the tokens in this table, and which of them it holds."""
    row = s["tokens"].long() - s["case"]["first"]
    return row, (row >= 0) & (row < s["case"]["rows"])


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s["pieces"][0], c["kind"])
    if c["op"] == "clip":
        norm = _plain_norm(s["pieces"][0], c["kind"])
        factor = (c["max_norm"] / (norm + EPS)).clamp(max=1.0)
        pairs = [(p, o) for ps, os in zip(s["pieces"], s["out_pieces"]) for p, o in zip(ps, os)]
        _ = [torch.mul(p, factor, out=o) if p.dtype == o.dtype == torch.float32 else o.copy_(p.float() * factor)
             for p, o in pairs]
        return norm, s["out"]
    row, inside = _inside(s)
    if c["op"] == "lookup":
        x = s["table"][row.clamp(0, c["rows"] - 1)].float() * s["scale"]
        return (x * inside[:, None]).to(s["out"].dtype)
    inside = inside & (s["tokens"] != s["padding"])
    x = s["dout"].float() * s["scale"] * inside[:, None]
    row = row.clamp(0, c["rows"] - 1)
    if c["accumulate"]:
        return s["grad"].index_add_(0, row, x)
    full = torch.zeros(c["rows"], c["width"], dtype=torch.float32, device=x.device).index_add_(0, row, x)
    return full.to(s["grad"].dtype)


def _own(s):
    import bucketed_gradient_all_amd as ddp
    c = s["case"]
    stream = torch.cuda.current_stream().cuda_stream
    if c["op"] == "norm":
        ddp.ddp_grad_norm(s["grads"], s["kind"], s["norm"].data_ptr(), stream)
        return s["norm"]
    if c["op"] == "clip":
        ddp.ddp_clip_grad_norm(s["grads"], s["kind"], c["max_norm"], s["norm"].data_ptr(), stream)
        return s["norm"], s["out"]
    if c["op"] == "lookup":
        ddp.ddp_embedding_lookup(s["desc"], s["table"].data_ptr(), s["tokens"].data_ptr(), c["tokens"],
                                 s["out"].data_ptr(), stream)
        return s["out"]
    ddp.ddp_embedding_grad(s["desc"], s["dout"].data_ptr(), s["tokens"].data_ptr(), c["tokens"],
                           s["grad"].data_ptr(), c["accumulate"], s["work"].data_ptr(), s["work"].numel(), stream)
    return s["grad"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2, "": 0}
    if c["op"] in ("norm", "clip"):
        n = sum(_sizes(c))
        if c["op"] == "norm":
            return {"bytes": n * size[c["dtype"]] + 4, "flops": 2 * n}
        # in place below the bound nothing has to be written, and only the norm's copy is read
        moved = n * c["copies"] * (size[c["dtype"]] + size[c["out"]]) if c["out"] else n * size[c["dtype"]]
        return {"bytes": moved + 4, "flops": 2 * n + n * c["copies"]}
    n, width = c["tokens"], c["width"]
    cdf, v = _cdf(c)
    p = torch.diff(cdf, prepend=torch.zeros(1, dtype=torch.float64))
    share = c["rows"] / v                                       # of the tokens this table holds
    real = n * (1.0 - c["pad"])
    used = float((1.0 - (1.0 - p) ** real).sum()) * share       # rows that occur
    index = n * (4 if c["index"] == "i32" else 8)
    if c["op"] == "lookup":
        return {"bytes": used * width * size[c["table"]] + n * width * size[c["act"]] + index, "flops": n * width}
    read = real * share * width * size[c["act"]]
    wrote = 2 * used * width * size[c["grad"]] if c["accumulate"] else c["rows"] * width * size[c["grad"]]
    return {"bytes": read + wrote + index, "flops": 2 * real * share * width}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] in ("norm", "clip"):
        x = s["in"][0].double()                                 # gaps between tensors hold zeros
        norm = {0: lambda: x.abs().max(), 1: lambda: x.abs().sum(), 2: lambda: torch.linalg.vector_norm(x)}[c["kind"]]()
        if c["op"] == "norm":
            return norm
        x.mul_(min(1.0, c["max_norm"] / (float(norm) + EPS)))
        return norm, [x for _ in s["in"]]
    where = s["tokens"].cpu().long() - c["first"]
    held = (where >= 0) & (where < c["rows"])
    if c["op"] == "lookup":
        out = torch.zeros(c["tokens"], c["width"], dtype=torch.float64, device="cuda")
        keep = held.nonzero()[:, 0].cuda()
        out[keep] = s["table"].double()[where[held].cuda()] * s["scale"]
        return out
    held &= s["tokens"].cpu().long() != s["padding"]
    # sums over sorted tokens: differences of a running sum lose too much, so rows go in by their turn
    at = held.nonzero()[:, 0]
    rows, order = torch.sort(where[at], stable=True)
    begin = torch.searchsorted(rows, rows)                      # first place of the same row
    turn = torch.arange(rows.numel()) - begin
    total = s["grad"].double() if c["accumulate"] else torch.zeros_like(s["grad"], dtype=torch.float64)
    rows, source, turn = rows.cuda(), at[order].cuda(), turn.cuda()
    few = int(turn.max()) + 1 if rows.numel() else 0
    for k in range(min(few, 64)):                               # every row once per turn: no two writes meet
        now = turn == k
        total[rows[now]] += s["dout"][source[now]].double() * s["scale"]
    late = turn >= 64
    for r in rows[late].unique().tolist() if few > 64 else ():  # the frequent rows' remainders
        total[r] += s["dout"][source[late & (rows == r)]].double().sum(0) * s["scale"]
    return total
