"""The optimizer's step and the layer norm as measured cases.

Four operators, each with its plain form in elementary torch operations and the
call a user makes of the library:

  adamw      one AdamW step over many tensors, the moments held in 32 bits; the
             gradients scaled by min(1, max_norm / (norm + 1e-6)) as they are read
  adamw8     the same with the moments held in 8 bits: blocks of 128 values, one
             scale a block, e4m3 codes of the first moment and of the root of the
             second
  layernorm  rows normalised by mean and variance, or by their mean square, with
             the residual added before
  layergrad  its backward pass: the rows' gradient, and the weight's and bias's,
             added to what the gradient buffer holds or written over it

`own` selects the side `run` takes; it is set from outside.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "": 0}
CLIP_EPS = 1e-6      # added to the norm before the division, as gradient clipping usually does
BLOCK = 128          # values of the 8-bit states with one scale
TOP = 448.0          # the largest e4m3 number
TINY = 2.0 ** -100   # a block whose largest value is below it is held as zeros
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8

# sizes of the eight-tensor list: weights and biases of a few small layers
PATTERN = (4096, 64, 16384, 128, 8192, 256, 2048, 32)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small network's first step: latency of one call
        {"name": "adamw_small", "op": "adamw", "layout": "pattern", "tensors": 8, "unit": 1, "odd": 0, "packed": False,
         "flat": False, "grad": "f32", "param": "f32", "copy": "", "bits": 32, "lr": 1e-3, "decay": 0.01, "step": 1,
         "clip": "", "sigma": 1e-2},
        # the encoder's flat fp32 buffer after the reduction, norm below the bound
        {"name": "adamw_encoder", "op": "adamw", "layout": "encoder", "layers": 24, "hidden": 1024, "ffn": 4096,
         "vocab": 30522, "packed": True, "flat": True, "grad": "f32", "param": "f32", "copy": "", "bits": 32,
         "lr": 1e-4, "decay": 0.01, "step": 1000, "clip": "below", "sigma": 1e-4},
        # bf16 weight gradients of a 1B decoder, fp32 parameters and the bf16 copy the next forward reads, clipped
        {"name": "adamw_decoder", "op": "adamw", "layout": "decoder", "layers": 16, "hidden": 2048, "ffn": 5632,
         "vocab": 32000, "packed": False, "flat": False, "grad": "bf16", "param": "f32", "copy": "bf16", "bits": 32,
         "lr": 3e-4, "decay": 0.1, "step": 2000, "clip": "above", "sigma": 1e-3},
        # odd tensors back to back, fp16 throughout but for the fp32 parameters
        {"name": "adamw8_odd", "op": "adamw", "layout": "pattern", "tensors": 161, "unit": 40, "odd": 1,
         "packed": True, "flat": False, "grad": "f16", "param": "f32", "copy": "f16", "bits": 8, "lr": 1e-3,
         "decay": 0.01, "step": 10, "clip": "above", "sigma": 1e-2},
        # the 1B decoder with the moments in 8 bits
        {"name": "adamw8_decoder", "op": "adamw", "layout": "decoder", "layers": 16, "hidden": 2048, "ffn": 5632,
         "vocab": 32000, "packed": False, "flat": False, "grad": "bf16", "param": "f32", "copy": "bf16", "bits": 8,
         "lr": 3e-4, "decay": 0.1, "step": 2000, "clip": "above", "sigma": 1e-3},
        # one of eight owners' shard of the encoder after a reduce-scatter: fp32 gradients, bf16 parameters alone
        {"name": "adamw8_shard", "op": "adamw", "layout": "shard", "numel": 41892352, "packed": True, "flat": True,
         "grad": "f32", "param": "bf16", "copy": "", "bits": 8, "lr": 1e-4, "decay": 0.01, "step": 1000, "clip": "",
         "sigma": 1e-4},
        # one new token of each of eight sequences, with the residual
        {"name": "layernorm_step", "op": "layernorm", "kind": "rms", "rows": 8, "width": 2048, "x": "bf16",
         "y": "bf16", "weight": "bf16", "add": True, "stats": False},
        # a batch of encoder sequences, fp32 throughout
        {"name": "layernorm_encoder", "op": "layernorm", "kind": "layer", "rows": 16384, "width": 1024, "x": "f32",
         "y": "f32", "weight": "f32", "add": True, "stats": True},
        # a training batch of the 1B decoder
        {"name": "layernorm_decoder", "op": "layernorm", "kind": "rms", "rows": 32768, "width": 2048, "x": "bf16",
         "y": "bf16", "weight": "bf16", "add": True, "stats": True},
        # a small encoder batch, the weight's gradient into the fp32 flat buffer
        {"name": "layergrad_encoder", "op": "layergrad", "kind": "layer", "rows": 2048, "width": 1024, "x": "f32",
         "y": "f32", "weight": "f32", "grad": "f32", "dz": True, "accumulate": True},
        # a training batch of the 1B decoder, the weight's gradient added to the fp32 main gradient
        {"name": "layergrad_decoder", "op": "layergrad", "kind": "rms", "rows": 32768, "width": 2048, "x": "bf16",
         "y": "bf16", "weight": "bf16", "grad": "f32", "dz": True, "accumulate": True},
        # odd sizes: an fp32 stream normalised into bf16, whole bf16 gradients for the reducer
        {"name": "layergrad_odd", "op": "layergrad", "kind": "layer", "rows": 8191, "width": 2047, "x": "f32",
         "y": "bf16", "weight": "f32", "grad": "bf16", "dz": False, "accumulate": False},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm evenly spread, odd ones among them."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v + rng.choice((0, 0, 1))))


def _draw_adamw(rng):
    kind = rng.choice(("pattern", "pattern", "decoder", "encoder", "shard"))
    if kind == "pattern":
        c = {"layout": kind, "tensors": _log(rng, 1, 400), "unit": _log(rng, 1, 200), "odd": rng.choice((0, 1)),
             "flat": False}
    elif kind == "decoder":
        hidden = 64 * rng.randint(4, 30)
        c = {"layout": kind, "layers": rng.randint(1, 16), "hidden": hidden, "ffn": 11 * hidden // 4,
             "vocab": _log(rng, 1000, 32000), "flat": rng.random() < 0.5}
    elif kind == "encoder":
        hidden = 64 * rng.randint(2, 16)
        c = {"layout": kind, "layers": rng.randint(1, 24), "hidden": hidden, "ffn": 4 * hidden,
             "vocab": _log(rng, 1000, 30522), "flat": rng.random() < 0.5}
    else:
        c = {"layout": kind, "numel": _log(rng, 1, 1 << 27), "flat": True}
    c["packed"] = rng.random() < 0.5
    c["grad"] = rng.choice(("f32", "f32", "bf16", "f16"))
    c["param"] = rng.choice(("f32", "f32", "f32", "bf16"))
    c["copy"] = rng.choice(("", "bf16", "f16")) if c["param"] == "f32" else ""
    c["bits"] = rng.choice((32, 8))
    c["lr"], c["decay"] = rng.choice((1e-4, 1e-3)), rng.choice((0.0, 0.01, 0.1))
    c["step"] = rng.choice((1, 10, 1000, 100000))
    c["clip"] = rng.choice(("", "above", "below"))
    c["sigma"] = rng.choice((1e-4, 1e-3, 1e-2))
    return c


def draw(rng):
    op = rng.choice(("adamw", "adamw", "layernorm", "layergrad"))
    if op == "adamw":
        return {"op": op, **_draw_adamw(rng)}
    width = rng.choice((_log(rng, 8, 16384), 64 * _log(rng, 1, 128), 8 * _log(rng, 1, 1024)))
    rows = _log(rng, 1, 65536)
    while rows * width > 16384 * 2048:
        rows = max(1, rows * 2 // 3)
    x = rng.choice(("f32", "bf16", "bf16", "f16"))
    c = {"op": op, "kind": rng.choice(("layer", "layer", "rms")), "rows": rows, "width": width, "x": x,
         "y": rng.choice(("f32", "bf16", "f16")) if x == "f32" else x, "weight": rng.choice(("f32", x))}
    if op == "layernorm":
        return {**c, "add": rng.random() < 0.5, "stats": rng.random() < 0.7}
    c["dz"], c["accumulate"] = rng.random() < 0.5, rng.random() < 0.6
    c["grad"] = "f32" if c["accumulate"] else rng.choice(("f32", c["weight"]))
    return c


# ------------------------------------------------------------------ the inputs
def _sizes(c):
    if c["layout"] == "shard":
        return [c["numel"]]
    if c["layout"] == "pattern":
        return [PATTERN[i % 8] * c["unit"] + (i % 61 if c["odd"] else 0) for i in range(c["tensors"])]
    h, f, v = c["hidden"], c["ffn"], c["vocab"]
    if c["layout"] == "decoder":   # embedding; per layer two norms, four projections, a gated block; norm, head
        s = [v * h] + [h, h * h, h * h, h * h, h * h, h, f * h, f * h, h * f] * c["layers"] + [h, v * h]
    else:
        s = ([v * h, 512 * h, 2 * h, h, h] + ([h * h, h] * 4 + [h, h, f * h, f, h * f, h, h, h]) * c["layers"]
             + [h * h, h])
    return [sum(s)] if c["flat"] else s


def _offsets(c):
    """Element offsets of the tensors in their buffer (back to back, or each on a boundary of 128) and its length."""
    at, offs = 0, []
    for n in _sizes(c):
        offs.append(at)
        at += n if c["packed"] else -(-n // 128) * 128
    return offs, at


def _blocks(n):
    return -(-n // BLOCK)


def _decays(c):
    """Weight decay of each tensor: none for vectors, which are the lists' small tensors."""
    sizes = _sizes(c)
    return [0.0 if n <= max(sizes) // 256 else c["decay"] for n in sizes]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2654435761 % (1 << 62) + 97)
    return g


def _normal(n, dtype, sigma, g):
    t = torch.empty(n, dtype=dtype, device="cuda")
    t.normal_(0.0, sigma, generator=g)
    return t


def _views(c, buf):
    return [buf[o:o + n] for o, n in zip(_offsets(c)[0], _sizes(c))]


def _scale_views(c, buf):
    at, out = 0, []
    for n in _sizes(c):
        out.append(buf[at:at + _blocks(n)])
        at += _blocks(n)
    return out


def _in_blocks(x):
    n = x.numel()
    return (torch.nn.functional.pad(x, (0, -n % BLOCK)) if n % BLOCK else x).view(-1, BLOCK)


def _encode(x, positive):
    """Codes and scales of fp32 values: the block's largest becomes 448. A positive value keeps a positive code where
    `positive` is true, so that a second moment never becomes zero beside a first one that is not."""
    n = x.numel()
    b = _in_blocks(x)
    top = b.abs().amax(1)
    none = top < TINY
    scale = torch.where(none, 0.0, top / TOP)
    code = (b * torch.where(none, 0.0, TOP / top)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if positive:
        code = torch.where((b > 0) & (code == 0), 1, code)
    return code.view(-1)[:n], scale


def _decode(code, scale):
    n = code.numel()
    return (_in_blocks(code).view(torch.float8_e4m3fn).float() * scale[:, None]).view(-1)[:n]


def _encode_into(x, positive, code, scale):
    new = _encode(x, positive)
    code.copy_(new[0])
    scale.copy_(new[1])


def _prepare_adamw(c, seed):
    g = _generator(seed)
    n = _offsets(c)[1]
    sigma, first = c["sigma"], c["step"] == 1
    s = {"case": c, "step": c["step"], "g": _normal(n, TYPES[c["grad"]], sigma, g),
         "p": _normal(n, TYPES[c["param"]], 0.02, g)}
    s["copy"] = s["p"].to(TYPES[c["copy"]]) if c["copy"] else None
    # moments as a run leaves them behind it, zero before the first step
    m = torch.zeros(n, device="cuda") if first else _normal(n, torch.float32, 0.3 * sigma, g)
    r = torch.zeros(n, device="cuda") if first else _normal(n, torch.float32, 0.2 * sigma, g).abs_().add_(0.8 * sigma)
    if c["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        blocks = sum(_blocks(k) for k in _sizes(c))
        s["m"], s["v"] = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["ms"], s["vs"] = (torch.zeros(blocks, device="cuda") for _ in range(2))
        for x, positive, code, scale in ((m, False, "m", "ms"), (r, True, "v", "vs")):
            for a, b, d in zip(_views(c, x), _views(c, s[code]), _scale_views(c, s[scale])):
                _encode_into(a, positive, b, d)
    # the norm of all of the model's gradients, which the step is given
    s["norm"] = torch.full((), sigma * math.sqrt(n), device="cuda") if c["clip"] else None
    s["max_norm"] = {"": 0.0, "above": 0.5, "below": 2.0}[c["clip"]] * sigma * math.sqrt(n)
    s["decay"] = _decays(c)
    s["pieces"] = [dict(zip(("g", "p", "copy", "m", "v", "ms", "vs"), t)) for t in zip(*(
        [None] * len(_sizes(c)) if s.get(k) is None else (_scale_views if k in ("ms", "vs") else _views)(c, s[k])
        for k in ("g", "p", "copy", "m", "v", "ms", "vs")))]
    if own:
        import bucketed_gradient_all_amd as ddp
        names = {"f32": ddp.DDP_F32, "bf16": ddp.DDP_BF16, "f16": ddp.DDP_F16}
        sizes = _sizes(c)

        def pointers(k):
            return [t[k].data_ptr() for t in s["pieces"]] if s.get(k) is not None else None

        s["opt"] = ddp.make_adamw(
            sizes, pointers("g"), pointers("p"), pointers("m"), pointers("v"),
            grad_dtype=[names[c["grad"]]] * len(sizes), param_dtype=[names[c["param"]]] * len(sizes),
            copy_ptrs=pointers("copy"), copy_dtype=[names[c["copy"]]] * len(sizes) if c["copy"] else None,
            state=ddp.DDP_STATE_F32 if c["bits"] == 32 else ddp.DDP_STATE_8BIT,
            m_scale_ptrs=pointers("ms"), v_scale_ptrs=pointers("vs"), weight_decay=s["decay"])
    return s


def _prepare_layernorm(c, seed):
    g = _generator(seed)
    rows, h, xt, yt = c["rows"], c["width"], TYPES[c["x"]], TYPES[c["y"]]
    layer = c["kind"] == "layer"
    s = {"case": c, "eps": 1e-5}
    # rows of different size, and a little off centre
    x = _normal(rows * h, torch.float32, 1.0, g).view(rows, h)
    x.mul_(torch.exp(_normal(rows, torch.float32, 0.5, g))[:, None]).add_(_normal(rows, torch.float32, 0.2, g)[:, None])
    s["weight"] = (1.0 + _normal(h, torch.float32, 0.1, g)).to(TYPES[c["weight"]])
    s["bias"] = _normal(h, torch.float32, 0.1, g).to(TYPES[c["weight"]]) if layer else None
    x = x.to(xt)
    if c["op"] == "layernorm":
        s["x"] = x
        s["add"] = _normal(rows * h, xt, 0.5, g).view(rows, h) if c["add"] else None
        s["z"] = torch.empty(rows, h, dtype=xt, device="cuda") if c["add"] else None
        s["out"] = torch.empty(rows, h, dtype=yt, device="cuda")
        s["mean"] = torch.empty(rows, device="cuda") if c["stats"] and layer else None
        s["rstd"] = torch.empty(rows, device="cuda") if c["stats"] else None
    else:
        s["z"] = x
        s["dy"] = _normal(rows * h, yt, 1e-3, g).view(rows, h)
        s["dz"] = _normal(rows * h, xt, 1e-3, g).view(rows, h) if c["dz"] else None
        s["dx"] = torch.empty(rows, h, dtype=xt, device="cuda")
        s["dweight"] = _normal(h, TYPES[c["grad"]], 1e-3, g)
        s["dbias"] = _normal(h, TYPES[c["grad"]], 1e-3, g) if layer else None
        # what the forward pass kept
        s["mean"], s["rstd"] = _stats64(x.double(), c, s["eps"])
        s["mean"], s["rstd"] = s["mean"].float()[:, 0] if layer else None, s["rstd"].float()[:, 0]
    if own:
        import bucketed_gradient_all_amd as ddp
        names = {"f32": ddp.DDP_F32, "bf16": ddp.DDP_BF16, "f16": ddp.DDP_F16}
        s["desc"] = ddp.LayerNormDesc(h, kind=ddp.DDP_LAYER_NORM if layer else ddp.DDP_RMS_NORM,
                                      x_dtype=names[c["x"]], y_dtype=names[c["y"]], weight_dtype=names[c["weight"]],
                                      grad_dtype=names[c.get("grad", "f32")], eps=s["eps"])
        if c["op"] == "layergrad":
            s["work"] = torch.empty(ddp.ddp_layernorm_grad_workspace_bytes(s["desc"], rows), dtype=torch.uint8,
                                    device="cuda")
    return s


def prepare(case, seed):
    return (_prepare_adamw if case["op"] == "adamw" else _prepare_layernorm)(case, seed)


# ------------------------------------------------------------------ one pass
def _outputs(s):
    c = s["case"]
    if c["op"] == "adamw":
        state = {"m": s["m"], "v": s["v"]} if c["bits"] == 32 else {
            "m": s["m"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "ms": s["ms"], "vs": s["vs"]}
        return {"p": s["p"], "copy": s["copy"], **state}
    if c["op"] == "layernorm":
        return {"y": s["out"], "z": s["z"], "mean": s["mean"], "rstd": s["rstd"]}
    return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}


def _scalars(s):
    c, t = s["case"], s["step"]
    return c["lr"] / (1.0 - BETA1 ** t), 1.0 / math.sqrt(1.0 - BETA2 ** t)


def _plain_adamw_piece(s, t, decay, factor):
    c = s["case"]
    size, root = _scalars(s)
    g = t["g"].float()
    if factor is not None:
        g = g * factor
    m = t["m"] if c["bits"] == 32 else _decode(t["m"], t["ms"])
    v = t["v"] if c["bits"] == 32 else _decode(t["v"], t["vs"]).square_()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    r = v.sqrt()
    p = t["p"].float() * (1.0 - c["lr"] * decay) - (m / (r * root + EPS)) * size
    t["p"].copy_(p)
    if c["copy"]:
        t["copy"].copy_(p)
    if c["bits"] == 32:
        t["m"].copy_(m)
        t["v"].copy_(v)
    else:
        _encode_into(m, False, t["m"], t["ms"])
        _encode_into(r, True, t["v"], t["vs"])


def _plain(s):
    c = s["case"]
    if c["op"] == "adamw":
        factor = (s["max_norm"] / (s["norm"] + CLIP_EPS)).clamp(max=1.0) if c["clip"] else None
        _ = [_plain_adamw_piece(s, t, d, factor) for t, d in zip(s["pieces"], s["decay"])]
        s["step"] += 1
        return _outputs(s)
    layer = c["kind"] == "layer"
    w = s["weight"].float()
    if c["op"] == "layernorm":
        z = s["x"]
        if c["add"]:
            z = s["z"].copy_(z.float() + s["add"].float())
        x = z.float()
        mean = x.mean(1, keepdim=True) if layer else None
        x = x - mean if layer else x
        rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"])
        y = x * rstd * w
        s["out"].copy_(y + s["bias"].float() if layer else y)
        if c["stats"]:
            s["rstd"].copy_(rstd[:, 0])
            if layer:
                s["mean"].copy_(mean[:, 0])
        return _outputs(s)
    x, dy, rstd = s["z"].float(), s["dy"].float(), s["rstd"][:, None]
    hat = (x - s["mean"][:, None] if layer else x) * rstd
    dw = (dy * hat).sum(0)
    db = dy.sum(0) if layer else None
    d = dy * w
    dx = d - hat * (d * hat).mean(1, keepdim=True)
    dx = (dx - d.mean(1, keepdim=True) if layer else dx) * rstd
    s["dx"].copy_(dx + s["dz"].float() if c["dz"] else dx)
    old = c["accumulate"]
    s["dweight"].copy_(s["dweight"].float() + dw if old else dw)
    if layer:
        s["dbias"].copy_(s["dbias"].float() + db if old else db)
    return _outputs(s)


def _ptr(t):
    return t.data_ptr() if t is not None else 0


def _own(s):
    import bucketed_gradient_all_amd as ddp
    c = s["case"]
    stream = torch.cuda.current_stream().cuda_stream
    if c["op"] == "adamw":
        ddp.ddp_adamw_step(s["opt"], c["lr"], s["step"], stream, beta1=BETA1, beta2=BETA2, eps=EPS,
                           max_norm=s["max_norm"], norm=_ptr(s["norm"]))
        s["step"] += 1
    elif c["op"] == "layernorm":
        ddp.ddp_layernorm(s["desc"], c["rows"], s["x"].data_ptr(), s["weight"].data_ptr(), _ptr(s["bias"]),
                          s["out"].data_ptr(), stream, add=_ptr(s["add"]), z=_ptr(s["z"]), mean=_ptr(s["mean"]),
                          rstd=_ptr(s["rstd"]))
    else:
        ddp.ddp_layernorm_grad(s["desc"], c["rows"], s["dy"].data_ptr(), s["z"].data_ptr(), s["weight"].data_ptr(),
                               _ptr(s["mean"]), s["rstd"].data_ptr(), s["dx"].data_ptr(), s["dweight"].data_ptr(),
                               _ptr(s["dbias"]), c["accumulate"], s["work"].data_ptr(), s["work"].numel(), stream,
                               dz=_ptr(s["dz"]))
    return _outputs(s)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(_sizes(c))
        blocks = sum(_blocks(k) for k in _sizes(c))
        states = 16 * n if c["bits"] == 32 else 4 * n + 16 * blocks      # both moments read and written
        return {"bytes": states + n * (SIZE[c["grad"]] + 2 * SIZE[c["param"]] + SIZE[c["copy"]]), "flops": 14 * n}
    n, h, rows = c["rows"] * c["width"], c["width"], c["rows"]
    vectors = 2 if c["kind"] == "layer" else 1                           # weight and bias, mean and 1 / deviation
    x, y = SIZE[c["x"]], SIZE[c["y"]]
    if c["op"] == "layernorm":
        moved = n * (x + y + (2 * x if c["add"] else 0)) + (4 * vectors * rows if c["stats"] else 0)
        return {"bytes": moved + vectors * h * SIZE[c["weight"]], "flops": 8 * n}
    moved = n * (2 * x + y + (x if c["dz"] else 0)) + 4 * vectors * rows + h * SIZE[c["weight"]]
    return {"bytes": moved + vectors * h * SIZE[c["grad"]] * (2 if c["accumulate"] else 1), "flops": 16 * n}


# ------------------------------------------------------------------ the definition, in 64 bits
def _stats64(x, c, eps):
    mean = x.sum(1, keepdim=True) / x.shape[1] if c["kind"] == "layer" else torch.zeros_like(x[:, :1])
    return mean, ((x - mean).square().sum(1, keepdim=True) / x.shape[1] + eps).pow(-0.5)


def _exact_codes(x, sizes, offs, positive):
    """Codes (in a buffer like x) and scales of x, block by block."""
    code, scales = torch.zeros_like(x), []
    for n, o in zip(sizes, offs):
        whole = n // BLOCK * BLOCK
        for a, b in ((o, o + whole), (o + whole, o + n)):
            if a == b:
                continue
            v = x[a:b].reshape(-1, min(BLOCK, b - a))
            top = v.abs().max(1, keepdim=True).values
            scale = torch.where(top < TINY, 0.0, top / TOP)
            q = torch.where(top < TINY, 0.0, v / scale)
            # e4m3: four exponent bits, three of fraction, steps of 2^-9 below 2^-6
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            q = torch.round(q / step) * step
            if positive:
                q = torch.where((v > 0) & (q == 0), 2.0 ** -9, q)
            code[a:b] = q.reshape(-1)
            scales.append(scale[:, 0])
    return code, torch.cat(scales)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = case
    if c["op"] == "adamw":
        offs, sizes = _offsets(c)[0], _sizes(c)
        used = torch.zeros(s["g"].numel(), dtype=torch.bool, device="cuda")
        keep = torch.ones(s["g"].numel(), dtype=torch.float64, device="cuda")
        old = {k: torch.zeros_like(keep) for k in ("m", "v")}
        at = 0
        for n, o, d in zip(sizes, offs, s["decay"]):
            used[o:o + n] = True
            keep[o:o + n] -= c["lr"] * d
            for k in ("m", "v"):
                x = s[k][o:o + n]
                if c["bits"] == 8:
                    scale = s[k + "s"][at:at + _blocks(n)].double().repeat_interleave(BLOCK)[:n]
                    x = x.view(torch.float8_e4m3fn).double() * scale
                    x = x if k == "m" else x * x
                old[k][o:o + n] = x.double()
            at += _blocks(n)
        g = s["g"].double() * (min(1.0, s["max_norm"] / (float(s["norm"]) + CLIP_EPS)) if c["clip"] else 1.0)
        m = BETA1 * old["m"] + (1.0 - BETA1) * g
        v = BETA2 * old["v"] + (1.0 - BETA2) * g * g
        del old, g
        t = c["step"]
        p0 = s["p"].double()
        p = p0 * keep - c["lr"] * (m / (1.0 - BETA1 ** t)) / (torch.sqrt(v / (1.0 - BETA2 ** t)) + EPS)
        out = {"p": torch.where(used, p, p0), "copy": torch.where(used, p, p0) if c["copy"] else None}
        if c["bits"] == 32:
            return {**out, "m": torch.where(used, m, s["m"].double()), "v": torch.where(used, v, s["v"].double())}
        out["m"], out["ms"] = _exact_codes(m, sizes, offs, False)
        out["v"], out["vs"] = _exact_codes(v.sqrt_(), sizes, offs, True)
        return out
    layer = c["kind"] == "layer"
    w = s["weight"].double()
    if c["op"] == "layernorm":
        z = s["x"].double()
        if c["add"]:
            z = (z + s["add"].double()).to(s["z"].dtype).double()
        mean, rstd = _stats64(z, c, s["eps"])
        y = (z - mean) * rstd * w
        return {"y": y + s["bias"].double() if layer else y, "z": z if c["add"] else None,
                "mean": mean[:, 0] if c["stats"] and layer else None, "rstd": rstd[:, 0] if c["stats"] else None}
    z, dy, rstd = s["z"].double(), s["dy"].double(), s["rstd"].double()[:, None]
    hat = (z - s["mean"].double()[:, None] if layer else z) * rstd
    d, h = dy * w, c["width"]
    # the derivative of each row's normalisation, as its Jacobian applied to d
    along = (d * hat).sum(1, keepdim=True) / h
    shift = d.sum(1, keepdim=True) / h if layer else 0.0
    dx = rstd * (d - shift - hat * along)
    dw, db = (dy * hat).sum(0), dy.sum(0)
    if c["accumulate"]:
        dw = dw + s["dweight"].double()
        db = db + s["dbias"].double() if layer else db
    return {"dx": dx + s["dz"].double() if c["dz"] else dx, "dweight": dw, "dbias": db if layer else None}
