"""The training-step operators around the compressor, as cases to be measured.

Three groups, each over the range of sizes that a data-parallel training run of
the layer tables of this repository meets:

  adamw       the clipped AdamW step on the flat buffers that decode writes,
              over many tensors at once, with float32 or 8-bit moments
  layer_norm  layer norm and its gradients, rows of a training batch down to
              the few rows of a decoding step
  scan        the gated linear recurrence along the sequence and its
              gradients, long sequences down to one new token

``run`` computes a case either in elementary torch operations (``own`` false)
or through the package's calls (``own`` true); ``exact`` computes it in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=100, scale=0.125, max_norm=1.0, seed=1234)
# the float32 values that a call's parameters hold
HYPER = {k: float(torch.tensor(x, dtype=torch.float32)) if isinstance(x, float) else x for k, x in HYPER.items()}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 32          # elements of one tensor that share a block scale of the 8-bit moments
E4M3_MAX_EXP = 8    # 448 = 1.75 * 2^8 is the largest e4m3 value


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one fully connected layer: the smallest optimizer call, latency counts
        {"name": "adamw f32 one layer", "op": "adamw", "table": "100x1000", "states": 32,
         "grad": "f32", "clip": False, "copy": False},
        # 16 square layers of the large flat gradient, decoded float32 sum, clipped
        {"name": "adamw f32 large", "op": "adamw", "table": "16*4096x4096", "states": 32,
         "grad": "f32", "clip": True, "copy": False},
        # 161 tensors from 64 to 2.4 million elements in one call, clipped, with the bf16 working copy
        {"name": "adamw 8-bit resnet50", "op": "adamw", "table": "resnet50", "states": 8,
         "grad": "f32", "clip": True, "copy": True},
        # the LSTM gate and FC layers with a bf16 gradient (summed without compression)
        {"name": "adamw 8-bit fc_lstm", "op": "adamw", "table": "4096x2048,4096x4096", "states": 8,
         "grad": "bf16", "clip": False, "copy": True},
        # the rows of one decoding step of a small batch
        {"name": "layer norm few rows", "op": "norm", "backward": False, "rows": 8, "cols": 1024,
         "dtype": "bf16"},
        # a training batch of 16384 tokens at width 4096
        {"name": "layer norm wide", "op": "norm", "backward": False, "rows": 16384, "cols": 4096,
         "dtype": "bf16"},
        # an odd number of float32 rows, a width that is no power of two
        {"name": "layer norm grad odd f32", "op": "norm", "backward": True, "rows": 4099,
         "cols": 1000, "dtype": "f32"},
        # many rows at width 1024: the weight's gradient sums over 32768 rows
        {"name": "layer norm grad rows", "op": "norm", "backward": True, "rows": 32768, "cols": 1024,
         "dtype": "bf16"},
        # one new token for 64 sequences: the state moves on by one step
        {"name": "scan one token", "op": "scan", "backward": False, "batch": 64, "length": 1,
         "channels": 2048, "dtype": "bf16", "sigmoid": True, "ragged": False},
        # a training batch
        {"name": "scan training batch", "op": "scan", "backward": False, "batch": 8, "length": 4096,
         "channels": 2048, "dtype": "bf16", "sigmoid": True, "ragged": False},
        # one long sequence with few channels: the length itself has to be shared out
        {"name": "scan grad long f32", "op": "scan", "backward": True, "batch": 1, "length": 65536,
         "channels": 256, "dtype": "f32", "sigmoid": False, "ragged": False},
        # padded sequences of different lengths, one of them empty, an odd width
        {"name": "scan grad ragged", "op": "scan", "backward": True, "batch": 16, "length": 2000,
         "channels": 1000, "dtype": "bf16", "sigmoid": True, "ragged": True},
    ]


def _size(rng, lo, hi):
    """Log-uniform over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    """An odd width, one of the layer tables' widths, or a multiple of 40 (16-byte rows in every type)."""
    return rng.choice([_size(rng, 16, 4100) | 1, rng.choice([64, 256, 512, 1000, 1024, 2048, 4096]),
                       40 * _size(rng, 1, 102)])


def draw(rng):
    op = rng.choice(["adamw", "adamw", "norm", "norm", "scan", "scan"])
    if op == "adamw":
        tensors = _size(rng, 1, 200)
        total = _size(rng, max(50000, 64 * tensors), 60_000_000)
        cols = _width(rng)
        rows = max(1, total // (tensors * cols))
        table = "%d*%dx%d" % (tensors, rows, cols) + rng.choice(["", ",%d" % cols, ",%d,%d" % (rows, cols)])
        return {"op": op, "table": table, "states": rng.choice([32, 8]),
                "grad": rng.choice(["f32", "bf16"]), "clip": rng.random() < 0.5,
                "copy": rng.random() < 0.5}
    if op == "norm":
        cols = _width(rng)
        rows = _size(rng, 1, max(1, min(65536, 60_000_000 // cols)))
        return {"op": op, "backward": rng.random() < 0.5, "rows": rows, "cols": cols,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    channels = _width(rng)
    length = _size(rng, 1, 40000)
    batch = _size(rng, 1, max(1, min(64, 50_000_000 // (channels * length))))
    return {"op": op, "backward": rng.random() < 0.5, "batch": batch, "length": length,
            "channels": channels, "dtype": rng.choice(["bf16", "f16", "f32"]),
            "sigmoid": rng.random() < 0.5, "ragged": batch > 1 and rng.random() < 0.4}


def _resnet50():
    """The 161 tensors of ResNet-50 in parameter order, as (rows, cols)."""
    out = []

    def layer(cout, fan_in):
        out.extend([(cout, fan_in), (1, cout), (1, cout)])

    layer(64, 3 * 49)
    cin = 64
    for width, blocks in ((64, 3), (128, 4), (256, 6), (512, 3)):
        for i in range(blocks):
            layer(width, cin)
            layer(width, 9 * width)
            layer(4 * width, width)
            if i == 0:
                layer(4 * width, cin)
            cin = 4 * width
    return out + [(1000, 2048), (1, 1000)]


def _shapes(table):
    if table == "resnet50":
        return _resnet50()
    out = []
    for part in table.split(","):
        times, _, shape = part.rpartition("*")
        dims = [int(x) for x in shape.split("x")]
        out += [(dims[0], dims[1]) if len(dims) == 2 else (1, dims[0])] * int(times or 1)
    return out


def _tensors(table):
    """(offset, numel, weight_decay, lr_scale) of each tensor; offsets are multiples of 4.
    Vectors (norm weights, biases) are not decayed."""
    out, at = [], 0
    for rows, cols in _shapes(table):
        out.append((at, rows * cols, 0.125 if rows > 1 else 0.0, 1.0 if rows > 1 else 0.5))
        at += (rows * cols + 3) // 4 * 4
    return out, at


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"adamw": _prepare_adamw, "norm": _prepare_norm, "scan": _prepare_scan}[case["op"]](case, seed, gen)


def _normal(gen, shape, scale=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).mul_(scale).to(dtype)


def _prepare_adamw(case, seed, gen):
    tensors, span = _tensors(case["table"])
    # gradients of which one element in 20 is 30 times larger; moments as after some
    # steps of such gradients
    burst = torch.rand(span, generator=gen, device=DEV).lt_(0.05).mul_(29.0).add_(1.0)
    grad = _normal(gen, span, 1e-3).mul_(burst)
    m = _normal(gen, span, 3e-4).mul_(burst)
    v = _normal(gen, span, 1e-3).mul_(burst).square_().add_(1e-8)
    del burst
    s = {"case": case, "tensors": tensors, "span": span, "weights": _normal(gen, span, 0.05),
         "grad": grad.to(DTYPES[case["grad"]]), "seed": HYPER["seed"] + seed,
         "copy": torch.zeros(span, dtype=torch.bfloat16, device=DEV) if case["copy"] else None,
         "clip": torch.zeros(2, device=DEV) if case["clip"] else None}
    # the table on the device: where each tensor (and each gap behind one) ends, and the
    # 32-element blocks of each tensor
    numel = torch.tensor([n for _, n, _, _ in tensors])
    pad = (4 - numel % 4) % 4
    s["runs"] = torch.stack([numel, pad], 1).reshape(-1).to(DEV)
    s["decay"] = torch.tensor([[d, 0.0] for _, _, d, _ in tensors]).reshape(-1).to(DEV)
    s["lr_scale"] = torch.tensor([[r, 0.0] for _, _, _, r in tensors]).reshape(-1).to(DEV)
    s["inside"] = torch.tensor([True, False] * len(tensors), device=DEV)
    if case["states"] == 32:
        s["m"], s["v"] = m, v
    else:
        blocks = (numel + BLOCK - 1) // BLOCK
        first = torch.cumsum(blocks, 0) - blocks
        offset = torch.tensor([o for o, _, _, _ in tensors])
        index = torch.arange(int(blocks.sum())) - first.repeat_interleave(blocks)
        s["start"] = (offset.repeat_interleave(blocks) + BLOCK * index).to(DEV)
        s["count"] = torch.minimum(numel.repeat_interleave(blocks) - BLOCK * index, torch.tensor(BLOCK)).to(DEV)
        s["nblocks"] = int(blocks.sum())
        s["m"] = torch.zeros(span, dtype=torch.float8_e4m3fn, device=DEV)
        s["v"] = torch.zeros(span, dtype=torch.float8_e4m3fn, device=DEV)
        s["scales"] = torch.zeros(2 * s["nblocks"], dtype=torch.uint8, device=DEV)
        at, real = _block_index(s)
        random16 = torch.randint(0, 65536, (2, s["nblocks"], BLOCK), generator=gen, device=DEV)
        for k, x in enumerate((m, v)):
            code, exponent = _quantise(_blocked(x.double(), at, real), random16[k], bool(k))
            _store_blocked(s["mv"[k]].view(torch.uint8), code, at, real)
            s["scales"][k::2] = exponent
    if own:
        import adaptive_residual_gradient_amd as A
        s["A"] = A
        s["opt"] = A.Optimizer(tensors)
        s["ws"] = s["opt"].norm_workspace(DEV)
    return s


def _prepare_norm(case, seed, gen):
    rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
    # activations with an offset and a few channels of larger scale
    gain = 1.0 + 4.0 * torch.rand(cols, generator=gen, device=DEV).lt(0.02)
    x = (_normal(gen, (rows, cols)) * gain + 0.3).to(dtype)
    s = {"case": case, "x": x, "weight": 1.0 + _normal(gen, cols, 0.2), "bias": _normal(gen, cols, 0.1),
         "mean": torch.empty(rows, device=DEV), "rstd": torch.empty(rows, device=DEV), "eps": 1e-5}
    s["out"] = torch.empty_like(x)
    if case["backward"]:
        s["dy"] = _normal(gen, (rows, cols), 0.01, dtype)
        f = x.double()
        s["mean"] = f.mean(1).float()
        s["rstd"] = (f.var(1, unbiased=False) + s["eps"]).rsqrt().float()
        s["dweight"], s["dbias"] = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    if own:
        import adaptive_residual_gradient_amd as A
        s["A"] = A
        s["ws"] = A.layer_norm_workspace(rows, cols, DEV) if case["backward"] else None
    return s


def _prepare_scan(case, seed, gen):
    B, T, D, dtype = case["batch"], case["length"], case["channels"], DTYPES[case["dtype"]]
    gate = _normal(gen, (B, T, D)) + 2.0            # forget gates open at first, as they are initialised
    gate = (gate if case["sigmoid"] else torch.sigmoid(gate)).to(dtype)
    s = {"case": case, "gate": gate, "x": _normal(gen, (B, T, D), 1.0, dtype),
         "h0": _normal(gen, (B, D), 0.5), "h_last": torch.empty(B, D, device=DEV), "lengths": None}
    if case["ragged"]:
        r = random.Random(seed)
        lengths = [r.randint(1, T) for _ in range(B)]
        lengths[0], lengths[-1] = 0, T
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    s["h"] = torch.empty(B, T, D, dtype=dtype, device=DEV)
    if case["backward"]:
        s["h"] = _plain_scan(s)[0]
        s["dh"] = _normal(gen, (B, T, D), 0.1, dtype)
        s["dh_last"], s["dh0"] = _normal(gen, (B, D), 0.1), torch.empty(B, D, device=DEV)
        s["dgate"], s["dx"] = torch.empty_like(gate), torch.empty_like(gate)
    if own:
        import adaptive_residual_gradient_amd as A
        s["A"] = A
        s["ws"] = A.gated_scan_workspace(B, T, D, DEV)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return {"adamw": _run_adamw, "norm": _run_norm, "scan": _run_scan}[state["case"]["op"]](state)


def _adamw_out(s):
    out = {"weights": s["weights"], "m": s["m"], "v": s["v"], "copy": s["copy"], "clip": s["clip"]}
    if s["case"]["states"] == 8:
        out["scales"] = s["scales"]
    return out


def _run_adamw(s):
    p = HYPER
    if not own:
        (_plain_adamw if s["case"]["states"] == 32 else _plain_adamw_8bit)(s)
        return _adamw_out(s)
    A = s["A"]
    if s["clip"] is not None:
        A.grad_norm(s["opt"], s["grad"], s["clip"], s["ws"], max_norm=p["max_norm"], scale=p["scale"])
    kw = dict(lr=p["lr"], beta1=p["beta1"], beta2=p["beta2"], eps=p["eps"], step=p["step"], scale=p["scale"],
              clip=s["clip"], weights_bf16=s["copy"])
    if s["case"]["states"] == 32:
        A.adamw(s["opt"], s["weights"], s["grad"], s["m"], s["v"], **kw)
    else:
        A.adamw_packed(s["opt"], s["weights"], s["grad"], s["m"], s["v"], s["scales"], seed=s["seed"], **kw)
    return _adamw_out(s)


def _run_norm(s):
    if not own:
        return _plain_norm_backward(s) if s["case"]["backward"] else _plain_norm(s)
    A = s["A"]
    if s["case"]["backward"]:
        A.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["out"], s["dweight"],
                              s["dbias"], s["ws"])
        return {"dx": s["out"], "dweight": s["dweight"], "dbias": s["dbias"]}
    A.layer_norm(s["x"], s["weight"], s["bias"], s["out"], s["mean"], s["rstd"], eps=s["eps"])
    return {"y": s["out"], "mean": s["mean"], "rstd": s["rstd"]}


def _run_scan(s):
    sigmoid = s["case"]["sigmoid"]
    if not own:
        if s["case"]["backward"]:
            dgate, dx, dh0 = _plain_scan_backward(s)
            return {"dgate": dgate, "dx": dx, "dh0": dh0}
        h, last = _plain_scan(s)
        return {"h": h, "h_last": last}
    A = s["A"]
    if s["case"]["backward"]:
        A.gated_scan_backward(s["gate"], s["x"] if sigmoid else None, s["h"], s["dh"], s["dgate"], s["dx"],
                              h0=s["h0"], dh_last=s["dh_last"], dh0=s["dh0"], lengths=s["lengths"],
                              sigmoid=sigmoid, ws=s["ws"])
        return {"dgate": s["dgate"], "dx": s["dx"], "dh0": s["dh0"]}
    A.gated_scan(s["gate"], s["x"], s["h"], h0=s["h0"], h_last=s["h_last"], lengths=s["lengths"],
                 sigmoid=sigmoid, ws=s["ws"])
    return {"h": s["h"], "h_last": s["h_last"]}


# ------------------------------------------------------------- plain forms

def _per_element(s, values):
    """One value of each tensor (and gap) to each element of the flat buffers."""
    return torch.repeat_interleave(values, s["runs"], output_size=s["span"])


def _plain_clip(s, inside):
    """Norm of the scaled gradient, its sum of squares in 64 bits, and the factor that brings
    it down to max_norm; the combined factor on the gradient."""
    p = HYPER
    if s["clip"] is None:
        return torch.full((), p["scale"], device=DEV), torch.ones((), device=DEV)
    g = torch.where(inside, s["grad"].double(), torch.zeros((), dtype=torch.float64, device=DEV))
    norm = (g * g).sum().sqrt() * p["scale"]
    s["clip"][0] = norm
    s["clip"][1] = torch.where(norm > p["max_norm"], p["max_norm"] / norm, torch.ones_like(norm))
    return s["clip"][1] * p["scale"], s["clip"][1]


def _steps(s, dtype):
    """Per element: step size lr / (1 - beta1^t) and decay factor 1 - lr * weight_decay."""
    p = HYPER
    lr = p["lr"] * _per_element(s, s["lr_scale"].double())
    keep = 1.0 - lr * _per_element(s, s["decay"].double())
    return (lr / (1.0 - p["beta1"] ** p["step"])).to(dtype), keep.to(dtype)


def _power_of_two(k):
    """2^k of whole numbers k in -1022..1023, made from its bits."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _plain_adamw(s):
    p = HYPER
    inside = _per_element(s, s["inside"])
    factor, _ = _plain_clip(s, inside)
    beta1, beta2 = p["beta1"], p["beta2"]
    size, keep = _steps(s, torch.float32)
    g = s["grad"].float() * factor
    m = beta1 * s["m"] + (1.0 - beta1) * g
    v = beta2 * s["v"] + (1.0 - beta2) * (g * g)
    denom = v.sqrt() * (1.0 - p["beta2"] ** p["step"]) ** -0.5 + p["eps"]
    w = s["weights"] * keep - size * (m / denom)
    for name, new in (("m", m), ("v", v), ("weights", w)):
        s[name].copy_(torch.where(inside, new, s[name]))
    if s["copy"] is not None:
        s["copy"].copy_(torch.where(inside, w.bfloat16(), s["copy"]))


def _fmix32(h):
    """The 32-bit finaliser of MurmurHash3 (Appleby), on int64 tensors."""
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random32(s, at):
    """The 32 random bits of each element: a hash of its place in the flat buffers, the
    call's seed and its step."""
    key = _fmix32(torch.tensor([s["seed"] & 0xFFFFFFFF], device=DEV)) ^ HYPER["step"]
    return _fmix32((at & 0xFFFFFFFF) ^ _fmix32(key ^ (((at >> 32) * 0x9E3779B9) & 0xFFFFFFFF)))


def _block_index(s):
    lane = torch.arange(BLOCK, device=DEV)
    real = lane < s["count"][:, None]
    return torch.where(real, s["start"][:, None] + lane, s["span"]), real


def _blocked(x, at, real):
    """Flat values as [blocks, 32], zero past a tensor's end."""
    return torch.where(real, x[at.clamp(max=x.numel() - 1)], torch.zeros((), dtype=x.dtype, device=DEV))


def _store_blocked(flat, blocks, at, real):
    spare = torch.cat([flat, flat.new_zeros(1)])
    spare.scatter_(0, at.reshape(-1), blocks.reshape(-1).to(flat.dtype))
    flat.copy_(spare[:-1])


def _quantise(x, random16, positive):
    """64-bit values [blocks, 32] to e4m3 codes and one power-of-two scale a block, rounded up
    with the probability of the remainder: the code is the top of the value's bits once a random
    number is added below it."""
    high = x.abs().view(torch.int64) >> 32
    top = high.amax(1)
    # the smallest scale under which the block's largest value rounds to 448 at most
    exponent = ((top + 0x3FFFF) >> 20) - 1023 - E4M3_MAX_EXP
    biased = (exponent + 127).clamp(0, 254)
    u = x.abs() * _power_of_two(127 - biased)[:, None]
    small = u < 2.0 ** -6
    u = torch.where(small, u + 2.0 ** -6, u)      # a subnormal code counts steps of 2^-9
    code = (((u.view(torch.int64) >> 32) + 2 * random16 + 1) >> 17) - (1023 - 7) * 8
    code = torch.where(small, code - 8, code)
    if positive:                                  # a second moment above zero never becomes zero
        code = torch.where((x > 0) & (code == 0), torch.ones_like(code), code)
    else:
        code = code | ((x < 0).to(torch.int64) << 7)
    return code, biased


def _plain_adamw_8bit(s):
    p = HYPER
    f64 = torch.float64
    beta1, beta2 = p["beta1"], p["beta2"]
    inside = _per_element(s, s["inside"])
    _, coef = _plain_clip(s, inside)
    at, real = _block_index(s)
    bits = _random32(s, at)
    # moments in 64 bits: the rounding to 8 bits must not hang on the order of a sum
    g = _blocked(s["grad"].to(f64), at, real) * (coef.to(f64) * p["scale"])
    scale = _power_of_two(s["scales"].to(torch.int64) - 127)
    m = _blocked(s["m"].to(f64), at, real) * scale[0::2, None]
    v = _blocked(s["v"].to(f64), at, real) * scale[1::2, None]
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * (g * g)
    size, keep = (_blocked(t, at, real) for t in _steps(s, torch.float32))
    denom = v.float().sqrt() * (1.0 - p["beta2"] ** p["step"]) ** -0.5 + p["eps"]
    w = _blocked(s["weights"], at, real) * keep - size * (m.float() / denom)
    _store_blocked(s["weights"], w, at, real)
    if s["copy"] is not None:
        _store_blocked(s["copy"], w.bfloat16(), at, real)
    code, s["scales"][0::2] = _quantise(m, bits & 0xFFFF, False)
    _store_blocked(s["m"].view(torch.uint8), code, at, real)
    code, s["scales"][1::2] = _quantise(v, bits >> 16, True)
    _store_blocked(s["v"].view(torch.uint8), code, at, real)


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = ((centred * centred).mean(1) + s["eps"]).rsqrt()
    y = centred * rstd[:, None] * s["weight"] + s["bias"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(s):
    dy = s["dy"].float()
    hat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * hat).sum(0, dtype=torch.float64).float(),
            "dbias": dy.sum(0, dtype=torch.float64).float()}


def _valid(s):
    """Which steps [batch, length, 1] lie within each sequence."""
    T = s["gate"].shape[1]
    if s["lengths"] is None:
        return torch.ones(s["gate"].shape[0], T, 1, dtype=torch.bool, device=DEV)
    return (torch.arange(T, device=DEV) < s["lengths"][:, None])[:, :, None]


def _gates(s):
    """Factor on the state, and on the input, of each step."""
    if not s["case"]["sigmoid"]:
        a = s["gate"].float()
        return a, torch.ones((), device=DEV)
    z = s["gate"].float()
    return torch.sigmoid(z), torch.sigmoid(-z)


def _prefix(a, b):
    """All h_t = a_t h_{t-1} + b_t from h = 0 by doubling: after k rounds each place holds the
    composition of the last 2^k steps."""
    k = 1
    while k < a.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_scan(s):
    a, k = _gates(s)
    ok = _valid(s)
    b = k * s["x"].float()
    first = torch.where(ok[:, :1], b[:, :1] + a[:, :1] * s["h0"][:, None], s["h0"][:, None])
    # past a sequence's end the state stays as it is
    a, b = torch.where(ok, a, torch.ones_like(a)), torch.where(ok, b, torch.zeros_like(b))
    b = torch.cat([first, b[:, 1:]], 1)
    h = _prefix(a, b)
    return torch.where(ok, h, torch.zeros_like(h)).to(s["gate"].dtype), h[:, -1].clone()


def _plain_scan_backward(s):
    a, k = _gates(s)
    ok = _valid(s)
    dh = torch.where(ok, s["dh"].float(), torch.zeros((), device=DEV))
    a = torch.where(ok, a, torch.ones_like(a))
    # the gradient that reaches step t from all later ones: l_t = dh_t + a_{t+1} l_{t+1}; past a
    # sequence's end a = 1 and dh = 0, so dh_last passes through to its last step
    dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_last"][:, None]], 1)
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    total = _prefix(later.flip(1), dh.flip(1)).flip(1)
    before = torch.cat([s["h0"][:, None], s["h"][:, :-1].float()], 1)
    if s["case"]["sigmoid"]:
        dgate = total * (before - s["x"].float()) * a * k
    else:
        dgate = total * before
    dx, dh0 = total * k, a[:, 0] * total[:, 0]
    zero = torch.zeros((), device=DEV)
    dtype = s["gate"].dtype
    return torch.where(ok, dgate, zero).to(dtype), torch.where(ok, dx, zero).to(dtype), dh0


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"adamw": _exact_adamw, "norm": _exact_norm, "scan": _exact_scan}[case["op"]](s)


def _exact_adamw(s):
    p = HYPER
    eight = s["case"]["states"] == 8
    coef, clip = 1.0, None
    if s["clip"] is not None:
        norm = p["scale"] * math.sqrt(sum(float(s["grad"][o:o + n].double().pow(2).sum())
                                          for o, n, _, _ in s["tensors"]))
        coef = min(1.0, p["max_norm"] / norm)
        clip = torch.tensor([norm, coef], dtype=torch.float64)
        coef = float(torch.tensor(coef, dtype=torch.float32))
    out = {"weights": s["weights"].double(), "m": s["m"].double(), "v": s["v"].double(),
           "copy": s["copy"].double() if s["copy"] is not None else None, "clip": clip}
    if eight:
        out["scales"] = None
    first = 0
    for offset, n, decay, lr_scale in s["tensors"]:
        part = slice(offset, offset + n)
        g = s["grad"][part].double() * (p["scale"] * coef)
        m, v = out["m"][part], out["v"][part]
        if eight:
            nb = (n + BLOCK - 1) // BLOCK
            both = _power_of_two(s["scales"][2 * first:2 * (first + nb)].long() - 127)
            m, v = m * both[0::2].repeat_interleave(BLOCK)[:n], v * both[1::2].repeat_interleave(BLOCK)[:n]
            first += nb
        m = m * p["beta1"] + g * (1 - p["beta1"])
        v = v * p["beta2"] + g ** 2 * (1 - p["beta2"])
        hat = m / (1 - p["beta1"] ** p["step"])
        root = (v / (1 - p["beta2"] ** p["step"])).sqrt()
        lr = p["lr"] * lr_scale
        w = out["weights"][part]
        w -= lr * (decay * w + hat / (root + p["eps"]))
        if out["copy"] is not None:
            out["copy"][part] = w
        if eight:
            place = torch.arange(offset, offset + n, device=DEV)
            bits = _random32(s, place)
            m, v = _exact_codes(m, bits % 65536), _exact_codes(v, bits // 65536, least=2.0 ** -9)
        out["m"][part], out["v"][part] = m, v
    return out


def _exact_codes(x, random16, least=0.0):
    """The e4m3 numbers that x is stored as, its block's scale divided out."""
    n = x.numel()
    size = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).reshape(-1, BLOCK).amax(1)
    part, exponent = torch.frexp(size)             # size = part * 2^exponent, part in [1/2, 1)
    # 448 = 0.875 * 2^9; a rounded value is told from it by its leading 21 bits
    exponent = exponent - 9 + (torch.floor(part * 2 ** 21) > 0.875 * 2 ** 21)
    exponent = exponent.clamp(-127, 127).repeat_interleave(BLOCK)[:n]
    u = x.abs() * _power_of_two(-exponent)
    step = _power_of_two((torch.frexp(u)[1] - 1).clamp(min=-6) - 3)
    up = torch.floor(u / step + (2 * random16 + 1).double() / 131072) * step
    up = torch.where((x != 0) & (up < least), torch.full_like(up, least), up)
    return torch.copysign(up, x)


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    if not s["case"]["backward"]:
        mean = x.sum(1) / x.shape[1]
        rstd = 1.0 / torch.sqrt((x ** 2).sum(1) / x.shape[1] - mean ** 2 + s["eps"])
        return {"y": torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), "mean": mean,
                "rstd": rstd}
    mean, rstd, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
    n = x.shape[1]
    hat = (x - mean[:, None]) * rstd[:, None]
    through = dy * w
    pull = through.sum(1) / n
    along = (through * hat).sum(1) / n
    return {"dx": (through - pull[:, None] - along[:, None] * hat) * rstd[:, None],
            "dweight": torch.sum(dy * hat, 0), "dbias": torch.sum(dy, 0)}


def _exact_scan(s):
    """Step by step along the sequence."""
    z, x = s["gate"].double(), s["x"].double()
    B, T, D = z.shape
    n = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=DEV)
    a, k = (1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))) if s["case"]["sigmoid"] else (z, torch.ones_like(z))
    if not s["case"]["backward"]:
        h, state = torch.zeros_like(z), s["h0"].double()
        for t in range(T):
            live = (t < n)[:, None]
            state = torch.where(live, a[:, t] * state + k[:, t] * x[:, t], state)
            h[:, t] = torch.where(live, state, torch.zeros_like(state))
        return {"h": h, "h_last": state}
    h, dh = s["h"].double(), s["dh"].double()
    dgate, dx, carry = torch.zeros_like(z), torch.zeros_like(z), s["dh_last"].double()
    for t in range(T - 1, -1, -1):
        live = (t < n)[:, None]
        here = dh[:, t] + carry
        before = h[:, t - 1] if t else s["h0"].double()
        slope = (before - x[:, t]) * a[:, t] * k[:, t] if s["case"]["sigmoid"] else before
        dgate[:, t] = torch.where(live, here * slope, torch.zeros_like(here))
        dx[:, t] = torch.where(live, here * k[:, t], torch.zeros_like(here))
        carry = torch.where(live, here * a[:, t], carry)
    return {"dgate": dgate, "dx": dx, "dh0": carry}


# -------------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once."""
    if case["op"] == "adamw":
        n = sum(r * c for r, c in _shapes(case["table"]))
        state = 16 if case["states"] == 32 else 4 + 2 * 2 / BLOCK
        size = torch.finfo(DTYPES[case["grad"]]).bits // 8
        return {"bytes": n * (8 + state + size + (2 if case["copy"] else 0)), "flops": 14 * n}
    size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    if case["op"] == "norm":
        n, rows, cols = case["rows"] * case["cols"], case["rows"], case["cols"]
        if case["backward"]:
            return {"bytes": 3 * n * size + 8 * rows + 12 * cols, "flops": 14 * n}
        return {"bytes": 2 * n * size + 8 * rows + 8 * cols, "flops": 7 * n}
    n, edge = case["batch"] * case["length"] * case["channels"], 4 * case["batch"] * case["channels"]
    if case["backward"]:
        return {"bytes": (6 if case["sigmoid"] else 5) * n * size + 3 * edge, "flops": 8 * n}
    return {"bytes": 3 * n * size + 2 * edge, "flops": 4 * n}
