"""Microscaled 4-bit (MXFP4) layers and the gated residual norm: their plain
forms in elementary torch operations beside the library's calls, and the cases
they are measured on.

The operators (x, y, o, h in bf16 or half; K = input features):
  quantize  x_r = x . blockdiag(R) in groups of g (g = 1: no rotation), each
            element's sum rounded once to fp32; per block of 32 elements of a
            row a scale 2^e, e = floor(log2 max|x_r|) - 2 clamped to
            [-127, 127], and 4-bit codes (sign, 0 0.5 1 1.5 2 3 4 6) of
            x_r / 2^e, ties to the even code, saturating at 6.
  dequant   W_hat = (code values * 2^e) . blockdiag(R)^T.
  gemm      y[m, n] = sum_k a[m, k] b[n, k] (+ bias[n]) over two such tensors.
  linear    y = gemm(quantize(x), w): the forward of a layer whose weight was
            quantized with the same rotation.
  norm      x' = x + gate * post(o), h = pre(x') * (1 + scale) + shift, with
            RMS or layer norms; pre() reads x' as it was rounded.
  block     norm with its h quantized at once, then the gemm of the next layer.

Layout of a quantized [rows, K] tensor: codes uint8 [rows, K/2], the even
element in the low nibble; scales uint8 [ceil(K/256), rows rounded up to 16, 8],
the biased exponent e + 127 of block 8 t + j of a row at [t, row, j].
"""

import math

import torch

own = False

ROT_SEED = 0xC0FFEE
_MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _dtype(case):
    return torch.float16 if case["dtype"] == "f16" else torch.bfloat16


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token entering a 5120-wide layer: the latency of a lone call
        {"name": "quantize-token", "op": "quantize", "m": 1, "k": 5120, "g": 256,
         "dtype": "bf16"},
        # the tokens of a whole video clip entering a feed-forward layer
        {"name": "quantize-clip", "op": "quantize", "m": 32760, "k": 5120, "g": 256,
         "dtype": "bf16"},
        # an attention projection read back for a 16-bit product
        {"name": "dequant-attn", "op": "dequant", "n": 3840, "k": 3840, "g": 256,
         "dtype": "bf16"},
        # a feed-forward weight read back, smaller groups, half
        {"name": "dequant-ffn", "op": "dequant", "n": 13824, "k": 5120, "g": 64,
         "dtype": "f16"},
        # a single token through a feed-forward weight: bound by the weight's bytes
        {"name": "gemm-token", "op": "gemm", "m": 1, "n": 13824, "k": 5120, "dtype": "bf16",
         "bias": False},
        # a ragged handful of text tokens, K not a whole number of tiles
        {"name": "gemm-ragged", "op": "gemm", "m": 333, "n": 9216, "k": 3872, "dtype": "f16",
         "bias": True},
        # the feed-forward product of a whole clip: bound by the matrix units
        {"name": "gemm-clip", "op": "gemm", "m": 32760, "n": 13824, "k": 5120,
         "dtype": "bf16", "bias": False},
        # a few tokens (a timestep or a pooled text embedding per sample)
        {"name": "linear-few", "op": "linear", "m": 9, "n": 3840, "k": 3840, "g": 256,
         "dtype": "bf16", "bias": True},
        # one image's tokens through an attention projection
        {"name": "linear-image", "op": "linear", "m": 4608, "n": 3840, "k": 3840, "g": 256,
         "dtype": "bf16", "bias": True},
        # a short text stream: residual, gate and sandwich norms of a few rows
        {"name": "norm-text", "op": "norm", "m": 77, "k": 3840, "samples": 1, "norm": "rms",
         "post": "rms", "weight": True, "modulated": True, "dtype": "bf16"},
        # two clips of a batch: gated residual, then a modulated layer norm
        {"name": "norm-clip", "op": "norm", "m": 32760, "k": 5120, "samples": 2,
         "norm": "layer", "post": "", "weight": False, "modulated": True, "dtype": "bf16"},
        # the step from one block's output into the next block's fused projection
        {"name": "block-image", "op": "block", "m": 4608, "n": 11520, "k": 3840, "g": 256,
         "samples": 1, "norm": "rms", "post": "rms", "weight": True, "modulated": True,
         "dtype": "bf16", "bias": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "dequant", "gemm", "linear", "norm", "block"))
    dtype = rng.choice(("bf16", "f16"))
    g = rng.choice((1, 4, 16, 64, 256))
    step = max(32, g)
    k = step * max(1, _log_int(rng, 256, 13824) // step)
    n = 16 * _log_int(rng, 4, 864)
    m = _log_int(rng, 1, 32760)
    bias = rng.random() < 0.5
    norms = {"samples": rng.choice((1, 2, 3)), "norm": rng.choice(("rms", "layer")),
             "post": rng.choice(("", "rms", "layer")), "weight": rng.random() < 0.5,
             "modulated": rng.random() < 0.7}
    most = 32760 * 5120
    m = max(1, min(m, most // k))
    if op in ("gemm", "linear", "block"):
        m = max(1, min(m, most // n, 32760 * 13824 // k * 5120 // n))
    if op in ("norm", "block"):
        m = norms["samples"] * max(1, m // norms["samples"])
    if op == "quantize":
        return {"op": op, "m": m, "k": k, "g": g, "dtype": dtype}
    if op == "dequant":
        return {"op": op, "n": min(n, most // k), "k": k, "g": g, "dtype": dtype}
    if op == "gemm":
        return {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias}
    if op == "linear":
        return {"op": op, "m": m, "n": n, "k": k, "g": g, "dtype": dtype, "bias": bias}
    if op == "norm":
        return {"op": op, "m": m, "k": k, "dtype": dtype, **norms}
    return {"op": op, "m": m, "n": n, "k": k, "g": g, "dtype": dtype, "bias": bias, **norms}


# ---- inputs ----------------------------------------------------------------

def _signs(g):
    """The rotation's signs d[0..g) for ROT_SEED (SplitMix64 in counter form)."""
    def mix(z):
        mask = (1 << 64) - 1
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        return z ^ (z >> 31)
    gamma = 0x9E3779B97F4A7C15
    outs = [mix((ROT_SEED + (i + 1) * gamma) & ((1 << 64) - 1)) for i in range(g)]
    return [1.0 if g == 1 or not (z >> 63) else -1.0 for z in outs]


def _rotation(g, device):
    """R = H_g . diag(d) / sqrt(g) in float64, H[i][j] = (-1)^popcount(i & j)."""
    i = torch.arange(g, device=device)
    a = i[:, None] & i[None, :]
    bits = a.unsqueeze(-1) >> torch.arange(8, device=device)
    odd = (bits & 1).sum(-1) & 1
    d = torch.tensor(_signs(g), dtype=torch.float64, device=device)
    return (1.0 - 2.0 * odd.double()) * d / math.sqrt(g)


def _tokens(m, k, gen, dtype):
    """Normal activations with a few strong channels, as a transformer's are."""
    x = torch.randn(m, k, device="cuda", generator=gen)
    strong = torch.randint(0, k, (max(1, k // 200),), device="cuda", generator=gen)
    x[:, strong] *= 30.0
    return x.to(dtype)


def _rows(*shape, gen, dtype, std=1.0, mean=0.0):
    return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt, k = case["op"], _dtype(case), case["k"]
    state = {"case": case, "g": case.get("g", 1)}
    state["rot"] = _rotation(state["g"], "cuda")
    if op in ("quantize", "linear"):
        state["x"] = _tokens(case["m"], k, gen, dt)
    if op == "gemm":
        state["xc"], state["xs"] = _plain_quantize(_tokens(case["m"], k, gen, dt), None)
    if op in ("dequant", "gemm", "linear", "block"):
        w = _rows(case["n"], k, gen=gen, dtype=torch.bfloat16, std=0.02)
        state["wc"], state["ws"] = _plain_quantize(w, None)
        state["bias"] = None
        if case.get("bias"):
            state["bias"] = _rows(case["n"], gen=gen, dtype=dt, std=0.1)
    if op in ("norm", "block"):
        m, b = case["m"], case["samples"]
        state["x"] = _tokens(m, k, gen, dt)
        state["o"] = _rows(m, k, gen=gen, dtype=dt)
        state["gate"] = state["scale"] = state["shift"] = None
        if case["modulated"]:
            # one projection of the timestep gives every modulation of a block: the
            # three used here are column ranges of one wide row per sample
            mod = _rows(b, 6 * k, gen=gen, dtype=dt, std=0.3)
            state["gate"] = mod[:, 2 * k:3 * k]
            state["scale"] = mod[:, 4 * k:5 * k]
            state["shift"] = mod[:, 3 * k:4 * k]
        state["weight"] = state["post_weight"] = None
        if case["weight"]:
            state["weight"] = _rows(k, gen=gen, dtype=dt, std=0.1, mean=1.0)
            if case["post"]:
                state["post_weight"] = _rows(k, gen=gen, dtype=dt, std=0.1, mean=1.0)
    return state


# ---- plain forms -----------------------------------------------------------

def _plain_rotate(x, rot):
    """x . blockdiag(R), each sum in 64 bits, rounded once to 32."""
    if rot is None or rot.shape[0] == 1:
        return x.float()
    g = rot.shape[0]
    return (x.double().reshape(-1, g) @ rot).float().reshape(x.shape)


def _plain_quantize(x, rot):
    """(codes, scales) of x [rows, k] in the layout above."""
    rows, k = x.shape
    v = _plain_rotate(x, rot).reshape(rows, k // 32, 32)
    top = v.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)  # top = f * 2^exponent, f in [1/2, 1)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    u = torch.ldexp(v, -e[..., None])
    a = u.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(u).to(torch.uint8) * 8
    code = code.reshape(rows, k // 2, 2)
    codes = code[..., 0] | (code[..., 1] << 4)
    tiles = -(-k // 256)
    padded = -(-rows // 16) * 16
    scales = torch.zeros(padded, tiles * 8, dtype=torch.uint8, device=x.device)
    scales[:rows, : k // 32] = (e + 127).to(torch.uint8)
    return codes, scales.reshape(padded, tiles, 8).transpose(0, 1).contiguous()


def _plain_values(codes, scales):
    """The values that codes and scales stand for, fp32 [rows, k]."""
    rows, half = codes.shape
    k = 2 * half
    table = torch.tensor(_MAGS + tuple(-a for a in _MAGS), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).reshape(rows, k // 32, 32)
    e = scales[:, :rows].transpose(0, 1).reshape(rows, -1)[:, : k // 32].int() - 127
    return torch.ldexp(table[pair.int()], e[..., None]).reshape(rows, k)


def _plain_norm(v, kind, weight, eps=1e-6):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps)
    return v if weight is None else v * weight.float()


def _per_row(mod, m):
    """A modulation row per sample, spread over the sample's rows."""
    return mod.float().repeat_interleave(m // mod.shape[0], 0)


def _plain_norm_residual(s):
    case, m = s["case"], s["case"]["m"]
    o = s["o"].float()
    if case["post"]:
        o = _plain_norm(o, case["post"], s["post_weight"])
    if s["gate"] is not None:
        o = o * _per_row(s["gate"], m)
    x = (s["x"].float() + o).to(s["x"].dtype)
    h = _plain_norm(x.float(), case["norm"], s["weight"])
    if s["scale"] is not None:
        h = h * (1 + _per_row(s["scale"], m)) + _per_row(s["shift"], m)
    return x, h.to(x.dtype)


def _plain_gemm(a, b, bias, dt):
    y = a @ b.t()
    return (y if bias is None else y + bias.float()).to(dt)


def _plain(s):
    case, op, dt = s["case"], s["case"]["op"], _dtype(s["case"])
    if op == "quantize":
        return _plain_values(*_plain_quantize(s["x"], s["rot"])).to(dt)
    if op == "norm":
        return _plain_norm_residual(s)
    w = _plain_values(s["wc"], s["ws"])
    if op == "dequant":
        g = s["g"]  # a sum of g values that are alike: 32 bits hold it
        return (w.reshape(-1, g) @ s["rot"].t().float()).reshape(w.shape).to(dt)
    if op == "gemm":
        return _plain_gemm(_plain_values(s["xc"], s["xs"]), w, s["bias"], dt)
    x, h = _plain_norm_residual(s) if op == "block" else (None, s["x"])
    a = _plain_values(*_plain_quantize(h, s["rot"]))
    y = _plain_gemm(a, w, s["bias"], dt)
    return (x, y) if op == "block" else y


# ---- the library's calls ---------------------------------------------------

def _own(s):
    import int8_gemm_amd as cr
    case, op, g, dt = s["case"], s["case"]["op"], s["g"], _dtype(s["case"])
    if op == "quantize":
        codes, scales = cr.convrot_quantize_mx4(s["x"], g, ROT_SEED)
        return cr.convrot_dequant_mx4(codes, scales, 1, dtype=dt)  # the values, still rotated
    if op == "dequant":
        return cr.convrot_dequant_mx4(s["wc"], s["ws"], g, ROT_SEED, dtype=dt)
    if op == "gemm":
        return cr.convrot_gemm_mx4(s["xc"], s["xs"], s["wc"], s["ws"], s["bias"], dtype=dt)
    if op == "linear":
        return cr.convrot_linear_mx4(s["x"], s["wc"], s["ws"], g, ROT_SEED, s["bias"])
    norms = {"gate": s["gate"], "post_norm": case["post"] or None,
             "post_weight": s["post_weight"], "norm": case["norm"], "weight": s["weight"],
             "scale": s["scale"], "shift": s["shift"]}
    if op == "norm":
        return cr.convrot_norm_residual(s["x"], s["o"], **norms)
    x, codes, scales = cr.convrot_norm_residual_mx4(s["x"], s["o"], g, ROT_SEED, **norms)
    return x, cr.convrot_gemm_mx4(codes, scales, s["wc"], s["ws"], s["bias"], dtype=dt)


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    op, k = case["op"], case["k"]
    m, n, g = case.get("m", 0), case.get("n", 0), case.get("g", 1)

    def quantized(rows):
        return rows * (k // 2 + k // 32)
    wide = 2 * m * k  # one 16-bit [m, k] tensor
    bias = 2 * n if case.get("bias") else 0
    product = {"bytes": quantized(n) + bias + 2 * m * n, "flops": 2 * m * n * k}
    rotate = int(math.log2(g)) if g > 1 else 0
    if op == "quantize":  # x in, the quantized form out and in, its values out
        return {"bytes": wide + 2 * quantized(m) + wide, "flops": m * k * (rotate + 4)}
    if op == "dequant":
        return {"bytes": quantized(n) + 2 * n * k, "flops": n * k * (rotate + 1)}
    if op == "gemm":
        return {"bytes": product["bytes"] + quantized(m), "flops": product["flops"]}
    if op == "linear":
        return {"bytes": product["bytes"] + wide,
                "flops": product["flops"] + m * k * (rotate + 2)}
    mods = 2 * k * (3 * case["samples"] if case["modulated"] else 0)
    mods += 2 * k * ((2 if case["post"] else 1) if case["weight"] else 0)
    if op == "norm":  # x and o in, x' and h out
        return {"bytes": 4 * wide + mods, "flops": 12 * m * k}
    return {"bytes": 3 * wide + mods + product["bytes"],
            "flops": product["flops"] + m * k * (14 + rotate)}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_rotate(v, g):
    """v . blockdiag(R): sums and differences of pairs (Sylvester's H), then the signs."""
    if g == 1:
        return v
    rows, k = v.shape
    t = v.reshape(-1, g)
    h = 1
    while h < g:
        t = t.reshape(-1, g // (2 * h), 2, h)
        t = torch.stack((t[:, :, 0] + t[:, :, 1], t[:, :, 0] - t[:, :, 1]), 2)
        t = t.reshape(-1, g)
        h *= 2
    d = torch.tensor(_signs(g), dtype=torch.float64, device=v.device)
    return (t * d / math.sqrt(g)).reshape(rows, k)


def _exact_fp4(v, g):
    """The values that the quantized form of v [rows, k] stands for. Between
    powers of two the 4-bit values are evenly spaced: spacing 1/2 up to 2, 1 up
    to 4, 2 above; a tie's even code is the even multiple of the spacing."""
    r = _exact_rotate(v, g).float().double()  # each rotated element is an fp32 number
    rows, k = r.shape
    r = r.reshape(rows, -1, 32)
    top = r.abs().amax(-1, keepdim=True)
    tiny = torch.finfo(torch.float64).tiny
    e = (torch.floor(torch.log2(top.clamp_min(tiny))) - 2).clamp(-127, 127)
    unit = torch.pow(torch.full_like(e, 2.0), e)
    a = r.abs() / unit
    space = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.minimum(torch.round(a / space) * space, torch.full_like(a, 6.0))
    return (torch.sign(r) * q * unit).reshape(rows, k)


def _exact_read(codes, scales):
    """Sign, exponent and mantissa of each code: (-1)^s 2^(x-1) (1 + m/2), or m/2."""
    rows, half = codes.shape
    c = torch.empty(rows, 2 * half, dtype=torch.int32, device=codes.device)
    c[:, 0::2] = codes.int() % 16
    c[:, 1::2] = codes.int() // 16
    s, x, f = c // 8, (c // 2) % 4, (c % 2).double()
    v = torch.where(x == 0, f / 2, torch.exp2(x.double() - 1) * (1 + f / 2))
    t = torch.arange(c.shape[1], device=codes.device) // 32
    e = scales[t // 8, :rows, t % 8].t().double() - 127
    return (1 - 2 * s) * v * torch.pow(torch.full_like(e, 2.0), e)


def _exact_norm(v, kind, weight):
    var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
    if kind == "rms":
        var, mean = var + mean * mean, 0.0
    v = (v - mean) / torch.sqrt(var + 1e-6)
    return v if weight is None else v * weight.double()


def _exact_norm_residual(s):
    case = s["case"]
    rows = torch.arange(case["m"], device="cuda") * case["samples"] // case["m"]
    t = s["o"].double()
    if case["post"]:
        t = _exact_norm(t, case["post"], s["post_weight"])
    if s["gate"] is not None:
        t = t * s["gate"].double()[rows]
    t = t + s["x"].double()
    h = _exact_norm(t.to(s["x"].dtype).double(), case["norm"], s["weight"])
    if s["scale"] is not None:
        h = h + h * s["scale"].double()[rows] + s["shift"].double()[rows]
    return t, h


def exact(case, seed):
    op = case["op"]
    if op not in ("quantize", "norm") and work(case)["flops"] > 4e14:
        return None  # the product in 64 bits would take too long
    s, g = prepare(case, seed), case.get("g", 1)
    if op == "quantize":
        return _exact_fp4(s["x"].double(), g)
    if op == "norm":
        return _exact_norm_residual(s)
    w = _exact_read(s["wc"], s["ws"])
    if op == "dequant":  # R^T undoes R: signs first, then the sums
        d = torch.tensor(_signs(g), dtype=torch.float64, device="cuda")
        flipped = (w.reshape(-1, g) * d).reshape(w.shape)
        return (_exact_rotate(flipped, g).reshape(-1, g) * d).reshape(w.shape)
    x = None
    if op == "gemm":
        a = _exact_read(s["xc"], s["xs"])
    elif op == "linear":
        a = _exact_fp4(s["x"].double(), g)
    else:
        x, h = _exact_norm_residual(s)
        a = _exact_fp4(h.to(s["x"].dtype).double(), g)
    y = torch.matmul(a, w.t())
    if s["bias"] is not None:
        y = y + s["bias"].double()
    return (x, y) if op == "block" else y
