"""The attention half of a transformer block: rotary positions with several
axes, norms of queries and keys with the rotation in the same pass, and
attention over packed sequences with grouped heads; their plain forms in
elementary torch operations beside the library's calls, and the cases they are
measured on.

The operators (T tokens, H heads of d elements, bf16 or half):
  table      positions [T, axes] -> fp32 [T, pairs, 2]: cos and sin of
             position * theta^(-2 j / n). An axis of `dims` elements owns dims / 2
             pairs; j and n count within the axis (n = its dims), or over all of
             them where the axes share one ladder (n = the sum of the dims).
  heads      q [T, Hq, d], k [T, Hk, d]: RMS or layer norm of each head, or of
             all heads of a token as one row, times a weight; then pair i of the
             first 2 pairs elements, (2i, 2i+1) or (i, i + pairs), is turned by
             its table entry: (a, b) -> (a cos - b sin, b cos + a sin). fp32
             throughout, rounded once.
  attention  out = softmax(scale q k^T) v per sequence and head; query head h
             reads key head h / (Hq / Hk). Causal: query i of Lq sees keys j <=
             i + Lk - Lq. A query that sees no key gives 0. lse [Hq, T] = log
             sum exp of its scores.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _ints(text):
    return [int(v) for v in text.split(",")]


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # the patches of one image behind its text tokens, three axes
        {"name": "table-image", "op": "table", "t": 4608, "dims": "32,48,48", "theta": 256.0,
         "shared": False},
        # a video clip: 21 frames of 30 x 52 patches
        {"name": "table-clip", "op": "table", "t": 32760, "dims": "44,42,42", "theta": 10000.0,
         "shared": False},
        # one new token, grouped heads: the latency of a lone call
        {"name": "heads-token", "op": "heads", "t": 1, "hq": 32, "hk": 8, "d": 128,
         "pairs": 64, "norm": "rms", "span": "head", "halves": True, "weight": True,
         "dtype": "bf16"},
        # a short stream of text tokens in half, half of each head turned
        {"name": "heads-text", "op": "heads", "t": 333, "hq": 24, "hk": 8, "d": 64, "pairs": 16,
         "norm": "layer", "span": "head", "halves": True, "weight": True, "dtype": "f16"},
        # one image's tokens, q and k being column ranges of the fused projection
        {"name": "heads-image", "op": "heads", "t": 4608, "hq": 30, "hk": 30, "d": 128,
         "pairs": 64, "norm": "rms", "span": "head", "halves": False, "weight": True,
         "dtype": "bf16"},
        # a clip, normed over all heads of a token
        {"name": "heads-clip", "op": "heads", "t": 32760, "hq": 40, "hk": 40, "d": 128,
         "pairs": 64, "norm": "rms", "span": "row", "halves": False, "weight": True,
         "dtype": "bf16"},
        # one token against a long cache: bound by the cache's bytes
        {"name": "attention-token", "op": "attention", "q_lens": "1", "k_lens": "30011",
         "cache": 32768, "hq": 32, "hk": 8, "d": 128, "causal": True, "lse": False,
         "dtype": "bf16"},
        # packed prompts of different lengths, causal, grouped heads, half
        {"name": "attention-packed", "op": "attention", "q_lens": "1,4095,333,17,2777,1000,64",
         "k_lens": "1,4095,333,17,2777,1000,64", "cache": 0, "hq": 32, "hk": 8, "d": 64,
         "causal": True, "lse": True, "dtype": "f16"},
        # a batch of single tokens over padded caches of different use
        {"name": "attention-batch", "op": "attention",
         "q_lens": "1,1,1,1,1,1,1,1,1,1,1,1", "cache": 8192,
         "k_lens": "8192,5000,1,77,6143,2500,8191,4096,301,7000,64,1025", "hq": 32, "hk": 8,
         "d": 128, "causal": True, "lse": False, "dtype": "bf16"},
        # one image's tokens, every token seeing every other
        {"name": "attention-image", "op": "attention", "q_lens": "4608", "k_lens": "4608",
         "cache": 0, "hq": 30, "hk": 30, "d": 128, "causal": False, "lse": False,
         "dtype": "bf16"},
        # a clip's tokens reading a prompt of 512
        {"name": "attention-cross", "op": "attention", "q_lens": "32760", "k_lens": "512",
         "cache": 0, "hq": 40, "hk": 40, "d": 128, "causal": False, "lse": False,
         "dtype": "bf16"},
        # a whole clip: bound by the matrix units
        {"name": "attention-clip", "op": "attention", "q_lens": "32760", "k_lens": "32760",
         "cache": 0, "hq": 40, "hk": 40, "d": 128, "causal": False, "lse": False,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("table", "heads", "attention", "attention"))
    dtype = rng.choice(("bf16", "f16"))
    d = rng.choice((64, 64, 72, 96, 128, 128, 128, 256))
    hk = rng.choice((1, 2, 4, 5, 8, 10, 24, 30, 40))
    group = rng.choice((1, 1, 2, 3, 4, 8)) if hk <= 10 else 1
    if op == "table":
        axes = rng.choice((1, 2, 3, 3, 4))
        dims = ",".join(str(2 * rng.randint(4, 32)) for _ in range(axes))
        return {"op": op, "t": _log_int(rng, 1, 32760), "dims": dims,
                "theta": rng.choice((256.0, 10000.0, 500000.0)),
                "shared": rng.random() < 0.3}
    if op == "heads":
        halves = rng.random() < 0.5
        step = 8 if halves else 4
        most = 32760 * 5120 // (hk * group * d)
        pairs = d // 2 // step * step if rng.random() < 0.7 else step * rng.randint(0, d // 2 // step)
        return {"op": op, "t": min(most, _log_int(rng, 1, 32760)), "hq": hk * group, "hk": hk,
                "d": d, "pairs": pairs, "norm": rng.choice(("", "rms", "rms", "layer")),
                "span": rng.choice(("head", "row")), "halves": halves,
                "weight": rng.random() < 0.7, "dtype": dtype}
    kind = rng.choice(("self", "cross", "cache"))
    batch = rng.choice((1, 1, 2, 3, 7, 16))
    top = _log_int(rng, 1, 16384)
    k_lens = [rng.randint(max(1, top // 3), top) for _ in range(batch)]
    cache = 0
    if kind == "self":
        q_lens = list(k_lens)
    elif kind == "cross":
        q_lens = [_log_int(rng, 1, 16384) for _ in range(batch)]
    else:
        cache = top + rng.randint(0, 200)
        q_lens = [min(k, _log_int(rng, 1, 9)) for k in k_lens]
    causal = kind == "cache" or rng.random() < 0.5
    # no more work than the largest listed case, and no more memory
    per_pair = hk * group * max(64, d)
    limit = 32760 * 32760 * 40 * 128
    while (sum(q * k for q, k in zip(q_lens, k_lens)) * per_pair > limit
           or (sum(q_lens) * group + sum(k_lens) + batch * cache) * hk * d > 8 * 32760 * 5120):
        q_lens = [max(1, q // 2) for q in q_lens]
        k_lens = [max(1, k // 2) for k in k_lens]
        cache //= 2
        cache = max(cache, max(k_lens)) if kind == "cache" else 0
    seen = all(q <= k for q, k in zip(q_lens, k_lens))  # else some queries see nothing
    return {"op": op, "q_lens": ",".join(map(str, q_lens)), "k_lens": ",".join(map(str, k_lens)),
            "cache": cache, "hq": hk * group, "hk": hk, "d": d, "causal": causal,
            "lse": (seen or not causal) and rng.random() < 0.5, "dtype": dtype}


# ---- inputs ----------------------------------------------------------------

def _positions(case, gen):
    """Patch positions (frame, row, column, ...) in their order, from an offset."""
    axes, t = len(_ints(case["dims"])), case["t"]
    at = torch.arange(t, device="cuda")
    cols = []
    size = 52
    for _ in range(axes - 1):
        cols.append(at % size)
        at = at // size
        size = 30
    cols.append(at)
    start = torch.randint(0, 1000, (axes,), device="cuda", generator=gen)
    return torch.stack(cols[::-1], 1) + start


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    op = case["op"]
    s = {"case": case}
    if op == "table":
        s["positions"] = _positions(case, gen)
        s["dims"] = _ints(case["dims"])
        return s
    dt, d, hq, hk = _DTYPES[case["dtype"]], case["d"], case["hq"], case["hk"]
    if op == "heads":
        t = case["t"]
        # q, k and v leave one projection; strong channels as a transformer's are
        qkv = randn(t, hq + 2 * hk, d)
        qkv *= 1 + 3 * torch.rand(hq + 2 * hk, d, device="cuda", generator=gen) ** 8
        qkv = qkv.to(dt)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"] = s["k_weight"] = s["table"] = None
        if case["weight"] and case["norm"]:
            row = case["span"] == "row"
            s["q_weight"] = (1 + 0.1 * randn(hq * d if row else d)).to(dt)
            s["k_weight"] = (1 + 0.1 * randn(hk * d if row else d)).to(dt)
        if case["pairs"]:
            angle = 1000 * torch.rand(t, case["pairs"], device="cuda", generator=gen)
            s["table"] = torch.stack((torch.cos(angle), torch.sin(angle)), -1)
        return s
    q_lens, k_lens = _ints(case["q_lens"]), _ints(case["k_lens"])
    batch = len(q_lens)
    rows = batch * case["cache"] or sum(k_lens)
    # heads of different temperature, from nearly flat to sharp
    heat = torch.linspace(0.5, 2.5, hq, device="cuda")[:, None]
    s["q"] = (randn(sum(q_lens), hq, d) * heat).to(dt)
    s["k"] = (randn(rows, hk, d) + 0.5 * randn(hk, d)).to(dt)
    s["v"] = randn(rows, hk, d).to(dt)
    s["q_offsets"] = _offsets(q_lens)
    s["used"] = None
    if case["cache"]:
        s["k_offsets"] = _offsets([case["cache"]] * batch)
        s["used"] = torch.tensor(k_lens, dtype=torch.int32, device="cuda")
    else:
        s["k_offsets"] = _offsets(k_lens)
    return s


def _spans(case):
    """(first query, queries, first key, keys) of each sequence."""
    q0 = k0 = 0
    for lq, lk in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
        yield q0, lq, k0, lk
        q0 += lq
        k0 += case["cache"] or lk


# ---- plain forms -----------------------------------------------------------

def _plain_table(s):
    case, dims = s["case"], s["dims"]
    angles, before, total = [], 0, sum(dims)
    for a, n in enumerate(dims):
        j = torch.arange(n // 2, device="cuda", dtype=torch.float64)
        power = (2 * (j + before)) / total if case["shared"] else 2 * j / n
        freq = torch.exp(-math.log(case["theta"]) * power)
        angles.append(s["positions"][:, a, None].double() * freq)
        before += n // 2
    angle = torch.cat(angles, 1)
    return torch.stack((torch.cos(angle), torch.sin(angle)), -1).float()


def _plain_norm(v, kind, weight):
    if not kind:
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
    return v if weight is None else v * weight.float()


def _plain_heads(s, x, weight):
    case = s["case"]
    t, h, d = x.shape
    v = x.float()
    if case["span"] == "row":
        v = _plain_norm(v.reshape(t, h * d), case["norm"], weight).reshape(t, h, d)
    else:
        v = _plain_norm(v, case["norm"], weight)
    p = case["pairs"]
    if p:
        c, n = s["table"][:, None, :, 0], s["table"][:, None, :, 1]
        if case["halves"]:
            a, b = v[..., :p], v[..., p:2 * p]
            turned = torch.cat((a * c - b * n, b * c + a * n), -1)
        else:
            a, b = v[..., 0:2 * p:2], v[..., 1:2 * p:2]
            turned = torch.stack((a * c - b * n, b * c + a * n), -1).reshape(t, h, 2 * p)
        v = torch.cat((turned, v[..., 2 * p:]), -1)
    return v.to(x.dtype)


def _plain_attention(s):
    case = s["case"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    group, scale = hq // hk, 1 / math.sqrt(d)
    out = torch.empty_like(s["q"])
    lse = torch.empty(hq, out.shape[0], device="cuda")
    for q0, lq, k0, lk in _spans(case):
        step = max(1, min(lq, (1 << 29) // (group * lk)))  # scores of at most 2 GB
        for h in range(hk):
            k = s["k"][k0:k0 + lk, h].float().t().contiguous()
            v = s["v"][k0:k0 + lk, h].float()
            heads = slice(h * group, (h + 1) * group)
            for i in range(0, lq, step):
                n = min(step, lq - i)
                q = s["q"][q0 + i:q0 + i + n, heads].float().reshape(n * group, d)
                p = (q @ k).mul_(scale)
                if case["causal"]:
                    row = torch.arange(i, i + n, device="cuda").repeat_interleave(group)
                    key = torch.arange(lk, device="cuda")
                    p.masked_fill_(key > row[:, None] + (lk - lq), -math.inf)
                top = p.amax(-1, keepdim=True)
                top = torch.where(top == -math.inf, torch.zeros_like(top), top)
                p.sub_(top).exp_()
                total = p.sum(-1, keepdim=True)
                o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
                out[q0 + i:q0 + i + n, heads] = o.reshape(n, group, d).to(out.dtype)
                if case["lse"]:
                    lse[heads, q0 + i:q0 + i + n] = (top + total.log()).reshape(n, group).t()
    return (out, lse) if case["lse"] else out


def _plain(s):
    op = s["case"]["op"]
    if op == "table":
        return _plain_table(s)
    if op == "heads":
        return _plain_heads(s, s["q"], s["q_weight"]), _plain_heads(s, s["k"], s["k_weight"])
    return _plain_attention(s)


# ---- the library's calls ---------------------------------------------------

def _own(s):
    import int8_gemm_amd as cr
    case = s["case"]
    if case["op"] == "table":
        return cr.convrot_rope_table(s["positions"], s["dims"], case["theta"],
                                     shared=case["shared"])
    if case["op"] == "heads":
        return cr.convrot_qk_norm_rope(s["q"], s["k"], s["table"], norm=case["norm"] or None,
                                       span=case["span"], q_weight=s["q_weight"],
                                       k_weight=s["k_weight"], halves=case["halves"])
    return cr.convrot_attention(s["q"], s["k"], s["v"], q_offsets=s["q_offsets"],
                                k_offsets=s["k_offsets"], k_lens=s["used"],
                                causal=case["causal"], return_lse=case["lse"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    op = case["op"]
    if op == "table":
        dims = _ints(case["dims"])
        pairs = sum(dims) // 2
        # an angle, its reduction, two series
        return {"bytes": case["t"] * (8 * len(dims) + 8 * pairs), "flops": case["t"] * pairs * 40}
    d, hq, hk = case["d"], case["hq"], case["hk"]
    if op == "heads":
        n = case["t"] * (hq + hk) * d
        weights = 0
        if case["weight"] and case["norm"]:
            weights = 2 * ((hq + hk) * d if case["span"] == "row" else 2 * d)
        return {"bytes": 4 * n + 8 * case["t"] * case["pairs"] + weights, "flops": 8 * n}
    pairs = keys = queries = 0
    for _, lq, _, lk in _spans(case):
        queries += lq
        if case["causal"]:
            # query i sees i + lk - lq + 1 keys, none below zero
            first, seen = max(1, lk - lq + 1), min(lq, lk)
            pairs += (first + lk) * seen // 2
            keys += lk
        else:
            pairs += lq * lk
            keys += lk if lq else 0
    bytes_ = 4 * queries * hq * d + 4 * keys * hk * d + (4 * queries * hq if case["lse"] else 0)
    return {"bytes": bytes_, "flops": 4 * pairs * hq * d}


# ---- the definitions in 64 bits --------------------------------------------

def _exact_table(s):
    case, dims = s["case"], s["dims"]
    axis = [a for a, n in enumerate(dims) for _ in range(n // 2)]
    if case["shared"]:
        power = [2 * i / sum(dims) for i in range(len(axis))]
    else:
        power = [2 * j / n for n in dims for j in range(n // 2)]
    freq = torch.tensor([case["theta"] ** -p for p in power], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, axis] * freq)
    return torch.view_as_real(turn)


def _exact_heads(s, x, weight):
    case = s["case"]
    t, h, d = x.shape
    v = x.double().reshape(t, -1) if case["span"] == "row" else x.double().reshape(t * h, d)
    if case["norm"]:
        var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
        if case["norm"] == "rms":
            var, mean = var + mean * mean, 0.0
        v = (v - mean) / torch.sqrt(var + 1e-6)
        if weight is not None:
            v = v * weight.double()
    v = v.reshape(t, h, d)
    p = case["pairs"]
    if p:
        turn = torch.view_as_complex(s["table"].double())[:, None]
        i = torch.arange(p, device="cuda")
        first, second = (i, i + p) if case["halves"] else (2 * i, 2 * i + 1)
        z = torch.complex(v[..., first], v[..., second]) * turn
        v[..., first], v[..., second] = z.real, z.imag
    return v


def _exact_attention(s):
    """Head by head, by softmax(x) = exp(x - logsumexp(x))."""
    case = s["case"]
    hq, d = case["hq"], case["d"]
    group = hq // case["hk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, out.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for q0, lq, k0, lk in _spans(case):
        for h in range(hq):
            k = s["k"][k0:k0 + lk, h // group].double()
            v = s["v"][k0:k0 + lk, h // group].double()
            # queries before `start` see nothing
            start = max(0, lq - lk) if case["causal"] else 0
            step = max(1, (1 << 28) // lk)
            for i in range(start, lq, step):
                at = slice(q0 + i, q0 + min(lq, i + step))
                x = torch.matmul(s["q"][at, h].double() / math.sqrt(d), k.t())
                if case["causal"]:
                    seen = torch.ones(x.shape, dtype=torch.bool, device="cuda")
                    x[~torch.tril(seen, diagonal=i + lk - lq)] = -math.inf
                z = torch.logsumexp(x, -1)
                lse[h, at] = z
                out[at, h] = torch.matmul(torch.exp(x - z[:, None]), v)
    return (out, lse) if case["lse"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "table":
        return _exact_table(s)
    if case["op"] == "heads":
        return (_exact_heads(s, s["q"], s["q_weight"]), _exact_heads(s, s["k"], s["k_weight"]))
    return _exact_attention(s)
