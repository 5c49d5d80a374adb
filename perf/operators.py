"""The expert operators' workloads: inputs, one pass, its algorithmic work and its 64-bit definition.

The operators work on the pairs (token, expert) of a mixture-of-experts layer, grouped by expert: group e holds
the rows offsets[e] .. offsets[e+1] of the pair order, any number of them, none included.

  forward    c[p] = a[r(p)] . b[e(p)]^T             grouped product; b is [experts, out, in], r the row gather
  backward   da[p] = dc[p] . b[e(p)]                 both gradients of that product
             db[e] = sum over the group of dc[p]^T a[r(p)]
  quantize   x -> blocks of 32 four-bit floats (sign, 2 exponent bits, 1 mantissa bit) with a power-of-two scale,
             and back
  mxfp4      the grouped product with both operands in that format
  swiglu     h = silu(gate) * up of the stacked product [gate | up]; swiglu_grad is its gradient

With `own` false a pass is computed with elementary torch operations in 32 bits; with `own` true by this
repository's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token through the stacked gate/up bank of the 256-expert top-6 layer: six weight matrices streamed
        {"name": "forward_one_token", "op": "forward", "dtype": "bf16", "tokens": 1, "top_k": 6, "experts": 256,
         "out": 4096, "in": 4096, "gather": True, "idle": 0.0},
        # the down product of a 2048-token prefill chunk: about 48 rows for each of the 256 experts
        {"name": "forward_prefill", "op": "forward", "dtype": "bf16", "tokens": 2048, "top_k": 6, "experts": 256,
         "out": 4096, "in": 2048, "gather": False, "idle": 0.0},
        # few large experts and a long ragged batch: the product is bound by arithmetic, not by the weights
        {"name": "forward_few_experts", "op": "forward", "dtype": "fp16", "tokens": 8191, "top_k": 2, "experts": 8,
         "out": 4096, "in": 4096, "gather": True, "idle": 0.0},
        # one training step's gradients of a GPU's share of the experts (64 of 256), a few of them without tokens
        {"name": "backward_train", "op": "backward", "dtype": "bf16", "tokens": 2048, "top_k": 6, "experts": 64,
         "out": 4096, "in": 4096, "gather": True, "idle": 0.05, "grad": "bf16"},
        # a small fine-tuned layer of odd widths, weight gradients kept in 32 bits for accumulation
        {"name": "backward_small_odd", "op": "backward", "dtype": "fp16", "tokens": 259, "top_k": 3, "experts": 13,
         "out": 1000, "in": 520, "gather": False, "idle": 0.1, "grad": "fp32"},
        # activations of a decode batch of 32 tokens
        {"name": "quantize_tokens", "op": "quantize", "dtype": "fp32", "rows": 32, "in": 4096},
        # a whole bank of 256 expert matrices at load time
        {"name": "quantize_bank", "op": "quantize", "dtype": "bf16", "rows": 256 * 2048, "in": 4096},
        # one decoded token through four-bit gate/up weights
        {"name": "mxfp4_one_token", "op": "mxfp4", "tokens": 1, "top_k": 6, "experts": 256, "out": 4096, "in": 4096,
         "gather": True, "idle": 0.0},
        # a decode batch of 32 tokens through four-bit down weights
        {"name": "mxfp4_batch", "op": "mxfp4", "tokens": 32, "top_k": 6, "experts": 256, "out": 4096, "in": 2048,
         "gather": False, "idle": 0.0},
        # an 8192-token prefill chunk through four-bit gate/up weights: 192 rows an expert
        {"name": "mxfp4_prefill", "op": "mxfp4", "tokens": 8192, "top_k": 6, "experts": 256, "out": 4096, "in": 4096,
         "gather": True, "idle": 0.0},
        # the activation of a decode batch of 32 tokens, top-6
        {"name": "swiglu_batch", "op": "swiglu", "dtype": "bf16", "rows": 192, "ffn": 2048},
        # its gradient for the pairs of an 8192-token training batch
        {"name": "swiglu_grad_train", "op": "swiglu_grad", "dtype": "bf16", "rows": 49152, "ffn": 2048},
    ]


def _spread(rng, lo, hi, step=1):
    """A size in [lo, hi], spread over its logarithm: a power of two now and then, an odd multiple of `step` else."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.3:
        return min(hi, max(lo, 1 << round(math.log2(x))))
    x = (int(x / step) // 2 * 2 + 1) * step
    return x if x <= hi else max(x - 2 * step, lo)


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "quantize", "mxfp4", "mxfp4", "swiglu", "swiglu_grad"])
    if op == "quantize":
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": _spread(rng, 1, 200000),
                "in": _spread(rng, 32, 8192, 32)}
    if op in ("swiglu", "swiglu_grad"):
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": _spread(rng, 1, 40000),
                "ffn": _spread(rng, 64, 2048, 8)}
    step = 32 if op == "mxfp4" else 8
    experts = _spread(rng, 1, 256)
    c = {"op": op, "tokens": _spread(rng, 1, 8192 if op == "mxfp4" else 2500), "top_k": rng.randint(1, min(6, experts)),
         "experts": experts, "out": _spread(rng, 64, 4096, 8), "in": _spread(rng, 64, 4096, step),
         "gather": rng.random() < 0.5, "idle": rng.choice([0.0, 0.0, 0.3])}
    if op != "mxfp4":
        c["dtype"] = rng.choice(["bf16", "fp16"])
    if op == "backward":
        c["experts"] = min(experts, 64)
        c["top_k"] = min(c["top_k"], c["experts"])
        c["grad"] = rng.choice([c["dtype"], "fp32"])
    return c


# ----------------------------------------------------------------- inputs
def _routing(c, g):
    """Top-k choices of a router with uneven experts, `idle` of which get no token: the token of each pair in
    pair order, the groups' offsets, and (for the plain form) the size of the largest group."""
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    bias = 0.5 * torch.randn(E, device="cuda", generator=g)
    bias[torch.randperm(E, device="cuda", generator=g)[: min(int(c["idle"] * E), E - k)]] = -1e9
    noise = -torch.log(-torch.log(torch.rand(T, E, device="cuda", generator=g).clamp(1e-6, 1 - 1e-6)))
    ids = (noise + bias).topk(k, dim=1).indices.reshape(-1)
    order = ids.sort(stable=True).indices
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return (order // k).to(torch.int32), offsets, int(counts.max())


def _normal(shape, scale, dtype, g):
    return torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(scale)


def _codes(shape, g):
    """Pairs of four-bit codes with the frequencies that normal values leave in a block."""
    low = [0, 1, 2, 3, 4, 4, 5, 6]
    high = [0, 1, 2, 3, 4, 4, 5, 7]
    table = [(low[b & 7] | (b & 8)) | ((high[b >> 4 & 7] | (b >> 4 & 8)) << 4) for b in range(256)]
    raw = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    table = torch.tensor(table, dtype=torch.uint8, device="cuda")
    return table[raw.int()]


def _scales(shape, middle, g):
    return torch.randint(middle - 1, middle + 2, shape, dtype=torch.uint8, device="cuda", generator=g)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "op": c["op"]}
    if c["op"] == "quantize":
        # rows of unlike magnitude, as tokens and weight rows have
        s["x"] = _normal((c["rows"], c["in"]), 1.0, DTYPES[c["dtype"]], g)
        s["x"] *= torch.exp(torch.randn(c["rows"], 1, device="cuda", generator=g)).to(s["x"].dtype)
        return s
    if c["op"] in ("swiglu", "swiglu_grad"):
        s["gu"] = _normal((c["rows"], 2 * c["ffn"]), 1.5, DTYPES[c["dtype"]], g)
        if c["op"] == "swiglu_grad":
            s["dh"] = _normal((c["rows"], c["ffn"]), 0.1, DTYPES[c["dtype"]], g)
        return s
    E, N, K = c["experts"], c["out"], c["in"]
    token, s["offsets"], s["most"] = _routing(c, g)
    s["rows"] = token if c["gather"] else None
    P = token.numel()
    R = c["tokens"] if c["gather"] else P
    if c["op"] == "mxfp4":
        s["a"], s["a_scales"] = _codes((R, K // 2), g), _scales((R, K // 32), 125, g)
        s["b"], s["b_scales"] = _codes((E, N, K // 2), g), _scales((E, N, K // 32), 120, g)
        return s
    dtype = DTYPES[c["dtype"]]
    s["a"] = _normal((R, K), 1.0, dtype, g)
    s["b"] = _normal((E, N, K), 1.0 / math.sqrt(K), dtype, g)
    if c["op"] == "backward":
        s["dc"] = _normal((P, N), 0.1, dtype, g)
        s["grad"] = DTYPES[c["grad"]]
    return s


# ------------------------------------------------------------- plain form
def _padded(s, x, gathered):
    """x's rows in a block of the largest group's size for each expert, zeros past a group's end, in 32 bits."""
    o = s["offsets"].long()
    at = o[:-1, None] + torch.arange(s["most"], device=o.device)
    inside = at < o[1:, None]
    at = at.clamp_max(int(s["rows"].numel()) - 1 if gathered else x.shape[0] - 1)
    if gathered:
        at = s["rows"].long()[at]
    return x[at].float() * inside[:, :, None]


def _ragged(s, y, pairs):
    """The rows of the groups in pair order, from the padded blocks."""
    e = _expert(s, pairs)
    return y[e, torch.arange(pairs, device=e.device) - s["offsets"].long()[e]]


def _expert(s, pairs):
    """The expert of each pair."""
    return torch.searchsorted(s["offsets"].long(), torch.arange(pairs, device=s["offsets"].device), right=True) - 1


def _values(codes, scales):
    """The numbers that codes and scales stand for, in 32 bits."""
    v = torch.tensor(MAGNITUDES + [-m for m in MAGNITUDES], device=codes.device)
    b = torch.arange(256, device=codes.device)
    two = torch.stack([v[b & 15], v[b >> 4]], 1)
    x = two[codes.int()].view(*scales.shape, 32)
    x *= torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)[..., None]
    return x.view(*codes.shape[:-1], codes.shape[-1] * 2)


def _round_trip(x):
    """x rounded to blocks of 32 four-bit floats: scale 2^(floor(log2 max|x|) - 2), ties to the even mantissa, past 6 to 6."""
    b = x.float().view(*x.shape[:-1], -1, 32)
    most = b.abs().amax(-1, keepdim=True)
    scale = torch.ldexp(torch.ones_like(most), (torch.frexp(most).exponent - 3).clamp_min(-127))
    m = (b / scale).abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp_max(6.0)
    return torch.copysign(m * scale, b).view(x.shape).to(x.dtype)


def _pairs(s):
    return s["case"]["tokens"] * s["case"]["top_k"]


def _product(s, a_of, b_of, dtype):
    """a . b^T by expert; where there are fewer pairs than experts only the pairs' own matrices are touched."""
    pairs, gathered = _pairs(s), s["rows"] is not None
    if pairs < s["case"]["experts"]:
        at = s["rows"].long() if gathered else slice(None)
        return torch.bmm(a_of(at)[:, None], b_of(_expert(s, pairs)).transpose(1, 2))[:, 0].to(dtype)
    a = _padded(s, a_of(slice(None)), gathered)
    return _ragged(s, torch.bmm(a, b_of(slice(None)).transpose(1, 2)), pairs).to(dtype)


def _forward_plain(s):
    return _product(s, lambda at: s["a"][at].float(), lambda e: s["b"][e].float(), s["a"].dtype)


def _backward_plain(s):
    dc = _padded(s, s["dc"], False)
    da = _ragged(s, torch.bmm(dc, s["b"].float()), _pairs(s)).to(s["a"].dtype)
    db = torch.bmm(dc.transpose(1, 2), _padded(s, s["a"], s["rows"] is not None))
    return {"da": da, "db": db.to(s["grad"])}


def _mxfp4_plain(s):
    return _product(s, lambda at: _values(s["a"][at], s["a_scales"][at]),
                    lambda e: _values(s["b"][e], s["b_scales"][e]), torch.bfloat16)


def _swiglu_plain(s):
    g, u = s["gu"].float().chunk(2, 1)
    return (g / (1 + torch.exp(-g)) * u).to(s["gu"].dtype)


def _swiglu_grad_plain(s):
    g, u = s["gu"].float().chunk(2, 1)
    dh, sig = s["dh"].float(), 1 / (1 + torch.exp(-g))
    return torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], 1).to(s["gu"].dtype)


PLAIN = {"forward": _forward_plain, "backward": _backward_plain, "quantize": lambda s: _round_trip(s["x"]),
         "mxfp4": _mxfp4_plain, "swiglu": _swiglu_plain, "swiglu_grad": _swiglu_grad_plain}


# ---------------------------------------------------------------- kernels
def _forward_own(qr, s):
    return qr.grouped_mm(s["a"], s["b"], s["offsets"], rows=s["rows"])


def _backward_own(qr, s):
    return {"da": qr.grouped_mm_grad_a(s["dc"], s["b"], s["offsets"]),
            "db": qr.grouped_mm_grad_b(s["dc"], s["a"], s["offsets"], rows=s["rows"], dtype=s["grad"])}


def _quantize_own(qr, s):
    codes, scales = qr.mxfp4_quantize(s["x"])
    return qr.mxfp4_dequantize(codes, scales, dtype=s["x"].dtype)


def _mxfp4_own(qr, s):
    return qr.mxfp4_grouped_mm(s["a"], s["a_scales"], s["b"], s["b_scales"], s["offsets"], rows=s["rows"],
                               dtype=torch.bfloat16)


OWN = {"forward": _forward_own, "backward": _backward_own, "quantize": _quantize_own, "mxfp4": _mxfp4_own,
       "swiglu": lambda qr, s: qr.swiglu(s["gu"]), "swiglu_grad": lambda qr, s: qr.swiglu_grad(s["dh"], s["gu"])}


def run(state):
    if own:
        import quantized_routed_moe_amd as qr
        return OWN[state["op"]](qr, state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "quantize":
        # x in; codes and scales out; the values they stand for out
        n = c["rows"] * c["in"]
        return {"bytes": n * (2 * size[c["dtype"]] + 0.5 + 1 / 32), "flops": 4 * n}
    if c["op"] == "swiglu":
        n = c["rows"] * c["ffn"]
        return {"bytes": 3 * n * size[c["dtype"]], "flops": 5 * n}
    if c["op"] == "swiglu_grad":
        n = c["rows"] * c["ffn"]
        return {"bytes": 5 * n * size[c["dtype"]], "flops": 12 * n}
    E, N, K, P = c["experts"], c["out"], c["in"], c["tokens"] * c["top_k"]
    R = c["tokens"] if c["gather"] else P
    # experts that get a token at all when each is as likely as the other; only their weights are read
    live = max(E - int(c["idle"] * E), c["top_k"])
    hit = live * (1 - (1 - c["top_k"] / live) ** c["tokens"])
    if c["op"] == "mxfp4":
        return {"bytes": (hit * N + R) * K * 17 / 32 + 2 * P * N, "flops": 2 * P * N * K}
    if c["op"] == "forward":
        return {"bytes": 2 * (hit * N * K + R * K + P * N), "flops": 2 * P * N * K}
    # dc, a and b in, da and every expert's db out
    return {"bytes": 2 * (P * N + R * K + hit * N * K + P * K) + size[c["grad"]] * E * N * K, "flops": 4 * P * N * K}


# ------------------------------------------------------ 64-bit definition
def _nearest(x):
    """Blocks of 32 rounded to the nearest representable number by comparing with the midpoints between them."""
    v = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    b = x.double().reshape(-1, 32)
    most = b.abs().amax(1, keepdim=True)
    exponent = torch.where(most > 0, torch.floor(torch.log2(most)), -125.0)
    # log2 rounds; the power of two at or below the largest magnitude is what is meant
    exponent += (torch.exp2(exponent + 1) <= most).double() - (torch.exp2(exponent) > most).double() * (most > 0)
    scale = torch.exp2((exponent - 2).clamp_min(-127))
    m = b.abs() / scale
    mid = (v[1:] + v[:-1]) / 2
    below, above = torch.bucketize(m, mid, right=False), torch.bucketize(m, mid, right=True)
    code = torch.where(below % 2 == 0, below, above)  # on a midpoint the two differ: the even code
    return (v[code] * scale * torch.where(b < 0, -1.0, 1.0)).reshape(x.shape)


def _wide(codes, scales):
    v = torch.tensor(MAGNITUDES + [-m for m in MAGNITUDES], dtype=torch.float64, device=codes.device)
    x = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = v[(codes & 15).int()], v[(codes >> 4).int()]
    return x * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        # the values are exact in every input type, so the type of run's output holds them
        y = torch.empty(s["x"].shape, dtype=s["x"].dtype, device="cuda")
        for i in range(0, case["rows"], 16384):
            y[i : i + 16384] = _nearest(s["x"][i : i + 16384]).to(y.dtype)
        return y
    if op == "swiglu":
        g, u = s["gu"][:, : case["ffn"]].double(), s["gu"][:, case["ffn"] :].double()
        return g * torch.sigmoid(g) * u
    if op == "swiglu_grad":
        g, u, dh = s["gu"][:, : case["ffn"]].double(), s["gu"][:, case["ffn"] :].double(), s["dh"].double()
        sig = torch.sigmoid(g)
        return torch.cat([dh * u * (sig + g * sig * (1 - sig)), dh * g * sig], 1)
    o = s["offsets"].tolist()
    rows = s["rows"].long() if s["rows"] is not None else torch.arange(_pairs(s), device="cuda")
    E, N, K = case["experts"], case["out"], case["in"]
    if op == "backward":
        da = torch.empty(rows.numel(), K, dtype=torch.float64, device="cuda")
        db = torch.empty(E, N, K, dtype=torch.float64, device="cuda")
        for e in range(E):
            i, j = o[e], o[e + 1]
            dc = s["dc"][i:j].double()
            da[i:j] = dc @ s["b"][e].double()
            db[e] = dc.t() @ s["a"][rows[i:j]].double()
        return {"da": da, "db": db}
    y = torch.empty(rows.numel(), N, dtype=torch.float64, device="cuda")
    for e in range(E):
        i, j = o[e], o[e + 1]
        if j > i:
            if op == "forward":
                a, b = s["a"][rows[i:j]].double(), s["b"][e].double()
            else:
                a, b = _wide(s["a"][rows[i:j]], s["a_scales"][rows[i:j]]), _wide(s["b"][e], s["b_scales"][e])
            y[i:j] = a @ b.t()
    return y
