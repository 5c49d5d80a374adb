"""Workloads of the operators that train an expert layer around its products: the router, the sum of a token's pairs
and the update of a bank, with one pass of each, its algorithmic work and its 64-bit definition.

  route        logits [T, E] -> the top_k experts of each token, their weights, and the pairs sorted by expert:
               scores are sigmoid or softmax, a bias for balance takes part in the choice only, groups of experts may be
               chosen first, weights may be renormalised over the chosen
  route_grad   the gradient of the logits from that of the weights
  combine      out[t] = sum over j of w[t, j] y[place[t, j]]: a token's pairs, weighted and summed
  combine_grad its gradients: of y and of w
  orthogonal   a matrix of the gradient's row and column space with singular values near 1, by Newton-Schulz products:
               X = g / |g|, then X <- a X + (b A + c A^2) X with A = X X^T, five times

With `own` false a pass is computed with elementary torch operations, in 32 bits (the router's scores in 64, where two
of them may lie close together); with `own` true by this repository's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


# ------------------------------------------------------------------ cases
def _route(name, op, dtype, tokens, experts, top_k, score, bias, groups, keep, renorm, scale, masked, padded):
    c = {"op": op, "dtype": dtype, "tokens": tokens, "experts": experts, "top_k": top_k, "score": score, "bias": bias,
         "groups": groups, "keep": keep, "renorm": renorm, "scale": scale, "masked": masked, "padded": padded}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decoded token through the router of the 256-expert top-6 layer
        _route("route_one_token", "route", "fp32", 1, 256, 6, "sigmoid", True, 1, 1, True, 1.0, 0.0, 0.0),
        # a prefill chunk of 8192 tokens, experts chosen within four of eight groups (a group on each of eight GPUs)
        _route("route_groups", "route", "bf16", 8192, 256, 6, "sigmoid", True, 8, 4, True, 2.5, 0.0, 0.0),
        # a training batch of odd length over few softmax-scored experts, some sequences padded
        _route("route_train_odd", "route", "fp32", 32771, 60, 4, "softmax", False, 1, 1, False, 1.0, 0.0, 0.03),
        # a large training batch of the 256-expert layer, a few experts taken out of service
        _route("route_train", "route", "fp32", 65536, 256, 6, "sigmoid", True, 1, 1, True, 1.0, 0.02, 0.0),
        # the backward pass of a large batch whose softmax weights are not renormalised: every logit has a gradient
        _route("route_grad_train", "route_grad", "bf16", 65536, 256, 6, "softmax", False, 1, 1, False, 1.0, 0.0, 0.0),
        # the backward pass of a small fine-tuned layer
        _route("route_grad_small", "route_grad", "fp32", 777, 100, 3, "sigmoid", True, 1, 1, True, 1.5, 0.0, 0.0),
        # the end of the layer for a decode batch of 32 tokens
        {"name": "combine_batch", "op": "combine", "dtype": "bf16", "tokens": 32, "top_k": 6, "hidden": 4096,
         "out": "fp32"},
        # and for a prefill chunk of 8192 tokens
        {"name": "combine_prefill", "op": "combine", "dtype": "bf16", "tokens": 8192, "top_k": 6, "hidden": 4096,
         "out": "bf16"},
        # the backward pass of a training batch
        {"name": "combine_grad_train", "op": "combine_grad", "dtype": "bf16", "tokens": 8192, "top_k": 6, "hidden": 4096,
         "out": "fp32"},
        # the backward pass of a small layer of odd width
        {"name": "combine_grad_odd", "op": "combine_grad", "dtype": "fp16", "tokens": 259, "top_k": 3, "hidden": 520,
         "out": "fp32"},
        # the update of sixteen experts' down matrices (a GPU's share of a bank of 256 over sixteen GPUs)
        {"name": "orthogonal_bank", "op": "orthogonal", "dtype": "bf16", "batch": 16, "rows": 4096, "cols": 2048,
         "idle": 1},
        # the update of a small layer's odd matrices from a momentum that is kept in 32 bits
        {"name": "orthogonal_odd", "op": "orthogonal", "dtype": "fp32", "batch": 13, "rows": 1000, "cols": 519,
         "idle": 0},
    ]


def _spread(rng, lo, hi, step=1):
    """A size in [lo, hi], spread over its logarithm: a power of two now and then, an odd multiple of `step` else."""
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.3:
        x = 1 << round(math.log2(x))
        if lo <= x <= hi and x % step == 0:
            return x
    x = (int(x / step) // 2 * 2 + 1) * step
    return x if x <= hi else max(x - 2 * step, lo)


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "combine", "combine_grad", "orthogonal", "orthogonal"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = max(_spread(rng, 2, 512) // groups, 1) * groups
        tokens = _spread(rng, 1, min(65536, 65536 * 256 // experts))
        keep = rng.randint(1, groups)
        top_k = rng.randint(1, min(8, keep * (experts // groups)))
        return _route(None, op, rng.choice(["bf16", "fp16", "fp32"]), tokens, experts, top_k,
                      rng.choice(["sigmoid", "softmax"]), rng.random() < 0.6, groups, keep, rng.random() < 0.6,
                      rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.1]), rng.choice([0.0, 0.0, 0.2]))
    if op in ("combine", "combine_grad"):
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "tokens": _spread(rng, 1, 4096),
                "top_k": rng.randint(1, 6), "hidden": _spread(rng, 64, 4096, 8), "out": rng.choice(["fp32", "same"])}
    rows, cols = _spread(rng, 8, 4096), _spread(rng, 8, 4096)
    m, n = min(rows, cols), max(rows, cols)
    most = 15 * 2048 * 2048 * (3 * 4096 + 2048) // (m * m * (3 * n + m))
    batch = _spread(rng, 1, max(1, min(most, 64)))
    return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "batch": batch, "rows": rows, "cols": cols,
            "idle": 1 if batch > 2 and rng.random() < 0.3 else 0}


# ----------------------------------------------------------------- inputs
def _normal(shape, scale, dtype, g):
    return torch.randn(shape, device="cuda", dtype=dtype, generator=g).mul_(scale)


def _prepare_route(c, g, s):
    T, E, dtype = c["tokens"], c["experts"], DTYPES[c["dtype"]]
    # some experts are liked more than others; the bias leans the other way, as the one that balances them does
    liked = torch.randn(E, device="cuda", generator=g)
    x = torch.randn(T, E, device="cuda", generator=g).mul_(1.5).add_(0.7 * liked)
    if c["masked"]:
        out = torch.randperm(E, device="cuda", generator=g)[: min(max(1, int(c["masked"] * E)), E - c["top_k"])]
        x[:, out] = -math.inf
    if c["padded"]:
        x[torch.rand(T, device="cuda", generator=g) < c["padded"]] = -math.inf
    s["logits"] = x.to(dtype)
    wide = 0.05 if c["score"] == "sigmoid" else 0.3 / E
    s["bias"] = -wide * liked if c["bias"] else None
    if c["op"] == "route_grad":
        s["ids"], s["w"] = _route_plain(s)[:2]
        s["dw"] = torch.randn(T, c["top_k"], device="cuda", generator=g)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c, "op": c["op"]}
    if c["op"] in ("route", "route_grad"):
        _prepare_route(c, g, s)
    elif c["op"] in ("combine", "combine_grad"):
        T, k, H, dtype = c["tokens"], c["top_k"], c["hidden"], DTYPES[c["dtype"]]
        s["out"] = dtype if c["out"] == "same" else DTYPES[c["out"]]
        s["y"] = _normal((T * k, H), 1.0, dtype, g)
        # where the pairs of 32 experts' groups stand: a token's pairs lie far apart
        expert = torch.rand(T, 32, device="cuda", generator=g).topk(k, dim=1).indices.reshape(-1)
        perm = expert.sort(stable=True).indices
        s["place"] = torch.empty_like(perm)
        s["place"][perm] = torch.arange(T * k, device="cuda")
        s["place"] = s["place"].view(T, k)
        w = torch.rand(T, k, device="cuda", generator=g) + 0.1
        s["w"] = w / w.sum(1, keepdim=True)
        if c["op"] == "combine_grad":
            s["dout"] = _normal((T, H), 0.1, s["out"], g)
    else:
        B, M, N = c["batch"], c["rows"], c["cols"]
        # the gradient that a batch of tokens leaves (a few strong directions), older ones below it; experts without
        # tokens have none
        tokens = max(1, min(M, N) // 4)
        x = torch.bmm(torch.randn(B, M, tokens, device="cuda", generator=g),
                      torch.randn(B, tokens, N, device="cuda", generator=g)).mul_(tokens**-0.5)
        x.add_(torch.randn(B, M, N, device="cuda", generator=g), alpha=0.3)
        x.mul_(1e-3 * torch.exp(torch.randn(B, 1, 1, device="cuda", generator=g)))
        if c["idle"]:
            x[: c["idle"]] = 0
        s["g"] = x.to(DTYPES[c["dtype"]])
    return s


# ------------------------------------------------------------- plain form
def _scores(s):
    """Scores in 64 bits: a choice between two of them must not hang on their rounding."""
    x = s["logits"].double()
    if s["case"]["score"] == "sigmoid":
        return x, 1 / (1 + torch.exp(-x))
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    z = e.sum(1, keepdim=True)
    return x, e / torch.where(z > 0, z, 1.0)


def _route_plain(s):
    """Chosen experts (-1: none left), their weights, and the pairs sorted by expert."""
    c = s["case"]
    T, E, k, G = c["tokens"], c["experts"], c["top_k"], c["groups"]
    x, score = _scores(s)
    key = score if s["bias"] is None else score + s["bias"]
    key = torch.where(x == -math.inf, -math.inf, key)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        some = best[:, :, 0] > -math.inf
        total = torch.where(some, torch.where(best == -math.inf, 0.0, best).sum(2), -math.inf)
        order = total.sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order[:, : c["keep"]], True)
        key = torch.where(kept[:, :, None], key.view(T, G, E // G), -math.inf).view(T, E)
    value, ids = key.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    there = value > -math.inf
    w = torch.where(there, score.gather(1, ids), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    ids = torch.where(there, ids, -1).to(torch.int32)
    return ids, (w * c["scale"]).float()


def _pairs_plain(ids, E):
    flat = ids.reshape(-1).long()
    flat = torch.where(flat < 0, E, flat)
    perm = flat.sort(stable=True).indices
    place = torch.empty_like(perm)
    place[perm] = torch.arange(perm.numel(), device=perm.device)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(
        0, flat, torch.ones_like(flat))[:E].cumsum(0)
    return {"perm": perm, "rows": (perm // ids.shape[1]).to(torch.int32), "place": place, "offsets": offsets}


def _route_all(s):
    ids, w = _route_plain(s)
    return {"ids": ids, "w": w, **_pairs_plain(ids, s["case"]["experts"])}


def _route_grad_plain(s):
    c, ids = s["case"], s["ids"].long()
    there = ids >= 0
    x = s["logits"].float()
    G = torch.where(there, s["dw"] * c["scale"], 0.0)
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        z = p.sum(1, keepdim=True)
        p = p / torch.where(z > 0, z, 1.0)
    chosen = torch.where(there, p.gather(1, ids.clamp_min(0)), 0.0)
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        G = torch.where(there, (G - (G * chosen).sum(1, keepdim=True) / total) / total, 0.0)
    d = torch.zeros_like(x).scatter_add_(1, ids.clamp_min(0), torch.where(there, G, 0.0))
    if c["score"] == "sigmoid":
        d = d * p * (1 - p)
    else:
        d = p * (d - (G * chosen).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _combine_plain(s):
    return (s["y"].float()[s["place"]] * s["w"][:, :, None]).sum(1).to(s["out"])


def _combine_grad_plain(s):
    d = s["dout"].float()
    dw = (s["y"].float()[s["place"]] * d[:, None]).sum(2)
    dy = torch.empty(s["y"].shape, device="cuda")
    dy[s["place"]] = s["w"][:, :, None] * d[:, None]
    return {"dy": dy.to(s["y"].dtype), "dw": dw}


def _orthogonal_plain(s):
    a, b, c = COEFFICIENTS
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        aa = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * aa + c * torch.bmm(aa, aa), x)
    return (x.transpose(1, 2) if tall else x).to(s["g"].dtype).contiguous()


PLAIN = {"route": _route_all, "route_grad": _route_grad_plain, "combine": _combine_plain,
         "combine_grad": _combine_grad_plain, "orthogonal": _orthogonal_plain}


# ---------------------------------------------------------------- kernels
def _route_own(qr, s):
    c = s["case"]
    r = qr.Routing.from_logits(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                               keep_groups=c["keep"], renormalize=c["renorm"], scale=c["scale"])
    return {"ids": r.ids, "w": r.w, "perm": r.perm, "rows": r.rows, "place": r.place, "offsets": r.offsets}


def _route_grad_own(qr, s):
    c = s["case"]
    return qr.route_grad(s["dw"], s["logits"], s["ids"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])


def _combine_grad_own(qr, s):
    dy, dw = qr.combine_grad(s["dout"], s["y"], s["place"], s["w"])
    return {"dy": dy, "dw": dw}


OWN = {"route": _route_own, "route_grad": _route_grad_own,
       "combine": lambda qr, s: qr.combine(s["y"], s["place"], s["w"], dtype=s["out"]), "combine_grad": _combine_grad_own,
       "orthogonal": lambda qr, s: qr.orthogonalize(s["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)}


def run(state):
    if own:
        import quantized_routed_moe_amd as qr
        return OWN[state["op"]](qr, state)
    return PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("route", "route_grad"):
        T, E, k, z = c["tokens"], c["experts"], c["top_k"], SIZE[c["dtype"]]
        if c["op"] == "route":
            # logits and bias in; ids and weights, the pairs' order (two of 8 bytes, one of 4) and the offsets out
            return {"bytes": T * E * z + 4 * E * c["bias"] + T * k * (8 + 20) + 4 * (E + 1), "flops": 8 * T * E}
        # the gradient of every logit out; the scores of a sigmoid are needed at the chosen experts only
        read = T * E * z if c["score"] == "softmax" and not c["renorm"] else T * k * z
        return {"bytes": read + T * E * z + 8 * T * k, "flops": 8 * T * E}
    if c["op"] in ("combine", "combine_grad"):
        T, k, H, z = c["tokens"], c["top_k"], c["hidden"], SIZE[c["dtype"]]
        o = z if c["out"] == "same" else SIZE[c["out"]]
        if c["op"] == "combine":
            return {"bytes": T * k * H * z + T * H * o + 12 * T * k, "flops": 2 * T * k * H}
        return {"bytes": 2 * T * k * H * z + T * H * o + 16 * T * k, "flops": 3 * T * k * H}
    B, m, n = c["batch"], min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
    # A and A^2 are symmetric: half of each; matrices of zeros need none
    return {"bytes": 2 * B * m * n * SIZE[c["dtype"]],
            "flops": STEPS * (B - c["idle"]) * (m * m * n + m * m * m + 2 * m * m * n)}


# ------------------------------------------------------ 64-bit definition
def _first(key, k):
    """The k first columns by (larger key, lower index) and whether each has a key above -inf, by counting for each
    column how many come before it."""
    T, E = key.shape
    at = torch.empty(T, k, dtype=torch.int64, device=key.device)
    col = torch.arange(E, device=key.device)
    for i in range(0, T, 1024):
        x = key[i : i + 1024]
        before = (x[:, None, :] > x[:, :, None]) | ((x[:, None, :] == x[:, :, None]) & (col < col[:, None]))
        rank = before.sum(2)
        at[i : i + 1024] = (rank[:, None, :] == torch.arange(k, device=key.device)[:, None]).int().argmax(2)
    return at, key.gather(1, at) != -math.inf


def _probabilities(c, logits):
    x = logits.double()
    if c["score"] == "sigmoid":
        return torch.sigmoid(x)
    return torch.nan_to_num(torch.exp(x - torch.logsumexp(x, 1, keepdim=True)), nan=0.0)


def _exact_route(c, s):
    E, k, G = c["experts"], c["top_k"], c["groups"]
    p = _probabilities(c, s["logits"])
    key = p + (0 if s["bias"] is None else s["bias"].double())
    key.masked_fill_(torch.isneginf(s["logits"]), -math.inf)
    if G > 1:
        total = torch.empty(key.shape[0], G, dtype=torch.float64, device=key.device)
        for j, part in enumerate(key.split(E // G, dim=1)):
            first = part.max(1, keepdim=True)
            rest = part.scatter(1, first.indices, -math.inf).max(1).values
            total[:, j] = first.values[:, 0] + torch.where(torch.isneginf(rest), 0.0, rest)
        at, _ = _first(total, c["keep"])
        owner = torch.arange(E, device=key.device) // (E // G)
        key.masked_fill_(~(owner[None, :, None] == at[:, None, :]).any(2), -math.inf)
    at, there = _first(key, k)
    w = p.gather(1, at) * there
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    ids = torch.where(there, at, -1)
    # the order of the pairs, from keys that no two of them share
    flat = torch.where(there, at, E).reshape(-1)
    n = flat.numel()
    order = (flat * n + torch.arange(n, device=flat.device)).argsort()
    place = torch.arange(n, device=flat.device)[order.argsort()]
    offsets = torch.searchsorted(flat[order], torch.arange(E + 1, device=flat.device))
    return {"ids": ids.to(torch.int32), "w": w * c["scale"], "perm": order,
            "rows": torch.div(order, k, rounding_mode="floor").to(torch.int32), "place": place,
            "offsets": offsets.to(torch.int32)}


def _exact_route_grad(c, s):
    p = _probabilities(c, s["logits"])
    T, E = p.shape
    # the weights' derivative by each score, summed over the chosen
    there = s["ids"] >= 0
    at = s["ids"].long().clamp_min(0)
    q, gw = p.gather(1, at) * there, s["dw"].double() * c["scale"] * there
    if c["renorm"]:
        z = q.sum(1, keepdim=True)
        z = torch.where(z > 0, z, torch.ones_like(z))
        gw = (gw / z - (gw * q).sum(1, keepdim=True) / z.square()) * there
    ds = torch.zeros(T, E, dtype=torch.float64, device=p.device)
    for j in range(c["top_k"]):
        ds[torch.arange(T, device=p.device), at[:, j]] += gw[:, j]
    if c["score"] == "sigmoid":
        return ds * (p - p * p)
    return ds * p - p * (ds * p).sum(1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "route":
        return _exact_route(c, s)
    if op == "route_grad":
        return _exact_route_grad(c, s)
    if op in ("combine", "combine_grad"):
        T, k, H = c["tokens"], c["top_k"], c["hidden"]
        w = s["w"].double()
        if op == "combine":
            out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
            for j in range(k):
                out += w[:, j : j + 1] * s["y"][s["place"][:, j]].double()
            return out
        d = s["dout"].double()
        dy = torch.empty(T * k, H, dtype=torch.float64, device="cuda")
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            dy[s["place"][:, j]] = w[:, j : j + 1] * d
            dw[:, j] = torch.linalg.vecdot(s["y"][s["place"][:, j]].double(), d)
        return {"dy": dy, "dw": dw}
    a, b, cc = COEFFICIENTS
    out = torch.empty(s["g"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["batch"]):
        x = s["g"][i].double()
        x = x / (torch.linalg.vector_norm(x) + EPS)
        for _ in range(STEPS):
            if c["rows"] > c["cols"]:
                t = x.t() @ x
                x = x @ (cc * (t @ t) + b * t) + a * x
            else:
                t = x @ x.t()
                x = (cc * (t @ t) + b * t) @ x + a * x
        out[i] = x
    return out
