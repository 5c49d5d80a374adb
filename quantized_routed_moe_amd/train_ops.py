"""Operators around the experts' products: the router with the order of its
pairs and its gradient, the sum of a token's pairs with its gradients, and the
orthogonalised update of a bank.

Argument checks and marshalling only, with the conventions of expert_ops: HIP
kernels behind the C ABI of include/moe.h, enqueued on `stream` (the current
one by default) without synchronising, results allocated for that stream.
The calls build no graph; Routing.from_logits, Routing.combine and expert_ffn
are the differentiable ones (Routing.combine by torch's operations where a
gradient is asked for, not by the kernels).
"""
from __future__ import annotations

import ctypes

import torch

from . import PairOrder, Router, _check, _layout, _lib
from .expert_ops import (DT, _dtype, _graph, _hold, _matrix, _new, _output, _plain, _pointer, _Refusal, _target,
                         _written)

SCORES = {"sigmoid": 1, "softmax": 2}
MAX_PAIRS = 1 << 20
MAX_EXPERTS = 1024
MAX_STEPS = 32
_FLOATS = tuple(DT)


def _rows(t, name, cols=None):
    """Row stride of a 2-d operand whose rows may be strided, element-aligned."""
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{name}: expected shape (rows, {'columns' if cols is None else cols}), got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: elements of a row must be consecutive")
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if stride < t.shape[1]:
        raise ValueError(f"{name}: row stride {stride} must cover a row")
    return stride


def _router(n_experts, top_k, score, renormalize, scale, bias=None, groups=1, keep_groups=None, group_best=2):
    if score not in SCORES:
        raise ValueError(f"score: expected one of {', '.join(SCORES)}, got {score!r}")
    keep = groups if keep_groups is None else keep_groups
    if (top_k | groups | keep | group_best) >> 31:  # would not be what the C call sees
        raise ValueError(f"top_k, groups, keep_groups, group_best: got {top_k}, {groups}, {keep}, {group_best}")
    return Router(n_experts, top_k, SCORES[score], groups, keep, group_best, 1 if renormalize else 0, scale, bias)


def _order(tokens, top_k, n_experts, like, stream):
    """New arrays for a pairs' order (perm, offsets, rows, place), its workspace and the C struct that names them."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _order(tokens, top_k, n_experts, like, None)
    new, pairs = like.new_empty, (tokens * top_k,)
    perm, place, rows = new(pairs, dtype=torch.int64), new(pairs, dtype=torch.int64), new(pairs, dtype=torch.int32)
    offsets = new((n_experts + 1,), dtype=torch.int32)
    n = _lib.moe_pair_order_bytes(tokens, n_experts)
    work = new((n,), dtype=torch.uint8) if n else None
    return (perm, offsets, rows, place), work, PairOrder(perm.data_ptr(), place.data_ptr(), rows.data_ptr(),
                                                         offsets.data_ptr(), work.data_ptr() if n else None, n)


def _route(call, logits, top_k, score, bias, groups, keep_groups, group_best, renormalize, scale, ordered, stream):
    """(ids, w, order tensors or None) of a checked call."""
    _dtype(logits, "logits", _FLOATS)
    ld = _rows(logits, "logits")
    T, E = logits.shape
    index, raw, side = _target(logits, "logits", stream)
    at = None
    if bias is not None:
        _layout(bias, "bias", torch.float32, (E,))
        at = _plain(bias, "bias", index)
    r = _router(E, top_k, score, renormalize, scale, at, groups, keep_groups, group_best)
    k = top_k if 0 < top_k <= E else 0  # else the call below refuses
    ids, w = _new(logits, (T, k), torch.int32, side), _new(logits, (T, k), torch.float32, side)
    order = work = struct = None
    if ordered and T * k <= MAX_PAIRS and 1 <= E <= MAX_EXPERTS:
        order, work, struct = _order(T, k, E, logits, side)
    _check(_lib.moe_route(ctypes.byref(r), DT[logits.dtype], logits.data_ptr(), ld, T, ids.data_ptr(), w.data_ptr(),
                          None if struct is None else ctypes.byref(struct), raw), call)
    _hold(side, logits, bias, work)
    return ids, w, order


def route(logits, top_k, score="sigmoid", bias=None, groups=1, keep_groups=None, group_best=2, renormalize=True,
          scale=1.0, stream=None):
    """(ids [T, top_k] int32, w [T, top_k] fp32): the experts that each token's logits [T, E] (fp32, bf16 or fp16)
    choose and their weights.

    Scores are "sigmoid" or "softmax" of the logits.  `bias` [E] fp32 is added for the choice only; an expert whose
    logit or bias is -inf is not there.  With groups > 1, of that many equal runs of experts the `keep_groups` with
    the largest sums of their `group_best` (1 or 2) largest keys stay.  Equal keys go to the lower index (a bias that
    is the same for every expert changes no order, nor does it make keys equal).  Weights are the chosen scores, with
    `renormalize` divided by their sum, times `scale`; where fewer than top_k experts are
    left, ids are -1 and weights 0."""
    graph = _graph("route", None, logits, instead="use Routing.from_logits")
    ids, w, _ = _route("moe_route", logits, top_k, score, bias, groups, keep_groups, group_best, renormalize, scale,
                       False, stream)
    return ids, w if graph is None else _Refusal.apply(graph, w, logits)


def route_grad(dw, logits, ids, score="sigmoid", renormalize=True, scale=1.0, out=None, stream=None):
    """The gradient of route's weights with respect to the logits: dlogits [T, E] in the logits' type from dw [T, k]
    fp32, the logits and the ids [T, k] int32 of the forward call (entries outside [0, E) have none)."""
    _dtype(logits, "logits", _FLOATS)
    ld = _rows(logits, "logits")
    T, E = logits.shape
    _layout(ids, "ids", torch.int32)
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids: expected [{T}, top_k], got {tuple(ids.shape)}")
    _layout(dw, "dw", torch.float32, tuple(ids.shape))
    index, raw, side = _target(logits, "logits", stream)
    r = _router(E, ids.shape[1], score, renormalize, scale)
    graph = _graph("route_grad", out, dw, logits, instead="use Routing.from_logits")
    if out is None:
        result = _new(logits, (T, E), logits.dtype, side)
    else:
        result = out
        _dtype(out, "out", (logits.dtype,))
        if tuple(out.shape) != (T, E):
            raise ValueError(f"out: expected shape {(T, E)}, got {tuple(out.shape)}")
    _check(_lib.moe_route_grad(ctypes.byref(r), DT[logits.dtype], logits.data_ptr(), ld, T, _plain(ids, "ids", index),
                               _plain(dw, "dw", index), _plain(result, "out", index), _rows(result, "out", E), raw),
           "moe_route_grad")
    if out is not None:
        _written(out)
    _hold(side, dw, logits, ids, out)
    return result if graph is None else _Refusal.apply(graph, result, dw, logits)


def sort_pairs(ids, n_experts, stream=None):
    """The order of the pairs (token, rank) of ids [T, k] (int32 or int64) by expert, those of an expert in their own
    order: (perm [T k] int64 the pair t * k + j at each place, offsets [n_experts + 1] int32 where each expert's begin,
    rows [T k] int32 the token at each place, place [T k] int64 each pair's place).  Entries outside [0, n_experts)
    are of no expert and come last."""
    _dtype(ids, "ids", (torch.int32, torch.int64))
    _layout(ids, "ids")
    if ids.dim() != 2:
        raise ValueError(f"ids: expected [tokens, k], got {tuple(ids.shape)}")
    T, k = ids.shape
    index, raw, side = _target(ids, "ids", stream)
    if T * k > MAX_PAIRS or not 1 <= n_experts <= MAX_EXPERTS:
        raise ValueError(f"ids: at most {MAX_PAIRS} pairs of 1 to {MAX_EXPERTS} experts, got {T * k} of {n_experts}")
    order, work, struct = _order(T, k, n_experts, ids, side)
    _check(_lib.moe_sort_pairs(ids.data_ptr(), ids.element_size(), T, k, n_experts, ctypes.byref(struct), raw),
           "moe_sort_pairs")
    _hold(side, ids, work)
    return order


def _pairs_of(place, w):
    _layout(place, "place", torch.int64)
    if place.dim() != 2:
        raise ValueError(f"place: expected [tokens, k], got {tuple(place.shape)}")
    _layout(w, "w", torch.float32, tuple(place.shape))
    return place.shape


def combine(y, place, w=None, out=None, dtype=torch.float32, stream=None):
    """out[t] = sum over j of w[t, j] * y[place[t, j]]: a token's pairs, weighted and summed.

    y [P, n] (fp32, bf16 or fp16; rows may be strided; n a multiple of 8), place [T, k] int64 (as Routing.place; an
    entry outside [0, P) adds nothing), w [T, k] fp32 (default: ones).  Returns [T, n] in `dtype`: y's type or fp32,
    for fp32 y any of the three."""
    _dtype(y, "y", _FLOATS)
    ldy = _matrix(y, "y", y.dtype, None, y.shape[-1])
    T, k = _pairs_of(place, w)
    P, n = y.shape
    index, raw, side = _target(y, "y", stream)
    graph = _graph("combine", out, y, *(() if w is None else (w,)), instead="use Routing.combine")
    allowed = _FLOATS if y.dtype is torch.float32 else (y.dtype, torch.float32)
    result, ldo = _output(out, (T, n), dtype, allowed, y, side)
    _check(_lib.moe_combine(DT[y.dtype], _pointer(y, "y", index), ldy, P, _plain(place, "place", index),
                            None if w is None else _plain(w, "w", index), T, k, n, _pointer(result, "out", index),
                            DT[result.dtype], ldo, raw), "moe_combine")
    if out is not None:
        _written(out)
    _hold(side, y, place, w, out)
    return result if graph is None else _Refusal.apply(graph, result, y, *(() if w is None else (w,)))


def _combine_grad(dout, y, place, w, pairs, dtype, dy, dw, stream):
    """The C call (dy, dw: outputs, None where not wanted); y is looked at for dw only."""
    T, k = _pairs_of(place, w)
    ldd = _matrix(dout, "dout", dout.dtype, T, dout.shape[-1])
    n = dout.shape[1]
    index, raw, side = _target(dout, "dout", stream)
    ldy = ldg = 0
    py = pw = pdy = pdw = None
    if dw is not None:
        ldy, py = _matrix(y, "y", dtype, pairs, n), _pointer(y, "y", index)
        _layout(dw, "dw", torch.float32, (T, k))
        pdw = _plain(dw, "dw", index)
    if dy is not None:
        ldg, pdy = _matrix(dy, "dy", dtype, pairs, n), _pointer(dy, "dy", index)
    if w is not None:
        pw = _plain(w, "w", index)
    _check(_lib.moe_combine_grad(DT[dtype], _pointer(dout, "dout", index), DT[dout.dtype], ldd, py, ldy, pairs,
                                 _plain(place, "place", index), pw, T, k, n, pdy, ldg, pdw, raw), "moe_combine_grad")
    _hold(side, dout, y, place, w, dy, dw)


def combine_grad(dout, y, place, w=None, dy=None, dw=None, stream=None):
    """The gradients of combine from dout [T, n] (y's type or fp32): (dy [P, n] in y's type, dw [T, k] fp32).

    place has to name every row of y once, as Routing.place does.  With a `dy` that is given it may leave rows out:
    they keep what they held; a row that two pairs name gets one of the two."""
    _dtype(y, "y", _FLOATS)
    _dtype(dout, "dout", (y.dtype, torch.float32))
    if y.dim() != 2 or dout.dim() != 2 or dout.shape[1] != y.shape[1]:
        raise ValueError(f"y and dout: expected [pairs, n] and [tokens, n], got {tuple(y.shape)}, {tuple(dout.shape)}")
    if place.dim() != 2:
        raise ValueError(f"place: expected [tokens, k], got {tuple(place.shape)}")
    P, shape = y.shape[0], tuple(place.shape)
    operands = (dout, y) if w is None else (dout, y, w)
    graph = None
    for t in {None} if dy is None and dw is None else (dy, dw):
        graph = _graph("combine_grad", t, *operands, instead="use Routing.combine") or graph
    given = [t for t in (dy, dw) if t is not None]
    if dy is None:
        if P != shape[0] * shape[1]:
            raise ValueError(f"place: names {shape[0] * shape[1]} of {P} rows of y (pass dy to leave rows out)")
        dy = _new(y, tuple(y.shape), y.dtype, stream)
    if dw is None:
        dw = _new(y, shape, torch.float32, stream)
    _combine_grad(dout, y, place, w, P, y.dtype, dy, dw, stream)
    _written(*given)
    if graph is None:
        return dy, dw
    return tuple(_Refusal.apply(graph, t, *operands) for t in (dy, dw))


# The odd quintic published by K. Jordan (2024): small singular values grow 3.4445 a step; all end in about 0.7 .. 1.2
QUINTIC = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, steps=5, coefficients=QUINTIC, eps=1e-7, out=None, stream=None):
    """The update that an orthogonalising optimiser makes of a gradient or its momentum g [.., rows, cols] (fp32, bf16
    or fp16, dense; a bank is a batch of matrices), each matrix by itself, in g's type.

    X = g / (|g| + eps) with the Frobenius norm, then `steps` times X <- a X + (b A + c A A) X with A = X X^T: the
    singular vectors of g, the singular values near 1.  `coefficients` is (a, b, c), or one such triple for each step.
    A matrix of zeros (an expert without tokens) gives zeros, one with a NaN or an infinity NaN throughout.  Values
    between the products have 22 bits.  `out` may be g itself."""
    _dtype(g, "g", _FLOATS)
    _layout(g, "g")
    if g.dim() < 2 or g.shape[-1] < 1 or g.shape[-2] < 1:
        raise ValueError(f"g: expected [.., rows, cols], got {tuple(g.shape)}")
    rows, cols = g.shape[-2:]
    batch = g.numel() // (rows * cols)
    if not 1 <= steps <= MAX_STEPS:
        raise ValueError(f"steps: expected 1 to {MAX_STEPS}, got {steps}")
    one = not hasattr(coefficients[0], "__len__")
    each = [tuple(coefficients)] * steps if one else [tuple(c) for c in coefficients]
    if len(each) != steps or any(len(c) != 3 for c in each):
        raise ValueError(f"coefficients: expected (a, b, c) or {steps} of them, got {coefficients!r}")
    index, raw, side = _target(g, "g", stream)
    graph = _graph("orthogonalize", out, g, instead="call it without gradients")
    if out is None:
        result = _new(g, tuple(g.shape), g.dtype, side)
    else:
        _layout(out, "out", g.dtype, tuple(g.shape))
        result = out
    n = _lib.moe_orthogonalize_bytes(batch, rows, cols)
    work = _new(g, (n,), torch.uint8, side) if n else None
    flat = (ctypes.c_float * (3 * steps))(*(x for c in each for x in c))
    _check(_lib.moe_orthogonalize(DT[g.dtype], g.data_ptr(), batch, rows, cols, steps, flat, eps,
                                  _plain(result, "out", index), work.data_ptr() if n else None, n, raw),
           "moe_orthogonalize")
    if out is not None:
        _written(out)
    _hold(side, g, work, out)
    return result if graph is None else _Refusal.apply(graph, result, g)
