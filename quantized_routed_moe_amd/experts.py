"""Expert FFNs built from the expert operators: a differentiable one on 16-bit
weights (`expert_ffn`) and one on four-bit weights (`Mxfp4Experts`).

Both take the routing of a `MoELayer` (`Routing.from_layer`, of its
`forward_debug`) or any top-k choice (`Routing.from_ids`) and compute, for
each token, sum over its experts of w * down_e(silu(gate_e x) * up_e x).
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from .expert_ops import (DT, _graph, _Refusal, grouped_mm, grouped_mm_grad_a, grouped_mm_grad_b, mxfp4_grouped_mm,
                         mxfp4_quantize, swiglu, swiglu_grad, swiglu_mxfp4)
from .train_ops import MAX_EXPERTS, MAX_PAIRS, _combine_grad, _route, combine, route_grad, sort_pairs


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t as the kernels take it: contiguous, 16-byte aligned."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _Route(torch.autograd.Function):
    """The weights of a choice, differentiable in the logits."""

    @staticmethod
    def forward(ctx, logits, bias, top_k, choice, kept):
        ids, w, order = _route("moe_route", logits, top_k, bias=bias, ordered=True, stream=None, **choice)
        kept.append((ids, order))
        ctx.save_for_backward(logits, ids)
        ctx.weights = {n: choice[n] for n in ("score", "renormalize", "scale")}
        return w

    @staticmethod
    def backward(ctx, dw):
        logits, ids = ctx.saved_tensors
        with torch.no_grad():
            d = route_grad(dw.contiguous(), logits, ids, **ctx.weights)
        if torch.is_grad_enabled():
            why = "a routing's weights cannot be differentiated twice: their gradient comes from a kernel without one"
            d = _Refusal.apply(why, d, dw, logits)
        return d, None, None, None, None


class Routing:
    """(token, expert) pairs sorted by expert: `perm` [T * k] the pair t * k + j at each place, `rows` its token,
    `offsets` [E + 1] where each expert's pairs begin, `place` [T * k] each pair's place, `w` [T, k] fp32; `ids` [T, k]
    where the routing was made of a choice."""

    def __init__(self, perm: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor):
        self.perm, self.offsets, self.w = perm.long(), offsets, w
        self.k = w.shape[1]
        self.rows = (self.perm // self.k).to(torch.int32)
        self.place = torch.empty_like(self.perm)
        self.place[self.perm] = torch.arange(self.perm.numel(), device=perm.device)
        self.ids = None

    def _tensors(self) -> tuple:
        return self.perm, self.offsets, self.rows, self.place

    @classmethod
    def _of(cls, tensors: tuple, w: torch.Tensor, ids: torch.Tensor | None = None) -> "Routing":
        """Of what _tensors() gave."""
        r = cls.__new__(cls)
        r.perm, r.offsets, r.rows, r.place = tensors
        r.w, r.k, r.ids = w, w.shape[1], ids
        return r

    @classmethod
    def from_layer(cls, debug: dict) -> "Routing":
        """Of what MoELayer.forward_debug returns."""
        return cls(debug["perm"], debug["offsets"], debug["w"])

    @classmethod
    def from_ids(cls, ids: torch.Tensor, w: torch.Tensor, n_experts: int, strict: bool = False) -> "Routing":
        """Of the experts [T, k] that a router chose and their weights [T, k]; pairs whose expert is outside
        [0, n_experts) are of none.  On the GPU the order is made by sort_pairs, without synchronising, for as many
        pairs and experts as the grouped products take and up to 1024 a token (of fewer than 64 tokens as much more).

        `strict` reads the ids first, which synchronises, and raises for one outside [-1, n_experts), which no router
        gives."""
        if strict and bool(((ids.long() < -1) | (ids.long() >= n_experts)).any()):
            raise ValueError(f"ids: expected experts below {n_experts}, or -1 for none")
        # sort_pairs cuts by tokens: 64 tokens of 512 / 1024 / 4096 / 16384 pairs, one workgroup's, take 71 / 138 / 579 /
        # 2429 us, torch's sort and count 125 / 131 / 211 / 332
        few = min(w.shape[0], 64) * w.shape[1] <= 1 << 16
        if ids.is_cuda and few and ids.numel() <= MAX_PAIRS and 1 <= n_experts <= MAX_EXPERTS:
            with torch.cuda.device(ids.device):
                choice = ids if ids.dtype in (torch.int32, torch.int64) else ids.long()
                return cls._of(sort_pairs(choice.reshape(w.shape).contiguous(), n_experts), w, ids)
        flat = ids.reshape(-1).long()
        flat = torch.where((flat < 0) | (flat >= n_experts), n_experts, flat)
        offsets = torch.zeros(n_experts + 1, dtype=torch.int32, device=ids.device)
        offsets[1:] = torch.bincount(flat, minlength=n_experts + 1)[:n_experts].cumsum(0)
        r = cls(flat.sort(stable=True).indices, offsets, w)
        r.ids = ids
        return r

    @classmethod
    def from_logits(cls, logits: torch.Tensor, top_k: int, score: str = "sigmoid", bias: torch.Tensor | None = None,
                    groups: int = 1, keep_groups: int | None = None, group_best: int = 2, renormalize: bool = True,
                    scale: float = 1.0) -> "Routing":
        """Of a router's logits [T, E] on the GPU, as `route` chooses and weights; `w` is differentiable in the logits
        (once; not in the bias, which takes no part in the weights)."""
        kept: list = []
        choice = dict(score=score, groups=groups, keep_groups=keep_groups, group_best=group_best,
                      renormalize=renormalize, scale=scale)
        if torch.is_grad_enabled() and logits.requires_grad:
            w = _Route.apply(logits, bias, top_k, choice, kept)
            (ids, order), = kept
        else:
            _graph("Routing.from_logits", None, logits)
            ids, w, order = _route("moe_route", logits, top_k, bias=bias, ordered=True, stream=None, **choice)
        return cls._of(order, w, ids)

    def to_pairs(self, x: torch.Tensor) -> torch.Tensor:
        """[T, n] -> [T * k, n]: each pair's token's row."""
        return x[self.rows.long()]

    def to_tokens(self, y: torch.Tensor) -> torch.Tensor:
        """[T * k, n] -> [T, k, n]: each token's pairs."""
        return y[self.place].view(-1, self.k, y.shape[1])

    def _by_kernel(self, *tensors) -> bool:
        """Whether combine's kernels take these operands (else torch's operations do, in whatever types)."""
        return all(t.is_cuda for t in tensors) and self.w.dtype is torch.float32 and self.place.numel() > 0

    def _places(self) -> torch.Tensor:
        return self.place.long().view(-1, self.k)

    def combine(self, y: torch.Tensor) -> torch.Tensor:
        """out [T, n] of the pairs' results y [T * k, n]: sum over a token's pairs of w * y.  Differentiable in w and
        y, by torch's operations; the kernel runs where no gradient is asked for."""
        if y.dim() != 2 or y.shape[0] != self.place.numel():
            raise ValueError(f"y: expected a row for each of {self.place.numel()} pairs, got {tuple(y.shape)}")
        graph = torch.is_grad_enabled() and (y.requires_grad or self.w.requires_grad)
        if graph or forward_ad._current_level >= 0 or not self._by_kernel(y, self.w) or y.shape[1] % 8 != 0 or (
                y.dtype not in DT):
            return (self.to_tokens(y).float() * self.w[:, :, None]).sum(1)
        return combine(_dense(y), self._places(), self.w.contiguous())


class _ExpertFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, gate_up, down, routing):
        gu = grouped_mm(x, gate_up, routing.offsets, rows=routing.rows)
        h = swiglu(gu)
        y = grouped_mm(h, down, routing.offsets)
        need_x, need_w, need_gate_up, need_down, _ = ctx.needs_input_grad
        ctx.save_for_backward(x, w, gate_up, down, gu if need_x or need_gate_up else None, h if need_down else None,
                              y if need_w else None, *routing._tensors())
        return routing.combine(y)

    @staticmethod
    def backward(ctx, dout):
        with torch.no_grad():
            grads = _ExpertFFN.gradients(ctx, dout)
        if not torch.is_grad_enabled():
            return (*grads, None)
        # create_graph: the kernels leave no graph, so a derivative of these would be wrong, not merely missing
        why = "expert_ffn cannot be differentiated twice: its gradients come from kernels without a derivative"
        sources = (dout, *ctx.saved_tensors[:4])
        return (*(g if g is None else _Refusal.apply(why, g, *sources) for g in grads), None)

    @staticmethod
    def gradients(ctx, dout):
        """Of x, w, gate_up and down; None, and nothing computed, for one that is not asked for."""
        x, w, gate_up, down, gu, h, y, *routing = ctx.saved_tensors
        need_x, need_w, need_gate_up, need_down, _ = ctx.needs_input_grad
        r = Routing._of(routing, w)
        dx = dw = d_gate_up = d_down = None
        need_y = need_x or need_gate_up or need_down
        kernel = r._by_kernel(dout, w)
        if kernel:
            dy = dout.new_empty((r.rows.numel(), dout.shape[1]), dtype=down.dtype) if need_y else None
            dw = w.new_empty(w.shape) if need_w else None
            _combine_grad(_dense(dout), y, r._places(), w.contiguous(), r.rows.numel(), down.dtype, dy, dw, None)
        else:
            if need_w:
                dw = (r.to_tokens(y).float() * dout[:, None]).sum(2)
            if need_y:
                dy = (r.to_pairs(dout) * w.reshape(-1)[r.perm][:, None]).to(down.dtype)
        if need_down:
            d_down = grouped_mm_grad_b(dy, h, r.offsets)
        if need_x or need_gate_up:
            dgu = swiglu_grad(grouped_mm_grad_a(dy, down, r.offsets), gu)
        if need_gate_up:
            d_gate_up = grouped_mm_grad_b(dgu, x, r.offsets, rows=r.rows)
        if need_x:
            # a token's gradient is the sum of its pairs', in fp32
            dx = grouped_mm_grad_a(dgu, gate_up, r.offsets, dtype=torch.float32)
            dx = combine(dx, r._places(), dtype=x.dtype) if kernel else r.to_tokens(dx).sum(1).to(x.dtype)
        return dx, dw, d_gate_up, d_down


def expert_ffn(x: torch.Tensor, routing: Routing, gate_up: torch.Tensor, down: torch.Tensor) -> torch.Tensor:
    """out [T, H] fp32 of x [T, H] (bf16 or fp16); gate_up [E, 2 F, H] with the gate rows first, down [E, H, F].
    Differentiable in x, routing.w, gate_up and down; a derivative of those gradients raises RuntimeError."""
    return _ExpertFFN.apply(x, routing.w, gate_up, down, routing)


class Mxfp4Experts:
    """The same FFN on four-bit weights, quantised once from 16- or 32-bit banks; activations are quantised on the
    way, x once for all its experts and the hidden activation as it is made.  Differentiable in routing.w only."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor):
        self.gate_up, self.down = mxfp4_quantize(gate_up), mxfp4_quantize(down)

    def forward(self, x: torch.Tensor, routing: Routing) -> torch.Tensor:
        """out [T, H] fp32 of x [T, H] (fp32, bf16 or fp16)."""
        graph = _graph("Mxfp4Experts", None, x)
        # The product is stored in bf16: half the traffic of fp32, and its rounding (2^-9) is lost beside the
        # activation's to four bits that follows.  256 experts top-6, 4096 -> 2048, normal weights and inputs, against
        # 64 bits on the unrounded weights: off by 0.2979 either way at 2048 tokens, 994 us against 1016.
        gu = mxfp4_grouped_mm(*mxfp4_quantize(x), *self.gate_up, routing.offsets, rows=routing.rows)
        y = mxfp4_grouped_mm(*swiglu_mxfp4(gu), *self.down, routing.offsets)
        if graph is not None:
            y = _Refusal.apply(graph, y, x)
        return routing.combine(y)

    __call__ = forward
