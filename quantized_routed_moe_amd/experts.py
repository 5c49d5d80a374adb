"""Expert FFNs built from the expert operators: a differentiable one on 16-bit
weights (`expert_ffn`) and one on four-bit weights (`Mxfp4Experts`).

Both take the routing of a `MoELayer` (`Routing.from_layer`, of its
`forward_debug`) or any top-k choice (`Routing.from_ids`) and compute, for
each token, sum over its experts of w * down_e(silu(gate_e x) * up_e x).
"""
from __future__ import annotations

import torch

from .expert_ops import (_graph, _Refusal, grouped_mm, grouped_mm_grad_a, grouped_mm_grad_b, mxfp4_grouped_mm,
                         mxfp4_quantize, swiglu, swiglu_grad, swiglu_mxfp4)


class Routing:
    """(token, expert) pairs sorted by expert: `perm` [T * k] the pair t * k + j at each place, `rows` its token,
    `offsets` [E + 1] where each expert's pairs begin, `place` [T * k] each pair's place, `w` [T, k] fp32."""

    def __init__(self, perm: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor):
        self.perm, self.offsets, self.w = perm.long(), offsets, w
        self.k = w.shape[1]
        self.rows = (self.perm // self.k).to(torch.int32)
        self.place = torch.empty_like(self.perm)
        self.place[self.perm] = torch.arange(self.perm.numel(), device=perm.device)

    def _tensors(self) -> tuple:
        return self.perm, self.offsets, self.rows, self.place

    @classmethod
    def _of(cls, tensors: tuple, w: torch.Tensor) -> "Routing":
        """Of what _tensors() gave."""
        r = cls.__new__(cls)
        r.perm, r.offsets, r.rows, r.place = tensors
        r.w, r.k = w, w.shape[1]
        return r

    @classmethod
    def from_layer(cls, debug: dict) -> "Routing":
        """Of what MoELayer.forward_debug returns."""
        return cls(debug["perm"], debug["offsets"], debug["w"])

    @classmethod
    def from_ids(cls, ids: torch.Tensor, w: torch.Tensor, n_experts: int) -> "Routing":
        """Of the experts [T, k] that a router chose and their weights [T, k]."""
        flat = ids.reshape(-1).long()
        offsets = torch.zeros(n_experts + 1, dtype=torch.int32, device=ids.device)
        offsets[1:] = torch.bincount(flat, minlength=n_experts).cumsum(0)
        return cls(flat.sort(stable=True).indices, offsets, w)

    def to_pairs(self, x: torch.Tensor) -> torch.Tensor:
        """[T, n] -> [T * k, n]: each pair's token's row."""
        return x[self.rows.long()]

    def to_tokens(self, y: torch.Tensor) -> torch.Tensor:
        """[T * k, n] -> [T, k, n]: each token's pairs."""
        return y[self.place].view(-1, self.k, y.shape[1])


class _ExpertFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, gate_up, down, routing):
        gu = grouped_mm(x, gate_up, routing.offsets, rows=routing.rows)
        h = swiglu(gu)
        y = grouped_mm(h, down, routing.offsets)
        need_x, need_w, need_gate_up, need_down, _ = ctx.needs_input_grad
        ctx.save_for_backward(x, w, gate_up, down, gu if need_x or need_gate_up else None, h if need_down else None,
                              y if need_w else None, *routing._tensors())
        return (routing.to_tokens(y).float() * w[:, :, None]).sum(1)

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
        if need_w:
            dw = (r.to_tokens(y).float() * dout[:, None]).sum(2)
        if need_x or need_gate_up or need_down:
            dy = (r.to_pairs(dout) * w.reshape(-1)[r.perm][:, None]).to(down.dtype)
        if need_down:
            d_down = grouped_mm_grad_b(dy, h, r.offsets)
        if need_x or need_gate_up:
            dgu = swiglu_grad(grouped_mm_grad_a(dy, down, r.offsets), gu)
        if need_gate_up:
            d_gate_up = grouped_mm_grad_b(dgu, x, r.offsets, rows=r.rows)
        if need_x:
            # a token's gradient is the sum of its pairs', in fp32
            dx = r.to_tokens(grouped_mm_grad_a(dgu, gate_up, r.offsets, dtype=torch.float32)).sum(1).to(x.dtype)
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
        return (routing.to_tokens(y).float() * routing.w[:, :, None]).sum(1)

    __call__ = forward
