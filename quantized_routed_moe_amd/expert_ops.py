"""Expert operators on 16-bit and four-bit weights: products grouped by expert
with their gradients, the microscaled four-bit format with its product, SwiGLU
with its gradient.

Argument checks and marshalling only; the operators are HIP kernels behind the
C ABI of include/moe.h.  Rows are (token, expert) pairs sorted by expert:
expert e owns rows offsets[e] .. offsets[e+1] - 1 (any number), `offsets` and
`rows` being int32 tensors on the GPU.  Work is enqueued on `stream` (the
current stream by default) without synchronising; a result that is not passed
in as `out` is allocated for that stream.  On a `stream` other than the one
that an operand was made on, the caller has that stream wait for it; the
operands' memory is not given to anyone else before the call has run.

The calls build no graph: expert_ffn is the differentiable one.  With an
operand that asks for a gradient the result can be used, but differentiating
through it raises (at once where it is written to `out` or the operand carries
a forward-mode tangent); codes and scales are integers, which torch does not
differentiate.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from . import Grouped, _check, _layout, _lib

DT = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
_HALF = (torch.bfloat16, torch.float16)


class _Refusal(torch.autograd.Function):
    """Passes a result on; differentiating through it raises.  `why` says what was asked for in vain."""

    @staticmethod
    def forward(ctx, why, out, *operands):
        ctx.why = why
        ctx.mark_dirty(out)
        return out

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(ctx.why)


def _graph(call, out, *operands):
    """None; where an operand asks for a gradient, why the result's derivative will be refused.  Raises where it could
    not be: the result is written to the caller's `out`, or an operand carries a forward-mode tangent."""
    if torch.is_grad_enabled():
        if out is not None and out.requires_grad:
            raise RuntimeError(f"{call} cannot write to an out that asks for a gradient")
        for t in operands:
            if t.requires_grad:
                why = f"{call} builds no graph, but an operand asks for a gradient (detach it, or use expert_ffn)"
                if out is not None:
                    raise RuntimeError(why)
                return why
    if forward_ad._current_level >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in operands):
        raise RuntimeError(f"{call} has no forward-mode derivative, but an operand carries a tangent")
    return None


def _dtype(t, name, allowed):
    if t.dtype not in allowed:
        raise ValueError(f"{name}: expected one of {', '.join(map(str, allowed))}, got {t.dtype}")


def _matrix(t, name, dtype, rows, cols):
    """Shape, type and layout of a 2-d operand whose rows may be strided; returns its row stride."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: expected shape ({'rows' if rows is None else rows}, {cols}), got {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.is_contiguous():
        stride = cols
        if shape[0] < 2:  # nothing lies behind a single row: any stride will do
            step = 16 // t.element_size()
            return (cols + step - 1) // step * step
    else:
        stride, inner = t.stride()
        if cols > 1 and inner != 1:
            raise ValueError(f"{name}: elements of a row must be consecutive")
    if stride < cols or stride * t.element_size() % 16:
        raise ValueError(f"{name}: row stride {stride} must cover a row and be a multiple of 16 bytes")
    return stride


def _pointer(t, name, index):
    """Device pointer of t on GPU `index`, 16-byte aligned."""
    if not t.is_cuda:
        raise ValueError(f"{name}: must be in GPU memory")
    p = t.data_ptr()
    if t.get_device() != index:
        raise ValueError(f"{name}: is on GPU {t.get_device()}, the call is on GPU {index}")
    if p & 15:
        raise ValueError(f"{name}: must start 16-byte aligned")
    return p


def _plain(t, name, index):
    """_pointer without the alignment."""
    if not t.is_cuda:
        raise ValueError(f"{name}: must be in GPU memory")
    if t.get_device() != index:
        raise ValueError(f"{name}: is on GPU {t.get_device()}, the call is on GPU {index}")
    return t.data_ptr()


def _target(first, name, stream):
    """(GPU, raw stream, stream to allocate for or None) of a call whose first operand is given."""
    if not first.is_cuda:
        raise ValueError(f"{name}: must be in GPU memory")
    index = first.get_device()
    if index != torch.cuda.current_device():
        raise ValueError(f"{name}: is on GPU {index}, the current GPU is {torch.cuda.current_device()}")
    if stream is None:
        # the handle alone: building a Stream object costs more than the rest of a small call
        return index, torch._C._cuda_getCurrentRawStream(index), None
    return index, stream.cuda_stream, stream


def _new(like, shape, dtype, stream):
    """A new tensor on like's GPU whose memory belongs to `stream` (None: the current one)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _hold(stream, *tensors):
    """Keeps the memory of a call's tensors from being reused, once they are dropped, before `stream` has run it."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _written(*outputs):
    """Tells autograd that the caller's tensors have been written to, as torch's own calls do: a graph that saved one
    refuses to use it."""
    for t in outputs:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _output(out, shape, dtype, allowed, like, stream):
    """(out, its row stride): a given output checked, or a new one."""
    if out is None:
        if dtype not in allowed:
            raise ValueError(f"out: expected one of {', '.join(map(str, allowed))}, got {dtype}")
        return _new(like, shape, dtype, stream), shape[-1]
    if out.dtype not in allowed:
        raise ValueError(f"out: expected one of {', '.join(map(str, allowed))}, got {out.dtype}")
    if len(shape) == 2:
        return out, _matrix(out, "out", out.dtype, *shape)
    _layout(out, "out", out.dtype, shape)
    return out, shape[-1]


def _groups(offsets, rows, src, n_experts, pairs, n, k, index):
    _layout(offsets, "offsets", torch.int32, (n_experts + 1,))
    at = _plain(offsets, "offsets", index)
    if rows is None:
        return Grouped(n_experts, n, k, pairs, at, None, 0)
    _layout(rows, "rows", torch.int32, (pairs,))
    # an empty tensor has no pointer; with no pairs nothing is read
    return Grouped(n_experts, n, k, pairs, at, _plain(rows, "rows", index) or at, src)


def _bank(b, name, dtype):
    if b.dim() != 3:
        raise ValueError(f"{name}: expected [experts, out, in], got {tuple(b.shape)}")
    _layout(b, name, dtype)
    return b.shape


def grouped_mm(a, b, offsets, rows=None, out=None, dtype=None, stream=None):
    """c[p] = a[rows[p]] @ b[e(p)].T for the pairs p of every expert e.

    a [R, K] bf16 or fp16 (rows may be strided), b [E, N, K] of the same type;
    rows [P] int32 names the row of a that each pair reads (default: P = R,
    pair p reads row p; an entry outside [0, R) reads zeros).  Returns c [P, N]
    in `dtype` (a's type or fp32).  Rows of no group come out as zeros."""
    _dtype(a, "a", _HALF)
    E, N, K = _bank(b, "b", a.dtype)
    lda = _matrix(a, "a", a.dtype, None, K)
    index, raw, side = _target(a, "a", stream)
    P = a.shape[0] if rows is None else rows.shape[0]
    g = _groups(offsets, rows, a.shape[0], E, P, N, K, index)
    graph = _graph("grouped_mm", out, a, b)
    result, ldc = _output(out, (P, N), dtype or a.dtype, (a.dtype, torch.float32), a, side)
    _check(_lib.moe_grouped_mm(ctypes.byref(g), DT[a.dtype], _pointer(a, "a", index), lda, _pointer(b, "b", index),
                               _pointer(result, "out", index), DT[result.dtype], ldc, raw), "moe_grouped_mm")
    if out is not None:
        _written(out)
    _hold(side, a, b, offsets, rows, out)
    return result if graph is None else _Refusal.apply(graph, result, a, b)


def grouped_mm_grad_a(dc, b, offsets, out=None, dtype=None, stream=None):
    """The gradient of grouped_mm with respect to each pair's row of a: da[p] = dc[p] @ b[e(p)].

    dc [P, N], b [E, N, K]; returns da [P, K] in `dtype` (dc's type or fp32).  Where pairs share a row of a,
    that row's gradient is the sum of theirs."""
    _dtype(dc, "dc", _HALF)
    E, N, K = _bank(b, "b", dc.dtype)
    ldd = _matrix(dc, "dc", dc.dtype, None, N)
    index, raw, side = _target(dc, "dc", stream)
    P = dc.shape[0]
    g = _groups(offsets, None, 0, E, P, N, K, index)
    graph = _graph("grouped_mm_grad_a", out, dc, b)
    result, lda = _output(out, (P, K), dtype or dc.dtype, (dc.dtype, torch.float32), dc, side)
    _check(_lib.moe_grouped_mm_grad_a(ctypes.byref(g), DT[dc.dtype], _pointer(dc, "dc", index), ldd,
                                      _pointer(b, "b", index), _pointer(result, "out", index), DT[result.dtype], lda,
                                      raw), "moe_grouped_mm_grad_a")
    if out is not None:
        _written(out)
    _hold(side, dc, b, offsets, out)
    return result if graph is None else _Refusal.apply(graph, result, dc, b)


def grouped_mm_grad_b(dc, a, offsets, rows=None, out=None, dtype=None, stream=None):
    """The gradient of grouped_mm with respect to b: db[e] = sum over e's pairs of dc[p].T @ a[rows[p]].

    dc [P, N], a [R, K] of the same type; returns db [E, N, K] in `dtype` (dc's type or fp32), zeros for an
    expert without pairs."""
    _dtype(dc, "dc", _HALF)
    ldd = _matrix(dc, "dc", dc.dtype, None, dc.shape[-1])
    P, N = dc.shape
    lda = _matrix(a, "a", dc.dtype, None if rows is not None else P, a.shape[-1])
    K = a.shape[1]
    index, raw, side = _target(dc, "dc", stream)
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets: expected [experts + 1], got {tuple(offsets.shape)}")
    E = offsets.shape[0] - 1
    g = _groups(offsets, rows, a.shape[0], E, P, N, K, index)
    graph = _graph("grouped_mm_grad_b", out, dc, a)
    result, _ = _output(out, (E, N, K), dtype or dc.dtype, (dc.dtype, torch.float32), dc, side)
    _check(_lib.moe_grouped_mm_grad_b(ctypes.byref(g), DT[dc.dtype], _pointer(dc, "dc", index), ldd,
                                      _pointer(a, "a", index), lda, _pointer(result, "out", index), DT[result.dtype],
                                      raw), "moe_grouped_mm_grad_b")
    if out is not None:
        _written(out)
    _hold(side, dc, a, offsets, rows, out)
    return result if graph is None else _Refusal.apply(graph, result, dc, a)


def _code_outputs(shape, codes, scales, like, stream):
    c, s = (*shape[:-1], shape[-1] // 2), (*shape[:-1], shape[-1] // 32)
    if codes is None:
        codes = _new(like, c, torch.uint8, stream)
    else:
        _layout(codes, "codes", torch.uint8, c)
    if scales is None:
        scales = _new(like, s, torch.uint8, stream)
    else:
        _layout(scales, "scales", torch.uint8, s)
    return codes, scales


def _rows_of(x, name):
    """x as (rows, cols, row stride): two dimensions with strided rows, or any number of them dense."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name}: expected rows of at least one element, got {tuple(x.shape)}")
    cols = x.shape[-1]
    if x.dim() == 2:
        return x.shape[0], cols, _matrix(x, name, x.dtype, None, cols)
    _layout(x, name)
    return x.numel() // cols, cols, cols


def mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """x [.., n] (fp32, bf16 or fp16; n a multiple of 32) as (codes [.., n/2], scales [.., n/32]), both uint8.

    The format is described in include/moe.h (moe_mxfp4_quantize)."""
    _dtype(x, "x", tuple(DT))
    rows, cols, ld = _rows_of(x, "x")
    if cols % 32:
        raise ValueError(f"x: rows of {cols} elements are not made of blocks of 32")
    index, raw, side = _target(x, "x", stream)
    given = codes, scales
    codes, scales = _code_outputs(x.shape, codes, scales, x, side)
    _check(_lib.moe_mxfp4_quantize(DT[x.dtype], _pointer(x, "x", index), ld, rows, cols,
                                   _pointer(codes, "codes", index), _plain(scales, "scales", index), raw),
           "moe_mxfp4_quantize")
    _written(*given)
    _hold(side, x, codes, scales)
    return codes, scales


def _format(codes, scales, c_name, s_name):
    _layout(codes, c_name, torch.uint8)
    if codes.dim() < 1 or codes.shape[-1] % 16 or codes.shape[-1] < 16:
        raise ValueError(f"{c_name}: expected rows of a multiple of 16 bytes, got {tuple(codes.shape)}")
    _layout(scales, s_name, torch.uint8, (*codes.shape[:-1], codes.shape[-1] // 16))
    return codes.shape[-1] * 2


def mxfp4_dequantize(codes, scales, out=None, dtype=torch.float32, stream=None):
    """The values that codes [.., n/2] and scales [.., n/32] stand for, [.., n] in `dtype`."""
    cols = _format(codes, scales, "codes", "scales")
    shape = (*codes.shape[:-1], cols)
    index, raw, side = _target(codes, "codes", stream)
    _graph("mxfp4_dequantize", out)
    result, ld = _output(out, shape, dtype, tuple(DT), codes, side)
    _check(_lib.moe_mxfp4_dequantize(_pointer(codes, "codes", index), _plain(scales, "scales", index),
                                     codes.numel() * 2 // cols, cols, DT[result.dtype], _pointer(result, "out", index),
                                     ld, raw), "moe_mxfp4_dequantize")
    if out is not None:
        _written(out)
    _hold(side, codes, scales, out)
    return result


def mxfp4_grouped_mm(a_codes, a_scales, b_codes, b_scales, offsets, rows=None, out=None, dtype=torch.bfloat16,
                     stream=None):
    """grouped_mm with both operands in the four-bit format (a [R, K], b [E, N, K]); returns c [P, N] in `dtype`
    (bf16 or fp32)."""
    K = _format(a_codes, a_scales, "a_codes", "a_scales")
    if a_codes.dim() != 2:
        raise ValueError(f"a_codes: expected two dimensions, got {tuple(a_codes.shape)}")
    E, N, half = _bank(b_codes, "b_codes", torch.uint8)
    if _format(b_codes, b_scales, "b_codes", "b_scales") != K:
        raise ValueError(f"b_codes: rows of {2 * half} elements, a has {K}")
    index, raw, side = _target(a_codes, "a_codes", stream)
    R = a_codes.shape[0]
    P = R if rows is None else rows.shape[0]
    g = _groups(offsets, rows, R, E, P, N, K, index)
    _graph("mxfp4_grouped_mm", out)
    result, ldc = _output(out, (P, N), dtype, (torch.bfloat16, torch.float32), a_codes, side)
    _check(_lib.moe_mxfp4_grouped_mm(ctypes.byref(g), _pointer(a_codes, "a_codes", index),
                                     _plain(a_scales, "a_scales", index), _pointer(b_codes, "b_codes", index),
                                     _plain(b_scales, "b_scales", index), _pointer(result, "out", index),
                                     DT[result.dtype], ldc, raw), "moe_mxfp4_grouped_mm")
    if out is not None:
        _written(out)
    _hold(side, a_codes, a_scales, b_codes, b_scales, offsets, rows, out)
    return result


def _gate_up(gu):
    _dtype(gu, "gu", tuple(DT))
    if gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError(f"gu: expected [rows, 2 * ffn], got {tuple(gu.shape)}")
    return gu.shape[0], gu.shape[1] // 2, _matrix(gu, "gu", gu.dtype, None, gu.shape[1])


def swiglu(gu, out=None, stream=None):
    """h = silu(gate) * up of gu [rows, 2 F] = [gate | up] (fp32, bf16 or fp16), [rows, F] of the same type."""
    rows, ffn, ldg = _gate_up(gu)
    index, raw, side = _target(gu, "gu", stream)
    graph = _graph("swiglu", out, gu)
    result, ldh = _output(out, (rows, ffn), gu.dtype, (gu.dtype,), gu, side)
    _check(_lib.moe_swiglu(DT[gu.dtype], _pointer(gu, "gu", index), ldg, rows, ffn, _pointer(result, "out", index), ldh,
                           raw), "moe_swiglu")
    if out is not None:
        _written(out)
    _hold(side, gu, out)
    return result if graph is None else _Refusal.apply(graph, result, gu)


def swiglu_mxfp4(gu, codes=None, scales=None, stream=None):
    """swiglu with its result in the four-bit format: (codes [rows, F/2], scales [rows, F/32])."""
    rows, ffn, ldg = _gate_up(gu)
    if ffn % 32:
        raise ValueError(f"gu: rows of {ffn} outputs are not made of blocks of 32")
    index, raw, side = _target(gu, "gu", stream)
    given = codes, scales
    codes, scales = _code_outputs((rows, ffn), codes, scales, gu, side)
    _check(_lib.moe_swiglu_mxfp4(DT[gu.dtype], _pointer(gu, "gu", index), ldg, rows, ffn,
                                 _pointer(codes, "codes", index), _plain(scales, "scales", index), raw), "moe_swiglu_mxfp4")
    _written(*given)
    _hold(side, gu, codes, scales)
    return codes, scales


def swiglu_grad(dh, gu, out=None, stream=None):
    """The gradient of swiglu: dgu [rows, 2 F] = [dgate | dup] from dh [rows, F] and the gu of the forward call."""
    rows, ffn, ldg = _gate_up(gu)
    ldd = _matrix(dh, "dh", gu.dtype, rows, ffn)
    index, raw, side = _target(gu, "gu", stream)
    graph = _graph("swiglu_grad", out, dh, gu)
    result, ldo = _output(out, (rows, 2 * ffn), gu.dtype, (gu.dtype,), gu, side)
    _check(_lib.moe_swiglu_grad(DT[gu.dtype], _pointer(dh, "dh", index), ldd, _pointer(gu, "gu", index), ldg, rows,
                                ffn, _pointer(result, "out", index), ldo, raw), "moe_swiglu_grad")
    if out is not None:
        _written(out)
    _hold(side, dh, gu, out)
    return result if graph is None else _Refusal.apply(graph, result, dh, gu)
