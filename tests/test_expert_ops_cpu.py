"""Refusals of the expert operators, on the host: the C calls reject bad
arguments before anything is enqueued, the binding rejects tensors the C ABI
cannot judge.  No GPU is needed: every call here ends in its checks."""
import ctypes

import pytest
import torch

import quantized_routed_moe_amd as qr

L = qr._lib
OK, INVALID, UNSUPPORTED, TOO_MANY = 0, -1, -2, -3
FAKE = 1 << 30  # 16-byte aligned host integers: never dereferenced
A, B, C, OFF, ROWS = FAKE, FAKE * 2, FAKE * 40, FAKE * 60, FAKE * 61
BF16, FP16, FP32 = 2, 3, 1


def grp(**kw):
    base = dict(n_experts=8, out_features=64, in_features=128, pairs=100, offsets=OFF, rows=None, src_rows=0)
    base.update(kw)
    return qr.Grouped(*(base[f] for f, _ in qr.Grouped._fields_))


def mm(g=None, dtype=BF16, a=A, lda=None, b=B, c=C, cdt=BF16, ldc=None, **kw):
    g = grp(**kw) if g is None else g
    return L.moe_grouped_mm(ctypes.byref(g), dtype, a, lda or g.in_features, b, c, cdt, ldc or g.out_features, None)


def grad_a(dtype=BF16, dc=A, ldd=None, b=B, da=C, dt=BF16, lda=None, **kw):
    g = grp(**kw)
    return L.moe_grouped_mm_grad_a(ctypes.byref(g), dtype, dc, ldd or g.out_features, b, da, dt, lda or g.in_features,
                                   None)


def grad_b(dtype=BF16, dc=A, ldd=None, a=B, lda=None, db=C, dt=BF16, **kw):
    g = grp(**kw)
    return L.moe_grouped_mm_grad_b(ctypes.byref(g), dtype, dc, ldd or g.out_features, a, lda or g.in_features, db, dt,
                                   None)


def mm4(a=A, sa=FAKE * 30, b=B, sb=FAKE * 31, c=C, cdt=BF16, ldc=None, **kw):
    g = grp(**kw)
    return L.moe_mxfp4_grouped_mm(ctypes.byref(g), a, sa, b, sb, c, cdt, ldc or g.out_features, None)


@pytest.mark.parametrize("call", [mm, grad_a, grad_b, mm4])
def test_group_refusals(call):
    for bad in (dict(n_experts=0), dict(n_experts=-3), dict(pairs=-1), dict(out_features=0), dict(in_features=0),
                dict(offsets=None), dict(offsets=OFF + 2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(n_experts=1025), dict(out_features=65544), dict(in_features=65568), dict(out_features=60),
                dict(in_features=132)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(pairs=(1 << 20) + 1) == TOO_MANY
    for bad in (dict(rows=ROWS + 1, src_rows=10), dict(rows=ROWS, src_rows=-1)):
        assert call(**bad) == INVALID, bad


def test_grouped_null_struct():
    assert L.moe_grouped_mm(None, BF16, A, 128, B, C, BF16, 64, None) == INVALID
    assert L.moe_grouped_mm_grad_a(None, BF16, A, 64, B, C, BF16, 128, None) == INVALID
    assert L.moe_grouped_mm_grad_b(None, BF16, A, 64, B, 128, C, BF16, None) == INVALID
    assert L.moe_mxfp4_grouped_mm(None, A, A, B, B, C, BF16, 64, None) == INVALID


@pytest.mark.parametrize("call,names", [(mm, ("a", "b", "c")), (grad_a, ("dc", "b", "da")), (grad_b, ("dc", "a", "db"))])
def test_grouped_operand_refusals(call, names):
    for n in names:
        assert call(**{n: None}) == INVALID, n            # missing
        assert call(**{n: FAKE * 20 + 8}) == INVALID, n   # misaligned
    out_dt = "cdt" if call is mm else "dt"
    for bad in (dict(dtype=FP32), dict(dtype=0), dict(dtype=7), {out_dt: FP16}, {out_dt: 0},
                {"dtype": FP16, out_dt: BF16}):
        assert call(**bad) == INVALID, bad
    assert call(**{names[2]: A + 16}) == INVALID          # output overlaps an input
    assert call(**{names[2]: B}) == INVALID


def test_strides():
    assert mm(lda=120) == INVALID and mm(lda=132) == INVALID and mm(ldc=60) == INVALID
    assert mm(lda=(1 << 21) + 8) == UNSUPPORTED and mm(ldc=(1 << 21) + 8) == UNSUPPORTED
    assert grad_a(ldd=56) == INVALID and grad_a(lda=124) == INVALID
    assert grad_b(ldd=56) == INVALID and grad_b(lda=124) == INVALID
    assert mm4(ldc=60) == INVALID


def test_gathered_source_past_its_limit():
    # 2^31 bytes and more cannot be addressed by a gather; without one they can
    assert mm(rows=ROWS, src_rows=1 << 23, c=1 << 45) == UNSUPPORTED
    assert grad_b(rows=ROWS, src_rows=1 << 23, a=1 << 44, db=1 << 45) == UNSUPPORTED
    assert mm4(rows=ROWS, src_rows=1 << 25, c=1 << 45) == UNSUPPORTED


def test_mxfp4_product_refusals():
    for bad in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(a=A + 8),
                dict(b=B + 4), dict(c=C + 2), dict(cdt=FP16), dict(cdt=9), dict(c=A), dict(c=FAKE * 31)):
        assert mm4(**bad) == INVALID, bad
    assert mm4(in_features=136) == UNSUPPORTED


def test_nothing_to_do():
    assert mm(pairs=0, a=None, c=None) == OK
    assert grad_a(pairs=0, dc=None, da=None) == OK
    assert mm4(pairs=0, a=None, sa=None, c=None) == OK
    assert L.moe_mxfp4_quantize(FP32, None, 64, 0, 64, None, None, None) == OK
    assert L.moe_mxfp4_dequantize(None, None, 0, 64, FP32, None, 64, None) == OK
    assert L.moe_swiglu(BF16, None, 64, 0, 32, None, 32, None) == OK
    assert L.moe_swiglu_mxfp4(BF16, None, 64, 0, 32, None, None, None) == OK
    assert L.moe_swiglu_grad(BF16, None, 32, None, 64, 0, 32, None, 64, None) == OK


def test_quantize_and_swiglu_refusals():
    def q(dt=FP32, x=A, ld=64, rows=4, cols=64, codes=B, scales=C):
        return L.moe_mxfp4_quantize(dt, x, ld, rows, cols, codes, scales, None)

    def dq(dt=FP32, x=A, ld=64, rows=4, cols=64, codes=B, scales=C):
        return L.moe_mxfp4_dequantize(codes, scales, rows, cols, dt, x, ld, None)

    for f in (q, dq):
        for bad in (dict(dt=0), dict(rows=-1), dict(cols=0), dict(x=None), dict(codes=None), dict(scales=None),
                    dict(x=A + 4), dict(codes=B + 8), dict(ld=62), dict(ld=66), dict(codes=A), dict(scales=A + 1)):
            assert f(**bad) == INVALID, bad
        for bad in (dict(cols=48), dict(cols=(1 << 21) + 32, ld=(1 << 21) + 32), dict(ld=(1 << 21) + 4)):
            assert f(**bad) == UNSUPPORTED, bad

    def sw(dt=BF16, gu=A, ldg=128, rows=4, ffn=64, h=B, ldh=64):
        return L.moe_swiglu(dt, gu, ldg, rows, ffn, h, ldh, None)

    def sg(dt=BF16, dh=C, ldd=64, gu=A, ldg=128, rows=4, ffn=64, h=B, ldh=128):
        return L.moe_swiglu_grad(dt, dh, ldd, gu, ldg, rows, ffn, h, ldh, None)

    for f in (sw, sg):
        for bad in (dict(dt=5), dict(rows=-2), dict(ffn=0), dict(gu=None), dict(h=None), dict(gu=A + 2), dict(ldg=126),
                    dict(ldg=132), dict(ldh=56), dict(h=A + 16)):
            assert f(**bad) == INVALID, bad
        assert f(ffn=60) == UNSUPPORTED
    assert sg(dh=None) == INVALID and sg(dh=B) == INVALID
    assert L.moe_swiglu_mxfp4(BF16, A, 96, 4, 48, B, C, None) == UNSUPPORTED
    assert L.moe_swiglu_mxfp4(BF16, A, 128, 4, 64, B, None, None) == INVALID
    assert L.moe_swiglu_mxfp4(BF16, A, 128, 4, 64, A + 32, C, None) == INVALID


def test_binding_checks_tensors():
    """Each bad tensor raises ValueError before the library is called (these are on the CPU, the last thing a good
    call is refused for)."""
    bf = torch.bfloat16
    a, b, o = torch.zeros(6, 16, dtype=bf), torch.zeros(3, 24, 16, dtype=bf), torch.zeros(4, dtype=torch.int32)
    dc, r = torch.zeros(6, 24, dtype=bf), torch.zeros(6, dtype=torch.int32)

    def refused(msg, f, *args, **kw):
        with pytest.raises(ValueError, match=msg):
            f(*args, **kw)

    refused("a: expected one of", qr.grouped_mm, a.float(), b, o)
    refused("b: expected torch.bfloat16", qr.grouped_mm, a, b.half(), o)
    refused("b: expected \\[experts", qr.grouped_mm, a, b[0], o)
    refused("b: must be contiguous", qr.grouped_mm, a, b.transpose(1, 2).contiguous().transpose(1, 2), o)
    refused("a: expected shape", qr.grouped_mm, a[:, :8], b, o)
    refused("elements of a row must be consecutive", qr.grouped_mm, torch.zeros(16, 6, dtype=bf).t(), b, o)
    refused("a: row stride", qr.grouped_mm, torch.zeros(6, 20, dtype=bf)[:, :16], b, o)
    refused("a: must be in GPU memory", qr.grouped_mm, a, b, o)
    refused("dc: expected shape", qr.grouped_mm_grad_a, a, b, o)
    refused("dc: must be in GPU memory", qr.grouped_mm_grad_a, dc, b, o)
    refused("a: expected shape", qr.grouped_mm_grad_b, dc, a[:5], o)
    refused("dc: must be in GPU memory", qr.grouped_mm_grad_b, dc, a[:5], o, rows=r)
    refused("x: expected one of", qr.mxfp4_quantize, a.double())
    refused("blocks of 32", qr.mxfp4_quantize, a)
    refused("x: must be in GPU memory", qr.mxfp4_quantize, torch.zeros(2, 64))
    codes, scales = torch.zeros(6, 16, dtype=torch.uint8), torch.zeros(6, 1, dtype=torch.uint8)
    refused("scales: expected shape", qr.mxfp4_dequantize, codes, scales[:3])
    refused("codes: expected torch.uint8", qr.mxfp4_dequantize, codes.int(), scales)
    refused("codes: expected rows", qr.mxfp4_dequantize, torch.zeros(6, 8, dtype=torch.uint8), scales)
    refused("codes: must be in GPU memory", qr.mxfp4_dequantize, codes, scales)
    bc, bs = torch.zeros(3, 24, 16, dtype=torch.uint8), torch.zeros(3, 24, 1, dtype=torch.uint8)
    refused("b_scales: expected shape", qr.mxfp4_grouped_mm, codes, scales, bc, bs[:2], o)
    refused("b_codes: rows of", qr.mxfp4_grouped_mm, codes, scales, torch.zeros(3, 24, 32, dtype=torch.uint8),
            torch.zeros(3, 24, 2, dtype=torch.uint8), o)
    refused("a_codes: expected two", qr.mxfp4_grouped_mm, bc, bs, bc, bs, o)
    refused("a_codes: must be in GPU memory", qr.mxfp4_grouped_mm, codes, scales, bc, bs, o)
    refused("gu: expected \\[rows", qr.swiglu, torch.zeros(4, 15))
    refused("gu: must be in GPU memory", qr.swiglu, torch.zeros(4, 16))
    refused("dh: expected shape", qr.swiglu_grad, torch.zeros(4, 16), torch.zeros(4, 16))
    refused("dh: expected torch.float32", qr.swiglu_grad, torch.zeros(4, 8, dtype=bf), torch.zeros(4, 16))
    refused("blocks of 32", qr.swiglu_mxfp4, torch.zeros(4, 16))


@pytest.mark.parametrize("rows", [1 << 40, 1 << 43, 1 << 44, 1 << 52, 1 << 56, 1 << 61, (1 << 62) + 1, (1 << 63) - 1])
def test_row_counts_past_the_address_space(rows):
    """Sizes whose bytes do not fit 64 bits, or wrap the operand's address, are refused like other impossible ones:
    nothing computed from them wraps into a range that looks right."""
    s = 1 << 21  # the longest stride
    for f in (lambda: mm(rows=ROWS, src_rows=rows, lda=s), lambda: grad_b(rows=ROWS, src_rows=rows, lda=s),
              lambda: mm(rows=ROWS, src_rows=rows), lambda: grad_b(rows=ROWS, src_rows=rows),
              lambda: mm4(rows=ROWS, src_rows=rows), lambda: mm4(rows=ROWS, src_rows=rows, in_features=65536)):
        assert f() in (INVALID, UNSUPPORTED)
    if rows >= 1 << 43:  # 2^21 fp32 elements a row: 2^23 bytes
        assert L.moe_mxfp4_quantize(FP32, A, s, rows, s, B, C, None) == INVALID
        assert L.moe_mxfp4_dequantize(A, B, rows, s, FP32, C, s, None) == INVALID
        assert L.moe_swiglu(FP32, A, s, rows, s // 2, B, s // 2, None) == INVALID
        assert L.moe_swiglu_mxfp4(FP32, A, s, rows, s // 2, B, C, None) == INVALID
        assert L.moe_swiglu_grad(FP32, A, s // 2, B, s, rows, s // 2, C, s, None) == INVALID
