"""The expert operators (grouped products and their gradients, the four-bit
format and its product, SwiGLU and its gradient) on the GPU, against plain
64-bit computations.

Tolerances.  A product's sum is held in fp32 and rounded once.  Its terms are
exact in fp32 (at most 11 + 11 significant bits, or 3 + 3 and powers of two),
so with D terms of absolute sum S the sum is off by at most D 2^-24 S when
every addition rounds to nearest; D 2^-23 S allows for additions that
truncate.  The output type adds half a unit of the last place: 2^-8 |y| for
bf16, 2^-11 |y| + 2^-25 for fp16, 2^-24 |y| for fp32.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, FP16, FP32, FP64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
UNIT = {BF16: 2.0**-8, FP16: 2.0**-11, FP32: 2.0**-24}
TINY = {BF16: 2.0**-130, FP16: 2.0**-25, FP32: 2.0**-149}


def _qr():
    import quantized_routed_moe_amd as qr
    return qr


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def offsets_of(sizes, head=0):
    o = [head]
    for n in sizes:
        o.append(o[-1] + n)
    return o


def close(got, want, mag, depth, where=""):
    """got within the bound above of the 64-bit want; mag: the sum of the terms' magnitudes."""
    got, u = got.cpu(), UNIT[got.dtype]
    err = (got.to(FP64) - want).abs()
    tol = u * want.abs() * (1 + 2.0**-10) + depth * 2.0**-23 * mag * (1 + u) + TINY[got.dtype]
    bad = ~(err <= tol)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max()):.3e} past its bound"


def grouped_ref(a, b, offsets, rows, pairs):
    """(c, sum of magnitudes) in 64 bits."""
    a, b = a.to(FP64), b.to(FP64)
    if rows is not None:
        ok = (rows >= 0) & (rows < a.shape[0])
        a = a[rows.long().clamp(0, a.shape[0] - 1)] * ok[:, None]
    c = torch.zeros(pairs, b.shape[1], dtype=FP64)
    m = torch.zeros_like(c)
    for e in range(b.shape[0]):
        i, j = offsets[e], offsets[e + 1]
        c[i:j] = a[i:j] @ b[e].t()
        m[i:j] = a[i:j].abs() @ b[e].abs().t()
    return c, m


def dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


# group sizes (rows before the first group, rows past the last one): empty groups, one row, odd sizes, whole tiles,
# groups longer than any tile, many groups, a single group, rows of no group
GROUPS = {
    "one_row": ([1], 0, 0),
    "one_of_many": ([0, 0, 1, 0], 0, 0),
    "ragged": ([3, 0, 17, 1, 64, 0, 130, 5], 0, 0),
    "whole_tiles": ([128, 256, 64], 0, 0),
    "long": ([700, 0, 333], 0, 0),
    "many": ([i % 4 for i in range(300)], 0, 0),
    "most_groups": ([1 if i % 7 == 0 else 0 for i in range(1024)], 0, 0),
    "rows_outside": ([5, 0, 40], 3, 9),
    "all_outside": ([0, 0], 0, 33),
    "singles": ([1] * 37, 0, 0),
}
WIDTHS = [(8, 8), (72, 40), (136, 264), (264, 520), (128, 1032)]


def make_case(name, n, k, dtype, gather, seed, pad=0):
    sizes, head, tail = GROUPS[name]
    g = gen(seed)
    offsets = offsets_of(sizes, head)
    pairs = offsets[-1] + tail
    src = 29 if gather else pairs
    a = torch.randn(src, k + pad, generator=g).to(dtype)
    b = (torch.randn(len(sizes), n, k, generator=g) / k**0.5).to(dtype)
    rows = torch.randint(0, src, (pairs,), generator=g, dtype=torch.int32) if gather else None
    return a, b, offsets, rows, pairs


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("gather", [False, True])
def test_forward(name, n, k, gather):
    qr = _qr()
    for dtype, out in ((BF16, BF16), (FP16, FP32)):
        a, b, offsets, rows, pairs = make_case(name, n, k, dtype, gather, seed=n + k)
        c = qr.grouped_mm(a.cuda(), b.cuda(), dev(offsets), rows=cuda(rows), dtype=out)
        assert c.dtype == out and c.shape == (pairs, n)
        want, mag = grouped_ref(a, b, offsets, rows, pairs)
        close(c, want, mag, k, f"{name} {dtype} -> {out}")


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("n,k", WIDTHS)
def test_grad_a(name, n, k):
    qr = _qr()
    for dtype, out in ((BF16, FP32), (FP16, FP16)):
        dc, b, offsets, _, pairs = make_case(name, k, n, dtype, False, seed=2 * n + k)  # dc [P, n]
        b = b.transpose(1, 2).contiguous()  # [E, n, k]
        da = qr.grouped_mm_grad_a(dc.cuda(), b.cuda(), dev(offsets), dtype=out)
        want, mag = grouped_ref(dc, b.transpose(1, 2), offsets, None, pairs)
        close(da, want, mag, n, f"{name} {dtype} -> {out}")


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("gather", [False, True])
def test_grad_b(name, n, k, gather):
    qr = _qr()
    if len(GROUPS[name][0]) * n * k > 3e7:
        n, k = 40, 72  # many experts: narrow matrices
    for dtype, out in ((BF16, BF16), (FP16, FP32)):
        a, _, offsets, rows, pairs = make_case(name, n, k, dtype, gather, seed=3 * n + k)
        dc = torch.randn(pairs, n, generator=gen(n * k)).to(dtype)
        db = qr.grouped_mm_grad_b(dc.cuda(), a.cuda(), dev(offsets), rows=cuda(rows), dtype=out).cpu()
        ra = (a if rows is None else a[rows.long()]).to(FP64)
        for e in range(len(offsets) - 1):
            i, j = offsets[e], offsets[e + 1]
            if j == i:
                assert not db[e].any()
                continue
            d = dc[i:j].to(FP64)
            close(db[e], d.t() @ ra[i:j], d.abs().t() @ ra[i:j].abs(), j - i, f"{name} {dtype} expert {e}")


def many_tiles(sizes, n, k, seed):
    """Operands on the GPU for groups of more tiles than there are CUs, with gathered rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    offsets = offsets_of(sizes)
    pairs, src = offsets[-1], 901
    a = torch.randn(src, k, device="cuda", generator=g).to(BF16)
    b = (torch.randn(len(sizes), n, k, device="cuda", generator=g) / k**0.5).to(BF16)
    dc = torch.randn(pairs, n, device="cuda", generator=g).to(BF16)
    rows = torch.randint(0, src, (pairs,), device="cuda", generator=g, dtype=torch.int32)
    return a, b, dc, rows, offsets


def close_each(got, want_of, sizes, offsets, depth_of, whole):
    """close() group by group, the 64-bit product on the GPU; whole: got[e] is a group's matrix, else rows of it."""
    for e, n in enumerate(sizes):
        if n or whole:
            x, y = want_of(e, slice(offsets[e], offsets[e + 1]))
            part = got[e] if whole else got[offsets[e] : offsets[e + 1]]
            close(part, (x @ y).cpu(), (x.abs() @ y.abs()).cpu(), max(depth_of(e), 1), f"group {e}")


MANY = [
    ([3000, 0, 517, 2100, 260, 1, 900], 2056, 200),                 # long groups: the largest tiles, several a workgroup
    ([2900, 1031], 2056, 72),                                       # tiles of two steps
    ([1200, 1900], 2824, 40),                                       # tiles of one step, the ring deeper than the tile
    ([(i * 37) % 61 for i in range(200)], 520, 328),                # short groups, many empty
    ([(i * 53) % 290 for i in range(64)], 1032, 136),               # groups around a tile's size
]


@pytest.mark.parametrize("sizes,n,k", MANY)
def test_more_tiles_than_workgroups(sizes, n, k):
    """Every workgroup takes several tiles in turn, of unlike groups: forward, both gradients."""
    qr = _qr()
    a, b, dc, rows, offsets = many_tiles(sizes, n, k, n + k)
    o, at = dev(offsets), rows.long()
    c = qr.grouped_mm(a, b, o, rows=rows)
    close_each(c, lambda e, s: (a[at[s]].double(), b[e].double().t()), sizes, offsets, lambda e: k, False)
    da = qr.grouped_mm_grad_a(dc, b, o, dtype=FP32)
    close_each(da, lambda e, s: (dc[s].double(), b[e].double()), sizes, offsets, lambda e: n, False)
    for gather in (True, False):
        x = a[at] if not gather else a
        db = qr.grouped_mm_grad_b(dc, x, o, rows=rows if gather else None)
        close_each(db, lambda e, s: (dc[s].double().t(), a[at[s]].double()), sizes, offsets, lambda e: sizes[e], True)


@pytest.mark.parametrize("sizes,n,k", [(s, n, 32 * k) for (s, n, _), k in zip(MANY, (7, 16, 25, 33, 17))])
def test_mxfp4_more_tiles_than_workgroups(sizes, n, k):
    """The same for the four-bit product, with one to five steps a tile (odd counts end in half a pair of scales)."""
    qr = _qr()
    a, b, _, rows, offsets = many_tiles(sizes, n, k, n + k)
    qa, qb = qr.mxfp4_quantize(a), qr.mxfp4_quantize(b)
    va, vb = qr.mxfp4_dequantize(*qa, dtype=BF16), qr.mxfp4_dequantize(*qb, dtype=BF16)
    at = rows.long()
    for out in (BF16, FP32):
        c = qr.mxfp4_grouped_mm(*qa, *qb, dev(offsets), rows=rows, dtype=out)
        close_each(c, lambda e, s: (va[at[s]].double(), vb[e].double().t()), sizes, offsets, lambda e: k, False)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_strided_operands_and_padding_are_not_read(dtype):
    """Rows of a, dc and of the outputs may be strided; what lies between them, NaN here, is neither read into a
    result nor written."""
    qr = _qr()
    n, k, pad = 136, 264, 24
    a, b, offsets, _, pairs = make_case("ragged", n, k, dtype, False, 5, pad=pad)
    a[:, k:] = float("nan")
    wide = torch.full((pairs, n + pad), float("nan"), dtype=dtype, device="cuda")
    qr.grouped_mm(a.cuda()[:, :k], b.cuda(), dev(offsets), out=wide[:, :n])
    want, mag = grouped_ref(a[:, :k], b, offsets, None, pairs)
    close(wide[:, :n], want, mag, k, "c")
    assert wide[:, n:].isnan().all()
    dc = torch.randn(pairs, n + pad, generator=gen(6)).to(dtype)
    dc[:, n:] = float("nan")
    d = dc[:, :n].to(FP64)
    wide = torch.full((pairs, k + pad), float("nan"), dtype=dtype, device="cuda")
    qr.grouped_mm_grad_a(dc.cuda()[:, :n], b.cuda(), dev(offsets), out=wide[:, :k])
    want, mag = grouped_ref(dc[:, :n], b.transpose(1, 2), offsets, None, pairs)
    close(wide[:, :k], want, mag, n, "da")
    assert wide[:, k:].isnan().all()
    db = qr.grouped_mm_grad_b(dc.cuda()[:, :n], a.cuda()[:, :k], dev(offsets), dtype=FP32)
    for e in range(len(offsets) - 1):
        i, j = offsets[e], offsets[e + 1]
        x, y = d[i:j], a[i:j, :k].to(FP64)
        close(db[e], x.t() @ y, x.abs().t() @ y.abs(), max(j - i, 1), f"db {e}")


def test_not_finite_values_stay_in_their_rows():
    """NaN and infinities in rows of no group, in other rows of the group and in experts without pairs reach no
    other row's result, and reach their own."""
    qr = _qr()
    n, k = 72, 104
    a, b, offsets, _, pairs = make_case("rows_outside", n, k, BF16, False, 7)
    want, mag = grouped_ref(a, b, offsets, None, pairs)
    bad = [0, 1, 4, 20, pairs - 1]
    a[bad] = float("nan")
    a[20] = float("inf")
    b[1] = float("nan")  # the empty group's matrix
    c = qr.grouped_mm(a.cuda(), b.cuda(), dev(offsets)).cpu()
    fine = torch.ones(pairs, dtype=torch.bool)
    fine[bad] = False
    close(c[fine], want[fine], mag[fine], k, "rows of finite values")
    assert c[4].isnan().all() and not c[20].isfinite().any()
    assert not c[[0, 1, pairs - 1]].any()  # rows of no group


def test_gathered_rows_out_of_range_read_zeros():
    qr = _qr()
    n, k = 72, 104
    for name in ("ragged", "singles"):
        a, b, offsets, rows, pairs = make_case(name, n, k, BF16, True, 8)
        rows[::5] = torch.tensor([-1, 29, 2**31 - 1, -(2**31), 1000], dtype=torch.int32).repeat(pairs)[: len(rows[::5])]
        c = qr.grouped_mm(a.cuda(), b.cuda(), dev(offsets), rows=rows.cuda())
        want, mag = grouped_ref(a, b, offsets, rows, pairs)
        close(c, want, mag, k, "c")
        dc = torch.randn(pairs, n, generator=gen(9)).to(BF16)
        db = qr.grouped_mm_grad_b(dc.cuda(), a.cuda(), dev(offsets), rows=rows.cuda(), dtype=FP32)
        ok = (rows >= 0) & (rows < 29)
        ra = a.to(FP64)[rows.long().clamp(0, 28)] * ok[:, None]
        for e in range(len(offsets) - 1):
            i, j = offsets[e], offsets[e + 1]
            x = dc[i:j].to(FP64)
            close(db[e], x.t() @ ra[i:j], x.abs().t() @ ra[i:j].abs(), max(j - i, 1), f"db {e}")


def test_offsets_are_clamped():
    """Offsets that run past the pairs or backwards leave the buffers alone; groups that lie inside come out right."""
    qr = _qr()
    n, k, pairs = 40, 72, 50
    a = torch.randn(pairs, k, generator=gen(10)).to(BF16)
    b = torch.randn(4, n, k, generator=gen(11)).to(BF16)
    c = qr.grouped_mm(a.cuda(), b.cuda(), dev([-7, 20, 20, 45, 900]))
    want, mag = grouped_ref(a, b, [0, 20, 20, 45, 50], None, pairs)
    close(c, want, mag, k, "clamped")
    c = qr.grouped_mm(a.cuda(), b.cuda(), dev([0, 30, 10, 10, 50]))
    assert c.shape == (pairs, n)
    qr.grouped_mm_grad_b(c, a.cuda(), dev([0, 30, 10, 10, 50]))
    torch.cuda.synchronize()


def running_maximum(offsets, pairs):
    """What offsets mean whatever they hold: each within [0, pairs] and no lower than the ones before it."""
    out, most = [], 0
    for o in offsets:
        most = max(most, min(max(o, 0), pairs))
        out.append(most)
    return out


def guarded(rows, cols, dtype):
    """(whole, inner): an output [rows, cols] inside a buffer of sevens, with rows before and past it and columns beside it."""
    whole = torch.full((rows + 6, cols + 16), 7.0, dtype=dtype, device="cuda")
    return whole, whole[3 : 3 + rows, :cols]


def guards_stand(whole, cols):
    w = whole.cpu()
    return bool((w[:3] == 7).all() and (w[-3:] == 7).all() and (w[:, cols:] == 7).all())


BACKWARD = [
    ([0, 30, 10, 10, 50], 50),                                  # a group that ends before it begins
    ([5, 0, 40, 2, 45], 50),
    ([50, 0, 50, 0, 50], 50),                                   # every other group the whole of it
    ([-9, 60, 3, 70, 20], 64),                                  # out of range as well
    ([0] + [(i * 97) % 301 for i in range(40)], 300),           # more bounds than a lane each of one group
    ([0, 700, 100, 650, 900, 20, 1100], 1100),                  # long groups
    ([(i * 389) % 1201 for i in range(401)], 1200),             # more groups than are held in registers
]


@pytest.mark.parametrize("offsets,pairs", BACKWARD)
@pytest.mark.parametrize("n,k", [(40, 96), (520, 160)])
def test_offsets_that_run_backwards(offsets, pairs, n, k):
    """An offset less than one before it counts as the largest of those: groups stay disjoint, every row has one
    writer, the results are defined and nothing beside the outputs is written."""
    qr = _qr()
    E, g = len(offsets) - 1, gen(pairs + n)
    o, held = dev(offsets), running_maximum(offsets, pairs)
    a, dc = torch.randn(pairs, k, generator=g).to(BF16), torch.randn(pairs, n, generator=g).to(BF16)
    b = (torch.randn(E, n, k, generator=g) / k**0.5).to(BF16)
    want, mag = grouped_ref(a, b, held, None, pairs)
    whole, c = guarded(pairs, n, BF16)
    qr.grouped_mm(a.cuda(), b.cuda(), o, out=c)
    close(c, want, mag, k, "c")
    assert guards_stand(whole, n)
    whole, da = guarded(pairs, k, FP32)
    qr.grouped_mm_grad_a(dc.cuda(), b.cuda(), o, out=da)
    close(da, *grouped_ref(dc, b.transpose(1, 2), held, None, pairs), n, "da")
    assert guards_stand(whole, k)
    whole = torch.full((E + 2, n, k), 7.0, device="cuda")
    qr.grouped_mm_grad_b(dc.cuda(), a.cuda(), o, out=whole[1:-1])
    assert (whole[0] == 7).all() and (whole[-1] == 7).all()
    db = whole[1:-1].cpu()
    for e in range(E):
        x, y = dc[held[e] : held[e + 1]].to(FP64), a[held[e] : held[e + 1]].to(FP64)
        close(db[e], x.t() @ y, x.abs().t() @ y.abs(), max(len(x), 1), f"db {e}")
    qa, qb = qr.mxfp4_quantize(a.cuda()), qr.mxfp4_quantize(b.cuda())
    va, vb = values_ref(*(t.cpu() for t in qa)), values_ref(*(t.cpu() for t in qb))
    whole, c = guarded(pairs, n, FP32)
    qr.mxfp4_grouped_mm(*qa, *qb, o, out=c)
    close(c, *grouped_ref(va, vb, held, None, pairs), k, "four-bit c")
    assert guards_stand(whole, n)


def test_no_pairs():
    qr = _qr()
    a, b = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.randn(3, 40, 64, device="cuda").to(BF16)
    o = dev([0, 0, 0, 0])
    assert qr.grouped_mm(a, b, o).shape == (0, 40)
    assert qr.grouped_mm_grad_a(torch.empty(0, 40, dtype=BF16, device="cuda"), b, o).shape == (0, 64)
    db = qr.grouped_mm_grad_b(torch.empty(0, 40, dtype=BF16, device="cuda"), a, o)
    assert db.shape == (3, 40, 64) and not db.any()
    assert qr.swiglu(torch.empty(0, 64, device="cuda")).shape == (0, 32)
    codes, scales = qr.mxfp4_quantize(torch.empty(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and qr.mxfp4_dequantize(codes, scales).shape == (0, 64)
    bc, bs = qr.mxfp4_quantize(b)
    assert qr.mxfp4_grouped_mm(codes, scales, bc, bs, o).shape == (0, 40)
    # pairs that all read from an empty source
    rows = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert not qr.grouped_mm(a, b, dev([0, 2, 2, 5]), rows=rows).any()


def test_a_bank_past_32_bits():
    """The last expert of a bank of more than 2^32 bytes and elements past 2^31: offsets that 32 bits do not hold."""
    qr = _qr()
    E, n, k = 132, 4096, 4096
    b = torch.zeros(E, n, k, dtype=BF16, device="cuda")
    assert b.numel() > 2**31
    last = (torch.randn(n, k, generator=gen(12)) / 64).to(BF16)
    b[-1] = last.cuda()
    for pairs in (2, 200):  # a few rows, and a tile and more
        a = torch.randn(pairs, k, generator=gen(13)).to(BF16)
        o = dev([0] * E + [pairs])
        c = qr.grouped_mm(a.cuda(), b, o, dtype=FP32)
        x, y = a.to(FP64), last.to(FP64)
        close(c, x @ y.t(), x.abs() @ y.abs().t(), k, f"c of {pairs}")
        da = qr.grouped_mm_grad_a(a.cuda(), b, o, dtype=FP32)
        close(da, x @ y, x.abs() @ y.abs(), n, f"da of {pairs}")
    dc = torch.randn(3, n, generator=gen(14)).to(BF16)
    qr.grouped_mm_grad_b(dc.cuda(), a[:3].cuda(), dev([0] * E + [3]), out=b)
    assert not b[:-1].any()
    x, y = dc.to(FP64), a[:3].to(FP64)
    close(b[-1], x.t() @ y, x.abs().t() @ y.abs(), 3, "db")


def test_gradients_against_differences():
    """The product is linear in a and in b, so a central difference of its fp32 output along a direction is the
    gradient's product with it, up to the sums' rounding.  Inputs are multiples of 1/4 and the step is 1/4: exact."""
    qr = _qr()
    sizes = [3, 0, 70, 1, 150]
    offsets, n, k, h = offsets_of(sizes), 72, 136, 0.25
    g = gen(15)
    pairs = offsets[-1]

    def grid(*shape):
        return (torch.randint(-8, 9, shape, generator=g) / 4).to(BF16).cuda()

    a, b, dc, o = grid(pairs, k), grid(len(sizes), n, k), grid(pairs, n), dev(offsets)
    da = qr.grouped_mm_grad_a(dc, b, o, dtype=FP32).double()
    db = qr.grouped_mm_grad_b(dc, a, o, dtype=FP32).double()

    def loss(x, y):
        return float((qr.grouped_mm(x, y, o, dtype=FP32).double() * dc.double()).sum())

    for seed in range(3):
        va = (torch.randint(0, 2, (pairs, k), generator=g) * 2 - 1).to(BF16).cuda()
        vb = (torch.randint(0, 2, (len(sizes), n, k), generator=g) * 2 - 1).to(BF16).cuda()
        for num, ana in (((loss(a + h * va, b) - loss(a - h * va, b)) / (2 * h), float((da * va.double()).sum())),
                         ((loss(a, b + h * vb) - loss(a, b - h * vb)) / (2 * h), float((db * vb.double()).sum()))):
            # products of multiples of 1/16 below 2^24: every sum here is exact
            assert num == ana


# -------------------------------------------------------- four-bit format
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantize_ref(x):
    """(codes, scales) by comparing with the midpoints of the representable values, in 64 bits."""
    b = x.to(FP64).reshape(-1, 32)
    amax = b.abs().amax(1)
    bad = ~amax.isfinite()  # NaN or infinity in the block
    _, e = torch.frexp(torch.where(bad, torch.zeros_like(amax), amax))
    s = torch.where(amax > 0, (e - 1 - 2 + 127).clamp(0, 254), torch.zeros_like(e))
    m = torch.where(bad[:, None], torch.zeros_like(b), b.abs() / torch.exp2(s.to(FP64) - 127)[:, None])
    v = torch.tensor(VALUES, dtype=FP64)
    mid = (v[1:] + v[:-1]) / 2
    lo, hi = torch.bucketize(m, mid, right=False), torch.bucketize(m, mid, right=True)
    code = torch.where(lo % 2 == 0, lo, hi) | (torch.signbit(x.reshape(-1, 32)).int() << 3)
    s = torch.where(bad, torch.full_like(s, 255), s)
    code = code.reshape(*x.shape[:-1], -1, 2)
    return (code[..., 0] | code[..., 1] << 4).to(torch.uint8), s.reshape(*x.shape[:-1], -1).to(torch.uint8), bad


def values_ref(codes, scales):
    v = torch.tensor(VALUES + [-x for x in VALUES], dtype=FP64)
    x = torch.stack([v[(codes & 15).long()], v[(codes >> 4).long()]], -1).reshape(*scales.shape, 32)
    s = torch.exp2(scales.to(FP64) - 127)
    s[scales == 255] = float("nan")
    return (x * s[..., None]).reshape(*codes.shape[:-1], -1)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (7, 96), (130, 352), (5, 4096), (1000, 32)])
def test_quantize_is_exact(dtype, rows, cols):
    qr = _qr()
    g = gen(rows + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g).float())
    x = x.to(dtype)
    codes, scales = qr.mxfp4_quantize(x.cuda())
    wc, ws, _ = quantize_ref(x)
    assert torch.equal(codes.cpu(), wc) and torch.equal(scales.cpu(), ws)
    for out in (FP32, BF16, FP16):
        y = qr.mxfp4_dequantize(codes, scales, dtype=out).cpu()
        assert torch.equal(y, values_ref(wc, ws).to(out))


def test_quantize_ties_extremes_and_not_finite():
    """Every tie and its neighbours at scales from the smallest to the largest, zeros of both signs, subnormals,
    values past 6, blocks with NaN or infinity; the block beside stays as it is."""
    qr = _qr()
    pts = [0.0, -0.0]
    for i in range(7):
        m = (VALUES[i] + VALUES[i + 1]) / 2
        pts += [m, -m, VALUES[i + 1], -VALUES[i + 1], m * (1 + 2.0**-20), m * (1 - 2.0**-20)]
    pts += [7.0, -7.0, 7.999, 5.0000005]
    pts = torch.tensor(pts, dtype=FP64)
    blocks = []
    for e in (-149, -140, -130, -127, -126, -125, -60, -1, 0, 1, 60, 124, 125):
        for i in range(0, len(pts), 31):
            blk = torch.zeros(32, dtype=FP64)
            part = pts[i : i + 31]
            blk[: len(part)] = part
            blk[31] = 4.0  # fixes the scale at 2^e unless a larger value does not fit
            blocks.append((blk * 2.0**e).to(FP32))
    for bad in (float("nan"), float("inf"), -float("inf")):
        blk = torch.ones(32)
        blk[17] = bad
        blocks += [blk, torch.arange(32.0)]
    blocks.append(torch.zeros(32))
    blocks.append(torch.full((32,), torch.finfo(FP32).max))
    x = torch.stack(blocks)
    codes, scales = qr.mxfp4_quantize(x.cuda())
    wc, ws, bad = quantize_ref(x)
    codes, scales = codes.cpu(), scales.cpu()
    assert torch.equal(scales, ws)
    assert torch.equal(codes[~bad], wc[~bad])
    y = qr.mxfp4_dequantize(codes.cuda(), scales.cuda()).cpu()
    assert y[bad].isnan().all() and torch.equal(y[~bad], values_ref(wc, ws)[~bad].to(FP32))


def test_quantize_strided_rows_and_many_dimensions():
    qr = _qr()
    x = torch.randn(9, 160, generator=gen(16))
    codes, scales = qr.mxfp4_quantize(x.cuda()[:, :96])
    wc, ws, _ = quantize_ref(x[:, :96])
    assert torch.equal(codes.cpu(), wc) and torch.equal(scales.cpu(), ws)
    wide = torch.full((9, 128), 7.0, device="cuda")
    qr.mxfp4_dequantize(codes, scales, out=wide[:, :96])
    assert torch.equal(wide[:, :96].cpu(), values_ref(wc, ws).to(FP32)) and (wide[:, 96:] == 7).all()
    x = torch.randn(3, 5, 64, generator=gen(17)).to(BF16)
    codes, scales = qr.mxfp4_quantize(x.cuda())
    assert codes.shape == (3, 5, 32) and scales.shape == (3, 5, 2)
    wc, ws, _ = quantize_ref(x)
    assert torch.equal(codes.cpu(), wc) and torch.equal(scales.cpu(), ws)


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("n,k", [(8, 32), (72, 96), (136, 224), (264, 544), (128, 1024)])
@pytest.mark.parametrize("gather", [False, True])
def test_mxfp4_product(name, n, k, gather):
    qr = _qr()
    sizes, head, tail = GROUPS[name]
    offsets = offsets_of(sizes, head)
    pairs, g = offsets[-1] + tail, gen(n + k)
    src = 29 if gather else pairs
    ac = torch.randint(0, 256, (src, k // 2), generator=g, dtype=torch.uint8)
    as_ = torch.randint(118, 132, (src, k // 32), generator=g, dtype=torch.uint8)
    bc = torch.randint(0, 256, (len(sizes), n, k // 2), generator=g, dtype=torch.uint8)
    bs = torch.randint(118, 132, (len(sizes), n, k // 32), generator=g, dtype=torch.uint8)
    rows = torch.randint(0, src, (pairs,), generator=g, dtype=torch.int32) if gather else None
    want, mag = grouped_ref(values_ref(ac, as_), values_ref(bc, bs), offsets, rows, pairs)
    for out in (BF16, FP32):
        c = qr.mxfp4_grouped_mm(ac.cuda(), as_.cuda(), bc.cuda(), bs.cuda(), dev(offsets), rows=cuda(rows), dtype=out)
        close(c, want, mag, k, f"{name} {out}")


@pytest.mark.parametrize("pairs", [1, 5, 200])
def test_mxfp4_product_not_a_number_and_extreme_scales(pairs):
    """A block of scale 255 makes its row's (its column's) results NaN and no others; the smallest and the largest
    scales meet without under- or overflow of the product."""
    qr = _qr()
    n, k = 72, 160
    x, w = torch.randn(pairs, k, generator=gen(18)), torch.randn(2, n, k, generator=gen(19))
    (ac, as_), (bc, bs) = qr.mxfp4_quantize(x.cuda()), qr.mxfp4_quantize(w.cuda())
    o = dev([0, 0, pairs])
    want, mag = grouped_ref(values_ref(ac.cpu(), as_.cpu()), values_ref(bc.cpu(), bs.cpu()), [0, 0, pairs], None, pairs)
    bad_a, bad_b = as_.clone(), bs.clone()
    bad_a[0, 3], bad_b[1, 5, 4], bad_b[0] = 255, 255, 255
    c = qr.mxfp4_grouped_mm(ac, bad_a, bc, bad_b, o, dtype=FP32).cpu()
    assert c[0].isnan().all() and c[:, 5].isnan().all()
    keep = [i for i in range(n) if i != 5]
    close(c[1:, keep], want[1:, keep], mag[1:, keep], k, "others")
    low, high = torch.zeros_like(as_), torch.full_like(bs, 254)
    v = values_ref(ac.cpu(), torch.full_like(as_, 127).cpu()), values_ref(bc.cpu(), torch.full_like(bs, 127).cpu())
    want, mag = grouped_ref(*v, [0, 0, pairs], None, pairs)
    close(qr.mxfp4_grouped_mm(ac, low, bc, high, o, dtype=FP32), want, mag, k, "scales 0 and 254")


# ------------------------------------------------------------------ swiglu
def swiglu_ref(gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f].to(FP64), gu[:, f:].to(FP64)
    s = torch.sigmoid(g)
    return g, u, s


# exp and the division are good to a few units of 2^-24 and the argument's rounding adds |g| 2^-24 of e^-g, of which
# the sigmoid keeps at most the same share; the formula's further products round once each
def swiglu_tol(want, g, dtype, terms):
    return UNIT[dtype] * want.abs() * 1.001 + (12 + 2 * g.abs()) * 2.0**-23 * terms + TINY[dtype] + 2.0**-120


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("rows,ffn", [(1, 8), (3, 40), (65, 136), (192, 2048), (1000, 24)])
def test_swiglu_and_gradient(dtype, rows, ffn):
    qr = _qr()
    gu = (torch.randn(rows, 2 * ffn, generator=gen(rows + ffn)) * 4).to(dtype)
    dh = torch.randn(rows, ffn, generator=gen(rows * ffn)).to(dtype)
    g, u, s = swiglu_ref(gu)
    h = qr.swiglu(gu.cuda()).cpu()
    want = g * s * u
    assert ((h.to(FP64) - want).abs() <= swiglu_tol(want, g, dtype, want.abs())).all()
    dgu = qr.swiglu_grad(dh.cuda(), gu.cuda()).cpu().to(FP64)
    d = dh.to(FP64)
    du, dg = d * g * s, d * u * s * (1 + g * (1 - s))
    assert ((dgu[:, ffn:] - du).abs() <= swiglu_tol(du, g, dtype, du.abs())).all()
    terms = d.abs() * u.abs() * s * (1 + g.abs())  # 1 + g (1 - s) cancels for negative gates
    assert ((dgu[:, :ffn] - dg).abs() <= swiglu_tol(dg, g, dtype, terms)).all()


@pytest.mark.parametrize("deviation", [0.1, 1.5, 16.0, 40.0])
def test_swiglu_in_32_bits(deviation):
    """fp32 results keep their relative precision for gates of every size.  In units of 2^-24: e^-|g| is off by 3 (a
    unit of the last place of the exponential, a rounding), 1 + e and its reciprocal by 1 each, e / (1 + e) by 6 in
    all; h = g s u takes two products more: 8.  du = dh g s likewise; dg's factors dh u s by 8, 1 + g (1 - s) by 8 of
    its terms, their product by 1: 17 of the terms' magnitudes.  2^-120 covers what is below the normal range."""
    qr = _qr()
    g = gen(int(10 * deviation))
    gate = torch.randn(500, 256, generator=g) * deviation
    gate[0] = torch.linspace(-80, 80, 256)
    gate[1] = torch.linspace(-1, 1, 256)
    gu = torch.cat([gate, torch.randn(500, 256, generator=g)], 1)
    dh = torch.randn(500, 256, generator=g)
    h, dgu = qr.swiglu(gu.cuda()).cpu(), qr.swiglu_grad(dh.cuda(), gu.cuda()).cpu().to(FP64)
    gate, up, s = swiglu_ref(gu)
    rest, d, unit = torch.sigmoid(-gate), dh.to(FP64), 2.0**-24 * 1.001
    want = gate * s * up
    assert ((h.to(FP64) - want).abs() <= 8 * unit * want.abs() + 2.0**-120).all()
    want = d * gate * s
    assert ((dgu[:, 256:] - want).abs() <= 8 * unit * want.abs() + 2.0**-120).all()
    want, terms = d * up * s * (1 + gate * rest), (d * up).abs() * s * (1 + gate.abs() * rest)
    assert ((dgu[:, :256] - want).abs() <= 17 * unit * terms + 2.0**-120).all()


def test_swiglu_gradient_against_differences():
    """Central differences of the 64-bit formula with step 2^-12: the third derivative of silu is below 1, so they
    are within h^2 / 6 of the gradient (times dh and the other factor)."""
    qr = _qr()
    gu = torch.randn(20, 128, generator=gen(20)) * 3
    dh = torch.randn(20, 64, generator=gen(21))
    dgu = qr.swiglu_grad(dh.cuda(), gu.cuda()).cpu().to(FP64)
    h = 2.0**-12

    def f(x):
        g, u, s = swiglu_ref(x)
        return g * s * u * dh.to(FP64)

    x = gu.to(FP64)
    for half in range(2):
        v = torch.zeros_like(x)
        v[:, 64 * half : 64 * half + 64] = h
        num = (f(x + v) - f(x - v)) / (2 * h)
        other = x[:, :64] if half else x[:, 64:]
        tol = (h * h / 6 + 40 * 2.0**-23) * dh.abs().to(FP64) * (other.abs() + 1) * (1 + x[:, :64].abs()) + 1e-9
        assert ((dgu[:, 64 * half : 64 * half + 64] - num).abs() <= tol).all()


def test_swiglu_extreme_gates_and_strides():
    qr = _qr()
    gate = [0.0, -0.0, 88.0, -88.0, 100.0, -100.0, 1e4, -1e4]
    gu = torch.tensor([gate + [2.0] * 8])
    h = qr.swiglu(gu.cuda()).cpu()
    g, u, s = swiglu_ref(gu)
    assert ((h.to(FP64) - g * s * u).abs() <= 2.0**-20 * (g * s * u).abs() + 2.0**-120).all()
    dgu = qr.swiglu_grad(torch.ones(1, 8).cuda(), gu.cuda()).cpu()
    assert dgu.isfinite().all()
    want = torch.cat([u * s * (1 + g * (1 - s)), g * s], 1)
    assert ((dgu.to(FP64) - want).abs() <= 2.0**-18 * want.abs() + 1e-30).all()
    # strided rows in and out; NaN in between stays there
    wide = torch.full((5, 2 * 24 + 8), float("nan"), dtype=BF16)
    wide[:, :48] = torch.randn(5, 48, generator=gen(22)).to(BF16)
    out = torch.full((5, 40), float("nan"), dtype=BF16, device="cuda")
    qr.swiglu(wide.cuda()[:, :48], out=out[:, :24])
    assert out[:, :24].isfinite().all() and out[:, 24:].isnan().all()
    assert torch.equal(out[:, :24], qr.swiglu(wide.cuda()[:, :48].contiguous()))
    grad = torch.full((5, 56), float("nan"), dtype=BF16, device="cuda")
    dh = torch.randn(5, 32, generator=gen(23)).to(BF16).cuda()[:, :24]
    qr.swiglu_grad(dh, wide.cuda()[:, :48], out=grad[:, :48])
    assert grad[:, 48:].isnan().all()
    assert torch.equal(grad[:, :48], qr.swiglu_grad(dh.contiguous(), wide.cuda()[:, :48].contiguous()))


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("rows,ffn", [(1, 32), (7, 96), (130, 2048)])
def test_swiglu_to_four_bits(dtype, rows, ffn):
    """The four-bit result is the quantisation of the activation in fp32: it equals that of swiglu's fp32 output."""
    qr = _qr()
    gu = (torch.randn(rows, 2 * ffn, generator=gen(rows + ffn)) * 3).to(dtype)
    codes, scales = qr.swiglu_mxfp4(gu.cuda())
    wc, ws = qr.mxfp4_quantize(qr.swiglu(gu.float().cuda()))
    assert torch.equal(codes, wc) and torch.equal(scales, ws)


# ----------------------------------------------------------- calling them
def test_other_streams_graphs_and_repeated_calls():
    """A call on a side stream, the same call captured into a graph and replayed with eager work between, and
    repeated calls give the same bits."""
    qr = _qr()
    n, k = 264, 544
    a, b, offsets, rows, pairs = make_case("ragged", n, k, BF16, True, 24)
    a, b, rows, o = a.cuda(), b.cuda(), rows.cuda(), dev(offsets)
    bq = qr.mxfp4_quantize(b)
    gu = torch.randn(pairs, 256, device="cuda").to(BF16)

    def chain(stream=None):
        c = qr.grouped_mm(a, b, o, rows=rows, stream=stream)
        da = qr.grouped_mm_grad_a(c, b, o, stream=stream)
        db = qr.grouped_mm_grad_b(c, a, o, rows=rows, stream=stream)
        q = qr.mxfp4_quantize(a, stream=stream)
        c4 = qr.mxfp4_grouped_mm(*q, *bq, o, rows=rows, stream=stream)
        h = qr.swiglu(gu, stream=stream)
        dg = qr.swiglu_grad(h, gu, stream=stream)
        h4 = qr.mxfp4_dequantize(*qr.swiglu_mxfp4(gu, stream=stream), stream=stream)
        return [c, da, db, *q, c4, h, dg, h4]

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = chain(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for i in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), f"replay {i}"
        again = chain()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(again, want)), f"eager call {i}"


def test_operands_that_ask_for_a_gradient():
    """No call passes for a constant: its result has the same bits, and differentiating through it raises; so does an
    `out` that torch could not follow, and a forward-mode tangent."""
    from torch.autograd import forward_ad

    qr = _qr()
    a, b, offsets, rows, pairs = make_case("ragged", 40, 64, BF16, True, 25)
    a, b, rows, o = a.cuda(), b.cuda(), rows.cuda(), dev(offsets)
    dc = torch.randn(pairs, 40, generator=gen(26)).to(BF16).cuda()
    gu = torch.randn(pairs, 64, generator=gen(27)).cuda()
    dh = torch.randn(pairs, 32, generator=gen(28)).cuda()
    calls = [("grouped_mm", lambda x, y, **kw: qr.grouped_mm(x, y, o, rows=rows, **kw), a, b),
             ("grouped_mm_grad_a", lambda x, y, **kw: qr.grouped_mm_grad_a(x, y, o, **kw), dc, b),
             ("grouped_mm_grad_b", lambda x, y, **kw: qr.grouped_mm_grad_b(x, y, o, rows=rows, **kw), dc, a),
             ("swiglu_grad", lambda x, y, **kw: qr.swiglu_grad(x, y, **kw), dh, gu),
             ("swiglu", lambda x, y, **kw: qr.swiglu(y, **kw), dh, gu)]
    for name, f, x, y in calls:
        want = f(x, y)
        assert not want.requires_grad
        for which in (0, 1):
            if name == "swiglu" and which == 0:
                continue
            args = [t.detach().clone().requires_grad_(i == which) for i, t in enumerate((x, y))]
            got = f(*args)
            assert torch.equal(got, want)
            with pytest.raises(RuntimeError, match=f"{name} builds no graph"):
                (got.float().sum() + args[which].float().sum()).backward()
            with pytest.raises(RuntimeError, match=f"{name} builds no graph"):
                f(*args, out=torch.empty_like(want))
            with torch.no_grad():
                assert not f(*args, out=torch.empty_like(want)).requires_grad
            with forward_ad.dual_level():
                args = [forward_ad.make_dual(t, torch.ones_like(t)) if i == which else t for i, t in enumerate((x, y))]
                with pytest.raises(RuntimeError, match=f"{name} has no forward-mode"):
                    f(*args)
                assert torch.equal(f(x, y), want)
    experts = qr.Mxfp4Experts(b.new_zeros(3, 64, 64).requires_grad_(), b.new_zeros(3, 64, 32))
    w = torch.rand(5, 2, device="cuda").requires_grad_()
    r = qr.Routing.from_ids(torch.tensor([[0, 1]] * 5, device="cuda"), w, 3)
    x = a[:5].detach().clone().requires_grad_()
    with pytest.raises(RuntimeError, match="Mxfp4Experts builds no graph"):
        experts(x, r).sum().backward()
    experts(x.detach(), r).sum().backward()  # the weights' gradient is torch's own
    assert w.grad.shape == w.shape


def test_operands_dropped_while_a_side_stream_has_work():
    """Operands, and outputs passed in, that are dropped right after a call on another stream: their memory is not
    handed out again before the call has run."""
    qr = _qr()
    pairs, n, k = 300, 264, 4096
    g = torch.Generator(device="cuda").manual_seed(29)
    o = [0, 120, 120, pairs]
    big = torch.randn(4096, 4096, device="cuda", generator=g)

    def fresh(*shape, dtype=BF16):
        return torch.randn(*shape, device="cuda", generator=g).to(dtype)

    def codes(x):
        return list(qr.mxfp4_quantize(x))

    def rows():
        return torch.arange(pairs, device="cuda", dtype=torch.int32).flip(0)

    new = torch.empty
    calls = [
        (lambda s, a, b, o, r, out: qr.grouped_mm(a, b, o, rows=r, out=out, stream=s),
         lambda: [fresh(pairs, k), fresh(3, n, k), dev(o), rows(), new(pairs, n, device="cuda", dtype=BF16)]),
        (lambda s, d, b, o, out: qr.grouped_mm_grad_a(d, b, o, out=out, stream=s),
         lambda: [fresh(pairs, n), fresh(3, n, k), dev(o), new(pairs, k, device="cuda", dtype=BF16)]),
        (lambda s, d, a, o, r, out: qr.grouped_mm_grad_b(d, a, o, rows=r, out=out, stream=s),
         lambda: [fresh(pairs, n), fresh(pairs, k), dev(o), rows(), new(3, n, k, device="cuda", dtype=BF16)]),
        (lambda s, x, c, e: qr.mxfp4_quantize(x, c, e, stream=s),
         lambda: [fresh(pairs, k), *codes(fresh(pairs, k))]),
        (lambda s, c, e, out: qr.mxfp4_dequantize(c, e, out=out, stream=s),
         lambda: [*codes(fresh(pairs, k)), new(pairs, k, device="cuda")]),
        (lambda s, ac, ae, bc, be, o, r, out: qr.mxfp4_grouped_mm(ac, ae, bc, be, o, rows=r, out=out, stream=s),
         lambda: [*codes(fresh(pairs, k)), *codes(fresh(3, n, k)), dev(o), rows(),
                  new(pairs, n, device="cuda", dtype=BF16)]),
        (lambda s, gu, out: qr.swiglu(gu, out=out, stream=s),
         lambda: [fresh(pairs, 2 * k), new(pairs, k, device="cuda", dtype=BF16)]),
        (lambda s, gu, c, e: qr.swiglu_mxfp4(gu, c, e, stream=s),
         lambda: [fresh(pairs, 2 * k), *codes(fresh(pairs, k))]),
        (lambda s, d, gu, out: qr.swiglu_grad(d, gu, out=out, stream=s),
         lambda: [fresh(pairs, k), fresh(pairs, 2 * k), new(pairs, 2 * k, device="cuda", dtype=BF16)]),
    ]
    side = torch.cuda.Stream()
    for i, (call, operands) in enumerate(calls):
        held = operands()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.mm(big, big)
            busy = torch.cuda.Event()
            busy.record()
        result = call(side, *held)
        was = {(t.data_ptr(), t.shape, t.dtype) for t in held}
        like = [(t.shape, t.dtype) for t in held]
        del held, result
        again = [torch.empty(s, dtype=d, device="cuda") for s, d in like]
        assert not busy.query(), "the side stream was not kept busy"
        assert not was & {(t.data_ptr(), t.shape, t.dtype) for t in again}, f"call {i}"
        del again
        torch.cuda.synchronize()


def test_columns_of_one_matrix():
    """Operands and outputs that are columns of one wide matrix share no element and are accepted; columns that do
    share one, or rows of another stride over the same memory, are refused."""
    qr = _qr()
    rows, f = 70, 64
    wide = torch.randn(rows, 6 * f, generator=gen(30)).to(BF16).cuda()
    gu, dh = wide[:, f : 3 * f], wide[:, 3 * f : 4 * f]
    want_h, want_g = qr.swiglu(gu.contiguous()), qr.swiglu_grad(dh.contiguous(), gu.contiguous())
    b, o = (torch.randn(2, f, 2 * f, generator=gen(31)) / 11).to(BF16).cuda(), dev([0, 30, rows])
    want_c = qr.grouped_mm(gu.contiguous(), b, o)
    want_a = qr.grouped_mm_grad_a(dh.contiguous(), b, o)
    before = wide.clone()
    assert torch.equal(qr.swiglu(gu, out=wide[:, :f]), want_h)              # before the operand's columns
    assert torch.equal(qr.swiglu(gu, out=wide[:, 3 * f : 4 * f]), want_h)   # right after them
    wide[:, 3 * f : 4 * f] = before[:, 3 * f : 4 * f]
    assert torch.equal(qr.swiglu_grad(dh, gu, out=wide[:, 4 * f :]), want_g)
    assert torch.equal(qr.grouped_mm(gu, b, o, out=wide[:, 5 * f :]), want_c)
    assert torch.equal(qr.grouped_mm_grad_a(dh, b, o, out=wide[:, 4 * f :]), want_a)
    assert torch.equal(wide[:, f : 4 * f], before[:, f : 4 * f])
    for bad in (wide[:, 8 : f + 8], wide[:, f : 2 * f], wide[:, 3 * f - 8 : 4 * f - 8], wide.view(-1, 3 * f)[:rows, :f]):
        with pytest.raises(qr.MoEError):
            qr.swiglu(gu, out=bad)
    assert torch.equal(wide[:, f : 4 * f], before[:, f : 4 * f])
    # one row further down and at the edge of the next row's columns
    tall = torch.zeros(rows + 1, 4 * f, dtype=BF16, device="cuda")
    tall[:rows, 2 * f :] = gu
    assert torch.equal(qr.swiglu(tall[:rows, 2 * f :], out=tall[1:, :f]), want_h)
    with pytest.raises(qr.MoEError):
        qr.swiglu(tall[:rows, 2 * f :], out=tall[1:, f + 8 : 2 * f + 8])


# ------------------------------------- every kernel of the products, by the rule that chooses it
def typed(sizes, n, k, dtype, seed):
    """many_tiles in another type."""
    a, b, dc, rows, offsets = many_tiles(sizes, n, k, seed)
    return a.to(dtype), b.to(dtype), dc.to(dtype), rows, offsets


# 31 tiles of 256 rows by 9 of 256 columns, at least 96 rows a group on average: the largest tile; remainders of 1, 65,
# 129 and 193 rows (one to four live row blocks of a wave) and of a whole tile
LARGE = [769, 577, 385, 705, 0, 2048, 1, 952]


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP16, FP32)])
def test_largest_tiles(dtype, out):
    """Forward and both gradients by 256x256 tiles, each operand type into each output type."""
    qr = _qr()
    k, n = 200, 2056
    a, b, _, rows, offsets = typed(LARGE, n, k, dtype, 40)
    o, at = dev(offsets), rows.long()
    c = qr.grouped_mm(a, b, o, rows=rows, dtype=out)
    close_each(c, lambda e, s: (a[at[s]].double(), b[e].double().t()), LARGE, offsets, lambda e: k, False)
    _, b, dc, _, _ = typed(LARGE, k, n, dtype, 41)  # columns of da: 2056
    da = qr.grouped_mm_grad_a(dc, b, o, dtype=out)
    close_each(da, lambda e, s: (dc[s].double(), b[e].double()), LARGE, offsets, lambda e: k, False)
    sizes, n, k = [64, 0, 1, 63, 65, 193, 700, 128, 300], 1032, 1288  # 9 experts of 5 x 6 tiles
    a, _, dc, rows, offsets = typed(sizes, n, k, dtype, 42)
    at = rows.long()
    for gather in (True, False):
        db = qr.grouped_mm_grad_b(dc, a if gather else a[at], dev(offsets), rows=rows if gather else None, dtype=out)
        close_each(db, lambda e, s: (dc[s].double().t(), a[at[s]].double()), sizes, offsets, lambda e: sizes[e], True)


# (group sizes, columns): few rows, streamed, a workgroup taking one column tile or several (the last of them short);
# tiles of 64x128, where there are few tiles and where there are few rows a group; tiles of 128x256
FORMS = {
    "streamed": ([1, 0, 3], 136),
    "streamed_sweeps": ([16, 0, 31, 1, 17, 40, 0, 0, 60, 5, 9, 16, 20, 30, 11, 0], 1400),
    "few_tiles": ([200, 0, 45], 264),
    "few_rows_a_group": ([(i * 5) % 19 for i in range(60)], 1032),
    "largest_tile": ([130, 900, 0, 257, 1, 700, 64, 1300], 1800),
}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("k", [1024, 2048, 2080, 2304, 4096, 4128])
def test_mxfp4_long_rows(form, k):
    """Rows of more than one load of scales (2048 elements), whole loads and remainders, through each kernel.  The
    scale of every block is its own, so that one taken from another block shows."""
    qr = _qr()
    sizes, n = FORMS[form]
    offsets = offsets_of(sizes)
    pairs, src, E = offsets[-1], 97, len(sizes)
    g = torch.Generator(device="cuda").manual_seed(k + n)

    def rand(lo, hi, *shape):
        return torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)

    ac, as_, bc, bs = rand(0, 256, src, k // 2), rand(118, 132, src, k // 32), rand(0, 256, E, n, k // 2), rand(118, 132, E, n, k // 32)
    rows = torch.randint(0, src, (pairs,), device="cuda", generator=g, dtype=torch.int32)
    va, vb = qr.mxfp4_dequantize(ac, as_).double(), qr.mxfp4_dequantize(bc, bs)
    at = rows.long()
    for gather, out in ((True, BF16), (False, FP32)):
        c = qr.mxfp4_grouped_mm(*((ac, as_) if gather else (ac[at], as_[at])), bc, bs, dev(offsets),
                                rows=rows if gather else None, dtype=out)
        close_each(c, lambda e, s: (va[at[s]], vb[e].double().t()), sizes, offsets, lambda e: k, False)


@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (FP16, FP16)])
@pytest.mark.parametrize("k", [520, 2056])
def test_streamed_sweeps(dtype, out, k):
    """16-bit rows of few rows a group: workgroups that take several column tiles, the last of them short."""
    qr = _qr()
    sizes, n = FORMS["streamed_sweeps"]
    a, b, _, rows, offsets = typed(sizes, n, k, dtype, k)
    at = rows.long()
    c = qr.grouped_mm(a, b, dev(offsets), rows=rows, dtype=out)
    close_each(c, lambda e, s: (a[at[s]].double(), b[e].double().t()), sizes, offsets, lambda e: k, False)


# ------------------------------------------------------------ subnormals
@pytest.mark.parametrize("dtype,low,other", [(FP16, -24, 0), (FP16, -24, -14), (BF16, -133, 20)])
@pytest.mark.parametrize("pairs", [3, 300])
def test_subnormal_operands_keep_their_value(dtype, low, other, pairs):
    """One term a sum, one factor of it subnormal: the product is exact in fp32, in each direction and kernel."""
    qr = _qr()
    n = k = 136
    g = gen(pairs)

    def small(*shape):
        return (torch.randint(1, 8, shape, generator=g) * 2.0**low).to(dtype)

    def plain(*shape):
        return ((1 + torch.randint(0, 64, shape, generator=g) / 64) * 2.0**other).to(dtype)

    a, b, dc = torch.zeros(pairs, k, dtype=dtype), plain(1, n, k), torch.zeros(pairs, n, dtype=dtype)
    p = torch.arange(pairs)
    a[p, (p * 7) % k], dc[p, (p * 5) % n] = small(pairs), small(pairs)
    o = dev([0, pairs])
    want = a.double() @ b[0].double().t()
    assert want.abs().max() < 2.0 ** (low + other + 4) and (want != 0).all()
    assert torch.equal(qr.grouped_mm(a.cuda(), b.cuda(), o, dtype=FP32).cpu().double(), want)
    assert torch.equal(qr.grouped_mm_grad_a(dc.cuda(), b.cuda(), o, dtype=FP32).cpu().double(), dc.double() @ b[0].double())
    dc, x = dc[:1], plain(1, k)  # one pair: one term
    assert torch.equal(qr.grouped_mm_grad_b(dc.cuda(), x.cuda(), dev([0, 1]), dtype=FP32)[0].cpu().double(),
                       dc.double().t() @ x.double())


@pytest.mark.parametrize("pairs", [3, 300])
def test_sums_of_fp16_subnormals(pairs):
    """In a sum the matrix unit aligns an fp16 subnormal as if its exponent were that of the smallest normal number,
    2^-14: the bound of the sum's rounding is that of terms whose factors are at least that large."""
    qr = _qr()
    n, k = 264, 520
    a = (torch.randn(pairs, k, generator=gen(50)) * 2.0**-22).to(FP16)
    b = torch.randn(1, n, k, generator=gen(51)).to(FP16)
    c = qr.grouped_mm(a.cuda(), b.cuda(), dev([0, pairs]), dtype=FP32)
    x, y = a.double(), b[0].double()
    close(c, x @ y.t(), x.abs().clamp_min(2.0**-14) @ y.abs().clamp_min(2.0**-14).t(), k, "c")


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
def test_swiglu_to_four_bits_against_64_bits(dtype):
    """Codes and scales are those of the 64-bit activation, or of one that is off by the 8 units of 2^-24 that the
    fp32 activation may be off by."""
    qr = _qr()
    gu = (torch.randn(300, 512, generator=gen(52)) * 3).to(dtype)
    codes, scales = (t.cpu() for t in qr.swiglu_mxfp4(gu.cuda()))
    g, u, s = swiglu_ref(gu)
    near = [quantize_ref(g * s * u * (1 + d)) for d in (-8 * 2.0**-24 * 1.001, 0, 8 * 2.0**-24 * 1.001)]
    assert ((scales == near[0][1]) | (scales == near[2][1])).all()
    same = (near[0][1] == near[2][1]).repeat_interleave(16, 1)  # blocks of one possible scale
    assert same.float().mean() > 0.99
    for nibble in (lambda c: c & 15, lambda c: c >> 4):
        ok = torch.stack([nibble(codes) == nibble(c) for c, _, _ in near]).any(0)
        assert (ok | ~same).all()


def test_autograd_sees_what_is_written():
    """An output that a graph has saved is refused by that graph once a call has written to it, as torch's own calls
    have it; an output that asks for a gradient itself is refused by the call."""
    qr = _qr()
    a, b, offsets, _, pairs = make_case("ragged", 64, 64, BF16, False, 60)
    a, b, o = a.cuda(), b.cuda(), dev(offsets)
    gu = torch.randn(pairs, 64, generator=gen(61)).to(BF16).cuda()
    dh = gu[:, :32].contiguous()
    codes, scales = qr.mxfp4_quantize(a)
    bc, bs = qr.mxfp4_quantize(b)
    calls = [lambda out: qr.grouped_mm(a, b, o, out=out), lambda out: qr.grouped_mm_grad_a(a, b, o, out=out),
             lambda out: qr.grouped_mm_grad_b(a, a, o, out=out), lambda out: qr.mxfp4_dequantize(codes, scales, out=out),
             lambda out: qr.mxfp4_grouped_mm(codes, scales, bc, bs, o, out=out), lambda out: qr.swiglu(gu, out=out),
             lambda out: qr.swiglu_grad(dh, gu, out=out)]
    shapes = [(pairs, 64), (pairs, 64), (len(offsets) - 1, 64, 64), (pairs, 64), (pairs, 64), (pairs, 32), (pairs, 64)]
    for i, (call, shape) in enumerate(zip(calls, shapes)):
        out = torch.zeros(shape, dtype=BF16, device="cuda")
        w = torch.ones(shape, dtype=BF16, device="cuda", requires_grad=True)
        y = (out * w).sum()
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        with pytest.raises(RuntimeError, match="cannot write to an out"):
            call(w)
        assert (w == 1).all(), i
        with torch.inference_mode():
            assert torch.equal(call(torch.empty(shape, dtype=BF16, device="cuda")), out)
    for call, c, s in ((lambda c, s: qr.mxfp4_quantize(a, c, s), codes, scales),
                       (lambda c, s: qr.swiglu_mxfp4(torch.cat([a, a], 1), c, s), codes, scales)):
        for t in (c, s):
            w = torch.ones(t.shape, device="cuda", requires_grad=True)
            y = (w * t).sum()
            call(c, s)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.backward()
