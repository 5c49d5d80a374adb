"""The operators around the experts' products on the GPU, against plain 64-bit computations: the router with the order
of its pairs and its gradient, and the sum of a token's pairs with its gradients.

Tolerances, relative unless said otherwise.  A router's weights come from 64 bits and are rounded once: 2^-24 (a softmax
that is not renormalised has a sum of exponentials to 2^-31 below it; check_route allows it 2^-19).  The gradient of
such a softmax has fp32 exponentials: e^x is within 2 units of 2^-24 and, its argument being rounded, |x| <= 30 more, a
lane's sum has 16 additions: 2 + 30 + 16 < 2^6 units, 2^-18 of the magnitudes that it adds, and the output's rounding.
Weighted sums are in fp32: a unit for each term and one for the product, of the sum of magnitudes, and the output's
rounding.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, FP16, FP32, FP64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
UNIT = {BF16: 2.0**-8, FP16: 2.0**-11, FP32: 2.0**-24}
TINY = {BF16: 2.0**-130, FP16: 2.0**-25, FP32: 2.0**-149}
ALL = [FP32, BF16, FP16]


def _qr():
    import quantized_routed_moe_amd as qr
    return qr


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------- router
def scores_of(x, score):
    x = x.to(FP64)
    if score == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z > 0, z, 1.0)


def reference(x, k, score="sigmoid", bias=None, groups=1, keep_groups=None, group_best=2, renormalize=True, scale=1.0):
    """(ids, w) in 64 bits, on the host."""
    T, E = x.shape
    s = scores_of(x, score)
    gone = x == -math.inf
    if bias is not None:
        gone = gone | (bias == -math.inf)
        key = s + bias.to(FP64)
    else:
        key = x.to(FP64) + 0.0
    key = torch.where(gone, -math.inf, key)
    if groups > 1:
        g = (key if bias is not None else torch.where(gone, -math.inf, s)).view(T, groups, E // groups)
        best = g.sort(2, descending=True).values[:, :, :group_best]
        total = torch.where(best[:, :, 0] > -math.inf, torch.where(best > -math.inf, best, 0.0).sum(2), -math.inf)
        keep = total.sort(dim=1, descending=True, stable=True).indices[:, : keep_groups or groups]
        mask = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, keep, True)
        key = torch.where(mask.repeat_interleave(E // groups, 1), key, -math.inf)
    value, ids = key.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    there = value > -math.inf
    w = torch.where(there, s.gather(1, ids), 0.0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return torch.where(there, ids, -1).to(torch.int32), w * scale


def order_of(ids, E):
    flat = ids.reshape(-1).long()
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    perm = flat.sort(stable=True).indices
    place = torch.empty_like(perm)
    place[perm] = torch.arange(perm.numel())
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
    return perm, offsets, (perm // max(ids.shape[1], 1)).to(torch.int32), place


def check_order(got, ids, E):
    for name, a, b in zip(("perm", "offsets", "rows", "place"), got, order_of(ids, E)):
        assert a.dtype == b.dtype and torch.equal(a.cpu(), b), name


def check_route(x, k, n=None, **kw):
    """route and Routing.from_logits of host logits against the reference; returns the ids."""
    qr = _qr()
    bias = kw.get("bias")
    want, w = reference(x, k, **kw)
    xs = x.cuda()
    on = dict(kw, bias=None if bias is None else bias.cuda())
    ids, weights = qr.route(xs, k, **on)
    assert ids.dtype == torch.int32 and torch.equal(ids.cpu(), want), f"{int((ids.cpu() != want).any(1).sum())} rows differ"
    dense = kw.get("score") == "softmax" and not kw.get("renormalize", True)
    unit = 2.0**-19 if dense else 2.0**-24 * (1 + 2.0**-20)
    err = (weights.cpu().to(FP64) - w).abs()
    assert weights.dtype == FP32 and bool((err <= unit * w.abs() + 2.0**-149).all()), float((err / w.abs()).nan_to_num().max())
    r = qr.Routing.from_logits(xs, k, **on)
    assert torch.equal(r.ids, ids) and torch.equal(r.w, weights) and r.k == k
    check_order((r.perm, r.offsets, r.rows, r.place), want, x.shape[1])
    return want


def logits(T, E, dtype, seed):
    g = gen(seed)
    return (1.5 * torch.randn(T, E, generator=g) + 0.7 * torch.randn(E, generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("T,E,k", [(1, 256, 6), (1, 1, 1), (5, 8, 8), (67, 60, 4), (130, 64, 8), (65, 100, 3), (64, 128, 1),
                                   (33, 257, 8), (70, 512, 6), (19, 1000, 8), (40, 1024, 5)])
def test_route(dtype, T, E, k):
    bias = 0.3 * torch.randn(E, generator=gen(E))
    for seed, (score, b, renorm, scale) in enumerate([("sigmoid", bias, True, 1.0), ("sigmoid", None, False, 2.5),
                                                      ("softmax", None, True, 1.0), ("softmax", None, False, 1.0),
                                                      ("softmax", bias / E, False, 0.5)]):
        check_route(logits(T, E, dtype, seed), k, score=score, bias=b, renormalize=renorm, scale=scale)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("T,E,k,groups,keep", [(77, 256, 6, 8, 4), (65, 256, 8, 8, 1), (9, 16, 3, 16, 5), (66, 60, 2, 4, 2),
                                               (20, 512, 8, 16, 16), (30, 1024, 8, 8, 3), (12, 6, 4, 2, 2), (31, 96, 5, 3, 2)])
def test_route_groups(dtype, T, E, k, groups, keep):
    bias = 0.2 * torch.randn(E, generator=gen(E))
    for seed, (score, b, best) in enumerate([("sigmoid", bias, 2), ("sigmoid", None, 2), ("softmax", None, 1),
                                             ("softmax", bias / E, 2)]):
        check_route(logits(T, E, dtype, seed), k, score=score, bias=b, groups=groups, keep_groups=keep, group_best=best)


def test_route_many_tokens():
    """More than one pass of a workgroup, and more than one workgroup's chunk of the order."""
    bias = 0.1 * torch.randn(64, generator=gen(0))
    check_route(logits(20011, 64, BF16, 3), 6, bias=bias)
    check_route(logits(33001, 10, FP32, 4), 2, score="softmax", renormalize=False)
    check_route(logits(3001, 320, FP16, 5), 8, bias=0.1 * torch.randn(320, generator=gen(1)), groups=8, keep_groups=3)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties(dtype, score):
    """Few distinct logits: most choices are among equals, with and without a bias that keeps them so."""
    x = torch.randint(-3, 3, (200, 96), generator=gen(7)).to(dtype) / 2
    x[0], x[1], x[2, 5] = 0.0, -0.0, -0.0
    even = torch.full((96,), 0.25)
    steps = torch.randint(0, 3, (96,), generator=gen(8)).float() / 4
    for b in (None, torch.zeros(96), even, steps):
        check_route(x, 8, score=score, bias=b)
        check_route(x, 4, score=score, bias=b, groups=8, keep_groups=2)
        check_route(x, 4, score=score, bias=b, groups=4, keep_groups=3, group_best=1)


def test_route_keys_next_to_each_other():
    """Keys that fp32 cannot tell apart: logits a place apart, and a bias that makes up for a logit's difference."""
    g = gen(9)
    base = torch.randn(300, 1, generator=g)
    x = base.repeat(1, 64)
    for _ in range(2):
        x = torch.where(torch.rand(x.shape, generator=g) < 0.5, torch.nextafter(x, torch.tensor(9.0)), x)
    for b in (None, torch.zeros(64), 3 * torch.ones(64)):
        for score in ("sigmoid", "softmax"):
            check_route(x, 6, score=score, bias=b)
            check_route(x, 6, score=score, bias=b, groups=8, keep_groups=2)
    # keys all within a few units of 0.75: what is left of the score's rounding decides
    x = torch.randn(1, 64, generator=g).repeat(50, 1)
    bias = (0.75 - torch.sigmoid(x[0].double())).float()
    x = x + 1e-7 * torch.randn(50, 64, generator=g)
    check_route(x, 8, bias=bias)
    check_route(x, 8, bias=bias, groups=4, keep_groups=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", [(48, 1), (256, 1), (48, 8), (256, 8)])
def test_route_masked(score, E, groups):
    """Experts that are not there, rows with fewer than top_k of them, rows with none."""
    x = logits(60, E, FP32, 2)
    g = gen(3)
    x[torch.rand(x.shape, generator=g) < 0.5] = -math.inf
    x[:3] = -math.inf
    x[3, : E - 2] = -math.inf
    x[4, 1:] = -math.inf
    bias = torch.randn(E, generator=g)
    bias[::7] = -math.inf
    for b in (None, bias):
        ids = check_route(x, 6, score=score, bias=b, groups=groups, keep_groups=max(1, groups // 2))
        assert (ids[:3] == -1).all() and (ids[3] == -1).any()
        check_route(x, 6, score=score, bias=b, groups=groups, renormalize=False)
    lowest = torch.finfo(FP32).min
    x[x == -math.inf] = lowest  # a mask of the type's lowest value leaves the expert there, with score 0
    check_route(x, 6, score=score, groups=groups, keep_groups=max(1, groups // 2))


def test_route_far_logits():
    x = torch.tensor([[1e4, -1e4, 3.0, 88.0, -88.0, 0.0, 700.0, -700.0]]).repeat(3, 1)
    x[1] = -1e30
    x[2, 0] = 3e38
    for score in ("sigmoid", "softmax"):
        check_route(x, 5, score=score)
        check_route(x, 5, score=score, bias=torch.tensor([0.0, 9.0, -3.0, 0, 1e30, -1e30, 0, 0]))
    # scores below fp32's and below 64 bits' range: weights of 0
    x = torch.full((1, 8), -2000.0)
    ids, w = _qr().route(x.cuda(), 3)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.0, 0.0, 0.0]]


def test_route_not_a_number():
    """NaN ranks behind every number; ids stay distinct and in range."""
    qr = _qr()
    x = logits(40, 64, FP32, 11)
    bad = torch.rand(40, 64, generator=gen(1)) < 0.3
    x[bad] = math.nan
    ids, w = qr.route(x.cuda(), 6)
    assert not bad.gather(1, ids.cpu().long()).any() and not w.isnan().any()
    x[0], x[1, 3:] = math.nan, math.nan
    for kw in (dict(), dict(score="softmax"), dict(bias=torch.zeros(64).cuda()), dict(groups=8, keep_groups=2),
               dict(score="softmax", bias=torch.zeros(64).cuda(), groups=4, keep_groups=4)):
        ids = qr.route(x.cuda(), 6, **kw)[0].cpu()
        assert ((ids >= 0) & (ids < 64)).all() and all(len(set(r)) == 6 for r in ids.tolist())
    bias = torch.zeros(64)
    bias[5] = math.inf
    y = logits(3, 64, FP32, 12)
    assert (qr.route(y.cuda(), 2, bias=bias.cuda())[0][:, 0] == 5).all()


def test_route_strided_rows():
    qr = _qr()
    wide = logits(50, 201, BF16, 6).cuda()
    part = wide[:, 3:103]
    a, b = qr.route(part, 5), qr.route(part.contiguous(), 5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dw = torch.randn(50, 5, generator=gen(1)).cuda()
    out = torch.full((50, 230), 7.0, dtype=BF16, device="cuda")
    qr.route_grad(dw, part, a[0], out=out[:, 30:130])
    assert torch.equal(out[:, 30:130], qr.route_grad(dw, part.contiguous(), a[0]))
    assert (out[:, :30] == 7).all() and (out[:, 130:] == 7).all()
    one = wide[:1, 1:98]
    assert torch.equal(qr.route(one, 2)[0], qr.route(one.clone(), 2)[0])


# ----------------------------------------------------------------- gradient
def grad_reference(dw, x, ids, score, renormalize, scale):
    """(dlogits, the magnitudes it is a difference of) in 64 bits, by autograd of the formula on the chosen."""
    p = scores_of(x, score)
    there = (ids >= 0) & (ids < x.shape[1])
    at, slip = ids.long() * there, torch.zeros_like(dw, dtype=FP64)
    s, G = p.gather(1, at) * there, dw.to(FP64) * scale * there
    if renormalize:
        S = s.sum(1, keepdim=True)
        S = torch.where(S == 0, 1.0, S)
        c = (G * s).sum(1, keepdim=True) / S
        # the difference is formed in 64 bits: off by a few units of 2^-53 of its operands, as the kernel's is
        slip = 2.0**-27 * (G.abs() + (G.abs() * s).sum(1, keepdim=True) / S) / S * there
        G = (G - c) / S * there
    # an expert named several times has the sum of its terms, each rounded before: what that is relative to is the sum
    # of their magnitudes, which may be far above that of the sum
    d, m = torch.zeros_like(p), torch.zeros_like(p)
    for j in range(ids.shape[1]):
        d.scatter_add_(1, at[:, j : j + 1], G[:, j : j + 1])
        m.scatter_add_(1, at[:, j : j + 1], G[:, j : j + 1].abs() + slip[:, j : j + 1])
    if score == "sigmoid":
        rest = scores_of(-x.to(FP64), score)  # 1 - p, which 64 bits lose where p is near 1
        return d * p * rest, m * p * rest
    if renormalize:
        return d * p, m * p
    c = (G * s).sum(1, keepdim=True)
    return d * p - p * c, m * p + (p * c).abs()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 256, 6), (1, 1, 1), (67, 60, 4), (33, 257, 8), (9, 1024, 2), (515, 100, 3)])
def test_route_grad(dtype, score, renorm, T, E, k):
    qr = _qr()
    x = logits(T, E, dtype, T)
    if T > 8:
        x[2], x[3, 1:], x[5] = -math.inf, -math.inf, 40.0
    ids, _ = reference(x, k, score=score)
    if T > 8 and E > 8:
        ids[6, 0], ids[7] = E, 3  # of no expert; the same expert every time
    dw = torch.randn(T, k, generator=gen(1))
    want, mag = grad_reference(dw, x, ids, score, renorm, 1.5)
    got = qr.route_grad(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalize=renorm, scale=1.5)
    assert got.dtype == dtype
    dense = score == "softmax" and not renorm
    tol = UNIT[dtype] * (1 + 2.0**-10) * want.abs() + (2.0**-18 if dense else 2.0**-21) * mag + TINY[dtype]
    err = (got.cpu().to(FP64) - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


def test_route_grad_against_differences():
    """The weights' change along a direction, from 64 bits, is what the gradient says."""
    qr = _qr()
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            x = logits(12, 40, FP32, 5)
            dw = torch.randn(12, 5, generator=gen(2))
            ids, _ = reference(x, 5, score=score)
            d = qr.route_grad(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalize=renorm).cpu().to(FP64)
            step = torch.randn(12, 40, generator=gen(3), dtype=FP64)
            h = 2.0**-12

            def loss(v):
                s = scores_of(v, score).gather(1, ids.long())
                return ((s / s.sum(1, keepdim=True) if renorm else s) * dw.to(FP64)).sum()

            num = (loss(x.to(FP64) + h * step) - loss(x.to(FP64) - h * step)) / (2 * h)
            # the third derivative's part, h^2 / 6 of it, and the fp32 rounding of each entry
            assert abs(float((d * step).sum() - num)) <= 1e-6 * float((d * step).abs().sum()) + h * h * 100


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_from_logits_is_differentiable(score, renorm):
    qr = _qr()
    x = logits(30, 24, FP32, 8)
    leaf = x.cuda().requires_grad_()
    r = qr.Routing.from_logits(leaf, 3, score=score, renormalize=renorm, scale=2.0)
    dw = torch.randn(30, 3, generator=gen(4))
    got, = torch.autograd.grad(r.w, leaf, dw.cuda())
    want, mag = grad_reference(dw, x, r.ids.cpu(), score, renorm, 2.0)
    assert bool(((got.cpu().to(FP64) - want).abs() <= 2.0**-18 * mag + 2.0**-24 * want.abs() + 2.0**-149).all())
    r = qr.Routing.from_logits(leaf, 3, score=score)
    d, = torch.autograd.grad(r.w.square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiated twice"):
        torch.autograd.grad(d.sum(), leaf)


# --------------------------------------------------------------- pair order
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E", [(0, 6, 8), (1, 1, 1), (1, 6, 256), (64, 6, 256), (65, 6, 256), (3, 40, 7), (1000, 6, 1024),
                                   (4099, 3, 1000), (16385, 2, 2), (20000, 8, 128), (50001, 6, 300), (1 << 20, 1, 5)])
def test_sort_pairs(dtype, T, k, E):
    ids = torch.randint(-1, E + 1, (T, k), generator=gen(T), dtype=dtype)  # some of no expert
    check_order(_qr().sort_pairs(ids.cuda(), E), ids, E)


def test_sort_pairs_uneven():
    qr = _qr()
    same = torch.full((5000, 4), 3)
    check_order(qr.sort_pairs(same.cuda(), 9), same, 9)
    none = torch.full((500, 4), -1)
    check_order(qr.sort_pairs(none.cuda(), 9), none, 9)
    far = torch.tensor([[1 << 40, -(1 << 40)], [(1 << 32) + 1, 1]])
    check_order(qr.sort_pairs(far.cuda(), 4), far, 4)
    r = qr.Routing.from_ids(same.cuda(), torch.rand(5000, 4).cuda(), 9)
    check_order(r._tensors(), same, 9)
    byte = torch.randint(0, 9, (50, 2), generator=gen(1), dtype=torch.uint8)
    check_order(qr.Routing.from_ids(byte.cuda(), torch.rand(50, 2).cuda(), 9)._tensors(), byte, 9)


def test_from_ids_past_the_kernels_limits():
    """More experts than the kernels take: torch's own operations, the same order."""
    ids = torch.randint(0, 2000, (300, 3), generator=gen(2))
    check_order(_qr().Routing.from_ids(ids.cuda(), torch.rand(300, 3).cuda(), 2000)._tensors(), ids, 2000)


# ------------------------------------------------------------------ combine
def pairs(T, k, n, dtype, seed, extra=0):
    g = gen(seed)
    y = torch.randn(T * k + extra, n, generator=g).to(dtype)
    place = torch.randperm(T * k + extra, generator=g)[: T * k].view(T, k)
    return y, place, torch.rand(T, k, generator=g) - 0.3


@pytest.mark.parametrize("dtype,out", [(BF16, FP32), (BF16, BF16), (FP16, FP32), (FP16, FP16), (FP32, FP32), (FP32, BF16),
                                       (FP32, FP16)])
@pytest.mark.parametrize("T,k,n", [(1, 6, 4096), (1, 1, 8), (7, 3, 104), (33, 8, 2056), (5, 11, 72), (300, 2, 24), (40, 5, 520),
                                   (3, 4, 65536), (130, 7, 256)])
def test_combine(dtype, out, T, k, n):
    y, place, w = pairs(T, k, n, dtype, n)
    place[0, 0] = -1  # of no pair
    for weights in (w, None):
        f = torch.ones(T, k) if weights is None else weights
        there = (place >= 0)[:, :, None]
        terms = y.to(FP64)[place.clamp_min(0)] * f.to(FP64)[:, :, None] * there
        got = _qr().combine(y.cuda(), place.cuda(), None if weights is None else weights.cuda(), dtype=out)
        assert got.dtype == out and got.shape == (T, n)
        want = terms.sum(1)
        tol = UNIT[out] * (1 + 2.0**-10) * want.abs() + (k + 1) * 2.0**-24 * terms.abs().sum(1) + TINY[out]
        assert bool(((got.cpu().to(FP64) - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype,dd", [(BF16, FP32), (BF16, BF16), (FP16, FP32), (FP16, FP16), (FP32, FP32)])
@pytest.mark.parametrize("T,k,n", [(1, 6, 4096), (1, 1, 8), (7, 3, 104), (33, 8, 2056), (5, 11, 72), (300, 2, 24), (40, 5, 1032),
                                   (2, 17, 1024)])
def test_combine_grad(dtype, dd, T, k, n):
    y, place, w = pairs(T, k, n, dtype, n)
    d = torch.randn(T, n, generator=gen(1)).to(dd)
    for weights in (w, None):
        f = (torch.ones(T, k) if weights is None else weights).to(FP64)
        dy, dw = _qr().combine_grad(d.cuda(), y.cuda(), place.cuda(), None if weights is None else weights.cuda())
        assert dy.dtype == dtype and dw.dtype == FP32
        want = torch.empty(T * k, n, dtype=FP64)
        want[place] = f[:, :, None] * d.to(FP64)[:, None]
        tol = (UNIT[dtype] + 2.0**-24) * (1 + 2.0**-10) * want.abs() + TINY[dtype]
        assert bool(((dy.cpu().to(FP64) - want).abs() <= tol).all())
        terms = y.to(FP64)[place] * d.to(FP64)[:, None]
        err = (dw.cpu().to(FP64) - terms.sum(2)).abs()
        assert bool((err <= n * 2.0**-24 * terms.abs().sum(2) + 2.0**-149).all())


def test_combine_grad_rows_no_pair_names():
    """Rows behind the pairs, and a pair without a place: left as they were, weight gradient 0."""
    qr = _qr()
    y, place, w = pairs(9, 3, 64, BF16, 1, extra=5)
    place[4, 1], place[5, 2] = 9 * 3 + 5, -7
    d = torch.randn(9, 64, generator=gen(2))
    dy = torch.full((32, 64), 3.0, dtype=BF16, device="cuda")
    _, dw = qr.combine_grad(d.cuda(), y.cuda(), place.cuda(), w.cuda(), dy=dy)
    named = torch.zeros(32, dtype=torch.bool)
    named[place[(place >= 0) & (place < 32)]] = True
    assert (dy.cpu()[~named] == 3).all() and not (dy.cpu()[named] == 3).all(1).any()
    assert dw[4, 1] == 0 and dw[5, 2] == 0
    with pytest.raises(ValueError, match="place"):
        qr.combine_grad(d.cuda(), y.cuda(), place.cuda(), w.cuda())


def test_combine_strided_and_special_values():
    qr = _qr()
    wide = torch.randn(12, 200, generator=gen(3)).to(BF16).cuda()
    y, place = wide[:, 16:80], torch.randperm(12, generator=gen(4)).view(6, 2).cuda()
    w = torch.rand(6, 2, generator=gen(5)).cuda()
    out = torch.full((6, 128), 9.0, device="cuda")
    qr.combine(y, place, w, out=out[:, 32:96])
    assert torch.equal(out[:, 32:96], qr.combine(y.contiguous(), place, w))
    assert (out[:, :32] == 9).all() and (out[:, 96:] == 9).all()
    x = y.contiguous()
    x[place[2, 0], 7], x[place[3, 1], 0] = math.nan, math.inf
    got = qr.combine(x, place, w)
    assert got[2, 7].isnan() and got[3, 0] == math.inf
    assert int((~got.isfinite()).sum()) == 2


def test_routing_combine():
    """Kernels and torch's operations say the same; with a graph both gradients are there."""
    qr = _qr()
    ids = torch.stack([torch.randperm(9, generator=gen(i))[:3] for i in range(20)]).cuda()
    w = torch.rand(20, 3, generator=gen(1)).cuda()
    y = torch.randn(60, 48, generator=gen(2)).to(BF16).cuda()
    r = qr.Routing.from_ids(ids, w, 9)
    want = (r.to_tokens(y).double() * w.double()[:, :, None]).sum(1)
    assert (r.combine(y).double() - want).abs().max() <= 2.0**-21 * want.abs().max()
    leaf, wl = y.float().requires_grad_(), w.clone().requires_grad_()
    rg = qr.Routing.from_ids(ids, wl, 9)
    rg.combine(leaf).sum().backward()
    assert leaf.grad is not None and wl.grad is not None
    odd = torch.randn(60, 5, generator=gen(3)).cuda()  # a width the kernel does not take
    assert r.combine(odd).shape == (20, 5)


# ------------------------------------------------- streams, graphs, together
def test_other_stream_and_repeat():
    qr = _qr()
    x = logits(700, 128, BF16, 1).cuda()
    y, place, w = (t.cuda() for t in pairs(700, 4, 256, BF16, 2))
    d = torch.randn(700, 256, generator=gen(3)).cuda()
    bias = 0.1 * torch.randn(128, generator=gen(4)).cuda()
    base = (*qr.route(x, 4, bias=bias), qr.combine(y, place, w), *qr.combine_grad(d, y, place, w))
    grad = qr.route_grad(base[1], x, base[0])
    order = qr.sort_pairs(base[0], 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        got = (*qr.route(x, 4, bias=bias, stream=s), qr.combine(y, place, w, stream=s),
               *qr.combine_grad(d, y, place, w, stream=s))
        got += (qr.route_grad(base[1], x, base[0], stream=s), *qr.sort_pairs(base[0], 128, stream=s))
        s.synchronize()
        for a, b in zip(got, (*base, grad, *order)):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    """The router, the products' order and the sum in one graph, on new inputs each replay."""
    qr = _qr()
    g = gen(5)
    x = torch.randn(500, 64, generator=g).cuda()
    bank_in = torch.randn(500 * 4, 64, generator=g).to(BF16).cuda()
    dout = torch.randn(500, 64, generator=g).cuda()

    def step():
        r = qr.Routing.from_logits(x, 4)
        out = qr.combine(bank_in, r.place.view(500, 4), r.w)
        dy, dw = qr.combine_grad(dout, bank_in, r.place.view(500, 4), r.w)
        return r.ids, r.w, r.perm, r.offsets, r.rows, out, dy, dw, qr.route_grad(dw, x, r.ids)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(500, 64, generator=g))
        bank_in.copy_(torch.randn(500 * 4, 64, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Two calls at once have workspaces of their own."""
    qr = _qr()
    xs = [logits(30000, 64, FP32, i).cuda() for i in range(2)]
    want = [qr.Routing.from_logits(x, 6) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(qr.Routing.from_logits(x, 6))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.ids, b.ids) and torch.equal(a.perm, b.perm) and torch.equal(a.offsets, b.offsets)


def test_nothing_to_do():
    qr = _qr()
    ids, w = qr.route(torch.empty(0, 16).cuda(), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    r = qr.Routing.from_logits(torch.empty(0, 16).cuda(), 3)
    assert r.offsets.tolist() == [0] * 17 and r.perm.numel() == 0
    assert qr.route_grad(w, torch.empty(0, 16).cuda(), ids).shape == (0, 16)
    place = torch.empty(0, 3, dtype=torch.int64).cuda()
    assert qr.combine(torch.empty(0, 8).cuda(), place, w).shape == (0, 8)
    dy, dw = qr.combine_grad(torch.empty(0, 8).cuda(), torch.empty(0, 8).cuda(), place, w)
    assert dy.shape == (0, 8) and dw.shape == (0, 3)
    none = torch.full((4, 3), -1).cuda()
    assert (qr.combine(torch.empty(0, 8).cuda(), none, torch.rand(4, 3).cuda()) == 0).all()


def test_largest_calls():
    """As many pairs as there may be: of one expert a token and of eight, of four experts and of 1024."""
    qr = _qr()
    P = 1 << 20
    for T, k, E, dtype in ((P, 1, 4, FP32), (P // 8, 8, 1024, BF16)):
        g = torch.Generator(device="cuda").manual_seed(k)
        x = torch.randn(T, E, generator=g, device="cuda").to(dtype)
        r = qr.Routing.from_logits(x, k)
        # equal logits: the lower expert first, as a stable sort has it
        want = torch.cat([c.sort(dim=1, descending=True, stable=True).indices[:, :k] for c in x.split(1 << 14)])
        assert torch.equal(r.ids.long(), want)
        del want
        flat = r.ids.reshape(-1).long()
        perm = flat.sort(stable=True).indices
        assert torch.equal(r.perm, perm) and torch.equal(r.rows.long(), perm // k)
        assert torch.equal(r.place[perm], torch.arange(P, device="cuda"))
        assert torch.equal(r.offsets[1:].long(), torch.bincount(flat, minlength=E).cumsum(0))
        y = torch.randn(P, 8, generator=g, device="cuda")
        w = r.w
        terms = w.to(FP64)[:, :, None] * y.to(FP64)[r.place.view(T, k)]
        got = qr.combine(y, r.place.view(T, k), w).to(FP64)
        assert bool(((got - terms.sum(1)).abs() <= (k + 1) * 2.0**-24 * terms.abs().sum(1) + 2.0**-149).all())
        d = torch.randn(T, 8, generator=g, device="cuda")
        dy, dw = qr.combine_grad(d, y, r.place.view(T, k), w)
        assert torch.equal(dy[r.place].view(T, k, 8), w[:, :, None] * d[:, None])
        mags = y.to(FP64)[r.place.view(T, k)] * d.to(FP64)[:, None]
        assert bool(((dw.to(FP64) - mags.sum(2)).abs() <= 12 * 2.0**-24 * mags.abs().sum(2) + 2.0**-149).all())
    with pytest.raises(ValueError, match="pairs"):
        qr.sort_pairs(torch.zeros(P // 8 + 1, 8, dtype=torch.int32, device="cuda"), 1024)
    with pytest.raises(qr.MoEError):
        qr.route(torch.zeros(P + 1, 4, device="cuda"), 1)


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_layer_from_logits_to_gradients(dtype):
    """Router, experts and sum together, differentiated to the router's logits, against 64-bit autograd.  At most
    eight 16-bit roundings in a row, as in the experts alone, the router's part being in fp32."""
    qr = _qr()
    T, E, k, H, F = 40, 12, 3, 64, 48
    g = gen(6)
    router = torch.randn(E, H, generator=g) / H**0.5
    x = torch.randn(T, H, generator=g).to(dtype)
    gate_up = (torch.randn(E, 2 * F, H, generator=g) / H**0.5).to(dtype)
    down = (torch.randn(E, H, F, generator=g) / F**0.5).to(dtype)
    dout = torch.randn(T, H, generator=g)
    leaves = [t.to(FP64).requires_grad_() for t in (router, x, gate_up, down)]
    lo = leaves[1].detach() @ leaves[0].t()
    lo32 = lo.float()
    ids, _ = reference(lo32.detach(), k, groups=4, keep_groups=2)
    s = torch.sigmoid(lo).gather(1, ids.long())
    w = 1.5 * s / s.sum(1, keepdim=True)
    y = []
    for t in range(T):
        acc = 0
        for j in range(k):
            gu = leaves[2][ids[t, j]] @ leaves[1][t]
            acc = acc + w[t, j] * (leaves[3][ids[t, j]] @ (torch.nn.functional.silu(gu[:F]) * gu[F:]))
        y.append(acc)
    want = torch.stack(y)
    grads = torch.autograd.grad(want, leaves, dout.to(FP64))
    rr, xx, gg, dd = [t.cuda().requires_grad_() for t in (router, x, gate_up, down)]
    logit = lo32.detach().cuda() + (xx.detach().float() @ rr.t() - (xx.detach().float() @ rr.t()).detach())
    r = qr.Routing.from_logits(logit, k, groups=4, keep_groups=2, scale=1.5)
    assert torch.equal(r.ids.cpu(), ids)
    out = qr.expert_ffn(xx, r, gg, dd)
    out.backward(dout.cuda())
    tol = 8 * UNIT[dtype]
    for got, ref in zip((out, rr.grad, xx.grad, gg.grad, dd.grad), (want.detach(), *grads)):
        assert float((got.detach().cpu().to(FP64) - ref).norm() / ref.norm()) <= tol


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_a_training_step(dtype):
    """Router, experts, their gradients and the banks' orthogonalised updates, with padding (tokens without experts) and
    tokens that fewer experts than top_k are left to; then captured and replayed on new inputs."""
    qr = _qr()
    T, E, k, H, F = 50, 8, 3, 64, 40
    g = gen(8)

    def inputs():
        lo = torch.randn(T, E, generator=g)
        lo[:4] = -math.inf
        lo[4:7, 1:] = -math.inf
        return lo, torch.randn(T, H, generator=g).to(dtype)

    lo, x = inputs()
    gate_up = (torch.randn(E, 2 * F, H, generator=g) / H**0.5).to(dtype)
    down = (torch.randn(E, H, F, generator=g) / F**0.5).to(dtype)
    dout = torch.randn(T, H, generator=g)
    statics = [t.cuda() for t in (lo, x, gate_up, down)]
    d = dout.cuda()

    def step():
        leaves = [t.detach().requires_grad_() for t in statics]
        r = qr.Routing.from_logits(leaves[0], k, "softmax", scale=1.5)
        out = qr.expert_ffn(leaves[1], r, *leaves[2:])
        grads = torch.autograd.grad(out, leaves, d)
        return (r.ids, out.detach(), *grads, *(qr.orthogonalize(b) for b in grads[2:]))

    ids, out, *grads, up_gu, up_d = (t.cpu() for t in step())
    want_ids, _ = reference(lo, k, score="softmax")
    assert torch.equal(ids, want_ids) and (ids[:4] == -1).all() and (ids[4:7, 1:] == -1).all()
    leaves = [t.to(FP64).requires_grad_() for t in (lo, x, gate_up, down)]
    p = leaves[0].exp()
    rows = []
    for t in range(T):
        mine = [int(e) for e in ids[t] if e >= 0]
        acc = 0 * leaves[1][t]
        for e in mine:
            gu = leaves[2][e] @ leaves[1][t]
            y = leaves[3][e] @ (torch.nn.functional.silu(gu[:F]) * gu[F:])
            acc = acc + 1.5 * p[t, e] / sum(p[t, i] for i in mine) * y
        rows.append(acc)
    want = torch.stack(rows)
    ref = torch.autograd.grad(want, leaves, dout.to(FP64))
    assert (out[:4] == 0).all() and (grads[0][:7] == 0).all() and (grads[1][:4] == 0).all()
    for a, b in zip((out, *grads), (want.detach(), *ref)):
        assert float((a.to(FP64) - b).norm() / b.norm()) <= 8 * UNIT[dtype]
    for update, grad in ((up_gu, grads[2]), (up_d, grads[3])):
        for a, b in zip(update, newton_schulz(grad)):
            assert float((a.to(FP64) - b).norm()) <= orthogonal_bound(b, dtype, depth=80)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        res = step()
    for i in range(3):
        for t, new in zip(statics, inputs()):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in res]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), i


# ------------------------------------------------------ orthogonalised update
QUINTIC = (3.4445, -4.7750, 2.0315)


def newton_schulz(g, steps=5, coefficients=QUINTIC, eps=1e-7):
    """64 bits, on the host."""
    each = [coefficients] * steps if not isinstance(coefficients[0], tuple) else coefficients
    x = g.to(FP64)
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-2, -1) if tall else x
    for a, b, c in each:
        aa = x @ x.transpose(-2, -1)
        x = a * x + (b * aa + c * (aa @ aa)) @ x
    return x.transpose(-2, -1) if tall else x


def orthogonal_bound(want, dtype, steps=5, growth=3.4445, depth=1):
    """What the output may be off by, as a norm.  Every number between the products is off by 2^-22 of itself (or
    2^-39, where the scale ends), a product's sum by as much again (its terms' lo lo part, and fp32 additions, whose
    errors are independent of each other: sqrt(depth) 2^-24, 2^-18 at most for 4096 terms).  A step's P and X pass
    on what they get multiplied by at most `growth` and add three such errors of a matrix of |X| <= |want|:
    the last step's weigh 1, those of the one before `growth` of what X was then, which was that much smaller where
    it grew (singular values that have stopped growing are multiplied by at most 1.6, the derivative of the quintic
    on [0.7, 1.2]).  So 3 * steps * 1.6^4 * (2^-22 + sqrt(depth) 2^-24), and the output's rounding.  Of a matrix so
    small beside eps that its numbers fall below the scale's end, 2^-39 for each of X's elements and steps is left, times
    the growth of the steps after it: nothing but for results that are as small themselves."""
    floor = 2.0**-39 * steps * growth**steps * want.numel() ** 0.5
    return (3 * steps * 1.6**4 * (2.0**-22 + depth**0.5 * 2.0**-24) + UNIT[dtype]) * float(want.norm()) + floor


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (2, 3, 5), (33, 31), (64, 64), (5, 40, 130), (130, 40), (100, 257),
                                   (3, 2, 65, 129), (300, 520), (2, 513, 260), (129, 1000), (700, 700)])
def test_orthogonalize(dtype, shape):
    g = (torch.randn(shape, generator=gen(sum(shape))) * 1e-3).to(dtype)
    want = newton_schulz(g)
    got = _qr().orthogonalize(g.cuda())
    assert got.dtype == dtype and got.shape == g.shape
    got, want = got.cpu().to(FP64).reshape(-1, *shape[-2:]), want.reshape(-1, *shape[-2:])
    for a, b in zip(got, want):
        err, tol = float((a - b).norm()), orthogonal_bound(b, dtype, depth=max(shape[-2:]))
        assert err <= tol, (err / float(b.norm()), tol / float(b.norm()))


def test_orthogonalize_one_product():
    """X' = c0 X keeps X: each of the three roundings to 22 bits (of X, of the identity, of the product) is within 2^-22,
    and 2^-39 where the scale ends."""
    for shape in ((300, 300), (1000, 519), (64, 2000)):
        g = torch.randn(shape, generator=gen(1))
        got = _qr().orthogonalize(g.cuda(), steps=1, coefficients=(1.0, 0.0, 0.0)).cpu().to(FP64)
        want = g.to(FP64) / (g.to(FP64).norm() + 1e-7)
        assert bool(((got - want).abs() <= 3.1 * 2.0**-22 * want.abs() + 2.0**-37).all())


@pytest.mark.parametrize("rows,cols", [(200, 200), (519, 1000), (96, 3000), (700, 900)])
@pytest.mark.parametrize("coefficients", [(0.0, 1.0, 0.0), (1.5, -0.5, 0.0)])
def test_orthogonalize_two_products(rows, cols, coefficients):
    """Products of positive terms, where errors cannot hide behind a sum that cancels: a first step's A, P and X are off
    by 2^-22 for each of the two roundings of every operand (six), and by the fp32 sum's additions, of which no term
    meets more than one for each 16 elements of three products, twice: 2^-24 each at most."""
    g = torch.rand(rows, cols, generator=gen(2)) + 0.1
    want = newton_schulz(g, 1, coefficients)
    got = _qr().orthogonalize(g.cuda(), steps=1, coefficients=coefficients).cpu().to(FP64)
    x = g.to(FP64) / g.to(FP64).norm()
    a, b, _ = (abs(c) for c in coefficients)
    m = x if rows <= cols else x.t()
    mag = a * m + b * (m @ m.t()) @ m
    n = 3 * (rows + cols) / 16
    tol = (6 * 2.0**-22 + n * 2.0**-24) * (mag if rows <= cols else mag.t())
    assert bool(((got - want).abs() <= tol + 2.0**-37).all())


def test_orthogonalize_batches_and_steps():
    """Every way of cutting tiles: whole rounds and a tail, parts of one matrix; each number of steps."""
    qr = _qr()
    g = torch.randn(7, 600, 900, generator=gen(3)).to(BF16)
    one = [qr.orthogonalize(m.cuda()).cpu() for m in g]
    want = newton_schulz(g)
    got = qr.orthogonalize(g.cuda()).cpu()
    for a, b, w in zip(got, one, want):
        tol = orthogonal_bound(w, BF16, depth=900)
        assert float((a.to(FP64) - w).norm()) <= tol and float((b.to(FP64) - w).norm()) <= tol
    for steps in range(1, 9):
        x = torch.randn(2, 70, 150, generator=gen(steps))
        y = qr.orthogonalize(x.cuda(), steps=steps).cpu().to(FP64)
        for a, w in zip(y, newton_schulz(x, steps)):
            assert float((a - w).norm()) <= orthogonal_bound(w, FP32, steps, depth=150)
    each = [(3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]
    x = torch.randn(90, 260, generator=gen(4))
    y = qr.orthogonalize(x.cuda(), steps=3, coefficients=each).cpu().to(FP64)
    w = newton_schulz(x, 3, each)
    assert float((y - w).norm()) <= orthogonal_bound(w, FP32, 3, depth=260)
    many = torch.randn(300, 20, 33, generator=gen(5)).to(FP16)
    y, w = qr.orthogonalize(many.cuda()).cpu().to(FP64), newton_schulz(many)
    assert all(float((a - b).norm()) <= orthogonal_bound(b, FP16, depth=33) for a, b in zip(y, w))


def test_orthogonalize_large():
    """Tiles of 256 x 256, several rounds of them, both orders, against 64 bits on the GPU."""
    qr = _qr()
    for shape in ((6, 2048, 1024), (9, 1024, 2048), (5, 1792, 1800)):
        g = torch.randn(shape, generator=gen(6)).to(BF16).cuda()
        got = qr.orthogonalize(g)
        for a, b in zip(got, g):
            w = newton_schulz(b)
            assert float((a.to(FP64) - w).norm()) <= orthogonal_bound(w, BF16, depth=2048)
        again = qr.orthogonalize(g)
        assert torch.equal(got, again)


def test_orthogonalize_special_matrices():
    qr = _qr()
    g = torch.randn(6, 40, 70, generator=gen(7))
    g[0] = 0
    g[1, 3, 4], g[2, 0, 0] = math.nan, math.inf
    g[3] *= 1e30
    g[4] *= 1e-30
    got = qr.orthogonalize(g.cuda()).cpu()
    assert (got[0] == 0).all() and got[1].isnan().all() and got[2].isnan().all()
    want = newton_schulz(g[3:])
    for a, w in zip(got[3:], want):
        assert float((a.to(FP64) - w).norm()) <= orthogonal_bound(w, FP32, depth=70)
    # no eps: a matrix of zeros still gives zeros, a tiny one its singular vectors
    tiny = g[5:6] * 1e-38
    got = qr.orthogonalize(torch.cat([g[:1], tiny]).cuda(), eps=0.0).cpu()
    w = newton_schulz(tiny[0], eps=0.0)
    assert (got[0] == 0).all() and float((got[1].to(FP64) - w).norm()) <= orthogonal_bound(w, FP32, depth=70)
    # one direction only: the others stay nothing
    u, v = torch.randn(50, 1, generator=gen(8)), torch.randn(1, 90, generator=gen(9))
    got, w = qr.orthogonalize((u @ v).cuda()).cpu().to(FP64), newton_schulz(u @ v)
    # fp32's own rounding of u v is the other directions' content, which grows 3.4445 a step in both alike; so does the
    # 2^-22 that the first products add to it: 3.4445^4 of it at most
    assert float((got - w).norm()) <= 141 * 2.0**-22 * 6 * float(w.norm())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rank,rest", [(1, 1e-2), (1, 1e-4), (4, 1e-3), (32, 1e-4), (0, 0.0)])
def test_orthogonalize_few_directions(dtype, rank, rest):
    """A few singular values far above the others (rank 0: 1 / k^2), as momenta have.  Six roundings of 2^-22 of the
    first step's products put what the largest direction has into the others, which grow 3.4445 a step: 6 2^-22
    3.4445^4 of the norm, as far as they go.  Where two further steps are taken on squares (16-bit results), what those
    have lost grows by 3.4445^2 a step and goes through the derivative of P, at most 4.775: 6 2^-22 4.775 3.4445^4
    more.  Then the output's rounding."""
    m, n = 300, 520
    g = gen(rank)
    u = torch.linalg.qr(torch.randn(m, m, generator=g, dtype=FP64))[0]
    v = torch.linalg.qr(torch.randn(n, m, generator=g, dtype=FP64))[0]
    k = torch.arange(m, dtype=FP64)
    x = ((u * (torch.where(k < rank, 1.0, rest) if rank else 1 / (k + 1) ** 2)) @ v.t()).to(dtype)
    want = newton_schulz(x)
    got = _qr().orthogonalize(x.cuda()).cpu().to(FP64)
    grown = 6 * 2.0**-22 * 3.4445**4
    tol = UNIT[dtype] + grown * (1 if dtype is FP32 else 1 + 4.775)
    assert float((got - want).norm()) <= tol * float(want.norm())


def test_orthogonalize_steep_steps():
    """Steps that let small singular values grow faster, 6 and then 3.75 a step: as above, with what steps on squares lose
    held to an eighth of the output's rounding each for the six."""
    each = [(6.0, -14.0, 9.0)] + [(3.75, -3.418, 0.858)] * 4  # 1.6 at most
    m, n = 200, 420
    g = gen(12)
    u = torch.linalg.qr(torch.randn(m, m, generator=g, dtype=FP64))[0]
    v = torch.linalg.qr(torch.randn(n, m, generator=g, dtype=FP64))[0]
    s = torch.full((m,), 1e-4, dtype=FP64)
    s[0] = 1
    for dtype in ALL:
        x = ((u * s) @ v.t()).to(dtype)
        want = newton_schulz(x, 5, each)
        got = _qr().orthogonalize(x.cuda(), steps=5, coefficients=each).cpu().to(FP64)
        tol = (1 + 6 / 8) * UNIT[dtype] + 6 * 2.0**-22 * 6 * 3.75**3
        assert float((got - want).norm()) <= tol * float(want.norm()), dtype


def test_orthogonalize_extreme_shapes():
    """More matrices than a launch takes; the longest rows; a single row; a large square."""
    qr = _qr()
    for shape, dtype in (((66000, 2, 3), FP32), ((2, 65536, 24), BF16), ((24, 65536), FP16), ((1, 65536), FP32),
                         ((3, 4100, 1030), BF16)):
        g = torch.randn(shape, generator=gen(shape[-1])).to(dtype).cuda()
        want = newton_schulz(g)
        got = qr.orthogonalize(g)
        err = (got.to(FP64) - want).flatten(-2).norm(dim=-1).reshape(-1)
        size = want.flatten(-2).norm(dim=-1).reshape(-1)
        one = orthogonal_bound(torch.ones(1, dtype=FP64), dtype, depth=max(shape[-2:])) + 2.0**-22
        assert bool((err <= one * size).all()), (shape, float((err / size).max()))


def test_orthogonalize_in_place_streams_and_graphs():
    qr = _qr()
    g = torch.randn(3, 100, 300, generator=gen(10)).cuda()
    want = qr.orthogonalize(g)
    out = torch.empty_like(g)
    assert qr.orthogonalize(g, out=out) is out and torch.equal(out, want)
    same = g.clone()
    qr.orthogonalize(same, out=same)
    assert torch.equal(same, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = qr.orthogonalize(g, stream=s)
    s.synchronize()
    assert torch.equal(x, want)
    static = g.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        res = qr.orthogonalize(static)
    for i in range(3):
        static.copy_(torch.randn(3, 100, 300, generator=gen(20 + i)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, qr.orthogonalize(static)), i
    odd = torch.randn(1 + 3 * 35 * 41, generator=gen(11)).to(BF16).cuda()[1:].view(3, 35, 41)  # aligned to an element only
    assert torch.equal(qr.orthogonalize(odd), qr.orthogonalize(odd.clone()))
    assert qr.orthogonalize(torch.empty(0, 4, 5).cuda()).shape == (0, 4, 5)


# ------------------------------------------------ where the choice is close
def check_alone(x, k, **kw):
    """What a token gets does not depend on the tokens beside it."""
    qr = _qr()
    on = {n: v.cuda() if torch.is_tensor(v) else v for n, v in kw.items()}
    ids, w = qr.route(x.cuda(), k, **on)
    for t in range(x.shape[0]):
        one, ow = qr.route(x[t : t + 1].cuda(), k, **on)
        assert torch.equal(one[0], ids[t]) and torch.equal(ow[0].nan_to_num(), w[t].nan_to_num()), t
    return ids.cpu()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("even", [0.5, -0.5, 0.0])
def test_route_groups_beside_a_token_that_ties(score, even):
    """A token whose groups are far apart is settled in fp32, whatever the tokens of the same wave need."""
    gone, small = -math.inf, math.log(0.2)
    x = torch.tensor([[0.0, 0.0, 0.0, 0.0], [0.0, gone, small, small], [0.0, gone, -0.1, -0.1], [gone, gone, 1.0, -3.0],
                      [-8.0, -9.0, gone, 2.0], [gone] * 4, [1.0, 2.0, 1.0, 2.0]])
    bias = torch.full((4,), even)
    check_route(x, 2, score=score, bias=bias, groups=2, keep_groups=1)
    check_alone(x, 2, score=score, bias=bias, groups=2, keep_groups=1)
    g = gen(21)
    x = torch.randn(64, 32, generator=g).repeat(2, 1)
    x[torch.rand(x.shape, generator=g) < 0.6] = gone
    x[::3] = 0.25  # ties throughout
    check_route(x, 4, score=score, bias=torch.full((32,), even), groups=8, keep_groups=3)


def test_route_groups_with_a_nan_beside_a_token_that_ties():
    """A group of a number and a NaN is behind one of two numbers, beside a tie too."""
    x = torch.tensor([[0.0, 0.0, 0.0, 0.0], [5.0, math.nan, -1.0, -1.0], [-1.0, -2.0, math.nan, 7.0]])
    for kw in (dict(), dict(bias=torch.zeros(4)), dict(bias=torch.tensor([0.0, 0.25, 0.0, 0.25]))):
        ids = check_alone(x, 2, groups=2, keep_groups=1, **kw)
        assert sorted(ids[1].tolist()) == [2, 3] and sorted(ids[2].tolist()) == [0, 1]


@pytest.mark.parametrize("dtype", ALL)
def test_route_groups_of_unlike_counts_that_almost_tie(dtype):
    """Softmax and one bias for all: a group with one expert left counts the bias once, one with two counts it twice.
    The bias is put where the scores meet, and the numbers next to that on both sides."""
    x = torch.tensor([[0.0, -math.inf, -1.0, -1.25], [0.0, -math.inf, -0.5, -0.25], [-math.inf, 0.5, 0.25, 0.25]]).to(dtype)
    for row in x:
        p = scores_of(row[None], "softmax")[0]
        meet = (p[:2].sum() - p[2:].sum()).float()
        for b in (meet, torch.nextafter(meet, torch.tensor(9.0)), torch.nextafter(meet, torch.tensor(-9.0)), 2 * meet,
                  meet / 2, -meet):
            bias = b.expand(4).clone()
            check_route(x, 1, score="softmax", bias=bias, groups=2, keep_groups=1)
            check_alone(x, 1, score="softmax", bias=bias, groups=2, keep_groups=1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_groups_with_a_large_even_bias(score):
    """One bias for all, beside which the scores vanish even in 64 bits: it decides between groups that count it once and
    twice, and between others their scores do."""
    qr = _qr()
    x = torch.tensor([[0.1, 0.2, 0.3, 0.2, 1.0, -math.inf, 0.2, 0.1], [0.1, 0.2, 0.3, 0.2, 0.2, 0.2, 0.2, 0.1]]).cuda()
    for even, best, two in ((1e17, [2, 3], [2, 1, 3]), (-1e17, [4, -1], [4, 2, 3])):
        bias = torch.full((8,), even).cuda()
        assert qr.route(x[:1], 2, score=score, bias=bias, groups=4, keep_groups=1)[0].tolist() == [best]
        assert qr.route(x[:1], 3, score=score, bias=bias, groups=4, keep_groups=2)[0].tolist() == [two]
        assert qr.route(x[1:], 4, score=score, bias=bias, groups=4, keep_groups=2)[0].tolist() == [[2, 3, 4, 5]]
        check_alone(x.cpu(), 2, score=score, bias=bias.cpu(), groups=4, keep_groups=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_groups_of_lowest_keys(score):
    """Two keys whose sum is past fp32: the group is there all the same, and its sum counts."""
    lowest = torch.finfo(FP32).min
    x = torch.zeros(3, 8)
    x[:, :2] = -math.inf
    x[1] += torch.arange(8)
    bias = torch.tensor([0, 0, lowest, lowest, -2e38, -2e38, -3e38, -3e38])
    for keep, kept in ((1, {4, 5}), (2, {4, 5, 6, 7}), (3, {2, 3, 4, 5, 6, 7})):
        ids = check_route(x, 2 * keep if keep < 3 else 6, score=score, bias=bias, groups=4, keep_groups=keep)
        assert set(ids[0].tolist()) == kept
    far = torch.tensor([1e38, 1e38, 3e38, 2e38, 3e38, 1e38, 3e38, 3e38])  # and past it above
    check_route(x, 2, score=score, bias=far, groups=4, keep_groups=1)
    x[2, 2:] = math.nan  # a NaN is behind every number and before what is not there
    for b in (None, bias):
        ids = check_alone(x[2:], 2, score=score, groups=4, keep_groups=1, **({} if b is None else {"bias": b}))
        assert (ids >= 2).all()


@pytest.mark.parametrize("E", [256, 512, 1024])
@pytest.mark.parametrize("v", [-5.7663784, -16.6443996, -16.75])
def test_route_softmax_of_many_small_terms(E, v):
    """One logit of 0, the others so far below that each is lost, in part or whole, when it is added to a running fp32
    sum: the weights are to fp32 rounding all the same, and the choice is that of real numbers where the bias puts the
    others just ahead, or just behind."""
    x = torch.full((3, E), v)
    x[:, 0] = 0
    x[1, 3], x[2, E - 1] = -1.0, -0.5
    want, w = reference(x, 4, score="softmax", renormalize=False)
    ids, got = _qr().route(x.cuda(), 4, score="softmax", renormalize=False)
    assert torch.equal(ids.cpu(), want)
    # 64 bits but for the exponentials' polynomial (2^-30) and one rounding
    assert bool(((got.cpu().to(FP64) - w).abs() <= 2.0**-24 * (1 + 2.0**-5) * w).all())
    p = scores_of(x[:1], "softmax")[0]
    meet = (p[0] - p[1]).float()
    for b in (meet, torch.nextafter(meet, torch.tensor(9.0)), torch.nextafter(meet, torch.tensor(-9.0))):
        bias = b.expand(E).clone()
        bias[0] = 0
        check_route(x, 2, score="softmax", bias=bias)
        check_route(x, 1, score="softmax", bias=bias, groups=4, keep_groups=2)
        check_route(x, 8, score="softmax", bias=bias, renormalize=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_of_chosen_experts_that_are_not_there(score, renorm):
    """Ids that name experts of logit -inf: their scores are 0, and so are the gradients."""
    x = logits(6, 20, FP32, 3)
    x[0], x[1, 4:], x[2, :3] = -math.inf, -math.inf, -math.inf
    ids = torch.tensor([[0, 1, 2], [5, 6, 7], [0, 1, 2], [2, 1, 0], [-1, 20, -1], [3, 3, 3]], dtype=torch.int32)
    dw = torch.randn(6, 3, generator=gen(2))
    want, mag = grad_reference(dw, x, ids, score, renorm, 1.0)
    got = _qr().route_grad(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalize=renorm).cpu().to(FP64)
    assert (got[0] == 0).all() and (renorm is False or (got[1:3] == 0).all())
    assert bool(((got - want).abs() <= 2.0**-24 * want.abs() + 2.0**-18 * mag + 2.0**-149).all())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("E,k", [(8, 1), (60, 3), (256, 1), (256, 8), (700, 4)])
def test_route_grad_of_a_confident_token(dtype, E, k):
    """A softmax's gradient at the chosen is p_j sum_e (G_j - G_e) p_e, to a relative error, however near p_j is to 1:
    p (G - sum G p) would lose it.  An exponential's is two units of 2^-24 and its argument's, |x| <= 30, more; the sum
    of a lane's sixteen and of lanes is in 64 bits or shorter than that: 2^-18.  Then the output's rounding."""
    qr = _qr()
    x = 0.25 * torch.randn(8, E, generator=gen(E))
    x[torch.arange(8), torch.arange(8) % E] += torch.tensor([0.0, 4, 8, 12, 16, 20, 24, 28])
    x = x.to(dtype)
    ids, _ = reference(x, k, score="softmax")
    dw = torch.randn(8, k, generator=gen(1))
    p = scores_of(x, "softmax")
    G = torch.zeros(8, E, dtype=FP64).scatter_(1, ids.long(), 1.5 * dw.to(FP64))
    terms = p[:, :, None] * (G[:, :, None] - G[:, None, :]) * p[:, None, :]
    want, mag = terms.sum(2), terms.abs().sum(2)
    got = qr.route_grad(dw.cuda(), x.cuda(), ids.cuda(), score="softmax", renormalize=False, scale=1.5).cpu().to(FP64)
    err = (got - want).abs()
    tol = UNIT[dtype] * (1 + 2.0**-10) * want.abs() + 2.0**-18 * mag + TINY[dtype]
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [1, 2, 8])
def test_route_grad_where_one_of_the_chosen_has_all_the_weight(dtype, score, k):
    """Renormalised, a weight's gradient is q_j sum_i (G_j - G_i) q_i over the chosen, to a relative error of 64 bits,
    however near a q is to 1, and the output's rounding."""
    qr = _qr()
    x = 0.25 * torch.randn(9, 40, generator=gen(k)) - (60 if score == "sigmoid" else 0)
    x[torch.arange(9), torch.arange(9)] += torch.tensor([0.0, 4, 8, 16, 20, 28, 36, 44, 52])
    x = x.to(dtype)
    ids, _ = reference(x, k, score=score)
    dw = torch.randn(9, k, generator=gen(1))
    s = scores_of(x, score).gather(1, ids.long())
    q, G = s / s.sum(1, keepdim=True), 1.5 * dw.to(FP64)
    terms = q[:, :, None] * (G[:, :, None] - G[:, None, :]) * q[:, None, :]
    if score == "sigmoid":
        terms = terms * scores_of(-x.to(FP64), score).gather(1, ids.long())[:, :, None]
    want, mag = (torch.zeros(9, 40, dtype=FP64).scatter_(1, ids.long(), v) for v in (terms.sum(2), terms.abs().sum(2)))
    got = qr.route_grad(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalize=True, scale=1.5).cpu().to(FP64)
    tol = UNIT[dtype] * (1 + 2.0**-10) * want.abs() + 2.0**-24 * (want != 0) * mag + TINY[dtype]
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol.clamp_min(1e-300)).max())
    # scores at the end of what 64 bits hold
    x = -709.0 - torch.arange(40.0)[None] / 2 if score == "sigmoid" else 1000 * torch.randn(1, 40, generator=gen(2))
    ids = torch.arange(k, dtype=torch.int32)[None]
    assert qr.route_grad(dw[:1].cuda(), x.cuda(), ids.cuda(), score=score, renormalize=True).isfinite().all()


def test_combine_of_more_than_one_launch():
    """As many tokens as there may be of rows so long that their threads pass 2^32; exact: one pair a token, weights that
    are powers of two."""
    qr = _qr()
    T, n = 1 << 20, 30736
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randn(5, n, generator=g, device="cuda").to(BF16)
    place = torch.randint(0, 5, (T, 1), generator=g, device="cuda")
    w = 2.0 ** torch.randint(-2, 3, (T, 1), generator=g, device="cuda")
    out = qr.combine(y, place, w, dtype=BF16)
    for t in range(0, T, 1 << 14):
        assert torch.equal(out[t : t + (1 << 14)], y[place[t : t + (1 << 14), 0]] * w[t : t + (1 << 14)].to(BF16)), t
    del out
    torch.cuda.empty_cache()


def test_routing_combine_gradients():
    """Through Routing.combine, in y and in w, against 64 bits; pairs of no expert among them."""
    qr = _qr()
    ids = torch.stack([torch.randperm(9, generator=gen(i))[:3] for i in range(20)])
    ids[3, 1] = -1
    w, y = torch.rand(20, 3, generator=gen(1)), torch.randn(60, 48, generator=gen(2))
    d = torch.randn(20, 48, generator=gen(3))
    for dtype in ALL:
        leaf, wl = y.to(dtype).cuda().requires_grad_(), w.cuda().requires_grad_()
        r = qr.Routing.from_ids(ids.cuda(), wl, 9)
        out = r.combine(leaf)
        got = torch.autograd.grad(out, (leaf, wl), d.cuda())
        place = order_of(ids, 9)[3].view(20, 3)
        at = y.to(dtype).to(FP64)[place]
        dy = torch.empty(60, 48, dtype=FP64)
        dy[place] = w.to(FP64)[:, :, None] * d.to(FP64)[:, None]
        terms = at * d.to(FP64)[:, None]
        assert bool(((got[0].cpu().to(FP64) - dy).abs() <= (UNIT[dtype] + 2.0**-24) * 1.01 * dy.abs() + TINY[dtype]).all())
        assert bool(((got[1].cpu().to(FP64) - terms.sum(2)).abs() <= 48 * 2.0**-24 * terms.abs().sum(2)).all())
        mags = (at * w.to(FP64)[:, :, None]).abs().sum(1)
        want = (at * w.to(FP64)[:, :, None]).sum(1)
        assert bool(((out.detach().cpu().to(FP64) - want).abs() <= 4 * 2.0**-24 * mags).all())


def test_route_groups_whose_differences_round_to_ties():
    """Group sums of 2 + 7e-18, 2 and 2 + 1.6e-17, which 64 bits hold without the bias but not beside it: in this order
    the first and the second, and the second and the third, seem to tie, but the third is ahead of the first."""
    qr = _qr()
    gone = -math.inf
    x = torch.tensor([[gone, gone, -40.0, -40.5, 40.0, gone, -39.0, -40.0]]).cuda()
    bias = torch.ones(8).cuda()
    for keep, want in ((1, [6, 7]), (2, [6, 2, 7, 3])):
        assert qr.route(x, 2 * keep, bias=bias, groups=4, keep_groups=keep)[0].tolist() == [want]


@pytest.mark.parametrize("T,k", [(64, 1024), (64, 1025), (1, 1 << 16), (3, 40000), (70, 2000)])
def test_from_ids_of_many_pairs_a_token(T, k):
    """By the kernels and by torch's operations, which the longest of these take: the same order."""
    ids = torch.randint(-1, 12, (T, k), generator=gen(k))
    check_order(_qr().Routing.from_ids(ids.cuda(), torch.rand(T, k).cuda(), 12)._tensors(), ids, 12)


def test_from_ids_leaves_long_rows_to_torch(monkeypatch):
    """One workgroup orders the pairs of up to 64 tokens: beyond 2^16 of them torch's operations are faster."""
    qr = _qr()
    from quantized_routed_moe_amd import experts
    seen = []
    kernel = experts.sort_pairs
    monkeypatch.setattr(experts, "sort_pairs", lambda ids, n: seen.append(tuple(ids.shape)) or kernel(ids, n))
    for T, k in ((64, 1024), (64, 1025), (1, 1 << 16), (1, (1 << 16) + 1), (100000, 8), (500, 2000)):
        qr.Routing.from_ids(torch.zeros(T, k, dtype=torch.int64).cuda(), torch.rand(T, k).cuda(), 12)
    assert seen == [(64, 1024), (1, 1 << 16), (100000, 8)]
