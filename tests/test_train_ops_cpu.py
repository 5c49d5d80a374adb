"""The operators around the experts' products on the host: the C calls refuse bad arguments before anything is
enqueued, the binding refuses tensors that the C ABI cannot judge, and Routing's torch operations, which CPU tensors
take, give the order that the kernels give.  No GPU is needed."""
import ctypes

import pytest
import torch

import quantized_routed_moe_amd as qr

L = qr._lib
OK, INVALID, UNSUPPORTED, TOO_MANY, WORKSPACE = 0, -1, -2, -3, -4
FAKE = 1 << 30  # aligned host integers: never dereferenced
A, B, C, D = FAKE, FAKE * 4, FAKE * 8, FAKE * 12
FP32, BF16, FP16 = 1, 2, 3
NAN, INF = float("nan"), float("inf")


def router(**kw):
    base = dict(n_experts=64, top_k=6, score=1, groups=1, keep_groups=1, group_best=2, renormalize=1, scale=1.0, bias=None)
    base.update(kw)
    return qr.Router(*(base[f] for f, _ in qr.Router._fields_))


def order(tokens=100, E=64, **kw):
    base = dict(perm=FAKE * 20, place=FAKE * 21, rows=FAKE * 22, offsets=FAKE * 23, workspace=FAKE * 24,
                workspace_bytes=L.moe_pair_order_bytes(tokens, E))
    base.update(kw)
    return qr.PairOrder(*(base[f] for f, _ in qr.PairOrder._fields_))


def route(dtype=FP32, logits=A, ld=None, tokens=100, ids=B, w=C, o=None, r=None, **kw):
    r = router(**kw) if r is None else r
    return L.moe_route(ctypes.byref(r), dtype, logits, r.n_experts if ld is None else ld, tokens, ids, w,
                       None if o is None else ctypes.byref(o), None)


def grad(dtype=FP32, logits=A, ld=None, tokens=100, ids=B, dw=C, d=D, ldd=None, **kw):
    r = router(**kw)
    return L.moe_route_grad(ctypes.byref(r), dtype, logits, r.n_experts if ld is None else ld, tokens, ids, dw, d,
                            r.n_experts if ldd is None else ldd, None)


@pytest.mark.parametrize("call", [route, grad])
def test_router_refusals(call):
    for bad in (dict(n_experts=0), dict(top_k=0), dict(top_k=65), dict(score=0), dict(score=3), dict(renormalize=2),
                dict(tokens=-1), dict(dtype=0), dict(dtype=4), dict(ld=63), dict(logits=None), dict(ids=None),
                dict(logits=A + 2), dict(ids=B + 2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(n_experts=1025), dict(top_k=9), dict(ld=(1 << 21) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(tokens=(1 << 20) // 6 + 1) == TOO_MANY
    assert call(tokens=1 << 62) == TOO_MANY


def test_choice_refusals():
    for bad in (dict(groups=0), dict(groups=3), dict(groups=8, keep_groups=0), dict(groups=8, keep_groups=9),
                dict(groups=32, keep_groups=2), dict(group_best=0), dict(group_best=3), dict(bias=D + 1), dict(w=None),
                dict(w=C + 1), dict(ids=A), dict(w=A), dict(w=B), dict(w=D, bias=D), dict(ids=D + 4, bias=D)):
        assert route(**bad) == INVALID, bad
    assert route(groups=32, keep_groups=32) == UNSUPPORTED
    assert L.moe_route(None, FP32, A, 64, 1, B, C, None, None) == INVALID


def test_route_grad_refusals():
    for bad in (dict(dw=None), dict(dw=C + 2), dict(d=None), dict(d=D + 2), dict(ldd=63), dict(d=A), dict(d=B), dict(d=C)):
        assert grad(**bad) == INVALID, bad
    assert grad(ldd=(1 << 21) + 1) == UNSUPPORTED
    assert L.moe_route_grad(None, FP32, A, 64, 1, B, C, D, 64, None) == INVALID


def test_order_refusals():
    assert L.moe_pair_order_bytes(-1, 8) == 0 and L.moe_pair_order_bytes(5, 0) == 0
    assert L.moe_pair_order_bytes(5, 1025) == 0 and L.moe_pair_order_bytes((1 << 20) + 1, 8) == 0
    sizes = [L.moe_pair_order_bytes(t, 64) for t in (1, 64, 65, 1000, 20000, 1 << 20)]
    assert sizes[0] == sizes[1] == 0 and sizes[2] > 0 and sizes == sorted(sizes)

    def sort(ids=A, size=4, tokens=100, k=6, E=64, o=None):
        o = order(tokens, E) if o is None else o
        return L.moe_sort_pairs(ids, size, tokens, k, E, ctypes.byref(o), None)

    for call in (lambda o: route(o=o), lambda o: sort(o=o)):
        for bad in (dict(perm=None), dict(place=None), dict(rows=None), dict(offsets=None), dict(perm=FAKE * 20 + 4),
                    dict(rows=FAKE * 22 + 2), dict(place=FAKE * 20), dict(offsets=FAKE * 22), dict(rows=A), dict(perm=A),
                    dict(workspace=None), dict(workspace=FAKE * 20)):
            assert call(order(**bad)) == INVALID, bad
        assert call(order(workspace=FAKE * 24 + 128)) == WORKSPACE
        assert call(order(workspace_bytes=L.moe_pair_order_bytes(100, 64) - 1)) == WORKSPACE
    assert route(o=order(perm=B)) == INVALID and route(o=order(rows=C)) == INVALID
    for bad in (dict(ids=None), dict(ids=A + 2), dict(size=8, ids=A + 4), dict(size=2), dict(tokens=-1), dict(k=0), dict(E=0)):
        assert sort(**bad) == INVALID, bad
    assert sort(E=1025) == UNSUPPORTED
    assert sort(tokens=1 << 20, k=2) == TOO_MANY and sort(tokens=1 << 40, k=1 << 40) == TOO_MANY
    assert L.moe_sort_pairs(A, 4, 5, 2, 8, None, None) == INVALID


def combine(dt=BF16, y=A, ldy=64, pairs=600, place=B, w=C, tokens=100, k=6, n=64, out=D, odt=FP32, ldo=64):
    return L.moe_combine(dt, y, ldy, pairs, place, w, tokens, k, n, out, odt, ldo, None)


def combine_grad(dt=BF16, d=A, ddt=FP32, ldd=64, y=B, ldy=64, pairs=600, place=FAKE * 6, w=C, tokens=100, k=6, n=64, dy=D,
                 lddy=64, dw=FAKE * 16):
    return L.moe_combine_grad(dt, d, ddt, ldd, y, ldy, pairs, place, w, tokens, k, n, dy, lddy, dw, None)


@pytest.mark.parametrize("call", [combine, combine_grad])
def test_combine_refusals(call):
    for bad in (dict(dt=0), dict(dt=4), dict(pairs=-1), dict(tokens=-1), dict(k=0), dict(n=0), dict(y=None), dict(y=B + 8),
                dict(ldy=56), dict(ldy=68), dict(place=None), dict(place=B + 4), dict(w=C + 2)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(n=60), dict(n=65544), dict(ldy=(1 << 21) + 8)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(pairs=(1 << 20) + 1) == TOO_MANY and call(tokens=1 << 20) == TOO_MANY


def test_combine_output_refusals():
    for bad in (dict(odt=0), dict(odt=FP16), dict(dt=FP16, odt=BF16), dict(out=None), dict(out=D + 4), dict(ldo=60),
                dict(out=A), dict(out=B), dict(out=C)):
        assert combine(**bad) == INVALID, bad
    for bad in (dict(ddt=0), dict(ddt=FP16), dict(dt=FP32, ddt=BF16), dict(d=None), dict(d=A + 8), dict(ldd=60),
                dict(dy=D + 8), dict(lddy=60), dict(dw=FAKE * 16 + 2), dict(dy=A), dict(dy=B), dict(dy=C), dict(dw=A),
                dict(dw=B), dict(dw=C), dict(dw=D), dict(dy=FAKE * 6), dict(dw=FAKE * 6)):
        assert combine_grad(**bad) == INVALID, bad
    assert combine_grad(dy=None, dw=None) == OK  # nothing asked for


def orthogonal(dt=FP32, g=A, batch=4, rows=64, cols=96, steps=5, c=None, eps=1e-7, out=B, ws=C, n=None):
    c = [3.4445, -4.775, 2.0315] * max(steps, 1) if c is None else c
    n = L.moe_orthogonalize_bytes(batch, rows, cols) if n is None else n
    return L.moe_orthogonalize(dt, g, batch, rows, cols, steps, (ctypes.c_float * len(c))(*c), eps, out, ws, n, None)


def test_orthogonalize_refusals():
    for bad in (dict(dt=0), dict(dt=5), dict(batch=-1), dict(rows=0), dict(cols=0), dict(steps=0), dict(eps=-1.0),
                dict(eps=NAN), dict(eps=INF), dict(g=None), dict(g=A + 2), dict(out=None), dict(out=B + 1), dict(out=A + 64),
                dict(c=[NAN, 0, 0] * 5), dict(c=[1, INF, 0] * 5),
                dict(c=[3.4445, 4.775, 2.0315] * 5),   # singular values that run away
                dict(c=[100.0, 0, 0] * 5), dict(batch=1 << 60)):
        assert orthogonal(**bad) == INVALID, bad
    for bad in (dict(rows=65537, n=1 << 40), dict(rows=16385, cols=16385, n=1 << 40), dict(steps=33)):
        assert orthogonal(**bad) == UNSUPPORTED, bad
    assert orthogonal(ws=None) == WORKSPACE and orthogonal(ws=C + 64) == WORKSPACE
    assert orthogonal(n=L.moe_orthogonalize_bytes(4, 64, 96) - 1) == WORKSPACE
    assert orthogonal(ws=A) == INVALID and orthogonal(ws=B) == INVALID
    assert L.moe_orthogonalize(FP32, A, 1, 8, 8, 5, None, 0.0, B, C, 1 << 30, None) == INVALID
    assert orthogonal(batch=0, g=None, out=None, ws=None, n=0) == OK


def test_orthogonalize_workspace():
    assert L.moe_orthogonalize_bytes(0, 8, 8) == 0 and L.moe_orthogonalize_bytes(1, 0, 8) == 0
    assert L.moe_orthogonalize_bytes(1, 70000, 8) == 0 and L.moe_orthogonalize_bytes(1, 20000, 20000) == 0
    assert L.moe_orthogonalize_bytes(4, 64, 96) == L.moe_orthogonalize_bytes(4, 96, 64)
    # bounded for any batch: matrices are taken 4 GiB at a time
    many = [L.moe_orthogonalize_bytes(b, 4096, 4096) for b in (1, 4, 15, 256, 10000)]
    assert many == sorted(many) and many[-1] < (4 << 30) + (512 << 20)
    assert L.moe_orthogonalize_bytes(100000, 1, 1) > 0


def test_nothing_to_do():
    assert route(tokens=0, logits=None, ids=None, w=None) == OK
    assert grad(tokens=0, logits=None, ids=None, dw=None, d=None) == OK
    assert combine(tokens=0, pairs=0, y=None, place=None, w=None, out=None) == OK
    assert combine_grad(tokens=0, pairs=0, d=None, y=None, place=None, w=None, dy=None, dw=None) == OK


def test_binding_refusals():
    x, ids = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    place, w, y = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2), torch.zeros(8, 16)
    refused = [
        lambda: qr.route(x, 2), lambda: qr.Routing.from_logits(x, 2), lambda: qr.route_grad(w, x, ids),
        lambda: qr.sort_pairs(ids, 8), lambda: qr.combine(y, place, w), lambda: qr.combine_grad(x, y, place, w),
        lambda: qr.orthogonalize(x),                                               # host tensors
        lambda: qr.route(x.double(), 2), lambda: qr.route(x[0], 2), lambda: qr.route(x.t(), 2),
        lambda: qr.route_grad(w, x, ids.long()), lambda: qr.route_grad(w.double(), x, ids),
        lambda: qr.route_grad(w[:, :1], x, ids), lambda: qr.route_grad(w, x, ids[:2]),
        lambda: qr.sort_pairs(ids.float(), 8), lambda: qr.sort_pairs(ids[0], 8), lambda: qr.sort_pairs(ids.t(), 8),
        lambda: qr.combine(y, place.int(), w), lambda: qr.combine(y, place[0], w), lambda: qr.combine(y, place, w[:2]),
        lambda: qr.combine(y, place, w.double()), lambda: qr.combine(y.double(), place, w),
        lambda: qr.combine_grad(x.double(), y, place, w), lambda: qr.combine_grad(x[:, :8], y, place, w),
        lambda: qr.orthogonalize(x[0]), lambda: qr.orthogonalize(x.double()), lambda: qr.orthogonalize(x.t()),
        lambda: qr.orthogonalize(x, coefficients=(1.0, 2.0)), lambda: qr.orthogonalize(x, 2, [(1.0, 0.0, 0.0)]),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            print(i)


def order_of(ids, E):
    flat = [int(e) if 0 <= int(e) < E else E for e in ids.reshape(-1)]
    perm = sorted(range(len(flat)), key=lambda p: (flat[p], p))
    place = [0] * len(perm)
    for at, p in enumerate(perm):
        place[p] = at
    return perm, [sum(e < x for e in flat) for x in range(E + 1)], [p // ids.shape[1] for p in perm], place


@pytest.mark.parametrize("E", [1, 5, 40])
def test_from_ids_on_the_host(E):
    ids = torch.randint(-1, E + 1, (13, 3), generator=torch.Generator().manual_seed(E))
    r = qr.Routing.from_ids(ids, torch.rand(13, 3), E)
    for got, want in zip((r.perm, r.offsets, r.rows, r.place), order_of(ids, E)):
        assert got.tolist() == want
    assert r.ids is ids and r.perm.dtype == r.place.dtype == torch.int64 and r.offsets.dtype == torch.int32


def test_combine_on_the_host_is_differentiable():
    ids = torch.tensor([[0, 2], [1, 0], [2, 1]])
    w = torch.rand(3, 2, requires_grad=True)
    y = torch.randn(6, 4, requires_grad=True)
    r = qr.Routing.from_ids(ids, w, 3)
    out = r.combine(y)
    want = torch.stack([sum(w[t, j] * y[r.place[2 * t + j]] for j in range(2)) for t in range(3)])
    assert torch.allclose(out, want)
    for a, b in zip(torch.autograd.grad(out.square().sum(), (w, y)), torch.autograd.grad(want.square().sum(), (w, y))):
        assert torch.allclose(a, b)


def test_numbers_that_do_not_fit_are_refused():
    from quantized_routed_moe_amd import train_ops
    for bad in (dict(top_k=1 + (1 << 32)), dict(groups=1 + (1 << 32)), dict(keep_groups=1 << 40), dict(group_best=-1)):
        with pytest.raises(ValueError):
            train_ops._router(**{"n_experts": 8, "top_k": 2, "score": "sigmoid", "renormalize": True, "scale": 1.0, **bad})
    for steps in (0, -1, 33, 5 + (1 << 32)):
        with pytest.raises(ValueError, match="steps"):
            qr.orthogonalize(torch.zeros(2, 3), steps=steps)


def test_combine_wants_a_row_for_each_pair():
    """A missing row is no pair without an expert: the kernel would leave it out of the sum."""
    r = qr.Routing.from_ids(torch.tensor([[0, 2], [1, 0], [2, 1]]), torch.rand(3, 2), 3)
    for y in (torch.ones(5, 8), torch.ones(7, 8), torch.ones(3, 2, 8), torch.ones(6)):
        with pytest.raises(ValueError, match="row for each of 6 pairs"):
            r.combine(y)
    assert r.combine(torch.ones(6, 8)).shape == (3, 8)


def test_from_ids_strict():
    """An id that no router gives is reported where that is asked for; -1 stands for none."""
    w = torch.rand(2, 2)
    for bad in ([[0, 4], [1, 2]], [[0, -2], [1, 2]], [[0, 1 << 40], [1, 2]]):
        with pytest.raises(ValueError, match="experts below 4"):
            qr.Routing.from_ids(torch.tensor(bad), w, 4, strict=True)
        assert qr.Routing.from_ids(torch.tensor(bad), w, 4).offsets.tolist()[-1] == 3
    r = qr.Routing.from_ids(torch.tensor([[0, -1], [3, 2]]), w, 4, strict=True)
    assert r.offsets.tolist() == [0, 1, 1, 2, 3]
    byte = torch.tensor([[0, 1], [3, 2]], dtype=torch.uint8)
    assert qr.Routing.from_ids(byte, w, 4, strict=True).offsets.tolist() == [0, 1, 2, 3, 4]
