"""expert_ffn's autograd on the host: the operators are replaced by 64-bit
computations of the same formulas, so what is tested is what the function
saves, computes and refuses around them."""
import pytest
import torch

import quantized_routed_moe_amd as qr
from quantized_routed_moe_amd import experts

T, K, E, H, F = 6, 2, 4, 8, 5


def groups(offsets):
    o = offsets.tolist()
    return [(e, slice(o[e], o[e + 1])) for e in range(len(o) - 1)]


def grouped_mm(a, b, offsets, rows=None, dtype=None):
    a = a if rows is None else a[rows.long()]
    c = torch.zeros(a.shape[0], b.shape[1], dtype=a.dtype)
    for e, s in groups(offsets):
        c[s] = a[s] @ b[e].t()
    return c


def grouped_mm_grad_a(dc, b, offsets, dtype=None):
    return grouped_mm(dc, b.transpose(1, 2), offsets)


def grouped_mm_grad_b(dc, a, offsets, rows=None, dtype=None):
    a = a if rows is None else a[rows.long()]
    return torch.stack([dc[s].t() @ a[s] for _, s in groups(offsets)])


def swiglu(gu):
    g, u = gu.chunk(2, 1)
    return g * torch.sigmoid(g) * u


def swiglu_grad(dh, gu):
    g, u = gu.chunk(2, 1)
    s = torch.sigmoid(g)
    return torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], 1)


@pytest.fixture
def calls(monkeypatch):
    """Puts the stand-ins in place; the names of the operators called, in order."""
    made = []

    def counted(f):
        def call(*args, **kw):
            made.append(f.__name__)
            with torch.no_grad():  # as the kernels: no graph
                return f(*args, **kw)
        return call

    for f in (grouped_mm, grouped_mm_grad_a, grouped_mm_grad_b, swiglu, swiglu_grad):
        monkeypatch.setattr(experts, f.__name__, counted(f))
    return made


def leaves(*frozen):
    g = torch.Generator().manual_seed(3)
    shapes = {"x": (T, H), "w": (T, K), "gate_up": (E, 2 * F, H), "down": (E, H, F)}
    return {n: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(n not in frozen) for n, s in shapes.items()}


IDS = torch.tensor([[0, 3], [3, 1], [0, 1], [1, 0], [3, 0], [1, 3]])  # nothing for expert 2


def own(v):
    r = qr.Routing.from_ids(IDS, v["w"], E)
    return qr.expert_ffn(v["x"], r, v["gate_up"], v["down"])


def formula(v):
    gu = torch.einsum("tkfh,th->tkf", v["gate_up"][IDS], v["x"])
    g, u = gu.chunk(2, 2)
    y = torch.einsum("tkhf,tkf->tkh", v["down"][IDS], g * torch.sigmoid(g) * u)
    return (y * v["w"][:, :, None]).sum(1)


def near(a, b):
    return torch.allclose(a.double(), b.double(), rtol=1e-5, atol=1e-4)  # sums over pairs are in 32 bits


def test_first_derivatives(calls):
    v = leaves()
    for create in (False, True):
        got = torch.autograd.grad(own(v).square().sum(), list(v.values()), create_graph=create)
        want = torch.autograd.grad(formula(v).square().sum(), list(v.values()))
        for n, a, b in zip(v, got, want):
            assert near(a, b), n


@pytest.mark.parametrize("first", ["x", "w", "gate_up", "down"])
@pytest.mark.parametrize("linear", [True, False])  # whether the gradient that comes in depends on the inputs itself
def test_a_second_derivative_is_refused(calls, first, linear):
    """The kernels leave no graph, so a gradient's derivative would lack their part: asking for it raises."""
    v = leaves()
    out = own(v)
    loss = out.sum() if linear else out.square().sum()
    d, = torch.autograd.grad(loss, v[first], create_graph=True)
    with pytest.raises(RuntimeError, match="expert_ffn.*twice"):
        torch.autograd.grad(d.square().sum(), list(v.values()), allow_unused=True)


NEEDED = {  # operators of the backward pass that each gradient cannot do without
    "w": set(),
    "x": {"swiglu_grad", "grouped_mm_grad_a"},
    "gate_up": {"swiglu_grad", "grouped_mm_grad_a", "grouped_mm_grad_b"},
    "down": {"grouped_mm_grad_b"},
}


@pytest.mark.parametrize("wanted", [("x",), ("w",), ("gate_up",), ("down",), ("x", "w"), ("gate_up", "down"),
                                    ("w", "down"), ("x", "gate_up")])
def test_only_the_gradients_asked_for_are_computed(calls, wanted):
    """Frozen banks cost nothing in the backward pass: neither their products nor the memory of their gradients."""
    v = leaves(*(n for n in ("x", "w", "gate_up", "down") if n not in wanted))
    loss = own(v).square().sum()
    del calls[:]
    loss.backward()
    assert set(calls) == set().union(*(NEEDED[n] for n in wanted))
    assert calls.count("grouped_mm_grad_b") == ("gate_up" in wanted) + ("down" in wanted)
    assert calls.count("grouped_mm_grad_a") == ("x" in wanted) + ("x" in wanted or "gate_up" in wanted)
    f = {n: t.detach().clone().requires_grad_() for n, t in v.items()}
    formula(f).square().sum().backward()
    for n, t in v.items():
        assert near(t.grad, f[n].grad) if n in wanted else t.grad is None, n


@pytest.mark.parametrize("name", ["perm", "offsets", "rows", "place"])
def test_routing_rewritten_between_forward_and_backward(calls, name):
    """Written into, the backward pass raises as torch does for any saved tensor; with another tensor put in its
    place, the forward call's own is used."""
    v = leaves()
    want = torch.autograd.grad(own(v).square().sum(), list(v.values()))
    r = qr.Routing.from_ids(IDS, v["w"], E)
    out = qr.expert_ffn(v["x"], r, v["gate_up"], v["down"])
    setattr(r, name, getattr(r, name).flip(0))
    for a, b in zip(torch.autograd.grad(out.square().sum(), list(v.values())), want):
        assert torch.equal(a, b)
    r = qr.Routing.from_ids(IDS, v["w"], E)
    out = qr.expert_ffn(v["x"], r, v["gate_up"], v["down"])
    getattr(r, name).copy_(getattr(r, name).flip(0))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.square().sum().backward()
