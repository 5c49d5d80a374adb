"""The expert FFNs that run the expert operators together: expert_ffn with all
its gradients against 64-bit autograd, Mxfp4Experts against the same steps in
64 bits, and both on the routing of a MoELayer, whose own (int8) output they
come close to.

Tolerances are relative norms.  Each 16-bit rounding is within 2^-8 (bf16) or
2^-11 (fp16) of its value; a result sees at most six of them in a row (h's
input, h, y, dy, dh, dgu), whose effects add at most linearly: 6 units.  The
sums' fp32 rounding is far below.
"""
import numpy as np
import pytest

import moe_synth as ms

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, FP16, FP64 = torch.bfloat16, torch.float16, torch.float64


def _qr():
    import quantized_routed_moe_amd as qr
    return qr


def off(got, want):
    return float((got.detach().cpu().to(FP64) - want).norm() / want.norm())


def reference(x, w, ids, gate_up, down):
    """The FFN in 64 bits, token by token and expert by expert."""
    f = down.shape[2]
    out = []
    for t in range(x.shape[0]):
        acc = 0
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            gu = gate_up[e] @ x[t]
            acc = acc + w[t, j] * (down[e] @ (torch.nn.functional.silu(gu[:f]) * gu[f:]))
        out.append(acc)
    return torch.stack(out)


def case(T, k, E, H, F, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    w = torch.rand(T, k, generator=g) + 0.1
    x = torch.randn(T, H, generator=g).to(dtype)
    gate_up = (torch.randn(E, 2 * F, H, generator=g) / H**0.5).to(dtype)
    down = (torch.randn(E, H, F, generator=g) / F**0.5).to(dtype)
    return ids, w, x, gate_up, down


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 4, 64, 32), (7, 3, 5, 104, 72), (60, 2, 3, 128, 264)])
def test_expert_ffn_and_its_gradients(dtype, T, k, E, H, F):
    qr = _qr()
    ids, w, x, gate_up, down = case(T, k, E, H, F, dtype, T)
    leaves = [t.to(FP64).requires_grad_() for t in (x, w, gate_up, down)]
    want = reference(leaves[0], leaves[1], ids, leaves[2], leaves[3])
    dout = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(FP64)
    grads = torch.autograd.grad(want, leaves, dout)
    xs, ws, gs, ds = [t.cuda().requires_grad_() for t in (x, w, gate_up, down)]
    r = qr.Routing.from_ids(ids.cuda(), ws, E)
    out = qr.expert_ffn(xs, r, gs, ds)
    out.backward(dout.float().cuda())
    tol = 6 * (2.0**-8 if dtype == BF16 else 2.0**-11)
    assert off(out, want.detach()) <= tol
    for got, ref, name in zip((xs.grad, ws.grad, gs.grad, ds.grad), grads, ("x", "w", "gate_up", "down")):
        assert got.shape == ref.shape and off(got, ref) <= tol, name


@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 4, 64, 32), (9, 3, 5, 96, 160), (70, 2, 3, 256, 128)])
def test_mxfp4_experts(T, k, E, H, F):
    """Against the same steps on the values that the codes stand for.  A value of the hidden activation that lies at
    a rounding boundary may take its other neighbour, a third of it away at most; the product it was made from is in
    bf16, so about one in a hundred is near enough to one: 0.33 * sqrt(0.01) of h, and bf16 roundings beside it."""
    qr = _qr()
    ids, w, x, gate_up, down = case(T, k, E, H, F, BF16, T + 1)
    experts = qr.Mxfp4Experts(gate_up.cuda(), down.cuda())
    r = qr.Routing.from_ids(ids.cuda(), w.cuda(), E)
    out = experts(x.cuda(), r)

    def rounded(t):
        return qr.mxfp4_dequantize(*qr.mxfp4_quantize(t.cuda())).cpu().to(FP64)

    xq, gq, dq = rounded(x), rounded(gate_up), rounded(down)
    want = []
    for t in range(T):
        acc = 0
        for j in range(k):
            e = int(ids[t, j])
            gu = (gq[e] @ xq[t]).to(BF16).to(FP64)
            h = rounded((torch.nn.functional.silu(gu[:F]) * gu[F:]).float()[None])[0]
            acc = acc + w[t, j].to(FP64) * (dq[e] @ h)
        want.append(acc)
    assert off(out, torch.stack(want)) <= 0.33 * 0.1 + 3 * 2.0**-8


def test_routing_of_a_layer():
    """A MoELayer's routing drives both FFNs on its own weights: the bf16 one comes within the layer's int8
    activation error (two quantisations of half a step of 1/127 of a block's maximum, about 1/250 of a value each,
    and bf16's roundings), the four-bit one within its formats' (three values rounded to 2 significant bits, about
    0.1 each)."""
    qr = _qr()
    cfg = ms.LayerConfig("experts", 512, 16, 3, 256, 24, shared=False, seed=77)
    inp = ms.make_inputs(cfg)
    layer = qr.MoELayer(cfg.hidden, cfg.n_experts, cfg.top_k, cfg.ffn, False, cfg.routed_fmt, cfg.route).load(inp)
    x = torch.from_numpy(inp["x"]).cuda()
    r = layer.forward_debug(x)
    want = r["out"].cpu().to(FP64)

    def bank(name, rows, cols):  # Q8 blocks: fp16 scale, 32 codes
        raw = np.ascontiguousarray(inp[name]).view(np.uint8).reshape(-1, 34)
        d = raw[:, :2].copy().view(np.float16).astype(np.float32)
        return torch.from_numpy(d * raw[:, 2:].view(np.int8)).view(cfg.n_experts, rows, cols)

    H, F = cfg.hidden, cfg.ffn
    gate_up = torch.cat([bank("gate", F, H), bank("up", F, H)], 1)
    down = bank("down", H, F)
    routing = qr.Routing.from_layer(r)
    with torch.no_grad():
        out = qr.expert_ffn(x.to(BF16), routing, gate_up.to(BF16).cuda(), down.to(BF16).cuda())
    assert off(out, want) <= 2 / 250 + 5 * 2.0**-8
    four = qr.Mxfp4Experts(gate_up.cuda(), down.cuda())(x, routing)
    assert off(four, want) <= 3 * 0.12


@pytest.mark.parametrize("wanted", [("x", "w"), ("down",), ("w",)])
def test_frozen_operands(wanted):
    """The gradients that are asked for are the bits of the full backward pass; the others are None and their banks'
    gradients are never allocated."""
    qr = _qr()
    T, k, E, H, F = 40, 2, 32, 512, 256
    ids, w, x, gate_up, down = case(T, k, E, H, F, BF16, 5)
    dout = torch.randn(T, H, generator=torch.Generator().manual_seed(6)).cuda()

    def grads(asked):
        v = {n: t.cuda().requires_grad_(n in asked) for n, t in zip(("x", "w", "gate_up", "down"), (x, w, gate_up, down))}
        out = qr.expert_ffn(v["x"], qr.Routing.from_ids(ids.cuda(), v["w"], E), v["gate_up"], v["down"])
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out.backward(dout)
        return {n: t.grad for n, t in v.items()}, torch.cuda.max_memory_allocated() - before

    whole, _ = grads(("x", "w", "gate_up", "down"))
    got, peak = grads(wanted)
    for n, g in got.items():
        assert torch.equal(g, whole[n]) if n in wanted else g is None, n
    if "down" not in wanted:
        assert peak < down.numel() * 2  # the smaller bank's gradient


def test_no_tokens():
    """A batch without tokens: empty results, zero gradients of the banks."""
    qr = _qr()
    ids, w, x, gate_up, down = (t[:0] if i < 3 else t for i, t in enumerate(case(3, 2, 4, 64, 32, BF16, 7)))
    xs, ws, gs, ds = [t.cuda().requires_grad_() for t in (x, w, gate_up, down)]
    r = qr.Routing.from_ids(ids.cuda(), ws, 4)
    out = qr.expert_ffn(xs, r, gs, ds)
    assert out.shape == (0, 64) and out.dtype == torch.float32
    out.backward(torch.zeros(0, 64, device="cuda"))
    assert xs.grad.shape == (0, 64) and ws.grad.shape == (0, 2)
    assert gs.grad.shape == gs.shape and not gs.grad.any() and ds.grad.shape == ds.shape and not ds.grad.any()
    assert qr.Mxfp4Experts(gate_up.cuda(), down.cuda())(x.cuda(), r).shape == (0, 64)
