"""The gate and the Muon step within the layer: routing from x, the whole forward, training steps, on the GPU."""
import math

import pytest
import torch

from expert_ffn_layer_amd import native as N
from expert_ffn_layer_amd.layer import TrainableLayer, pack
from inputgen import layers as L

from _gpu import act_torch, build, say
from _muon import gate_gradient, step_errors
from _train import DT, half_step

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

SPECS = [
    L.LayerSpec("gated-f32", T=40, H=256, E=8, k=2, I=128, act="f32", w_routed="f32", w_shared="f32", seed=71),
    L.LayerSpec("gated-bf16-shared", T=33, H=512, E=24, k=4, I=256, shared=True, seed=72),
    L.LayerSpec("gated-bf16-one", T=1, H=256, E=256, k=8, I=128, seed=73),
    L.LayerSpec("gated-bf16-many", T=2100, H=512, E=64, k=6, I=256, shared=True, seed=74),
]
IDS = [s.name for s in SPECS]


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def out(*shape, dtype=torch.float32):
    return torch.full(shape, -7, dtype=dtype, device=DEV)


def routed(spec, pl, x, rule, bias, logits=True):
    r = {"logits": out(spec.T, spec.E) if logits else None, "idx": out(spec.T, spec.k, dtype=torch.int32), "w": out(spec.T, spec.k)}
    N.moe_route_gated(pl.shape, rule, x, pl.Wr, bias, r["logits"], r["idx"], r["w"], pl.ws)
    return r


@pytest.mark.parametrize("spec", SPECS, ids=IDS)
def test_route(spec):
    say("route", spec.name)
    lay, pl = build(spec, DEV)
    dtype = act_torch(spec)
    x = lay["x"].view(dtype)
    bias = torch.randn(spec.E, generator=gen_of(1), device=DEV) * 0.1
    rule = N.make_gate("sigmoid", groups=4, top_groups=2, group_top=2, scale=2.5)
    r = routed(spec, pl, x, rule, bias)
    # a sum of H products in fp32
    wr = lay["Wr"].view(dtype).reshape(spec.H, spec.E).double()
    want, size = x.double() @ wr, x.double().abs() @ wr.abs()
    assert ((r["logits"].double() - want).abs() <= spec.H * 2.0 ** -24 * size).all()
    idx, w = out(spec.T, spec.k, dtype=torch.int32), out(spec.T, spec.k)
    N.moe_gate(pl.shape, rule, r["logits"], bias, idx, w)
    assert torch.equal(idx, r["idx"]) and torch.equal(w, r["w"])
    again = routed(spec, pl, x, rule, bias, logits=False)
    assert torch.equal(again["idx"], idx) and torch.equal(again["w"], w)
    # the router's own rule is the renormalised softmax's
    r = routed(spec, pl, x, N.make_gate(), None)
    N.moe_route(pl.shape, x, pl.Wr, None, idx, w, pl.ws)
    assert torch.equal(idx, r["idx"]) and (w - r["w"]).abs().max() <= 1e-5


@pytest.mark.parametrize("spec", SPECS, ids=IDS)
def test_forward_is_its_stages(spec):
    """With experts that are off, so that some pairs are skipped; on the second stream where a shared expert runs there."""
    lay, pl = build(spec, DEV)
    dtype = act_torch(spec)
    x = lay["x"].view(dtype)
    bias = torch.zeros(spec.E, device=DEV)
    bias[:-(spec.k - 1)] = -math.inf  # one expert too few
    for b in (None, bias):
        rule = N.make_gate("sigmoid", scale=1.5)
        y, idx, w = out(spec.T, spec.H, dtype=dtype), out(spec.T, spec.k, dtype=torch.int32), out(spec.T, spec.k)
        pl.forward_gated(x, rule, b, y, idx, w)
        r = routed(spec, pl, x, rule, b)
        off, slot, pair = out(spec.E + 1, dtype=torch.int32), out(spec.T * spec.k, dtype=torch.int32), out(spec.T * spec.k, dtype=torch.int32)
        N.moe_permute(pl.shape, r["idx"], off, slot, pair, pl.ws)
        yp, ys = out(spec.T * spec.k, spec.H, dtype=dtype), out(spec.T, spec.H, dtype=dtype) if spec.shared else None
        N.moe_grouped_ffn(pl.shape, x, off, slot, pl.routed, pl.shared, yp, ys, pl.ws)
        want = torch.empty_like(y)
        N.moe_combine(pl.shape, yp, pair, r["w"], ys, want)
        assert torch.equal(idx, r["idx"]) and torch.equal(w, r["w"]) and torch.equal(y, want)
        assert torch.isfinite(y.float()).all()
        assert (idx == -1).any() == (b is not None and spec.k > 1)


def test_captured_forward():
    spec = SPECS[1]
    lay, pl = build(spec, DEV)
    _, other = build(spec, DEV)
    x = lay["x"].view(act_torch(spec)).clone()
    rule, bias = N.make_gate("sigmoid", groups=4, top_groups=2, group_top=2), torch.zeros(spec.E, device=DEV)
    y, idx, w = out(spec.T, spec.H, dtype=x.dtype), out(spec.T, spec.k, dtype=torch.int32), out(spec.T, spec.k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pl.forward_gated(x, rule, bias, y, idx, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pl.forward_gated(x, rule, bias, y, idx, w)
    for i in range(4):
        x.copy_(x.flip(0) * (1.0 + 0.25 * i))
        bias.copy_(torch.randn(spec.E, generator=gen_of(i), device=DEV))
        graph.replay()
        want = [torch.empty_like(t) for t in (y, idx, w)]
        other.forward_gated(x, rule, bias, *want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, idx, w), want)), "replay %d" % i


def matrices(gen, spec, *lead):
    dtype = DT[spec.act]
    size = {"gate": (spec.H, spec.I), "up": (spec.H, spec.I), "down": (spec.I, spec.H)}
    return {n: (torch.randn((*lead, *z), generator=gen, device=DEV) * z[0] ** -0.5).to(dtype) for n, z in size.items()}


LAYERS = [
    L.LayerSpec("gated-train-f32", T=24, H=256, E=6, k=2, I=128, act="f32", w_routed="f32", w_shared="f32", seed=81),
    L.LayerSpec("gated-train-bf16", T=100, H=512, E=8, k=3, I=256, shared=True, seed=82),
]


@pytest.mark.parametrize("spec", LAYERS, ids=[s.name for s in LAYERS])
@pytest.mark.parametrize("rule", [dict(score="sigmoid", groups=2, top_groups=1, group_top=2, scale=2.5), dict(score="softmax", renormalize=False)],
                         ids=["sigmoid", "softmax"])
@pytest.mark.parametrize("side", [False, True])
def test_training_steps(spec, rule, side):
    """Forward, backward with the router's gradient, and Muon, two steps, against 64-bit autograd of the same choice of
    experts; on the current stream and on another."""
    say("training", spec.name, rule, side)
    gen, dtype = gen_of(spec.seed), DT[spec.act]
    H, E, k, T = spec.H, spec.E, spec.k, spec.T
    master = spec.act == "bf16"
    routed_, shared = matrices(gen, spec, E), matrices(gen, spec) if spec.shared else None
    Wr = (torch.randn(H, E, generator=gen, device=DEV) * H ** -0.5).to(dtype)
    bias = torch.randn(E, generator=gen, device=DEV) * 0.1
    lay = TrainableLayer(spec, Wr, routed_, shared, master=master, rule=N.make_gate(**rule), optimizer="muon")
    stream = torch.cuda.Stream() if side else None
    un = half_step(dtype)
    for step in range(2):
        x, dy = ((torch.randn(T, H, generator=gen, device=DEV)).to(dtype) for _ in range(2))
        torch.cuda.synchronize()
        y = lay.forward(x, bias, stream=stream)
        dx, dlogits = lay.backward(dy, stream=stream)
        torch.cuda.synchronize()
        leaves = {"x": x.double().requires_grad_(), "l": (x.double() @ Wr.double()).requires_grad_()}
        for tag, m in (("r", routed_), ("s", shared)):
            if m is not None:
                leaves |= {tag + n: t.double().requires_grad_() for n, t in m.items()}
        s = torch.sigmoid(leaves["l"]) if rule["score"] == "sigmoid" else torch.softmax(leaves["l"], 1)
        w = s.gather(1, lay.idx.long())
        if rule.get("renormalize", True):
            w = w / w.sum(1, keepdim=True)
        w = w * rule.get("scale", 1.0)
        rows = []
        for e in range(E):
            g = leaves["x"] @ leaves["rgate"][e]
            rows.append((g * torch.sigmoid(g) * (leaves["x"] @ leaves["rup"][e])) @ leaves["rdown"][e])
        want = (torch.stack(rows, 1).gather(1, lay.idx.long()[:, :, None].expand(T, k, H)) * w[:, :, None]).sum(1)
        if shared is not None:
            g = leaves["x"] @ leaves["sgate"]
            want = want + (g * torch.sigmoid(g) * (leaves["x"] @ leaves["sup"])) @ leaves["sdown"]
        want.backward(dy.double())
        got = {"x": dx, "l": dlogits} | {"r" + n: t for n, t in lay.grads[0].items()}
        if shared is not None:
            got |= {"s" + n: t for n, t in lay.grads[1].items()}
        # up to 8 roundings of half a step on each path (g, u, h, y_perm, dy_perm, dg, du, the output), in norm
        tol = 8 * un + 1e-5

        def far(a, b):
            return ((a.double() - b).norm() / b.norm()).item()
        assert far(y, want.detach()) <= tol
        for n, t in got.items():
            assert far(t, leaves[n].grad) <= tol, n
        # the step by these gradients
        lr, mu, wd = 0.02, 0.9, 0.1
        ps, gs, ms, copies = lay.optimizer.keep
        before = [(t if copies is None else copies[i]).double().clone() for i, t in enumerate(ps)]
        moment = [mu * m.double() + g.double() for m, g in zip(ms, gs)]
        lay.muon_step(lr, mu, True, wd, stream=stream)
        torch.cuda.synchronize()
        for i, p in enumerate(ps):
            z = p.shape if p.dim() == 3 else (1, *p.shape)
            o, e = step_errors((gs[i].double() + mu * moment[i]).reshape(z), dtype)
            scale = lr * 0.2 * math.sqrt(max(z[1:]))
            new = before[i].reshape(z) * (1 - lr * wd) - scale * o
            at = (p if copies is None else copies[i]).double().reshape(z)
            d = ((at - new).abs() - 2.0 ** -22 * (new.abs() + (scale * o).abs())).clamp(min=0)
            assert (d.square().sum((1, 2)).sqrt() <= scale * e * o.square().sum((1, 2)).sqrt()).all(), i


def test_router_step():
    """What a user does with dlogits: the router's own gradient and step, by a matrix of E columns."""
    T, H, E, k = 50, 256, 40, 4
    gen = gen_of(5)
    x, W = torch.randn(T, H, generator=gen, device=DEV), torch.randn(H, E, generator=gen, device=DEV) * H ** -0.5
    packed, _ = pack("f32", W.reshape(1, H, E), None, H, E)
    shape = N.make_shape(T, H, E, k, 128, act="f32", w_routed="f32")
    ws = torch.empty(N.moe_workspace_size(shape), dtype=torch.uint8, device=DEV)
    rule = N.make_gate("sigmoid", scale=2.0)
    logits, idx, w = torch.empty(T, E, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    N.moe_route_gated(shape, rule, x, packed, None, logits, idx, w, ws)
    dw = torch.randn(T, k, generator=gen, device=DEV)
    want, bound = gate_gradient(logits, idx, dw, "sigmoid", True, 2.0)
    N.moe_gate_backward(shape, rule, logits, idx, dw, logits)
    assert ((logits.double() - want).abs() <= bound).all()
    grad, m = x.t() @ logits, torch.zeros(H, E, device=DEV)
    table = N.muon_tensors([W], [grad], [m], scale=[1.0])
    before = W.double().clone()
    N.moe_muon(table, torch.empty(N.moe_muon_workspace_size(table), dtype=torch.uint8, device=DEV), lr=0.1, momentum=0.5, nesterov=False)
    o, e = step_errors(grad.double()[None], torch.float32)
    assert torch.equal(m, grad)
    d = ((W.double() - before + 0.1 * o[0]).abs() - 2.0 ** -22 * (before.abs() + 0.1 * o[0].abs())).clamp(min=0)
    assert d.norm() <= 0.1 * e[0] * o.norm()


@pytest.mark.parametrize("spec", LAYERS, ids=[s.name for s in LAYERS])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_training_with_experts_that_are_off(spec, score, renormalize):
    """Fewer experts than k: pairs that are nobody's, in memory that held NaN, reach neither the outputs nor the gradients."""
    say("experts off", spec.name, score, renormalize)
    gen, dtype = gen_of(spec.seed + 1), DT[spec.act]
    H, E, k, T = spec.H, spec.E, spec.k, spec.T
    routed_, shared = matrices(gen, spec, E), matrices(gen, spec) if spec.shared else None
    Wr = (torch.randn(H, E, generator=gen, device=DEV) * H ** -0.5).to(dtype)
    lay = TrainableLayer(spec, Wr, routed_, shared, rule=N.make_gate(score, renormalize=renormalize))
    x, dy = ((torch.randn(T, H, generator=gen, device=DEV)).to(dtype) for _ in range(2))
    for on in (1, 0, k - 1):
        bias = torch.zeros(E, device=DEV)
        bias[torch.randperm(E, generator=gen, device=DEV)[:E - on]] = -math.inf
        for t in (*lay.y, *lay.dx, lay.dy_perm, *[p for pair in lay.pre for p in pair]):
            t.fill_(math.nan)
        y = lay.forward(x, bias)
        dx, dlogits = lay.backward(dy)
        assert (lay.idx[:, on:] == -1).all() and (lay.idx[:, :on] >= 0).all()
        l = (x.double() @ Wr.double()).requires_grad_()
        leaves = {"x": x.double().requires_grad_()} | {"r" + n: t.double().requires_grad_() for n, t in routed_.items()}
        if shared is not None:
            leaves |= {"s" + n: t.double().requires_grad_() for n, t in shared.items()}
        s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
        w = s.gather(1, lay.idx[:, :on].long())
        if renormalize and on:
            w = w / w.sum(1, keepdim=True)

        def ffn(tag, e):
            g = leaves["x"] @ leaves[tag + "gate"][e]
            return (g * torch.sigmoid(g) * (leaves["x"] @ leaves[tag + "up"][e])) @ leaves[tag + "down"][e]
        rows = torch.stack([ffn("r", e) for e in range(E)], 1)
        want = (rows.gather(1, lay.idx[:, :on].long()[:, :, None].expand(T, on, H)) * w[:, :, None]).sum(1)
        if shared is not None:
            want = want + ffn("s", ...)
        want.backward(dy.double())
        got = {"x": dx} | {"r" + n: t for n, t in lay.grads[0].items()} | ({"s" + n: t for n, t in lay.grads[1].items()} if shared is not None else {})
        # up to 8 roundings of half a step on each path, in norm
        tol = 8 * half_step(dtype) + 1e-5

        def near(a, b):  # zeros have to be zeros
            return (a.double() - b).norm() <= tol * b.norm()
        assert near(y, want.detach())
        for n, t in got.items():
            assert near(t, leaves[n].grad), (on, n)
        if on == 0 or (on == 1 and renormalize):  # no weight, or one that is the scale
            assert (dlogits == 0).all()
        else:
            assert near(dlogits, l.grad)
