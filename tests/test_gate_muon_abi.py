"""The gate's, the orthogonalisation's and the Muon step's entry points check their arguments on the host before any
launch (no GPU)."""
import ctypes
import math

import pytest
import torch

from expert_ffn_layer_amd import layer, native as N
from inputgen import layers as L

P = ctypes.c_void_p
OK, M8, M2 = P(0x10000), P(0x10008), P(0x10002)  # aligned, 8 off a 16-byte boundary, 2 off; never read
BIG = 1 << 40


def at(i):
    return P(0x100000 * (i + 1))


def shape(**kw):
    base = dict(T=4, H=256, E=16, k=2, I=128, act="bf16", w_routed="bf16")
    base.update(kw)
    return N.make_shape(**base)


def error():
    return N.load().moe_last_error().decode()


def gate(s=None, r=None, logits=at(0), bias=at(1), idx=at(2), w=at(3)):
    return N.load().moe_gate(s or shape(), r or N.make_gate(), logits, bias, idx, w, None)


def gate_backward(s=None, r=None, logits=at(0), idx=at(1), dw=at(2), dl=at(3)):
    return N.load().moe_gate_backward(s or shape(), r or N.make_gate(), logits, idx, dw, dl, None)


def route(s=None, r=None, x=at(0), wr=at(1), bias=at(2), logits=at(3), idx=at(4), w=at(5), ws=at(6), size=BIG):
    return N.load().moe_route_gated(s or shape(), r or N.make_gate(), x, wr, bias, logits, idx, w, ws, size, None)


def layer_forward(s=None, r=None, x=at(0), ws=at(6), size=BIG):
    w = N.MoeWeights(0x10000, 0x10000, 0x10000)
    return N.load().moe_layer_forward_gated(s or shape(), r or N.make_gate(), x, at(1), None, w, None, at(5), None, None, ws, size, None)


CALLS = (gate, gate_backward, route, layer_forward)


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=3), dict(groups=-1), dict(groups=4, top_groups=0), dict(groups=4, top_groups=5),
                                dict(groups=16, top_groups=1), dict(group_top=0), dict(group_top=3), dict(scale=math.nan), dict(scale=math.inf)])
def test_rules(kw):
    for call in CALLS:
        assert call(r=N.make_gate(**kw)) == 1, call


def test_rule_fields():
    for name, value in (("score", 2), ("score", -1), ("renormalize", 2)):
        r = N.make_gate()
        setattr(r, name, value)
        for call in CALLS:
            assert call(r=r) == 1 and error()
    r = N.make_gate("sigmoid", groups=8, group_top=2)
    assert (r.score, r.groups, r.top_groups, r.group_top, r.renormalize, r.scale) == (1, 8, 8, 2, 1, 1.0)
    with pytest.raises(KeyError):
        N.make_gate("tanh")
    for call in CALLS:
        assert call(s=shape(E=256, k=2), r=N.make_gate(groups=128)) == 1 and "groups" in error()
        assert call(s=shape(E=0)) == 1 and call(s=shape(k=17, E=32)) == 1 and call(s=shape(T=-1)) == 1


def test_gate_pointers():
    none = P(None)
    for kw in (dict(logits=none), dict(idx=none), dict(w=none), dict(logits=M2), dict(bias=M2), dict(idx=M2), dict(w=M2)):
        assert gate(**kw) == 1, kw
    for kw in (dict(logits=none), dict(idx=none), dict(dw=none), dict(dl=none), dict(logits=M2), dict(idx=M2), dict(dw=M2), dict(dl=M2)):
        assert gate_backward(**kw) == 1, kw
    for kw in (dict(idx=at(0)), dict(w=at(0)), dict(w=at(1)), dict(idx=at(1)), dict(w=at(2))):
        assert gate(**kw) == 1 and "memory" in error(), kw
    # the last element of the logits, and one that begins before them
    assert gate(idx=P(0x100000 + 4 * 16 * 4 - 4)) == 1 and gate(w=P(0x100000 - 4)) == 1
    for kw in (dict(dl=at(1)), dict(dl=at(2)), dict(dl=P(0x100000 + 4))):
        assert gate_backward(**kw) == 1 and "memory" in error(), kw
    s = shape(T=0)
    assert gate(s, logits=none, idx=none, w=none) == 0 and gate_backward(s, logits=none, idx=none, dw=none, dl=none) == 0
    lib = N.load()
    assert lib.moe_gate(None, N.make_gate(), OK, OK, OK, OK, None) == 1 and lib.moe_gate(shape(), None, OK, OK, OK, OK, None) == 1
    assert lib.moe_gate_backward(shape(), None, OK, OK, OK, OK, None) == 1
    assert lib.moe_route_gated(shape(), None, OK, OK, OK, OK, OK, OK, OK, BIG, None) == 1


def test_route_pointers():
    none = P(None)
    for kw in (dict(x=none), dict(wr=none), dict(idx=none), dict(w=none), dict(x=M8), dict(wr=M8), dict(bias=M2), dict(logits=M2), dict(idx=M2),
               dict(w=M2), dict(ws=none), dict(ws=P(0x10010))):
        assert route(**kw) == 1, kw
    assert route(size=64) == 3 and layer_forward(size=64) == 3 and layer_forward(x=none) == 1
    for kw in (dict(logits=at(0)), dict(idx=at(1)), dict(w=at(2)), dict(w=at(4)), dict(logits=at(5)), dict(idx=at(6)), dict(ws=at(0))):
        assert route(**kw) == 1 and "memory" in error(), kw
    assert route(shape(T=0), x=none, wr=none, logits=none, idx=none, w=none) == 0


def test_gate_binding():
    r, s = N.make_gate(), shape()
    good = dict(logits=torch.zeros(4, 16), bias=torch.zeros(16), topk_idx=torch.zeros(4, 2, dtype=torch.int32), topk_w=torch.zeros(4, 2))
    for name, bad in (("logits", torch.zeros(4, 15)), ("logits", torch.zeros(4, 16).double()), ("bias", torch.zeros(15)),
                      ("bias", torch.zeros(16).bfloat16()), ("topk_idx", torch.zeros(4, 2, dtype=torch.int64)),
                      ("topk_idx", torch.zeros(4, 3, dtype=torch.int32)), ("topk_w", torch.zeros(8).half())):
        with pytest.raises(ValueError, match=name):
            N.moe_gate(s, r, **good | {name: bad})
    with pytest.raises(ValueError, match="GPU"):
        N.moe_gate(s, r, **good)
    good = dict(logits=torch.zeros(4, 16), topk_idx=torch.zeros(4, 2, dtype=torch.int32), dtopk_w=torch.zeros(4, 2), dlogits=torch.zeros(4, 16))
    for name, bad in (("logits", torch.zeros(3, 16)), ("topk_idx", torch.zeros(4, 2)), ("dtopk_w", torch.zeros(4)), ("dlogits", torch.zeros(4, 2))):
        with pytest.raises(ValueError, match=name):
            N.moe_gate_backward(s, r, **good | {name: bad})


def ns(steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7):
    return N.MoeNewtonSchulz(steps, a, b, c, eps)


def orthogonalize(p=None, kind="bf16", count=2, rows=40, cols=24, g=at(0), o=at(1), ws=at(2), size=BIG):
    return N.load().moe_orthogonalize(p or ns(), N.DTYPE[kind], count, rows, cols, g, o, ws, size, None)


def muon_config(**kw):
    base = dict(ns=ns(), p_type=1, g_type=1, lr=0.1, momentum=0.9, weight_decay=0.1, nesterov=1, lr_dev=None, grad_scale=None)
    base.update(kw)
    return N.MoeMuonConfig(*base.values())


def tensor(p=0x100000, g=0x200000, m=0x300000, master=None, count=2, rows=40, cols=24, scale=1.0):
    return N.MoeMuonTensor(p, g, m, master, count, rows, cols, scale)


def muon(*t, ws=at(20), size=BIG, count=None, **kw):
    arr = (N.MoeMuonTensor * max(1, len(t)))(*t)
    return N.load().moe_muon(muon_config(**kw), arr, len(t) if count is None else count, ws, size, None)


BAD_NS = [dict(steps=0), dict(steps=33), dict(a=math.nan), dict(b=math.inf), dict(c=-math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf)]
FAR_NS = [dict(a=4.0, b=0.0, c=0.0, steps=1), dict(a=0.0, b=15.0, c=0.0), dict(a=1.0, b=0.0, c=15.0), dict(a=-3.8, b=0.0, c=0.0),
          dict(a=1.5, b=0.0, c=0.0, steps=5), dict(a=3.4445, b=-4.7750, c=4.0)]


@pytest.mark.parametrize("kw", BAD_NS)
def test_bad_steps(kw):
    assert orthogonalize(ns(**kw)) == 1 and muon(tensor(), ns=ns(**kw)) == 1


@pytest.mark.parametrize("kw", FAR_NS)
def test_polynomials_that_leave_the_range(kw):
    """Singular values grow past what the steps' 16-bit numbers hold."""
    assert orthogonalize(ns(**kw)) == 2 and "singular" in error()
    assert muon(tensor(), ns=ns(**kw)) == 2


def test_orthogonalize_arguments():
    none = P(None)
    for kw in (dict(count=-1), dict(rows=-1), dict(cols=-3), dict(kind="fp8"), dict(g=none), dict(o=none), dict(g=M8), dict(o=M8), dict(ws=none),
               dict(ws=P(0x10010))):
        assert orthogonalize(**kw) == 1, kw
    for kw in (dict(o=at(0)), dict(ws=at(0)), dict(o=at(2)), dict(o=P(0x100000 + 2 * 40 * 24 * 2 - 16))):
        assert orthogonalize(**kw) == 1 and "memory" in error(), kw
    assert orthogonalize(size=64) == 3
    assert orthogonalize(rows=1 << 21, cols=1) == 2 and orthogonalize(rows=40000, cols=40000) == 2
    lib = N.load()
    assert lib.moe_orthogonalize(None, 1, 1, 1, 1, OK, at(1), at(2), BIG, None) == 1
    assert orthogonalize(count=0, g=none, o=none, ws=none) == 0
    b = ctypes.c_size_t()
    size = lib.moe_orthogonalize_workspace_size
    assert size(1, 1, 8, 8, None) == 1 and size(2, 1, 8, 8, ctypes.byref(b)) == 1 and size(1, -1, 8, 8, ctypes.byref(b)) == 1
    assert size(1, 1, 1 << 21, 8, ctypes.byref(b)) == 2
    sizes = [N.moe_orthogonalize_workspace_size("bf16", n, 7168, 2048) for n in (0, 1, 8, 1000, 100000)]
    assert sizes[0] == 0 < sizes[1] < sizes[2] < sizes[3] == sizes[4]  # long stacks are worked on in parts
    assert N.moe_orthogonalize_workspace_size("f32", 1, 300, 300) > N.moe_orthogonalize_workspace_size("bf16", 1, 300, 300)


def test_muon_arguments():
    for kw in (dict(p_type=2), dict(g_type=3), dict(lr=-1.0), dict(lr=math.nan), dict(momentum=1.0), dict(momentum=-0.1), dict(weight_decay=-0.1),
               dict(nesterov=2), dict(lr_dev=0x10002), dict(grad_scale=0x10001), dict(count=-1), dict(ws=P(None)), dict(ws=P(0x10010))):
        assert muon(tensor(), **kw) == 1, kw
    for kw in (dict(p=None), dict(g=None), dict(m=None), dict(p=0x100008), dict(g=0x200008), dict(m=0x300004), dict(master=0x400004),
               dict(scale=math.nan), dict(count=-1), dict(rows=-1)):
        assert muon(tensor(**kw)) == 1, kw
    assert muon(tensor(rows=1 << 21)) == 2
    assert muon(tensor(master=0x400000), p_type=0) == 1  # fp32 parameters take no copies
    assert muon(tensor(master=0x400000), tensor(0x500000, 0x600000, 0x700000)) == 1
    assert muon(tensor(), size=64) == 3
    for kw in (dict(g=0x100000), dict(m=0x100000), dict(g=0x300000), dict(master=0x300000), dict(p=0x200000)):
        assert muon(tensor(**kw)) == 1 and "overlap" in error(), kw
    assert muon(tensor(), tensor(0x100000, 0x600000, 0x700000)) == 1 and "overlap" in error()
    assert muon(tensor(), ws=P(0x300000)) == 1 and "overlap" in error()
    assert muon(tensor(), lr_dev=0x300000) == 1 and muon(tensor(), grad_scale=0x100000) == 1
    assert muon(tensor(g=at(20).value)) == 1  # a gradient in the workspace
    assert muon(count=0) == 0 and muon(tensor(None, None, None, count=0)) == 0 and muon(tensor(None, None, None, rows=0), ws=P(None)) == 0
    lib = N.load()
    assert lib.moe_muon(None, None, 0, None, 0, None) == 1 and lib.moe_muon(muon_config(), None, 2, None, 0, None) == 1
    b = ctypes.c_size_t()
    assert lib.moe_muon_workspace_size(1, None, 1, ctypes.byref(b)) == 1 and lib.moe_muon_workspace_size(1, None, 0, None) == 1
    assert lib.moe_muon_workspace_size(3, None, 0, ctypes.byref(b)) == 1


def test_muon_workspace_counts_a_class_together():
    def need(*t):
        arr, b = (N.MoeMuonTensor * len(t))(*t), ctypes.c_size_t()
        assert N.load().moe_muon_workspace_size(1, arr, len(t), ctypes.byref(b)) == 0
        return b.value
    one, both = need(tensor(rows=300, cols=400)), need(tensor(rows=300, cols=400), tensor(rows=400, cols=300))
    assert both > one and need(tensor(rows=300, cols=400, count=4)) == both
    assert need(tensor(rows=300, cols=400), tensor(rows=8, cols=8)) == one  # one class after the other
    assert need(tensor(count=0)) == 0 and need(tensor(rows=64, cols=128)) == 0  # a workgroup each needs none


def test_muon_binding():
    w = torch.zeros(3, 4, 5)
    for p, g, m in (([w], [], [w]), ([w], [w, w], [w]), ([w], [w[:, :3]], [w]), ([w], [w], [w.bfloat16()]), ([w.half()], [w], [w]), ([w], [w.double()], [w]),
                    ([w, w.bfloat16()], [w, w], [w, w]), ([w[0, 0]], [w[0, 0]], [w[0, 0]]), ([w], [w], [w])):
        with pytest.raises(ValueError):
            N.muon_tensors(p, g, m)  # the last one: not on a GPU
    with pytest.raises(ValueError):
        N.muon_tensors([w], [w], [w], scale=[])
    for g, o in ((w, w.bfloat16()), (w, w[:2]), (w.half(), w.half()), (w[0, 0], w[0, 0])):
        with pytest.raises(ValueError):
            N.moe_orthogonalize(g, o, w)
    empty = N.muon_tensors([], [], [])
    N.moe_muon(empty, None)
    assert N.moe_muon_workspace_size(empty) == 0


def test_layer_refuses():
    spec = L.LayerSpec("optimizers", T=8, H=256, E=4, k=2, I=128, act="f32", w_routed="f32", w_shared="f32", seed=1)
    for kw in (dict(optimizer="sgd"), dict(optimizer="muon", state="e4m3")):
        with pytest.raises(ValueError, match="optimizer"):
            layer.TrainableLayer(spec, None, None, **kw)
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    with pytest.raises(ValueError, match="muon"):
        lay.muon_step(0.1)
    lay.muon_ws = torch.zeros(1)
    with pytest.raises(ValueError, match="Muon"):
        lay.step(0.1)
