"""The training entry points check their arguments on the host before any launch (no GPU)."""
import ctypes

import pytest
import torch

from expert_ffn_layer_amd import layer, native as N

P = ctypes.c_void_p
OK, M8, M2 = P(0x10000), P(0x10008), P(0x10002)  # aligned, 8 off a 16-byte boundary, 2 off; never read
BIG = 1 << 40


def shape(**kw):
    base = dict(T=4, H=256, E=8, k=2, I=128, act="bf16", w_routed="bf16")
    base.update(kw)
    return N.make_shape(**base)


def weights(*at):
    return N.MoeWeights(*(at or (0x10000,) * 3), None, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(H=100), 1), (dict(I=64), 1), (dict(E=0), 1), (dict(k=9), 1), (dict(T=-1), 1), (dict(act="fp8"), 1),
    (dict(w_routed="fp8"), 2), (dict(w_routed="mxfp4"), 2), (dict(act="f32"), 2), (dict(I_shared=128), 2)])
def test_shapes(kw, status):
    with pytest.raises(N.MoeError) as e:
        N.moe_train_workspace_size(shape(**kw))
    assert e.value.status == status


def test_workspace_size():
    lib = N.load()
    assert lib.moe_train_workspace_size(ctypes.byref(shape()), None) == 1
    a, b = (N.moe_train_workspace_size(shape(T=t)) for t in (4, 400))
    assert 0 < N.moe_train_workspace_size(shape(T=0)) < a < b
    assert b >= 400 * 2 * 128 * 3 * 2  # h, dg and du of every row


def ffn(s, x=OK, off=OK, slot=OK, w=None, g=OK, u=OK, y=OK, ws=OK, size=BIG):
    w = weights() if w is None else w
    return N.load().moe_gated_ffn(ctypes.byref(s), x, off, slot, ctypes.byref(w), g, u, y, ws, size, None)


def ffn_backward(s, x=OK, off=OK, slot=OK, w=None, g=OK, u=OK, dy=OK, dx=OK, grads=(0x10000,) * 3, ws=OK, size=BIG):
    w = weights() if w is None else w
    gr = None if grads is None else ctypes.byref(N.MoeWeightGrads(*grads))
    return N.load().moe_gated_ffn_backward(ctypes.byref(s), x, off, slot, ctypes.byref(w), g, u, dy, dx, gr, ws, size, None)


def test_block_refuses():
    s = shape()
    for fn in (ffn, ffn_backward):
        assert fn(s, x=None) == 1 and fn(s, x=M8) == 1
        assert fn(s, off=None) == 1                      # NULL offsets with 8 experts
        assert fn(s, off=M2) == 1 and fn(s, slot=M2) == 1
        assert fn(s, w=weights(0x10000, None, 0x10000)) == 1 and fn(s, w=weights(0x10000, 0x10008, 0x10000)) == 1
        assert fn(s, ws=None) == 1 and fn(s, ws=P(0x10010)) == 1 and fn(s, size=16) == 3
        assert fn(s, g=None) == 1 and fn(s, g=M8) == 1 and fn(s, u=M8) == 1
    assert ffn(s, y=None) == 1 and ffn(s, y=M8) == 1
    assert ffn_backward(s, dy=None) == 1 and ffn_backward(s, dy=M8) == 1 and ffn_backward(s, dx=M8) == 1
    assert ffn_backward(s, dx=None, grads=None) == 1
    assert ffn_backward(s, grads=(0x10000, None, 0x10000)) == 1 and ffn_backward(s, grads=(0x10000, 0x10000, 0x10008)) == 1
    assert ffn(shape(T=0), x=None, y=None, g=None, u=None) == 0  # nothing to do
    apart = dict(x=P(0x20000), g=P(0x30000), u=P(0x40000), y=P(0x50000))
    for a, b in (("g", "u"), ("g", "y"), ("u", "y"), ("y", "x"), ("g", "x")):
        assert ffn(s, **apart | {a: apart[b]}) == 1 and "memory" in N.load().moe_last_error().decode()
    apart = dict(x=P(0x20000), g=P(0x30000), u=P(0x40000), dy=P(0x50000), dx=P(0x60000), grads=(0x70000, 0x80000, 0x90000))
    for name in ("x", "g", "u", "dy"):
        assert ffn_backward(s, **apart | {"dx": apart[name]}) == 1 and "memory" in N.load().moe_last_error().decode()
        assert ffn_backward(s, **apart | {"grads": (0x70000, apart[name].value, 0x90000)}) == 1
    for grads in ((0x70000, 0x70000, 0x90000), (0x70000, 0x80000, 0x60000), (0x10000, 0x80000, 0x90000)):
        assert ffn_backward(s, **apart | {"grads": grads}) == 1 and "memory" in N.load().moe_last_error().decode()
    lib = N.load()
    assert lib.moe_gated_ffn(None, OK, OK, OK, ctypes.byref(weights()), OK, OK, OK, OK, BIG, None) == 1
    assert lib.moe_gated_ffn(ctypes.byref(s), OK, OK, OK, None, OK, OK, OK, OK, BIG, None) == 1


def test_combine_backward_refuses():
    s = shape()

    def call(s=s, **kw):
        a = dict(dy=OK, y=P(0x20000), slot=OK, w=OK, rows=P(0x30000), dw=OK) | kw
        return N.load().moe_combine_backward(ctypes.byref(s), *a.values(), None)
    for name in ("dy", "y", "slot", "w", "rows", "dw"):
        assert call(**{name: None}) == 1
    assert call(dy=M8) == 1 and call(y=M8) == 1 and call(rows=M8) == 1
    assert call(slot=M2) == 1 and call(w=M2) == 1 and call(dw=M2) == 1
    assert call(rows=P(0x20000)) == 1 and call(rows=OK) == 1  # in place
    assert call(shape(T=0)) == 0
    assert call(shape(H=100)) == 1


def config(**kw):
    a = dict(p_type=1, g_type=1, state=0, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1) | kw
    return N.MoeAdamwConfig(**a)


def tensor(**kw):
    a = dict(p=0x10000, g=0x20000, m=0x30000, v=0x40000, n=64) | kw
    return N.MoeAdamwTensor(**a)


def adamw(c, *tensors, count=None):
    arr = (N.MoeAdamwTensor * max(1, len(tensors)))(*tensors)
    return N.load().moe_adamw(ctypes.byref(c), arr, len(tensors) if count is None else count, None)


def test_adamw_refuses():
    for kw in (dict(p_type=2), dict(g_type=3), dict(state=2), dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0),
               dict(beta1=-0.1), dict(beta2=1.5), dict(beta2=float("nan")), dict(eps=-1e-8), dict(weight_decay=-0.1),
               dict(step=0), dict(lr_dev=0x10002), dict(step_dev=0x10004), dict(grad_scale=0x10001)):
        assert adamw(config(**kw), tensor()) == 1, kw
    for kw in (dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(n=-1), dict(n=1 << 41), dict(p=0x10008),
               dict(g=0x20004), dict(m=0x30002), dict(v=0x40008), dict(master=0x50008)):
        assert adamw(config(), tensor(**kw)) == 1, kw
    assert adamw(config(state=1), tensor()) == 1  # scales missing
    assert adamw(config(state=1), tensor(m_scale=0x50002, v_scale=0x60000)) == 1
    assert adamw(config(p_type=0), tensor(master=0x50000)) == 1
    assert adamw(config(), tensor(), tensor(p=0x50000, master=0x60000)) == 1  # one with a master copy
    assert adamw(config(), tensor(), tensor()) == 1  # the same tensor twice
    assert "overlap" in N.load().moe_last_error().decode()
    assert adamw(config(), tensor(), tensor(p=0x10040)) == 1  # inside the first one's 128 bytes
    assert adamw(config(), tensor(m=0x40000)) == 1  # m is v
    assert adamw(config(), tensor(), tensor(p=0x50000, m=0x60000, v=0x300C0)) == 1  # v inside the first one's m
    assert adamw(config(), tensor(master=0x40080)) == 1  # a master copy inside v
    assert adamw(config(), tensor(), count=-1) == 1
    assert adamw(config(), count=0) == 0 and adamw(config(), tensor(n=0, p=None)) == 0
    assert N.load().moe_adamw(None, None, 0, None) == 1 and N.load().moe_adamw(ctypes.byref(config()), None, 1, None) == 1


def test_adamw_table_refuses_mismatched_lists():
    f, b = torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16)
    for args in (([f], [], [f], [f]), ([f], [f], [b], [f]), ([f], [torch.zeros(9)], [f], [f]), ([f.double()], [f], [f], [f]),
                 ([f], [f], [f], [f], None, [f], None), ([f], [f], [f], [f], None, [f[:1]], [f[:1]]),
                 ([f], [f], [f], [f])):  # the last: not on a GPU
        with pytest.raises(ValueError):
            N.adamw_tensors(*args)
    assert len(N.adamw_tensors([], [], [], []).array) == 0


def test_binding_refuses_tensors_off_the_gpu():
    """A host tensor's address never reaches a kernel."""
    b, i = torch.zeros(8, 256, dtype=torch.bfloat16), torch.zeros(16, dtype=torch.int32)
    w = {n: b for n in ("gate", "up", "down")}
    with pytest.raises(ValueError):
        N.moe_gated_ffn(shape(), b, i, i, w, b, b, b, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        N.moe_gated_ffn_backward(shape(), b, i, i, w, b, b, b, b, w, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        N.moe_combine_backward(shape(), b, b, i, b, b, b)
    f = torch.zeros(8)
    table = N.AdamwTensors((N.MoeAdamwTensor * 1)(tensor()), [[f]], "f32", "f32", 0)
    for kw in ({}, dict(lr_dev=f.double()), dict(step_dev=f), dict(grad_scale=f[:0])):
        with pytest.raises(ValueError):
            N.moe_adamw(table, **kw)


def test_layer_refuses_other_sizes_types_and_strides():
    t = torch.zeros(4, 8)
    layer._need("x", t, torch.float32, (4, 8))
    layer._need("x", t, torch.float32, (8, 4), (4, 8))
    for bad in (t[:3], t.double(), torch.zeros(8, 4).T, t[None]):
        with pytest.raises(ValueError):
            layer._need("x", bad, torch.float32, (4, 8))
