"""What TrainableLayer and the training entry points refuse before any launch (no GPU)."""
import contextlib
import ctypes
import types

import numpy as np
import pytest
import torch

from expert_ffn_layer_amd import layer, native as N
from inputgen import layers as L

from _train import chain_error

SPEC = L.LayerSpec("train-refusals", T=8, H=256, E=4, k=2, I=128, act="f32", w_routed="f32", w_shared="f32", seed=1)


def mats(dtype=torch.float32, device="cpu"):
    return {"gate": torch.zeros(4, 256, 128, dtype=dtype, device=device), "up": torch.zeros(4, 256, 128, dtype=dtype, device=device),
            "down": torch.zeros(4, 128, 256, dtype=dtype, device=device)}


def test_layer_refuses_router_weights_of_another_type_or_size():
    """The packing kernel reads H E elements of the activations' type at the address."""
    for bad in (torch.zeros(256, 4, dtype=torch.bfloat16), torch.zeros(4, 256), torch.zeros(4, 256).T, torch.zeros(1024)):
        with pytest.raises(ValueError, match="Wr"):
            layer.TrainableLayer(SPEC, bad, mats())


def test_layer_refuses_tensors_off_its_gpu():
    """A host tensor's address, or another GPU's, never reaches a kernel."""
    with pytest.raises(ValueError, match="GPU"):
        layer.TrainableLayer(SPEC, torch.zeros(256, 4), mats())
    t = torch.zeros(4, 8)
    for device in (torch.device("cpu"), torch.device("meta"), torch.device("cuda:0")):
        with pytest.raises(ValueError, match="GPU"):
            layer._need("x", t, torch.float32, (4, 8), device=device)
    # forward and backward check against the router weights' device before they call anything
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    lay.T, lay.H, lay.E, lay.dtype, lay.x = 4, 8, 3, torch.float32, t
    lay.Wr = types.SimpleNamespace(device=torch.device("cuda:0"))
    for call in (lay.forward, lay.backward):
        with pytest.raises(ValueError, match="GPU"):
            call(t)


def test_layer_refuses_a_bias_of_another_size_or_type():
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    lay.T, lay.H, lay.E, lay.dtype = 4, 8, 3, torch.float32
    good = types.SimpleNamespace(shape=(4, 8), dtype=torch.float32, is_contiguous=lambda: True, device="gpu", is_cuda=True)
    lay.Wr = types.SimpleNamespace(device="gpu")
    for bad in (torch.zeros(2), torch.zeros(3, dtype=torch.bfloat16), torch.zeros(6)[::2]):
        with pytest.raises(ValueError, match="bias"):
            lay.forward(good, bad)


def test_a_stream_of_another_gpu_is_refused():
    tensor = types.SimpleNamespace(get_device=lambda: 0, data_ptr=lambda: 16)
    stream = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=1)
    with pytest.raises(ValueError, match="stream"):
        N._run((tensor,), stream, lambda at, st: 0)
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    lay.Wr, lay.streams = types.SimpleNamespace(device=torch.device("cuda:0")), {}
    with pytest.raises(ValueError, match="stream"):
        lay._work_on(stream)


def test_layer_calls_with_its_own_gpu_as_the_current_one(monkeypatch):
    """Every call of the library is made under the layer's GPU, whichever one is current."""
    current, calls = ["cuda:0"], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    names = ("moe_route_permute", "moe_gated_ffn", "moe_combine", "moe_combine_backward", "moe_gated_ffn_backward")
    for name in names:
        monkeypatch.setattr(N, name, lambda *a, name=name: calls.append((name, current[0])))
    monkeypatch.setattr(layer, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(layer, "_result", lambda *a: None)
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    for n in "T H E dtype w idx off slot_token pair_slot ws ones dy_perm".split():
        setattr(lay, n, None)
    lay.Wr, lay._work_on = types.SimpleNamespace(device="cuda:1", get_device=lambda: 1), lambda *a: None
    lay.shapes, lay.weights, lay.y, lay.dx, lay.grads, lay.pre = [1, 2], [{}, {}], [1, 2], [1, 2], [{}, {}], [[1, 1], [2, 2]]
    lay.forward("x")
    lay.backward("dy")
    assert {n for n, _ in calls} == set(names) and {d for _, d in calls} == {"cuda:1"}


def test_a_failed_forward_leaves_nothing_to_go_back_through(monkeypatch):
    """Part of what backward reads is the new batch's then, part the old one's."""
    def failing(*a):
        raise N.MoeError(4, "launch")
    monkeypatch.setattr(layer.TrainableLayer, "_gpu", lambda self: contextlib.nullcontext())
    monkeypatch.setattr(N, "moe_route_permute", lambda *a: None)
    monkeypatch.setattr(N, "moe_gated_ffn", failing)
    monkeypatch.setattr(layer, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(layer, "_result", lambda *a: None)
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    for n in "T H E dtype w idx off slot_token pair_slot ws".split():
        setattr(lay, n, None)
    lay.Wr, lay._work_on, lay.x = types.SimpleNamespace(device="cuda:0"), lambda *a: None, "the batch before"
    lay.shapes, lay.weights, lay.y, lay.pre = [1], [{}], [1], [[1, 1]]
    with pytest.raises(N.MoeError):
        lay.forward("x")
    with pytest.raises(RuntimeError):
        lay.backward("dy")


@pytest.mark.parametrize("fails_at", range(9))
def test_a_failed_set_tokens_leaves_a_layer_that_takes_no_batch(monkeypatch, fails_at):
    """Memory that runs out half way leaves buffers of two sizes, which no kernel may see."""
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    lay.H, lay.I, lay.E, lay.k, lay.act, lay.dtype, lay.weights = 256, 128, 4, 2, "f32", torch.float32, [{}]
    lay.Wr = torch.zeros(4)
    lay.set_tokens(4)
    lay.x = torch.zeros(4, 256)
    empty, left = torch.empty, [fails_at]

    def failing(*a, **kw):
        left[0] -= 1
        if left[0] < 0:
            raise MemoryError("no memory")
        return empty(*a, **kw)
    monkeypatch.setattr(torch, "empty", failing)
    with pytest.raises(MemoryError):
        lay.set_tokens(8)
    monkeypatch.undo()
    for T in (4, 8):
        with pytest.raises(ValueError, match="x:"):
            lay.forward(torch.zeros(T, 256))
    with pytest.raises(RuntimeError):
        lay.backward(torch.zeros(8, 256))
    lay.set_tokens(8)
    assert lay.T == 8 and lay.pre[0][0].shape == (16, 128)


# ------------------------------------------------------------------------------------------------
# arrays that overlap; addresses are never read

def adamw(*tensors, state=0, p_type=1, g_type=1, **kw):
    c = N.MoeAdamwConfig(p_type=p_type, g_type=g_type, state=state, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, **kw)
    arr = (N.MoeAdamwTensor * len(tensors))(*[N.MoeAdamwTensor(**t) for t in tensors])
    rc = N.load().moe_adamw(ctypes.byref(c), arr, len(tensors), None)
    return rc, N.load().moe_last_error().decode()


def tensor(at, n=600, q8=False, **kw):
    t = dict(p=at, g=at + 0x1000, m=at + 0x2000, v=at + 0x3000, n=n)
    if q8:
        t |= dict(m_scale=at + 0x4000, v_scale=at + 0x5000)
    return t | kw


# 600 elements take 1200 bytes of bf16, 2400 of fp32, 600 of codes and 12 of scales
@pytest.mark.parametrize("state,other", [
    (1, dict(v_scale=0x24000)), (1, dict(v_scale=0x24008)), (1, dict(m_scale=0x23FF8, v_scale=0x24000)),
    (1, dict(m_scale=0x14000)), (1, dict(v_scale=0x14008)), (1, dict(m_scale=0x15004)), (1, dict(m_scale=0x12254)),
    (1, dict(p=0x14000)), (1, dict(m=0x15000)),
    (0, dict(g=0x20000)), (0, dict(g=0x22000)), (0, dict(g=0x10000)), (0, dict(g=0x104A0)), (0, dict(g=0x0FFF0)),
    (0, dict(g=0x12950)), (0, dict(g=0x13000)), (1, dict(g=0x14000)), (1, dict(g=0x14FF0))])
def test_adamw_refuses_overlapping_arrays(state, other):
    q8 = state == 1
    rc, text = adamw(tensor(0x10000, q8=q8), tensor(0x20000, q8=q8, **other), state=state)
    assert rc == 1 and "overlap" in text


@pytest.mark.parametrize("kw", [dict(lr_dev=0x10010), dict(step_dev=0x12000), dict(grad_scale=0x12950), dict(step_dev=0x104A8)])
def test_adamw_refuses_device_values_inside_updated_arrays(kw):
    rc, text = adamw(tensor(0x10000), **kw)
    assert rc == 1 and "overlap" in text


@pytest.mark.parametrize("eps", [2.0 ** -1074, 1e-44, 1e-39, 2.0 ** -127])
def test_adamw_refuses_an_eps_below_the_normal_numbers(eps):
    c = N.MoeAdamwConfig(p_type=1, g_type=1, state=0, lr=1e-3, beta1=0.9, beta2=0.95, eps=eps, step=1)
    arr = (N.MoeAdamwTensor * 1)(N.MoeAdamwTensor(**tensor(0x10000)))
    assert N.load().moe_adamw(ctypes.byref(c), arr, 1, None) == 1 and "eps" in N.load().moe_last_error().decode()


P = ctypes.c_void_p
# T 4, k 2, E 2, H 256, I 128 in bf16: x 2048 bytes, rows of H 4096, of I 2048, a weight 131072, offsets 12, slots 32,
# workspace under 0x10000
BLOCK = dict(x=0x100000, off=0x110000, slot=0x120000, gate=0x200000, up=0x300000, down=0x400000, g=0x500000, u=0x510000,
             dy=0x520000, y=0x600000, dgate=0x700000, dup=0x800000, ddown=0x900000, ws=0xA00000)


def block(gradient, **kw):
    a = BLOCK | kw
    s = N.make_shape(4, 256, 2, 2, 128)
    w = N.MoeWeights(a["gate"], a["up"], a["down"], None, None, None)
    ws, size = P(a["ws"]), N.moe_train_workspace_size(s)
    assert size < 0x10000
    if gradient:
        grads = N.MoeWeightGrads(a["dgate"], a["dup"], a["ddown"])
        rc = N.load().moe_gated_ffn_backward(ctypes.byref(s), P(a["x"]), P(a["off"]), P(a["slot"]), ctypes.byref(w), P(a["g"]),
                                             P(a["u"]), P(a["dy"]), P(a["y"]), ctypes.byref(grads), ws, size, None)
    else:
        rc = N.load().moe_gated_ffn(ctypes.byref(s), P(a["x"]), P(a["off"]), P(a["slot"]), ctypes.byref(w), P(a["g"]), P(a["u"]),
                                    P(a["y"]), ws, size, None)
    return rc, N.load().moe_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(u=0x5007F0), dict(g=0x5107F0), dict(y=0x5007F0), dict(y=0x4FF010), dict(y=0x1007F0), dict(y=0x21FFF0), dict(y=0x300000),
    dict(g=0x41FFF0), dict(g=0x400000), dict(y=0x10FFF0), dict(y=0x11F010), dict(y=0xA00000), dict(g=0xA00800), dict(u=0x9FF810),
    dict(ws=0x300000), dict(ws=0x5FFF00), dict(ws=0x100700), dict(ws=0x110000)])
def test_block_refuses_overlapping_outputs(kw):
    rc, text = block(False, **kw)
    assert rc == 1 and "memory" in text


@pytest.mark.parametrize("kw", [
    dict(y=0x520FF0), dict(y=0x51F010), dict(y=0x5007F0), dict(y=0x1007F0), dict(y=0x21FFF0), dict(dgate=0x4E0010),
    dict(dup=0x71FFF0), dict(ddown=0x7E0010), dict(dgate=0x5FFFF0), dict(dup=0x520FF0), dict(ddown=0x3FFFF0),
    dict(dgate=0x0E0010), dict(dup=0x110000), dict(dgate=0xA00000), dict(y=0xA00800), dict(ws=0x900000), dict(ws=0x500700),
    dict(ws=0x120000), dict(ws=0x200000)])
def test_block_gradient_refuses_overlapping_outputs(kw):
    rc, text = block(True, **kw)
    assert rc == 1 and "memory" in text


# T 4, k 2, H 256 in bf16: dy 2048 bytes, rows 4096, slots and weights 32
@pytest.mark.parametrize("kw", [
    dict(rows=0x200FF0), dict(rows=0x1FF010), dict(rows=0x1007F0), dict(rows=0x2FFFF0), dict(rows=0x400010 - 0x1000), dict(dw=0x2007F0),
    dict(dw=0x100000), dict(dw=0x300010), dict(dw=0x40001C), dict(dw=0x3FFFE4), dict(dw=0x500FF0)])
def test_combine_gradient_refuses_overlapping_outputs(kw):
    a = dict(dy=0x100000, y=0x200000, slot=0x300000, w=0x400000, rows=0x500000, dw=0x600000) | kw
    s = N.make_shape(4, 256, 2, 2, 128)
    rc = N.load().moe_combine_backward(ctypes.byref(s), *[P(v) for v in a.values()], None)
    assert rc == 1 and "memory" in N.load().moe_last_error().decode()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_the_path_does_not_matter_to_training(act):
    """H = 256 and I = 128 have no prefill kernel, nor have f32 weights: that is the inference forward's matter."""
    sizes = {N.moe_train_workspace_size(N.make_shape(4, 256, 2, 2, 128, act=act, w_routed=act, path=path))
             for path in ("auto", "decode", "prefill")}
    assert len(sizes) == 1


# ------------------------------------------------------------------------------------------------
# the bound on the error of fp32 products, against sums made in other ways

def summed(a, b, round_length):
    """a [K, m], b [K, n]: sum_k a[k, :, None] b[k, None, :], each addition rounded to fp32, sums of round_length
    elements added to a total."""
    total = np.zeros((a.shape[1], b.shape[1]), np.float32)
    for k0 in range(0, len(a), round_length):
        acc = np.zeros_like(total)
        for k in range(k0, min(k0 + round_length, len(a))):
            acc = (acc + np.outer(a[k].astype(np.float64), b[k])).astype(np.float32)
        total = total + acc
    return total


@pytest.mark.parametrize("K", [4096, 20000])
def test_error_bound_tells_the_ways_of_summing_apart(K):
    rng = np.random.default_rng(K)
    a, b = (rng.standard_normal((K, 24)).astype(np.float32) for _ in range(2))
    want = a.astype(np.float64).T @ b

    def far(x):
        return np.linalg.norm(x - want) / np.linalg.norm(want)
    half = [torch.from_numpy(t).bfloat16().float().numpy() for t in (a, b)]
    assert far(summed(a, b, 128)) <= chain_error(K)
    assert far(summed(a, b, K)) > chain_error(K)           # one chain
    assert far(summed(*half, 128)) > 100 * chain_error(K)  # bf16 operands
