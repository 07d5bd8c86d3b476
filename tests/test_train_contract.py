"""What TrainableLayer and the training entry points refuse before any launch (no GPU)."""
import contextlib
import ctypes
import types

import pytest
import torch

from expert_ffn_layer_amd import layer, native as N
from inputgen import layers as L

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
    lay.Wr, lay.streams = types.SimpleNamespace(device=torch.device("cuda:0")), set()
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
    names = ("moe_route_permute", "moe_gated_ffn", "moe_combine", "moe_combine_backward", "moe_gated_ffn_backward")
    for name in names:
        monkeypatch.setattr(N, name, lambda *a, name=name: calls.append((name, current[0])))
    monkeypatch.setattr(layer, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(layer, "_result", lambda *a: None)
    lay = layer.TrainableLayer.__new__(layer.TrainableLayer)
    for n in "T H E dtype w idx off slot_token pair_slot ws ones dy_perm".split():
        setattr(lay, n, None)
    lay.Wr, lay._work_on = types.SimpleNamespace(device="cuda:1"), lambda *a: None
    lay.shapes, lay.weights, lay.y, lay.dx, lay.grads, lay.pre = [1, 2], [{}, {}], [1, 2], [1, 2], [{}, {}], [[1, 1], [2, 2]]
    lay.forward("x")
    lay.backward("dy")
    assert {n for n, _ in calls} == set(names) and {d for _, d in calls} == {"cuda:1"}


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
