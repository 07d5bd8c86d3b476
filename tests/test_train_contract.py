"""What TrainableLayer and the training entry points refuse before any launch (no GPU)."""
import types

import pytest
import torch

from expert_ffn_layer_amd import layer
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
