"""What LayerStep checks and keeps on the host, without a GPU: the calls of the library are replaced."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def layer():
    if not os.path.exists(os.path.join(ROOT, "balanced_token_dispatch_amd", "libmoe.so")):
        pytest.skip("libmoe.so not built")
    from balanced_token_dispatch_amd import layer
    return layer


def step_of(layer, **attrs):
    """A LayerStep of R2 S4 K2 E6 B1 H32 H'16 with the given attributes, none of its buffers made."""
    L = layer.LayerStep.__new__(layer.LayerStep)
    L.s, L.rank = layer.Shape(2, 4, 2, 6, 1, 32, 16), 1
    L.topk_idx, L.topk_w = torch.zeros(2, 4, 2, dtype=torch.int32), torch.zeros(2, 4, 2)
    for k, v in attrs.items():
        setattr(L, k, v)
    return L


def test_route_takes_logits_of_this_layers_experts(layer, monkeypatch):
    """More columns than experts would make ids that no expert has, fewer would leave experts out."""
    seen = []
    monkeypatch.setattr(layer, "moe_router_topk", lambda *a: seen.append(a))
    monkeypatch.setattr(layer, "moe_router_backward", lambda *a: seen.append(a))
    L = step_of(layer, dtopk_w=torch.zeros(8))
    for shape in ((4, 7), (4, 5), (5, 6), (24,), (1, 4, 6)):
        x = torch.zeros(shape)
        with pytest.raises(layer.MoeError, match="logits"):
            L.route(x)
        with pytest.raises(layer.MoeError, match="logits"):
            L.route_backward(x, torch.zeros_like(x))
    assert not seen
    x = torch.zeros(4, 6)
    L.route(x)
    L.route_backward(x, torch.zeros_like(x))
    assert len(seen) == 2
