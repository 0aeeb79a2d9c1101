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


def clipping_step(layer, monkeypatch):
    """A LayerStep whose clipping is computed by torch."""
    def sumsq(grads, out, ws):
        out.fill_(sum(float(g.double().square().sum()) for g in grads))

    def clip(grads, total, max_norm, norm):
        norm.copy_(total.sqrt())
        for g in grads:
            g.mul_(float(min(1.0, max_norm / (total.sqrt() + 1e-6))))

    monkeypatch.setattr(layer, "moe_grad_sumsq", sumsq)
    monkeypatch.setattr(layer, "moe_grad_clip", clip)
    return step_of(layer, dw_up=torch.ones(7, 32, 16), dw_down=torch.ones(7, 16, 32), clip_ws=None,
                   sumsq=torch.zeros(1, dtype=torch.float64), grad_norm=torch.zeros(1))


def test_clipping_has_no_norm_over_ranks(layer, monkeypatch):
    """An expert with replicas has a part of its gradient on each rank that holds one, and nothing in the step
    brings them together: the squares of the parts do not add up to the square of their sum."""
    L = clipping_step(layer, monkeypatch)
    with pytest.raises(TypeError):
        L.clip_gradients(1.0, group=object())
    assert (L.dw_up == 1.0).all()
    L.clip_gradients(1.0)
    assert float(L.dw_up[:6].double().square().sum() + L.dw_down[:6].double().square().sum()) == pytest.approx(1.0, rel=1e-6)


def test_a_kept_norm_stays(layer, monkeypatch):
    L = clipping_step(layer, monkeypatch)
    first = L.clip_gradients(1.0)
    value = first.item()
    assert value == pytest.approx((2 * 6 * 32 * 16) ** 0.5)
    second = L.clip_gradients(0.5)
    assert first.item() == value and second.item() == pytest.approx(1.0, rel=1e-6)
    assert L.grad_norm.item() == second.item()
