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


class Reached(Exception):
    """The step went on to its first call."""


def scaled_step(layer, monkeypatch, **attrs):
    """An 8-bit LayerStep with weights whose quantising is recorded and whose forward stops at the plan."""
    calls = []
    monkeypatch.setattr(layer, "moe_quant_weight", lambda *a: calls.append(a))

    def plan(*a):
        raise Reached
    monkeypatch.setattr(layer, "moe_plan", plan)
    w = dict(w_up=torch.ones(7, 32, 16), w_down=torch.ones(7, 16, 32))
    L = step_of(layer, scaled=True, plan_noalloc=False, counts=None, plan=None, status=None, ws=None, d=None,
                quantised_from=None, **w, **attrs)
    L.q_up, L.q_down = layer.QuantWeights(L.w_up), layer.QuantWeights(L.w_down)
    return L, calls


def test_forward_refuses_weights_changed_since_they_were_quantised(layer, monkeypatch):
    """An update in place (a whole tensor, a view of it, an optimizer's step on a parameter over it) or another tensor in
    the weights' place: forward() would run on the old 8-bit ones."""
    L, _ = scaled_step(layer, monkeypatch)

    def adam():
        p = torch.nn.Parameter(L.w_down)
        p.grad = torch.ones_like(p)
        torch.optim.AdamW([p]).step()

    def replaced():
        L.w_up = L.w_up.clone()

    def in_inference():
        with torch.inference_mode():
            L.w_down.mul_(2.0)

    for change in (lambda: L.w_up.add_(1.0), lambda: L.w_down[2].copy_(torch.zeros(16, 32)), adam, replaced, in_inference):
        L.quantise_weights()
        for _ in range(2):
            with pytest.raises(Reached):
                L.forward()
        change()
        with pytest.raises(ValueError, match="quantise_weights"):
            L.forward()
    L.quantise_weights()
    with pytest.raises(Reached):
        L.forward()


def test_weights_made_in_inference_mode(layer, monkeypatch):
    """They do not count their changes: the first quantising is asked for, later ones are the caller's."""
    with torch.inference_mode():
        L, _ = scaled_step(layer, monkeypatch)
        with pytest.raises(ValueError, match="quantise_weights"):
            L.forward()
        L.quantise_weights()
        with pytest.raises(Reached):
            L.forward()


@pytest.mark.parametrize("backward", [False, True])
def test_a_forward_only_layer_keeps_one_order_of_weights(layer, monkeypatch, backward):
    """The input gradients' order is neither held nor written nor moved to the slots without a backward."""
    L, calls = scaled_step(layer, monkeypatch, backward_enabled=backward)
    L.q_up, L.q_down = (layer.QuantWeights(w, dgrad=backward) for w in (L.w_up, L.w_down))
    L.quantise_weights()
    for (w, q, q_scale, qt, qt_scale), whole in zip(calls, (L.w_up, L.w_down)):
        assert w.shape[0] == qt.shape[0] == qt_scale.shape[0] == 6 and w.data_ptr() == whole.data_ptr()
        assert (q is not None) == (q_scale is not None) == backward
    assert [t is None for t in L.q_up.tensors()] == [not backward] * 2 + [False] * 2
    moved = []
    for name in ("moe_plan", "moe_dispatch_layout"):
        monkeypatch.setattr(layer, name, lambda *a: None)
    monkeypatch.setattr(layer, "moe_prefetch", lambda d, r, plan, t: moved.append(t))

    def rows(*a, **k):
        raise Reached
    monkeypatch.setattr(layer, "moe_quant_rows", rows)
    for name in ("cu", "dest", "src", "x_all", "xp", "xq"):
        setattr(L, name, layer.QuantRows(1, 16, torch.float8_e4m3fn, "cpu") if name == "xq" else None)
    with pytest.raises(Reached):
        L.forward()
    assert len(moved) == (8 if backward else 4) and all(t is not None for t in moved)


def test_weights_put_into_8_bits_elsewhere(layer, monkeypatch):
    """A caller that writes q_up and q_down itself (from a checkpoint in 8 bits) says so."""
    L, calls = scaled_step(layer, monkeypatch)
    L.weights_quantised = True
    assert not calls and L.weights_quantised
    with pytest.raises(Reached):
        L.forward()
    L.w_up.add_(1.0)
    assert not L.weights_quantised
    L.weights_quantised = True
    L.weights_quantised = False
    with pytest.raises(ValueError, match="quantise_weights"):
        L.forward()


def test_a_block_takes_rows_of_this_layer(layer, monkeypatch):
    """enter(), leave() and their gradients take [S, H] tensors, on a layer that was made with a norm."""
    seen = []
    for name in ("moe_layer_norm", "moe_layer_norm_backward", "moe_dropout"):
        monkeypatch.setattr(layer, name, lambda *a, **k: seen.append((a, k)))
    x = torch.zeros(4, 32)
    L = step_of(layer, norm="rms", backward_enabled=True, x_all=torch.zeros(8, 32), out=x.clone(), total=x.clone(), norm_mean=None,
                norm_rstd=torch.zeros(4), norm_ws=torch.zeros(8), dout_all=torch.zeros(8, 32))
    w = torch.ones(32)
    calls = (lambda L, t: L.enter(t, w), lambda L, t: L.enter(x, w, residual=t), lambda L, t: L.leave(t),
             lambda L, t: L.leave_backward(t), lambda L, t: L.enter_backward(t, w, x, w), lambda L, t: L.enter_backward(x, w, t, w),
             lambda L, t: L.enter_backward(x, w, x, w, dtotal=t), lambda L, t: L.enter_backward(x, w, x, w, dresidual=t))
    for call in calls:
        for bad in (torch.zeros(5, 32), torch.zeros(4, 31), torch.zeros(128)):
            with pytest.raises(layer.MoeError, match="expected"):
                call(L, bad)
        with pytest.raises(ValueError, match="without a norm"):
            call(step_of(layer, norm=None), x)
    forward_only = step_of(layer, norm="rms", backward_enabled=False)
    for call in calls[3:]:
        with pytest.raises(ValueError, match="without a backward"):
            call(forward_only, x)
    assert not seen
    for call in calls:
        call(L, x)
    assert len(seen) == len(calls)
    # the rank's own rows: [4, 8) of x_all and dout_all
    assert seen[0][0][2].data_ptr() == L.x_all[4:].data_ptr() and seen[3][0][1].data_ptr() == L.dout_all[4:].data_ptr()


def test_balance_loss_takes_logits_of_this_layers_experts(layer, monkeypatch):
    seen = []
    for name in ("moe_expert_counts", "moe_balance_loss", "moe_balance_loss_backward"):
        monkeypatch.setattr(layer, name, lambda *a, **k: seen.append(a))
    L = step_of(layer, seq_counts=torch.zeros(1, 6, dtype=torch.int32), balance_ws=None)
    for bad in (torch.zeros(4, 7), torch.zeros(5, 6), torch.zeros(24)):
        with pytest.raises(layer.MoeError, match="logits"):
            L.balance_loss(bad, torch.zeros(1))
        with pytest.raises(layer.MoeError, match="logits"):
            L.balance_loss_backward(bad, bad)
    assert not seen
    assert L.count_experts() is L.seq_counts
    L.balance_loss(torch.zeros(4, 6), torch.zeros(1))
    L.balance_loss_backward(torch.zeros(4, 6), torch.zeros(4, 6))
    assert len(seen) == 3 and seen[0][0].data_ptr() == L.topk_idx[1].data_ptr()


def test_norm_and_sequences_are_checked(layer):
    for kw in (dict(norm="batch"), dict(sequences=0)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            layer.LayerStep(layer.Shape(2, 4, 2, 6, 1, 32, 16), device="cpu", **kw)
