"""The dropouts of a block's step, without a GPU: the calls of the library are replaced."""
import torch

from test_layer_cpu import layer, step_of  # noqa: F401  (layer: a fixture)


def test_the_ways_in_and_out_draw_their_own_masks(layer, monkeypatch):  # noqa: F811
    """Both drop rows of the same shape, so with one rng only the offsets tell their masks apart: by default they do, in
    the same step and in others whose rng[1] has moved by one or more; each gradient takes its forward's."""
    seen = {}
    monkeypatch.setattr(layer, "moe_layer_norm", lambda *a, **k: seen.update(enter=k["offset"]))
    monkeypatch.setattr(layer, "moe_layer_norm_backward", lambda *a, **k: seen.update(enter_backward=k["offset"]))
    monkeypatch.setattr(layer, "moe_dropout", lambda *a, **k: seen.update(
        {"leave" if k.get("residual") is not None else "leave_backward": k["offset"]}))
    x, w, rng = torch.zeros(4, 32), torch.ones(32), torch.tensor([7, 0])
    L = step_of(layer, norm="rms", backward_enabled=True, x_all=torch.zeros(8, 32), out=x.clone(), total=x.clone(), norm_mean=None,
                norm_rstd=torch.zeros(4), norm_ws=torch.zeros(8), dout_all=torch.zeros(8, 32))
    L.enter(x, w, residual=x, p=0.1, rng=rng)
    L.leave(x.clone(), p=0.1, rng=rng)
    L.leave_backward(x, p=0.1, rng=rng)
    L.enter_backward(x, w, x.clone(), w, p=0.1, rng=rng)
    assert seen["enter"] == seen["enter_backward"] and seen["leave"] == seen["leave_backward"]
    apart = (seen["leave"] - seen["enter"]) % 2 ** 64
    assert 2 ** 32 <= apart <= 2 ** 64 - 2 ** 32
    # an offset that is given is taken as it is
    L.leave(x.clone(), p=0.1, rng=rng, offset=5)
    L.leave_backward(x, p=0.1, rng=rng, offset=-6)
    assert seen["leave"] == 5 and seen["leave_backward"] == -6
