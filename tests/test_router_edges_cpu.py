"""The router's definition in float64 where its scores leave the range of float64, against decimal
arithmetic of 60 digits."""
from decimal import Decimal, localcontext

import numpy as np
import pytest

from oracle import scaled_ref as ref


def exact_logistic_weights(c, d):
    """(weights, gradients of sum(d w) in the logits) of the chosen logits c, by their definition."""
    with localcontext() as ctx:
        ctx.prec, ctx.Emin, ctx.Emax = 60, -10 ** 12, 10 ** 12
        s = [1 / (1 + (-Decimal(float(x))).exp()) for x in c]
        total = sum(s)
        w = [v / total for v in s]
        inner = sum(Decimal(float(a)) * b for a, b in zip(d, w))
        g = [b * (Decimal(float(a)) - inner) * (1 - v) for a, b, v in zip(d, w, s)]
        return np.array([float(v) for v in w]), np.array([float(v) for v in g])


@pytest.mark.parametrize("c", [(-94.0, -95.0), (-100.0, -101.0, -130.5), (-720.0, -700.0), (-800.0, -801.0, -2000.0),
                               (-30.0, -94.0), (5.0, -94.0, -800.0), (0.5, -1.5, 3.0), (-1e4, -1e4, -1e4 - 1)])
def test_logistic_weights_of_far_logits(c):
    c = np.array(c)
    d = np.linspace(-1.0, 2.0, len(c)) ** 3
    w, g = exact_logistic_weights(c, d)
    got = ref.router_weights(c, range(len(c)), "sigmoid")
    assert np.allclose(got, w, rtol=1e-13, atol=1e-300)
    grad = ref.router_backward(c[None], np.arange(len(c))[None], d[None], "sigmoid")[0]
    assert np.allclose(grad, g, rtol=1e-12, atol=1e-14 * np.abs(d).sum())


def test_logistic_weights_of_masked_logits():
    """-inf weighs nothing, also where all are; the type's lowest value is a number like any other."""
    low = float(np.finfo(np.float32).min)
    w = lambda *c: list(ref.router_weights(np.array(c), range(len(c)), "sigmoid"))  # noqa: E731
    assert w(-np.inf, -np.inf) == [0.0, 0.0]
    assert w(-np.inf, -900.0) == [0.0, 1.0]
    assert w(low, low, low, low) == [0.25] * 4
    assert w(low, 1.0) == [0.0, 1.0]
    assert np.isnan(w(np.nan, 1.0)).all()


@pytest.mark.parametrize("score", ["softmax_topk", "softmax", "sigmoid"])
def test_bias_orders_a_fully_masked_row(score):
    """Where every logit is -inf every score is 0 (the logit itself for softmax_topk: no order but the ids), so the
    bias alone chooses; all weights are 0."""
    bias = np.array([0.5, -1.0, 2.0, 0.25, 2.0])
    ids, w = ref.router_topk(np.full((1, 5), -np.inf), 3, score, bias)
    assert list(ids[0]) == ([0, 1, 2] if score == "softmax_topk" else [2, 4, 0])
    assert (w == 0).all()
