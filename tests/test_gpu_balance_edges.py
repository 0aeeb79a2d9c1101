"""The balance loss of logits far below 0."""
import numpy as np
import pytest
import torch

from block_common import F32, U, exactly, tensor
from oracle import block_ref as ref
from test_gpu_balance import gradient, losses

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


@pytest.mark.parametrize("n", [64, 200])
@pytest.mark.parametrize("top", [-1.5, -8.0, -12.0, -16.0, -17.0, -18.0, -20.0, -40.0, -55.0, -59.0, -60.5, -80.0, -100.0, -1000.0])
def test_logistic_of_low_rows(m, top, n):
    """Two logits just below `top`, a sequence a token, all copies at the larger one: balance is 2 P_0.

    Only the distance of the logits (at most 1/4, exact) goes through an exponential that tells them apart, however low both
    are.  In U: the smaller one's exponential 1/4 of 2.25 (product, constant) and 2 for itself; 1 + t, with t in error by
    |m| (1.25) + 2 of its share, which is at most 1, and by 0.7 from the exponential, and rounded: 2.7; the reciprocal 2, the
    product 1: 5.7 and 8.3 for the two numerators.  P_0 is at least 1/2: half of their sum, 7, and 1 for the sum, 2 for
    its reciprocal, 1 for the product, 1 for the result: 12."""
    r = np.random.default_rng(int(-top * 8) + n)
    x = top - r.random((n, 1)) + np.array([[0.0, -1.0]]) * r.random((n, 1)) / 4
    x = tensor(x, F32)
    x[:, 1] = torch.minimum(x[:, 1], x[:, 0])
    counts = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda").repeat(n, 1)
    cu = list(range(n + 1))
    b, _ = losses(m, x, counts, cu, "sigmoid")
    want, _ = ref.balance_loss(exactly(x), exactly(counts), np.array(cu), "sigmoid")
    assert (np.abs(exactly(b) - want) <= 13 * U * want).all()
    # the gradient: P_0 (1 - P_0) (1 - logistic): 12 for P_0, 12 P_0 / (1 - P_0) <= 16 and a rounding for the difference, 5
    # for the rest, 3 products
    one = torch.ones(n, device="cuda")
    got = exactly(gradient(m, x, counts, cu, one, None, "sigmoid"))
    want = ref.balance_loss_backward(exactly(x), exactly(counts), np.array(cu), np.ones(n), np.zeros(n), "sigmoid")
    assert (np.abs(got - want) <= 40 * U * np.abs(want)).all()
