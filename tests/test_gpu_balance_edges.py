"""The balance loss where the logistic is steepest, and every kernel of it on bounds that are none."""
import numpy as np
import pytest
import torch

from block_common import F32, U, exactly, tensor
from oracle import block_ref as ref
from test_gpu_balance import counts_of, gradient, losses, on_gpu

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


class Guarded:
    """A tensor inside a larger one, whose other bytes are checked."""

    def __init__(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.n, self.all = n, torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        self.t = self.all[4096:4096 + n].view(dtype).view(shape)

    def untouched(self):
        return bool((self.all[:4096] == 0x5A).all() and (self.all[4096 + self.n:] == 0x5A).all())


@pytest.mark.parametrize("T,E,K,n", [(9000, 16, 8, 70), (70000, 600, 1, 65), (150000, 8, 1, 300), (5000, 300, 2, 3)])
def test_bounds_out_of_range_of_many_tokens(m, T, E, K, n):
    """Bounds that fall or leave the tokens, in the kernels of many tokens and sequences: nothing outside the outputs and the
    scratch is written, and every call ends."""
    r = np.random.default_rng(T)
    x, idx = torch.randn(T, E, device="cuda"), torch.from_numpy(r.integers(-1, E + 1, (T, K)).astype(np.int32)).cuda()
    one = torch.ones(n, device="cuda")
    lowest, highest = -(1 << 31), (1 << 31) - 1
    falling = np.linspace(T, 0, n + 1).astype(np.int64)
    for cu in (falling, falling + T // 2, falling - T // 2, np.full(n + 1, T + 5), np.full(n + 1, -5),
               r.integers(-T, 2 * T, n + 1), np.where(r.random(n + 1) < 0.5, lowest, highest),
               np.where(np.arange(n + 1) % 2, 0, T)):
        counts, ws = Guarded((n, E), torch.int32), Guarded((m.balance_loss_workspace_bytes(T, n),), torch.uint8)
        b, z, g = Guarded((n,), F32), Guarded((n,), F32), Guarded((T, E), F32)
        at = on_gpu([int(v) for v in cu])
        m.moe_expert_counts(idx, counts.t, cu_tokens=at)
        for score in ("softmax", "sigmoid"):
            m.moe_balance_loss(x, counts.t, b.t, ws.t, zloss=z.t, score=score, cu_tokens=at)
            m.moe_balance_loss_backward(x, counts.t, g.t, dbalance=one, dzloss=one, score=score, cu_tokens=at)
        torch.cuda.synchronize()
        assert all(t.untouched() for t in (counts, ws, b, z, g))
    # bounds that hold still give what they mean
    cu = [0] + sorted(int(v) for v in r.integers(0, T + 1, n - 1)) + [T]
    ids = idx.cpu().numpy()
    which = np.repeat(np.arange(n), np.diff(cu))
    want = np.bincount((which[:, None] * E + ids)[(ids >= 0) & (ids < E)], minlength=n * E).reshape(n, E)
    assert np.array_equal(counts_of(m, idx, E, cu).cpu().numpy(), want)
