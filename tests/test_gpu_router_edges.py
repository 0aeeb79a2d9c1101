"""The router where its other tests do not go, against float64."""
import numpy as np
import pytest
import torch

from oracle import scaled_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def topk(m, x, K, score, bias=None, factor=1.0):
    idx = torch.full((x.shape[0], K), -9, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], K), -9.0, device="cuda")
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    m.moe_router_topk(x, idx, w, score, b, factor)
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def backward(m, x, idx, dw, score, factor=1.0):
    d = torch.full_like(x, 3.0)
    m.moe_router_backward(x, torch.from_numpy(np.asarray(idx, np.int32)).cuda(),
                          torch.from_numpy(np.asarray(dw, np.float32)).cuda(), d, score, factor)
    return d


def weight_tol(x, n):
    """Relative error of a weight: the exponents' arguments are rounded once (2^-24 of the spread of the
    logits), exp, the two divisions, 1 + exp and the factor give at most two steps (2^-23) each, the sum of n
    terms one rounding each."""
    return (float(np.ptp(x)) + n + 16) * 2.0 ** -23


FAR = [-90.0, -94.0, -104.0, -150.0, -300.0, -700.0, -2000.0, -30000.0]


def far_rows(E, dtype):
    """Rows of logits within 8 of each other around far places, and rows that reach from ordinary ones to
    them, rounded to the given type."""
    r = np.random.default_rng(E)
    x = np.stack([at - r.integers(0, 9, E) for at in FAR] + [r.integers(-99, -60, E), r.integers(-95, 3, E),
                                                             np.where(np.arange(E) % 3, -100.0, -88.0)])
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(2, 2), (7, 3), (64, 6), (130, 20), (256, 8), (300, 40), (1024, 8)])
def test_logistic_of_far_logits(m, E, K, dtype, many):
    """Chosen logits so low that exp(-x) or the logistic itself leaves fp32: weights that sum to the factor, and their
    gradient.  many: more tokens than any device's 8 per compute unit."""
    x = far_rows(E, dtype)
    xd = x.double().numpy()
    rows = np.arange(8209) % len(xd) if many else np.arange(len(xd))
    xs = x[torch.from_numpy(rows)].cuda()
    idx, w = topk(m, xs, K, "sigmoid", factor=2.5)
    widx, ww = ref.router_topk(xd, K, "sigmoid", factor=2.5)
    assert np.array_equal(idx, widx[rows])
    assert np.array_equal(w, w[:len(xd)][rows])
    tol = np.array([weight_tol(r, K) for r in xd])[:, None]
    assert (np.abs(w[:len(xd)] - ww) <= tol * ww + 2.0 ** -125).all()
    assert (np.abs(w[:len(xd)].sum(1) - 2.5) <= 2.5 * tol[:, 0]).all()
    dw = np.random.default_rng(1).standard_normal((len(xd), K)).astype(np.float32)
    want = ref.router_backward(xd, widx, dw, "sigmoid", 1.5)
    d = backward(m, xs, widx[rows], dw[rows], "sigmoid", 1.5)
    assert torch.equal(d, d[:len(xd)][torch.from_numpy(rows).cuda()])
    # each entry: a weight times a difference of gradients of at most 1.5 sum |dw|, and 1 - logistic
    mag = 1.5 * np.abs(dw).astype(np.float64).sum(1, keepdims=True)
    half = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0
    assert (np.abs(d[:len(xd)].double().cpu().numpy() - want) <= 4 * tol * mag + half + 2.0 ** -125).all()


def test_logistic_of_far_logits_against_differences(m):
    """Central differences of the kernel's own weights, h = 1/16, at logits that hold every step exactly
    (multiples of 2^-10 above -2^9): off by h^2 / 12 of sum |dw| (the third derivative of a weight in one
    logit is below 1/2) and by the weights' own rounding over h."""
    T, E, K, h = 3, 12, 4, 1.0 / 16
    x = (np.random.default_rng(0).integers(-512, 512, (T, E)) / 1024.0).astype(np.float32)
    x[:, K:] -= 20.0
    x += np.array([-92.0, -120.0, -400.0], np.float32)[:, None]
    dw = np.random.default_rng(1).standard_normal((T, K)).astype(np.float32)
    d = backward(m, torch.from_numpy(x).cuda(), np.tile(np.arange(K), (T, 1)), dw, "sigmoid").cpu().numpy()

    def value(y):
        idx, w = topk(m, torch.from_numpy(y).cuda(), K, "sigmoid")
        return np.array([sum(w[t, k] * dw[t, idx[t, k]] for k in range(K)) for t in range(T)])

    tol = (h * h / 12 + 2 * weight_tol(x[0], K) / h) * np.abs(dw).sum(1)
    for e in range(K):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        assert (np.abs((value(up) - value(down)) / (2 * h) - d[:, e]) <= tol).all()
    assert (d[:, K:] == 0).all() and (np.abs(d[:, :K]).max(1) > 1e-2).all()


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("score", ["softmax_topk", "softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(3, 2), (64, 5), (130, 130), (256, 8), (300, 40), (1024, 8)])
def test_bias_orders_masked_rows(m, E, K, score, many):
    """Rows without a logit above -inf, with one, with half: the bias alone orders experts whose score is 0."""
    r = np.random.default_rng(E)
    x = r.standard_normal((7, E)).astype(np.float32)
    x[1] = -np.inf
    x[2, np.arange(E) != E // 2] = -np.inf
    x[4] = -np.inf
    x[5, ::2] = -np.inf
    bias = r.permutation(np.linspace(-1.0, 1.0, E)).astype(np.float32)
    rows = np.arange(8209) % 7 if many else np.arange(7)
    idx, w = topk(m, torch.from_numpy(x[rows]).cuda(), K, score, bias)
    widx, ww = ref.router_topk(x.astype(np.float64), K, score, bias)
    assert np.array_equal(idx, widx[rows])
    finite = np.where(np.isfinite(x), x, 0.0).astype(np.float64)
    assert (np.abs(w - ww[rows]) <= weight_tol(finite, E) * ww[rows]).all()
    assert (w[rows == 1] == 0).all() and (w[rows == 4] == 0).all()
