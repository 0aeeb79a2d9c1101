"""The router and its gradient on the GPU against float64."""
import numpy as np
import pytest
import torch

from oracle import scaled_ref as ref

pytestmark = pytest.mark.gpu
SCORES = ["softmax_topk", "softmax", "sigmoid"]
SHAPES = [(1, 1, 1), (1, 2, 2), (5, 7, 3), (33, 64, 6), (9, 65, 8), (17, 256, 8), (4, 257, 12), (6, 384, 8),
          (3, 513, 1), (2, 1024, 16), (2, 100, 100), (1, 1024, 1024)]


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def logits_of(seed, T, E, dtype):
    """Normal logits (with repeats, so that ties are met) as the given type."""
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32))
    x[:, ::5] = (x[:, ::5] * 2).round() / 2
    return x.to(dtype).cuda()


def topk(m, x, K, score, bias=None, factor=1.0):
    idx = torch.full((x.shape[0], K), -9, dtype=torch.int32, device="cuda")
    w = torch.full((x.shape[0], K), -9.0, device="cuda")
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    m.moe_router_topk(x, idx, w, score, b, factor)
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def weight_tol(x, n):
    """Relative error of a weight: the exponent's argument is rounded once (2^-24 of its size, at most
    the spread of the logits, or their size for the logistic), exp, the division and the factor give
    at most two steps (2^-23) each, the sum of n terms one rounding each."""
    x = x[np.isfinite(x)]
    spread = max(float(np.ptp(x)), float(np.abs(x).max())) if x.size else 0.0
    return (spread + n + 16) * 2.0 ** -23


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_topk(m, score, T, E, K, dtype):
    x = logits_of(T * E + K, T, E, dtype)
    idx, w = topk(m, x, K, score, factor=2.5)
    xd = x.double().cpu().numpy()
    widx, ww = ref.router_topk(xd, K, score, factor=2.5)
    assert np.array_equal(idx, widx)
    assert (np.abs(w - ww) <= weight_tol(xd, E) * ww).all()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,K", [(5, 7, 3), (17, 256, 8), (6, 384, 8), (2, 1000, 16)])
def test_topk_bias(m, score, T, E, K):
    x = logits_of(3, T, E, torch.float32)
    bias = np.random.default_rng(4).standard_normal(E).astype(np.float32)
    bias[::3] = 0.0
    idx, w = topk(m, x, K, score, bias)
    xd = x.double().cpu().numpy()
    widx, ww = ref.router_topk(xd, K, score, bias)
    assert np.array_equal(idx, widx)
    assert (np.abs(w - ww) <= weight_tol(xd, E) * ww).all()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E", [4, 64, 130, 300, 900])
def test_topk_masked(m, score, E):
    """Masked experts (-inf, or the type's lowest value), rows with fewer left than K, rows with none,
    all equal, signed zeros."""
    K = min(E, 8)
    x = np.random.default_rng(E).standard_normal((8, E)).astype(np.float32)
    x[0, ::2] = -np.inf
    x[1, 1:] = -np.inf
    x[2, :] = -np.inf
    x[3, :] = np.finfo(np.float32).min
    x[4, : E // 2] = np.finfo(np.float32).min
    x[5, :] = 1.5
    x[6, :] = np.where(np.arange(E) % 2, 0.0, -0.0)
    x[7, E - 1] = 60.0
    idx, w = topk(m, torch.from_numpy(x).cuda(), K, score)
    widx, ww = ref.router_topk(x.astype(np.float64), K, score)
    assert np.array_equal(idx, widx)
    assert np.isfinite(w).all()
    finite = np.where(np.abs(x) < 1e30, x, 0.0).astype(np.float64)
    assert (np.abs(w - ww) <= weight_tol(finite, E) * ww + 2.0 ** -126).all()


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E,K", [(3, 3), (64, 5), (65, 8), (128, 8), (130, 130), (251, 8), (256, 16), (300, 8), (512, 12),
                                 (513, 70), (1024, 8)])
def test_topk_many_tokens(m, score, E, K, bias):
    """More tokens than any device's 8 per compute unit, not a multiple of a wave's: normal rows between
    masked, equal, tied, NaN and infinite ones, which share waves with them."""
    r = np.random.default_rng(E + K)
    x = r.standard_normal((37, E)).astype(np.float32)
    x[:, ::5] = np.round(x[:, ::5] * 2) / 2
    x[3] = -np.inf
    x[8] = 0.25
    x[11, ::2] = -np.inf
    x[17, E // 2] = np.nan
    x[20] = np.finfo(np.float32).min
    T = 8209
    rows = np.arange(T) % 37
    b = r.standard_normal(E).astype(np.float32) if bias else None
    keep = np.ones(37, bool)
    if bias and score == "softmax":
        keep[[3, 17]] = False   # scores of NaN over all experts: no order to compare
    idx, w = topk(m, torch.from_numpy(x[rows]).cuda(), K, score, b)
    assert (idx.min(1) >= 0).all() and (idx.max(1) < E).all()
    k = keep[rows]
    assert np.array_equal(idx[k], idx[:37][rows][k]) and np.array_equal(w[k], w[:37][rows][k], equal_nan=True)
    widx, ww = ref.router_topk(x[keep].astype(np.float64), K, score, b)
    assert np.array_equal(idx[:37][keep], widx)
    finite = np.where(np.abs(x) < 1e30, x, 0.0).astype(np.float64)
    finite[np.isnan(x)] = 0.0
    got = w[:37][keep]
    assert np.array_equal(np.isnan(got), np.isnan(ww))
    ok = ~np.isnan(ww)
    assert (np.abs(got - ww)[ok] <= (weight_tol(finite, E) * ww + 2.0 ** -126)[ok]).all()


def test_topk_nan_first(m):
    x = np.zeros((2, 70), np.float32)
    x[0, 65] = np.nan
    x[0, 3] = np.inf
    x[1, 9] = 2.0
    idx, w = topk(m, torch.from_numpy(x).cuda(), 3, "softmax_topk")
    assert list(idx[0][:2]) == [65, 3] and np.isnan(w[0]).all()
    assert idx[1][0] == 9 and np.isfinite(w[1]).all()


def run_backward(m, x, idx, dw, score, factor=1.0):
    d = torch.full_like(x, 3.0)
    m.moe_router_backward(x, torch.from_numpy(np.asarray(idx, np.int32)).cuda(),
                          torch.from_numpy(np.asarray(dw, np.float32)).cuda(), d, score, factor)
    return d


def grad_close(d, want, xd, dw, factor, dtype):
    """Errors of d against want: each term is a weight (see weight_tol) times a gradient, the terms are
    added in fp32; their magnitudes are at most factor * sum |dw|."""
    E = xd.shape[1]
    mag = factor * np.abs(dw).astype(np.float64).sum(1, keepdims=True)
    tol = 4 * weight_tol(xd, E) * mag + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0)
    return (np.abs(d.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(m, score, T, E, K, dtype):
    x = logits_of(T + E + K, T, E, dtype)
    xd = x.double().cpu().numpy()
    idx, _ = ref.router_topk(xd, K, score)
    dw = np.random.default_rng(2).standard_normal((T, K)).astype(np.float32)
    want = ref.router_backward(xd, idx, dw, score, 1.5)
    assert grad_close(run_backward(m, x, idx, dw, score, 1.5), want, xd, dw, 1.5, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E,K", [(3, 3), (64, 5), (65, 8), (128, 20), (130, 130), (251, 8), (256, 16), (300, 40), (512, 12),
                                 (513, 70), (1024, 8)])
def test_backward_many_tokens(m, score, E, K, dtype):
    """More tokens than any device's 8 per compute unit: masked rows, ids twice and more and outside the
    experts, among rows that share their waves."""
    r = np.random.default_rng(E * K)
    x = torch.from_numpy(r.standard_normal((37, E)).astype(np.float32)).to(dtype)
    x[3] = -float("inf")
    x[11, ::2] = -float("inf")
    xd = x.double().numpy()
    idx, _ = ref.router_topk(xd, K, score)
    idx[5, :] = idx[5, 0]
    idx[6, ::2] = idx[6, 0]
    idx[7, 1:] = E
    idx[8] = -1
    idx[9, K - 1] = idx[9, 0]
    dw = r.standard_normal((37, K)).astype(np.float32)
    rows = np.arange(8209) % 37
    d = run_backward(m, x[torch.from_numpy(rows)].cuda(), idx[rows], dw[rows], score, 1.5)
    first = d[:37]
    assert torch.equal(d, first[torch.from_numpy(rows).cuda()])   # finite, and the same in every wave
    want = ref.router_backward(xd, idx, dw, score, 1.5)
    assert grad_close(first, want, np.where(np.isfinite(xd), xd, 0.0), dw, 1.5, dtype)


@pytest.mark.parametrize("score", SCORES)
def test_backward_odd_ids(m, score):
    """Ids outside the experts, the same id twice, rows with no valid id, masked logits."""
    x = logits_of(8, 6, 70, torch.float32)
    x[3, 10:] = -float("inf")
    x[4] = -float("inf")
    idx = np.array([[0, 69, 5], [5, 5, 6], [-1, 70, 4], [1, 2, 30], [0, 1, 2], [-1, -1, 1 << 30]])
    dw = np.random.default_rng(3).standard_normal((6, 3)).astype(np.float32)
    xd = x.double().cpu().numpy()
    want = ref.router_backward(xd, idx, dw, score)
    d = run_backward(m, x, idx, dw, score)
    assert grad_close(d, want, np.where(np.isfinite(xd), xd, 0.0), dw, 1.0, torch.float32)
    assert (d[5] == 0).all()


@pytest.mark.parametrize("score", SCORES)
def test_backward_against_differences(m, score):
    """Central differences of the kernel's own weights in the logits, the choice held by a wide
    margin: sum(dw * w) changes by the gradient.  Step h = 1/16 on chosen logits of size about 1: the
    third derivative of a weight in one logit is below 1/2, so differences are off by at most h^2 / 12 of
    sum |dw|, and by the weights' own rounding over h."""
    T, E, K = 2, 20, 4
    x = np.random.default_rng(0).uniform(-1, 1, (T, E)).astype(np.float32)
    x[:, :K] += 8.0
    dw = np.random.default_rng(1).standard_normal((T, K)).astype(np.float32)
    d = run_backward(m, torch.from_numpy(x).cuda(), np.tile(np.arange(K), (T, 1)), dw, score).cpu().numpy()
    h = 1.0 / 16

    def value(y):
        idx, w = topk(m, torch.from_numpy(y).cuda(), K, score)
        out = np.zeros(T)
        for t in range(T):
            for k in range(K):
                out[t] += w[t, k] * dw[t, idx[t, k]]
        return out

    tol = (h * h / 12 + 2 * weight_tol(x, E) / h) * np.abs(dw).sum(1)
    for e in range(E):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        assert (np.abs((value(up) - value(down)) / (2 * h) - d[:, e]) <= tol).all()


def test_many_tokens(m):
    """More tokens than one launch has waves for."""
    x = torch.randn(70001, 16, device="cuda")
    idx = torch.empty((70001, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((70001, 2), device="cuda")
    m.moe_router_topk(x, idx, w)
    want = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :2]
    assert torch.equal(idx.long(), want)
