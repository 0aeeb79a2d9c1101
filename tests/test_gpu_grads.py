"""The global gradient norm and clipping on the GPU against float64."""
import numpy as np
import pytest
import torch

from oracle import scaled_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def tensors(seed, sizes, kinds, scale=1.0):
    rng = np.random.default_rng(seed)
    return [(torch.from_numpy(rng.standard_normal(n).astype(np.float32)) * scale).to(kinds[i % len(kinds)]).cuda()
            for i, n in enumerate(sizes)]


def sumsq_of(m, grads):
    s = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    ws = torch.full((m.grad_sumsq_workspace_bytes(),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_grad_sumsq(grads, s, ws)
    return s


def check(m, grads, max_norm, in_place):
    before = [g.double().cpu().numpy() for g in grads]
    norm, coef = ref.grad_clip(before, max_norm)
    s = sumsq_of(m, grads)
    # squares in 64 bits: two roundings of 2^-53 a term at most
    assert abs(s.item() - norm * norm) <= 1e-12 * norm * norm
    out = grads if in_place else [torch.full_like(g, 9.0) for g in grads]
    n32 = torch.full((1,), -1.0, device="cuda")
    m.moe_grad_clip(grads, s, max_norm, n32, None if in_place else out)
    assert abs(n32.item() - norm) <= 2.0 ** -24 * norm + 1e-45
    for b, o in zip(before, out):
        # the factor and the product are rounded once each (2^-24), bf16 once more (2^-8)
        tol = 2.0 ** -22 + (2.0 ** -8 if o.dtype == torch.bfloat16 else 0.0)
        assert (np.abs(o.double().cpu().numpy() - coef * b) <= tol * np.abs(coef * b) + 1e-40).all()


F, B = torch.float32, torch.bfloat16
LISTS = {
    "one_value": ([1], [F]), "one_bf16": ([1], [B]), "odd": ([3, 5, 1025, 7, 16384, 16385], [F, B]),
    "empty_among": ([0, 4, 0, 0, 33], [F, B]), "many": (list(range(1, 400, 2)), [B, F]),
    "exact_batch": ([40000] * 64, [F]), "batch_and_one": ([100] * 65, [F]),
    "small_then_large": ([10] * 64 + [5000001], [F]), "large_then_small": ([5000001] + [10] * 70, [B]),
    "one_chunk": ([16384], [F]), "two_chunks": ([16385], [B]), "two_tensors": ([100, 16384], [F, B]),
    "two_then_empty": ([9, 0, 12] + [0] * 70, [F, B]), "three_chunks": ([1, 2, 3], [B, F]),
    "over_parts": ([1 << 14] * 40 + [(1 << 26) + 3], [F]),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("limit", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("name", list(LISTS))
def test_clip(m, name, limit, in_place):
    sizes, kinds = LISTS[name]
    check(m, tensors(len(sizes), sizes, kinds), limit, in_place)


def test_unaligned(m):
    """Gradients that begin at any element of a flat buffer, clipped into others that begin elsewhere."""
    for dtype in (F, B):
        flat = torch.randn(100000, device="cuda").to(dtype)
        dst = torch.full((100100,), 5.0, device="cuda", dtype=dtype)
        cuts = [1, 8, 13, 1000, 1003, 33333, 99999]
        grads = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
        outs = [dst[a + 3:b + 3] for a, b in zip(cuts, cuts[1:])]
        s = sumsq_of(m, grads)
        norm, coef = ref.grad_clip([g.double().cpu().numpy() for g in grads], 1.0)
        assert abs(s.item() - norm * norm) <= 1e-12 * norm * norm
        m.moe_grad_clip(grads, s, 1.0, out=outs)
        got = dst[4:100002].double().cpu().numpy()
        want = coef * flat[1:99999].double().cpu().numpy()
        tol = 2.0 ** -22 + (2.0 ** -8 if dtype == B else 0.0)
        assert (np.abs(got - want) <= tol * np.abs(want) + 1e-40).all()
        assert (dst[:4] == 5.0).all() and (dst[100002:] == 5.0).all()


def test_large_and_small_values(m):
    """Squares that fp32 cannot hold, and values far below the largest."""
    g = [torch.tensor([3e38, -1e30, 1.0], device="cuda"), torch.full((1000,), 1e-30, device="cuda")]
    check(m, g, 1.0, False)
    check(m, [torch.full((777,), 1e-25, device="cuda")], 1.0, False)


def test_zero_and_empty(m):
    check(m, [torch.zeros(100, device="cuda")], 1.0, True)
    s = sumsq_of(m, [])
    n = torch.full((1,), 7.0, device="cuda")
    m.moe_grad_clip([], s, 1.0, n)
    assert s.item() == 0.0 and n.item() == 0.0
    e = [torch.empty(0, device="cuda")]
    n.fill_(7.0)
    m.moe_grad_clip(e, sumsq_of(m, e), 1.0, n)
    assert n.item() == 0.0


def test_not_finite(m):
    """A NaN anywhere makes norm and gradients NaN; an infinity makes the norm infinite, the finite
    gradients 0 and the infinite one NaN (inf * 0)."""
    g = tensors(1, [100, 200], [F])
    g[1][7] = float("nan")
    s, n = sumsq_of(m, g), torch.zeros(1, device="cuda")
    m.moe_grad_clip(g, s, 1.0, n)
    assert torch.isnan(n).all() and all(torch.isnan(x).all() for x in g)
    g = tensors(1, [100, 200], [F])
    g[1][7] = float("inf")
    m.moe_grad_clip(g, sumsq_of(m, g), 1.0, n)
    assert torch.isinf(n).all() and (g[0] == 0).all() and torch.isnan(g[1][7]) and (g[1][:7] == 0).all()


def test_same_bits_again(m):
    g = tensors(2, [123457, 99, 1 << 20], [F, B])
    assert torch.equal(sumsq_of(m, g), sumsq_of(m, g))


def test_over_32_bits(m):
    """A tensor whose bytes pass 2^32 (its elements 2^31)."""
    n = (1 << 31) + 5
    g = torch.zeros(n, dtype=B, device="cuda")
    g[0], g[n // 2], g[n - 1] = 3.0, 4.0, 12.0
    s, norm = sumsq_of(m, [g]), torch.zeros(1, device="cuda")
    m.moe_grad_clip([g], s, 6.5, norm)
    assert norm.item() == 13.0
    assert [g[0].item(), g[n // 2].item(), g[n - 1].item(), g[n - 2].item()] == [1.5, 2.0, 6.0, 0.0]


def test_refused_lists(m):
    """A tensor listed twice to be clipped, outputs of another type or number, a strided gradient."""
    g = tensors(4, [100, 200], [F])
    s = sumsq_of(m, g + g)            # the sum may count a tensor twice
    for grads, out in ((g + g[:1], None), (g, [g[0], g[0]]), (g, g[:1]), (g, [g[0].bfloat16(), g[1]]), (g, [g[0], g[1][:10]])):
        with pytest.raises(m.MoeError):
            m.moe_grad_clip(grads, s, 1.0, out=out)
    with pytest.raises(m.MoeError):
        m.moe_grad_sumsq([g[0][::2]], s, torch.empty(m.grad_sumsq_workspace_bytes(), dtype=torch.uint8, device="cuda"))
    with pytest.raises(m.MoeError):
        m.moe_grad_sumsq(g, s, torch.empty(8, dtype=torch.uint8, device="cuda"))
