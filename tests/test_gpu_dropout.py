"""moe_dropout on the GPU against the mask's definition."""
import numpy as np
import pytest
import torch

from block_common import BF16, F32, U, exactly, rng_of, rounding, tensor
from oracle import block_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


@pytest.mark.parametrize("seed,offset", [(0, 0), ((1 << 64) - 1, (1 << 64) - 1), (0x0123456789ABCDEF, 1 << 33)])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2047, 2048, 2055, 100001])
def test_mask(m, n, seed, offset):
    """The kept elements are the definition's, one by one; ones show the scale."""
    for dtype in (F32, BF16):
        for p in (0.1, 0.5, 0.999):
            x = torch.ones(n, dtype=dtype, device="cuda")
            out = torch.full_like(x, 9.0)
            m.moe_dropout(x, out, p, rng_of(seed, offset))
            assert np.array_equal(exactly(out) != 0, ref.kept(n, p, seed, offset))
            scale = 65536 / (65536 - ref.below(p))
            got = exactly(out)[exactly(out) != 0]
            assert (np.abs(got - scale) <= (rounding(dtype) + 2 * U) * scale).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1), (6, 1408), (33, 257), (3, 5, 7), (1, 7168)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.25, 1.0])
def test_values(m, shape, dtype, residual, p):
    r = np.random.default_rng(1)
    x = tensor(r.standard_normal(shape), dtype)
    res = tensor(r.standard_normal(shape), dtype) if residual else None
    out = torch.full_like(x, 9.0)
    m.moe_dropout(x, out, p, rng_of(3, 4), residual=res, offset=-2)
    xs = ref.drop(exactly(x), p, 3, 2)
    want = xs + (exactly(res) if residual else 0.0)
    e = 2 * U * np.abs(xs) + U * np.abs(want)
    assert (np.abs(exactly(out) - want) <= e + rounding(dtype) * (np.abs(want) + e)).all()
    if p == 0.0 and not residual or p == 1.0 and residual:
        assert torch.equal(out, res if residual else x)


def test_gradient(m):
    """The same call on the gradient: zero where dropped, scaled elsewhere, whatever the values were."""
    x, dout = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    out, dx = torch.empty_like(x), torch.empty_like(x)
    rng = rng_of(8, 9)
    m.moe_dropout(x, out, 0.4, rng, offset=3)
    m.moe_dropout(dout, dx, 0.4, rng, offset=3)
    assert torch.equal(dx == 0, out == 0)
    # out is linear in x: <dout, out> = <dx, x>, each term rounded twice on either side
    a, b = (dout.double() * out.double()), (dx.double() * x.double())
    assert abs(float(a.sum() - b.sum())) <= 4 * U * float(a.abs().sum())


def test_offsets_are_added(m):
    x = torch.ones(4096, device="cuda")
    a, b, c = (torch.empty_like(x) for _ in range(3))
    m.moe_dropout(x, a, 0.5, rng_of(5, 10), offset=7)
    m.moe_dropout(x, b, 0.5, rng_of(5, 17))
    m.moe_dropout(x, c, 0.5, rng_of(5, 18))
    assert torch.equal(a, b) and not torch.equal(b, c)


def test_in_place_and_unaligned(m):
    r = np.random.default_rng(2)
    for dtype in (F32, BF16):
        flat = torch.full((3000,), 5.0, dtype=dtype, device="cuda")
        x, res = tensor(r.standard_normal(1003), dtype), tensor(r.standard_normal(1003), dtype)
        want = torch.empty_like(x)
        m.moe_dropout(x, want, 0.3, rng_of(1, 1), residual=res)
        at = flat[11:1014]
        at.copy_(x)
        m.moe_dropout(at, at, 0.3, rng_of(1, 1), residual=res)
        assert torch.equal(at, want) and (flat[:11] == 5).all() and (flat[1014:] == 5).all()
        at.copy_(res)
        m.moe_dropout(x, at, 0.3, rng_of(1, 1), residual=at)
        assert torch.equal(at, want)


def test_dropped_values_do_not_matter(m):
    """NaN and infinities in dropped places are gone, in kept ones they stay."""
    x = torch.randn(512, device="cuda")
    rng = rng_of(4, 4)
    base = torch.empty_like(x)
    m.moe_dropout(x, base, 0.5, rng)
    gone = torch.from_numpy(~ref.kept(512, 0.5, 4, 4)).cuda()
    for v in (float("nan"), float("inf")):
        y, out = torch.where(gone, torch.full_like(x, v), x), torch.empty_like(x)
        m.moe_dropout(y, out, 0.5, rng)
        assert torch.equal(out, base)
        y[:] = v
        m.moe_dropout(y, out, 0.5, rng)
        assert (out[gone] == 0).all() and not torch.isfinite(out[~gone]).any()


def test_over_32_bits(m):
    """Elements past 2^32: the tail's mask is the definition's there."""
    n = (1 << 32) + 77
    x = torch.ones(n, dtype=BF16, device="cuda")
    m.moe_dropout(x, x, 0.5, rng_of(6, 7))
    assert np.array_equal(exactly(x[-100:]) != 0, ref.kept(100, 0.5, 6, 7, first=n - 100))
    assert np.array_equal(exactly(x[:64]) != 0, ref.kept(64, 0.5, 6, 7))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_than_the_caches_hold(m, dtype, residual):
    """A call that streams past the caches begins and ends as calls on those parts alone do."""
    n = (320 << 20) // (2 if dtype == BF16 else 4) + 5
    x, rng = torch.randn(n, device="cuda").to(dtype), rng_of(12, 13)
    res = torch.randn(n, device="cuda").to(dtype) if residual else None
    out, few = torch.empty_like(x), torch.empty(100003, dtype=dtype, device="cuda")
    m.moe_dropout(x, out, 0.2, rng, residual=res)
    m.moe_dropout(x[:100003], few, 0.2, rng, residual=res[:100003] if residual else None)
    assert torch.equal(out[:100003], few)
    xs = np.where(ref.kept(77, 0.2, 12, 13, first=n - 77), exactly(x[-77:]) * 65536 / (65536 - ref.below(0.2)), 0.0)
    want = xs + (exactly(res[-77:]) if residual else 0.0)
    e = 2 * U * np.abs(xs) + U * np.abs(want)
    assert (np.abs(exactly(out[-77:]) - want) <= e + rounding(dtype) * (np.abs(want) + e)).all()


def test_captured_and_replayed(m):
    x, out, want = torch.ones(5000, device="cuda"), torch.empty(5000, device="cuda"), torch.empty(5000, device="cuda")
    rng = rng_of(2, 0)
    m.moe_dropout(x, out, 0.5, rng)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_dropout(x, out, 0.5, rng)
    seen = []
    for rep in range(3):
        rng[1] += 1
        out.fill_(7.0)
        g.replay()
        m.moe_dropout(x, want, 0.5, rng)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1])


def test_refused_and_empty(m):
    x, rng = torch.zeros(64, device="cuda"), rng_of(1, 2)
    out = torch.zeros_like(x)
    for call in (lambda: m.moe_dropout(x.half(), out, 0.1, rng), lambda: m.moe_dropout(x[::2], out[:32], 0.1, rng),
                 lambda: m.moe_dropout(x, out[:63], 0.1, rng), lambda: m.moe_dropout(x, out.bfloat16(), 0.1, rng),
                 lambda: m.moe_dropout(x, out, 1.5, rng), lambda: m.moe_dropout(x, out, 0.1, None),
                 lambda: m.moe_dropout(x, out, 0.1, rng.cpu()), lambda: m.moe_dropout(x, out, 0.1, rng[:1]),
                 lambda: m.moe_dropout(x[:32], x[16:48], 0.1, rng), lambda: m.moe_dropout(x, out, 0.1, rng, residual=out[:1])):
        with pytest.raises(m.MoeError):
            call()
    m.moe_dropout(x[:0], out[:0], 0.5, rng)
    m.moe_dropout(x, out, 0.0, None)
