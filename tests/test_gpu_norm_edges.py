"""moe_layer_norm and its gradient on rows of very large values and of infinities."""
import pytest
import torch

from block_common import BF16, F32, rng_of
from test_gpu_norm import Rows, forward

pytestmark = pytest.mark.gpu
# one of each kernel and width of row that are told apart
WIDTHS = [5, 33, 200, 300, 513, 1001, 7168, 8193, 12001, 16384, 20000]


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def run(m, x, residual, kind, p, rng, w):
    t = dict(y=torch.empty_like(x), total=torch.empty_like(x), rstd=torch.empty(len(x), device="cuda"))
    if kind == "layer":
        t["mean"] = torch.empty(len(x), device="cuda")
    m.moe_layer_norm(x, w, t["y"], eps=0.0, kind=kind, residual=residual, total=t["total"], mean=t.get("mean"), rstd=t["rstd"],
                     p=p, rng=rng)
    return t


@pytest.mark.parametrize("kind,residual,p", [("layer", False, 0.0), ("layer", True, 0.25), ("rms", True, 0.0), ("rms", False, 0.25)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", WIDTHS)
def test_rows_whose_squares_leave_fp32(m, width, dtype, kind, residual, p):
    """Without eps a row scaled by a power of two has the same y, bit for bit, and its statistics are scaled by it: also where
    the sum of its squares (from 2^53 at the widest row) or their mean (from 2^64) does not fit fp32.  The rows beside
    it, which share its wave or its workgroup, are as they were."""
    g = torch.Generator().manual_seed(width)
    x = (torch.randn(6, width, generator=g) + 0.5).to(dtype).cuda()
    r = torch.randn(6, width, generator=g).to(dtype).cuda() if residual else None
    w, rng = torch.ones(width, device="cuda"), rng_of(3, 4) if p else None
    base = run(m, x, r, kind, p, rng, w)
    for e in (50, 54, 56, 57, 58, 60, 62, 63, 64, 66, 90, 100):
        s = torch.ones(6, 1, device="cuda")
        s[1] = s[4] = 2.0 ** e
        t = run(m, (x.float() * s).to(dtype), None if r is None else (r.float() * s).to(dtype), kind, p, rng, w)
        s = s.view(-1)
        assert torch.equal(t["y"], base["y"]), e
        assert torch.equal(t["rstd"] * s, base["rstd"]), e
        assert torch.equal(t["total"].float(), base["total"].float() * s[:, None]), e
        if kind == "layer":
            assert torch.equal(t["mean"], base["mean"] * s), e


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("width", WIDTHS)
def test_gradient_of_large_rows(m, width, kind):
    """From the statistics that such a row's forward left: dx is scaled by the power's inverse, bit for bit."""
    x, dy = torch.randn(3, width, device="cuda") + 0.5, torch.randn(3, width, device="cuda")
    w = torch.ones(width, device="cuda")
    dx = []
    for scale in (1.0, 2.0 ** 60, 2.0 ** 70):
        t = run(m, x * scale, None, kind, 0.0, None, w)
        out = torch.empty_like(dy)
        m.moe_layer_norm_backward(t["total"], w, t["rstd"], dy, out, mean=t.get("mean"), kind=kind)
        dx.append(out * scale)
    assert torch.isfinite(dx[0]).all() and torch.equal(dx[0], dx[1]) and torch.equal(dx[0], dx[2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", WIDTHS)
def test_rows_that_are_not_finite(m, width, dtype):
    """A NaN takes its whole row, an infinity too where a mean is taken; without one, 1 / sqrt(infinity) is 0: the infinite
    column is NaN (infinity times 0), the others the bias.  Other rows are as they were."""
    inf, nan = float("inf"), float("nan")
    for kind in ("layer", "rms"):
        c = Rows(1, 7, width, dtype, kind, False)
        c.b = torch.linspace(-1, 1, width, device="cuda")
        base = forward(m, c)
        others = torch.tensor([0, 1, 3, 4, 6], device="cuda")
        for v in (nan, inf, -inf):
            x = c.x.clone()
            c.x[2, width // 2], c.x[5, width - 1] = v, v
            t = forward(m, c)
            c.x = x
            for k in base:
                assert torch.equal(t[k][others], base[k][others])
            for row, at in ((2, width // 2), (5, width - 1)):
                if kind == "layer" or v != v:
                    assert torch.isnan(t["y"][row]).all() and torch.isnan(t["rstd"][row])
                else:
                    rest = torch.arange(width, device="cuda") != at
                    assert t["rstd"][row] == 0 and torch.isnan(t["y"][row, at])
                    assert torch.equal(t["y"][row, rest], c.b.to(dtype)[rest])
