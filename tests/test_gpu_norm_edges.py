"""moe_layer_norm and its gradient: rows of very large values, infinities, every kernel in place, a row among others, and
the borders of the short gradients."""
import numpy as np
import pytest
import torch

import test_gpu_norm as norm
from block_common import BF16, F32, U, exactly, rng_of
from test_gpu_norm import Rows, forward, gradients

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


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", WIDTHS)
def test_in_place_in_every_kernel(m, width, dtype, kind):
    """y and total in the places of x and residual, dx and dresidual in those of dy and dtotal, either way round: as
    without, bit for bit, also where the moved-back end of a row is two threads'."""
    rows = 9
    c = Rows(3, rows, width, dtype, kind, True)
    rng = rng_of(5, 6)
    t = forward(m, c, 0.2, rng)
    for y_in_x in (True, False):
        x, res = c.x.clone(), c.residual.clone()
        y, total = (x, res) if y_in_x else (res, x)
        m.moe_layer_norm(x, c.w, y, bias=c.b, kind=kind, residual=res, total=total, p=0.2, rng=rng)
        assert torch.equal(y, t["y"]) and torch.equal(total, t["total"])
    dy, dt = torch.randn_like(c.x), torch.randn_like(c.x)
    g = gradients(m, c, t["total"], t.get("mean"), t["rstd"], dy, dt, 0.2, rng)
    ws = torch.empty(m.layer_norm_backward_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")
    mean = exactly(t["mean"])[:, None] if kind == "layer" else 0.0
    xh, d = (exactly(t["total"]) - mean) * exactly(t["rstd"])[:, None], np.abs(exactly(dy))
    for dx_in, dres_in in (("dy", "dtotal"), ("dtotal", "dy"), ("dy", None), ("dtotal", None), (None, "dtotal"), (None, "dy")):
        a, b = dy.clone(), dt.clone()
        place = {"dy": a, "dtotal": b}
        dx, dres = (torch.empty_like(dy) if k is None else place[k] for k in (dx_in, dres_in))
        dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
        m.moe_layer_norm_backward(t["total"], c.w, t["rstd"], a, dx, dw, ws, dbias=db, mean=t.get("mean"), kind=kind, dtotal=b,
                                  dresidual=dres, p=0.2, rng=rng)
        assert torch.equal(dx, g["dx"]) and torch.equal(dres, g["dresidual"]), (dx_in, dres_in)
        # the sums of columns may be added up in another order: each is off by at most rows + 8 roundings of the magnitudes
        assert (np.abs(exactly(dw) - exactly(g["dweight"])) <= 2 * (rows + 8) * U * (d * np.abs(xh)).sum(0)).all()
        if kind == "layer":
            assert (np.abs(exactly(db) - exactly(g["dbias"])) <= 2 * (rows + 8) * U * d.sum(0)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", WIDTHS)
def test_a_row_alone_is_the_row_among_others(m, width, dtype):
    """Bit for bit: few rows and one go through the same kernel."""
    c = Rows(8, 40, width, dtype, "layer", True)
    whole = forward(m, c)
    one = Rows(8, 40, width, dtype, "layer", True)
    one.x, one.residual = c.x[17:18].clone(), c.residual[17:18].clone()
    alone = forward(m, one)
    for k in whole:
        assert torch.equal(alone[k], whole[k][17:18]), k


@pytest.mark.parametrize("kind,dtot,p,accumulate", [("layer", True, 0.3, True), ("rms", False, 0.0, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", [(292, 7168), (293, 7168), (512, 4096), (513, 4096)])
def test_borders_of_the_short_gradients(m, rows, width, dtype, kind, dtot, p, accumulate):
    """The last rows and widths whose columns are summed beside the rows, and the first that are not (2^21 values)."""
    norm.test_backward(m, rows, width, dtype, kind, dtot, p, accumulate)
