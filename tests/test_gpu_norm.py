"""moe_layer_norm and its gradient on the GPU against float64."""
import numpy as np
import pytest
import torch

from block_common import BF16, F32, U, exactly, norm_backward_bound, norm_bound, rng_of, rounding, tensor
from oracle import block_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5
# rows, width: one value, part of a run of 8, the borders of every width that the kernels tell apart
SHAPES = [(1, 1), (3, 5), (2, 8), (7, 33), (5, 512), (3, 513), (2, 1001), (4, 1024), (3, 1032), (2, 2048), (2, 2049), (1, 4096),
          (3, 4100), (2, 7168), (1, 8192), (2, 8193), (1, 16384), (2, 16391), (1, 40000), (300, 64), (1100, 40),
          (5, 200), (9, 256), (3, 129), (8200, 24),
          (512, 30), (513, 30), (384, 1409), (385, 1409), (146, 7168), (147, 7168)]  # and of its short gradients


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


class Rows:
    """Inputs of one call: rows of a residual stream with a mean and a few large columns."""

    def __init__(self, seed, rows, width, dtype, kind, residual, w_dtype=None):
        r = np.random.default_rng(seed)
        self.kind, self.dtype = kind, dtype
        big = np.where(r.random(width) < 0.02, 12.0, 1.0)
        self.x = tensor(r.standard_normal((rows, width)), dtype)
        self.residual = tensor(r.standard_normal((rows, width)) * big + 0.3, dtype) if residual else None
        self.w = tensor(1 + 0.2 * r.standard_normal(width), w_dtype or F32)
        self.b = tensor(0.2 * r.standard_normal(width), w_dtype or F32) if kind == "layer" else None


def forward(m, c, p=0.0, rng=None, offset=0, **out):
    t = {"y": torch.full_like(c.x, 9.0), "rstd": torch.full((c.x.shape[0],), -1.0, device="cuda")}
    if c.kind == "layer":
        t["mean"] = torch.full((c.x.shape[0],), -1.0, device="cuda")
    if c.residual is not None or p > 0:
        t["total"] = torch.full_like(c.x, 9.0)
    t.update(out)
    m.moe_layer_norm(c.x, c.w, t["y"], bias=c.b, eps=EPS, kind=c.kind, residual=c.residual, p=p, rng=rng,
                     offset=offset, **{k: v for k, v in t.items() if k != "y"})
    return t


def check_forward(c, t, p, seed, offset):
    x = exactly(c.x)
    xs = ref.drop(x, p, seed, offset)
    h = xs + (exactly(c.residual) if c.residual is not None else 0.0)
    eh = 2 * U * np.abs(xs) * (p > 0) + (U * np.abs(h) if c.residual is not None else 0.0)
    y, mean, rstd = ref.layer_norm(h, exactly(c.w), None if c.b is None else exactly(c.b), EPS, c.kind)
    by, bm, br = norm_bound(h, eh, y, mean, rstd, exactly(c.w), EPS, c.kind, c.dtype)
    assert (np.abs(exactly(t["y"]) - y) <= by).all()
    assert (np.abs(exactly(t["rstd"]) - rstd) <= br).all()
    if c.kind == "layer":
        assert (np.abs(exactly(t["mean"]) - mean) <= bm + U * np.abs(mean)).all()
    if "total" in t:
        assert (np.abs(exactly(t["total"]) - h) <= eh + rounding(c.dtype) * (np.abs(h) + eh)).all()


@pytest.mark.parametrize("kind,residual,p", [("layer", False, 0.0), ("layer", True, 0.3), ("rms", True, 0.0), ("rms", False, 0.5)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_forward(m, rows, width, dtype, kind, residual, p):
    c = Rows(rows * width, rows, width, dtype, kind, residual, w_dtype=dtype)
    seed, offset = (1 << 63) + width, (1 << 40) + rows
    t = forward(m, c, p, rng_of(seed, offset) if p else None, offset=7)
    check_forward(c, t, p, seed, offset + 7)


def gradients(m, c, h, mean, rstd, dy, dtotal, p, rng, offset=0, accumulate=False, sums=True):
    rows, width = h.shape
    t = {"dx": torch.full_like(dy, 9.0), "dresidual": torch.full_like(dy, 9.0)}
    if sums:
        t["dweight"] = torch.full((width,), 2.0, device="cuda")
        if c.kind == "layer":
            t["dbias"] = torch.full((width,), -3.0, device="cuda")
    ws = torch.full((m.layer_norm_backward_workspace_bytes(rows, width),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_layer_norm_backward(h, c.w, rstd, dy, t["dx"], t.get("dweight"), ws if sums else None, dbias=t.get("dbias"), mean=mean,
                              kind=c.kind, dtotal=dtotal, dresidual=t["dresidual"], accumulate=accumulate, p=p, rng=rng,
                              offset=offset)
    return t


@pytest.mark.parametrize("kind,dtot,p,accumulate", [("layer", False, 0.0, False), ("layer", True, 0.3, True),
                                                    ("rms", True, 0.0, False), ("rms", False, 0.5, True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_backward(m, rows, width, dtype, kind, dtot, p, accumulate):
    c = Rows(rows + width, rows, width, dtype, kind, True, w_dtype=dtype)
    r = np.random.default_rng(rows)
    h, dy = c.residual, tensor(r.standard_normal((rows, width)) * 2.0 ** -6, dtype)
    dtotal = tensor(r.standard_normal((rows, width)) * 2.0 ** -6, dtype) if dtot else None
    hd, w = exactly(h), exactly(c.w)
    _, mean, rstd = ref.layer_norm(hd, w, None, EPS, kind)
    mean_t, rstd_t = tensor(mean, F32) if kind == "layer" else None, tensor(rstd, F32)
    mean, rstd = exactly(mean_t) if kind == "layer" else None, exactly(rstd_t)  # what the call is given, exactly
    seed, offset = 99 + width, 3
    t = gradients(m, c, h, mean_t, rstd_t, dy, dtotal, p, rng_of(seed, offset) if p else None, accumulate=accumulate)
    dh, dw, db = ref.layer_norm_backward(hd, w, mean, rstd, exactly(dy), kind)
    if dtot:
        dh = dh + exactly(dtotal)
    bh, bw, bb = norm_backward_bound(hd, w, mean, rstd, exactly(dy), exactly(dtotal) if dtot else None, dh, kind, dtype)
    assert (np.abs(exactly(t["dresidual"]) - dh) <= bh).all()
    dx = ref.drop(dh, p, seed, offset)
    scale = 65536 / (65536 - ref.below(p))
    assert (np.abs(exactly(t["dx"]) - dx) <= scale * bh + 3 * U * np.abs(dx)).all()
    assert (exactly(t["dx"])[dx == 0] == 0).all() or p == 0
    was_w, was_b = (2.0, -3.0) if accumulate else (0.0, 0.0)
    assert (np.abs(exactly(t["dweight"]) - dw - was_w) <= bw + U * np.abs(dw + was_w)).all()
    if kind == "layer":
        assert (np.abs(exactly(t["dbias"]) - db - was_b) <= bb + U * np.abs(db + was_b)).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(m, kind):
    """<dx, v> and <dweight, v> against the loss moved along v, worked out by the forward kernel in fp32."""
    rows, width = 6, 200
    c = Rows(5, rows, width, F32, kind, False)
    r = np.random.default_rng(6)
    dy = tensor(r.standard_normal((rows, width)), F32)
    t = forward(m, c)
    g = gradients(m, c, c.x, t.get("mean"), t["rstd"], dy, None, 0.0, None)
    step = 2.0 ** -7
    for name, of in (("dx", "x"), ("dweight", "w")):
        at = getattr(c, of)
        v = tensor(r.standard_normal(tuple(at.shape)), F32)
        side = []
        for sign in (1, -1):
            setattr(c, of, at + sign * step * v)
            side.append(float((forward(m, c)["y"].double() * dy.double()).sum()))
        setattr(c, of, at)
        got, want = (side[0] - side[1]) / (2 * step), float((g[name].double() * v.double()).sum())
        # central differences: step^2 / 6 of a third derivative, at most some tens of |v|^3 |dy| over sqrt(rows width) independent
        # signs; rounding: 2^-22 of each of the rows * width terms of order 1, as independent, over the step
        size = np.sqrt(rows * width)
        assert abs(got - want) <= step ** 2 / 6 * 60 * size + 4 * 2.0 ** -22 * size / step


def test_sixteen_bit_weights_on_fp32_rows(m):
    c = Rows(11, 30, 1408, F32, "layer", True, w_dtype=BF16)
    check_forward(c, forward(m, c), 0.0, 0, 0)
    f = forward(m, c)
    dy = torch.randn_like(c.x)
    t = gradients(m, c, f["total"], f["mean"], f["rstd"], dy, None, 0.0, None)
    h, mean, rstd = exactly(f["total"]), exactly(f["mean"]), exactly(f["rstd"])
    dh, dw, db = ref.layer_norm_backward(h, exactly(c.w), mean, rstd, exactly(dy), "layer")
    bh, bw, bb = norm_backward_bound(h, exactly(c.w), mean, rstd, exactly(dy), None, dh, "layer", F32)
    assert (np.abs(exactly(t["dx"]) - dh) <= bh).all() and (np.abs(exactly(t["dweight"]) - dw) <= bw + U * np.abs(dw)).all()


@pytest.mark.parametrize("width", [40, 2048, 1001, 20000])
def test_total_of_rows_alone_is_their_copy(m, width):
    """Without residual and dropout h is x, bit for bit (the sign of a zero too)."""
    x = torch.randn(3, width, device="cuda").bfloat16()
    x[0, ::3] = -0.0
    y, total = torch.empty_like(x), torch.empty_like(x)
    m.moe_layer_norm(x, torch.ones(width, device="cuda"), y, kind="rms", total=total)
    assert torch.equal(total.view(torch.int16), x.view(torch.int16))


def test_one_token_matches_many(m):
    """A row's result is its own: alone or among others, bit for bit where the kernel is the same, else within the bound."""
    c = Rows(8, 40, 7168, BF16, "layer", True)
    whole = forward(m, c)
    one = Rows(8, 40, 7168, BF16, "layer", True)
    one.x, one.residual = c.x[17:18].clone(), c.residual[17:18].clone()
    check_forward(one, forward(m, one), 0.0, 0, 0)
    check_forward(c, whole, 0.0, 0, 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unaligned_rows(m, dtype):
    """Tensors that begin at any element of a larger one; nothing behind or before them is written."""
    rows, width = 5, 1003
    flat = {k: torch.full((rows * width + 40,), 5.0, dtype=dtype, device="cuda") for k in ("x", "res", "total", "y")}
    c = Rows(4, rows, width, dtype, "layer", True)
    cut = lambda k, o: flat[k][o:o + rows * width].view(rows, width)  # noqa: E731
    x, res, total, y = cut("x", 1), cut("res", 3), cut("total", 7), cut("y", 13)
    x.copy_(c.x), res.copy_(c.residual)
    c.x, c.residual = x, res
    t = forward(m, c, 0.25, rng_of(3, 4), total=total, y=y)
    check_forward(c, t, 0.25, 3, 4)
    for k, o in (("total", 7), ("y", 13)):
        assert (flat[k][:o] == 5.0).all() and (flat[k][o + rows * width:] == 5.0).all()


@pytest.mark.parametrize("width", [7168, 1001, 20000])
def test_in_place(m, width):
    """The sum in the residual's place and the rows in x's; the gradients in dy's and dtotal's."""
    rows = 9
    c = Rows(3, rows, width, BF16, "layer", True)
    rng = rng_of(5, 6)
    t = forward(m, c, 0.2, rng)
    x, res = c.x.clone(), c.residual.clone()
    m.moe_layer_norm(x, c.w, x, bias=c.b, residual=res, total=res, p=0.2, rng=rng)
    assert torch.equal(x, t["y"]) and torch.equal(res, t["total"])
    dy, dt = torch.randn_like(c.x), torch.randn_like(c.x)
    g = gradients(m, c, t["total"], t["mean"], t["rstd"], dy, dt, 0.2, rng)
    a, b = dy.clone(), dt.clone()
    ws = torch.empty(m.layer_norm_backward_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    m.moe_layer_norm_backward(t["total"], c.w, t["rstd"], a, a, dw, ws, dbias=db, mean=t["mean"], dtotal=b, dresidual=b, p=0.2,
                              rng=rng)
    assert torch.equal(a, g["dx"]) and torch.equal(b, g["dresidual"])
    # the sums of columns of so few rows are added up in another order where dy keeps its place: each is off by at most
    # rows + 8 additions' roundings of the sum of magnitudes
    xh = (exactly(t["total"]) - exactly(t["mean"])[:, None]) * exactly(t["rstd"])[:, None]
    d = np.abs(exactly(dy))
    assert (np.abs(exactly(dw) - exactly(g["dweight"])) <= 2 * (rows + 8) * U * (d * np.abs(xh)).sum(0)).all()
    assert (np.abs(exactly(db) - exactly(g["dbias"])) <= 2 * (rows + 8) * U * d.sum(0)).all()


@pytest.mark.parametrize("width", [300, 7168, 33000])
def test_rows_of_one_value_and_of_large_ones(m, width):
    """A constant row has variance 0: y is the bias.  A mean of 10^4 spreads: its digits do not reach the differences."""
    w, b = torch.ones(width, device="cuda"), torch.full((width,), 0.5, device="cuda")
    x = torch.full((2, width), 3.0, device="cuda")
    y = torch.empty_like(x)
    m.moe_layer_norm(x, w, y, bias=b)
    # the mean of equal values is off by the additions' roundings; sqrt(eps) = 2^-8.3 turns u into 316 u
    assert (np.abs(exactly(y) - 0.5) <= 3.0 * (64 + width // 1024 + 3) * U * EPS ** -0.5).all()
    c = Rows(2, 2, width, F32, "layer", False)
    c.x = (c.x + 8192.0).contiguous()
    check_forward(c, forward(m, c), 0.0, 0, 0)


@pytest.mark.parametrize("width", [100, 1408, 7168, 20000])
def test_small_rows_without_eps(m, width):
    """Scaled by an even power of two, rows give the same y bit for bit, down to squares of 2^-120."""
    x = torch.randn(3, width, device="cuda")
    w, y, z = torch.ones(width, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    m.moe_layer_norm(x, w, y, kind="rms", eps=0.0)
    for e in (-20, -46, -60):
        m.moe_layer_norm(x * 2.0 ** e, w, z, kind="rms", eps=0.0)
        assert torch.equal(y, z), e


def test_not_finite(m):
    """A NaN or infinity takes its own row, no other; where the dropout takes it away it is gone."""
    c = Rows(1, 4, 1000, F32, "layer", True)
    base = forward(m, c)["y"].clone()
    for v in (float("nan"), float("inf"), -float("inf")):
        c.x[2, 77] = v
        y = forward(m, c)["y"]
        assert torch.isnan(y[2]).all() and torch.equal(y[[0, 1, 3]], base[[0, 1, 3]])
    t = forward(m, c, 1.0, rng_of(1, 2))
    assert torch.equal(t["total"], c.residual) and torch.isfinite(t["y"]).all()


def test_without_rows_and_without_sums(m):
    c = Rows(1, 0, 64, BF16, "layer", False)
    forward(m, c)
    t = gradients(m, c, c.x, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), c.x.clone(), None, 0.0, None)
    assert (t["dweight"] == 0).all() and (t["dbias"] == 0).all()
    t = gradients(m, c, c.x, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), c.x.clone(), None, 0.0, None,
                  accumulate=True)
    assert (t["dweight"] == 2).all() and (t["dbias"] == -3).all()
    c = Rows(2, 5, 700, BF16, "layer", False)
    f = forward(m, c)
    dy = torch.randn_like(c.x)
    with_sums = gradients(m, c, c.x, f["mean"], f["rstd"], dy, None, 0.0, None)
    assert torch.equal(gradients(m, c, c.x, f["mean"], f["rstd"], dy, None, 0.0, None, sums=False)["dx"], with_sums["dx"])


def test_same_bits_again_and_on_other_streams(m):
    c = Rows(4, 700, 1408, BF16, "layer", True)
    rng = rng_of(5, 6)
    t = forward(m, c, 0.1, rng)
    dy = torch.randn_like(c.x)
    g = gradients(m, c, t["total"], t["mean"], t["rstd"], dy, None, 0.1, rng)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # two calls at once, each with a workspace of its own
        with torch.cuda.stream(s):
            f = forward(m, c, 0.1, rng)
            got.append((f, gradients(m, c, f["total"], f["mean"], f["rstd"], dy, None, 0.1, rng)))
    torch.cuda.synchronize()
    for f, h in got:
        assert all(torch.equal(f[k], t[k]) for k in t) and all(torch.equal(h[k], g[k]) for k in g)


def test_rows_over_32_bits(m):
    """Elements that pass 2^31 (their bytes 2^32): the last rows are those of a call on them alone."""
    width = 16384
    rows = (1 << 31) // width + 3
    x = torch.empty(rows, width, dtype=BF16, device="cuda").normal_()
    w = torch.ones(width, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    m.moe_layer_norm(x, w, y, kind="rms", rstd=rstd)
    small, few = torch.empty(4, width, dtype=BF16, device="cuda"), torch.empty(4, device="cuda")
    m.moe_layer_norm(x[-4:].clone(), w, small, kind="rms", rstd=few)
    # the same row by a kernel of other lanes: rstd by at most twice the additions' roundings, y by a step of its type
    assert ((y[-4:].float() - small.float()).abs() <= 2.0 ** -7 * small.float().abs() + 1e-30).all()
    assert ((rstd[-4:] - few).abs() <= 300 * U * few).all()
    dx = torch.empty_like(x)
    m.moe_layer_norm_backward(x, w, rstd, y, dx, kind="rms")
    tail = torch.empty_like(small)
    m.moe_layer_norm_backward(x[-4:].clone(), w, rstd[-4:].clone(), y[-4:].clone(), tail, kind="rms")
    # dx of y itself is 0 but for roundings: g - xh mean(g xh), both of size up to |xh|
    assert ((dx[-4:].float() - tail.float()).abs() <= 2.0 ** -7 * tail.float().abs() + 300 * U * 6).all()


@pytest.mark.parametrize("width,dtype", [(7168, BF16), (5121, F32), (12000, BF16)])
def test_more_than_the_caches_hold(m, width, dtype):
    """Calls that stream past the caches: their first rows are bit for bit those of a call on them alone, the sums over
    all rows those of float64."""
    rows = (300 << 20) // (width * (2 if dtype == BF16 else 4))
    c = Rows(7, 8, width, dtype, "layer", True)
    c.x = torch.randn(rows, width, device="cuda").to(dtype)
    c.residual = (torch.randn(rows, width, device="cuda") + 0.2).to(dtype)
    rng = rng_of(21, 22)
    t = forward(m, c, 0.1, rng)
    dy, dt = (torch.randn(rows, width, device="cuda").to(dtype) for _ in range(2))
    g = gradients(m, c, t["total"], t["mean"], t["rstd"], dy, dt, 0.1, rng)
    few = Rows(7, 8, width, dtype, "layer", True)
    few.x, few.residual = c.x[:70].clone(), c.residual[:70].clone()
    f = forward(m, few, 0.1, rng)
    h = gradients(m, few, f["total"], f["mean"], f["rstd"], dy[:70].clone(), dt[:70].clone(), 0.1, rng)
    for k in ("y", "total", "mean", "rstd"):
        assert torch.equal(t[k][:70], f[k]), k
    for k in ("dx", "dresidual"):
        assert torch.equal(g[k][:70], h[k]), k
    dw, db, mw, mb = (torch.zeros(width, dtype=torch.float64, device="cuda") for _ in range(4))
    for lo in range(0, rows, 4096):
        r = slice(lo, lo + 4096)
        xh = (t["total"][r].double() - t["mean"][r].double()[:, None]) * t["rstd"][r].double()[:, None]
        d = dy[r].double()
        dw += (d * xh).sum(0)
        db += d.sum(0)
        mw += (d * xh).abs().sum(0)
        mb += d.abs().sum(0)
    sums = (64 + rows // 64 + 8) * U
    assert ((g["dweight"] - dw).abs() <= sums * mw).all() and ((g["dbias"] - db).abs() <= sums * mb).all()


def test_refused(m):
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    y, f, b = torch.zeros_like(x), torch.ones(4, device="cuda"), torch.zeros(64, device="cuda")
    rng = rng_of(1, 2)
    ws = torch.empty(m.layer_norm_backward_workspace_bytes(4, 64), dtype=torch.uint8, device="cuda")
    e = m.MoeError
    fwd = lambda x=x, w=w, y=y, **k: m.moe_layer_norm(x, w, y, **k)  # noqa: E731
    bwd = lambda total=x, w=w, rstd=f, dy=y, dx=torch.zeros_like(x), dw=b, ws=ws, **k: m.moe_layer_norm_backward(  # noqa: E731
        total, w, rstd, dy, dx, dw, ws, **{"mean": f.clone(), **k})
    for call in (lambda: fwd(x=x.half()), lambda: fwd(x=x.t()), lambda: fwd(w=w[:63]), lambda: fwd(y=y.bfloat16()),
                 lambda: fwd(bias=b.bfloat16()), lambda: fwd(residual=y.clone()), lambda: fwd(p=0.1, total=x.clone()),
                 lambda: fwd(p=0.1, rng=rng), lambda: fwd(p=0.1, rng=rng.int(), total=x.clone()), lambda: fwd(kind="batch"),
                 lambda: fwd(mean=f, kind="rms"), lambda: fwd(mean=f[:3]), lambda: fwd(eps=-1.0), lambda: fwd(p=2.0),
                 lambda: fwd(residual=x.clone(), total=y), lambda: bwd(mean=None), lambda: bwd(ws=None),
                 lambda: bwd(ws=ws[:100]), lambda: bwd(dw=b.double()), lambda: bwd(dx=x), lambda: bwd(kind="rms"),
                 lambda: bwd(dresidual=y, dx=y), lambda: bwd(dbias=b), lambda: bwd(p=0.5)):
        with pytest.raises(e):
            call()
    fwd()
    bwd(dbias=b.clone())


def test_captured_and_replayed(m):
    """Forward and gradient in one graph: a replay draws the mask of what rng holds then, and reuses the workspace that an
    eager call in between writes too."""
    c = Rows(6, 130, 2048, BF16, "layer", True)
    rng, dy = rng_of(11, 0), torch.randn_like(c.x)
    rows, width = c.x.shape
    ws = torch.empty(m.layer_norm_backward_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")
    f32 = dict(dtype=F32, device="cuda")

    def buffers():
        return dict(total=torch.empty_like(c.x), y=torch.empty_like(c.x), mean=torch.empty(rows, **f32),
                    rstd=torch.empty(rows, **f32), dx=torch.empty_like(c.x), dres=torch.empty_like(c.x),
                    dw=torch.zeros(width, **f32), db=torch.zeros(width, **f32))

    def call(t):
        m.moe_layer_norm(c.x, c.w, t["y"], bias=c.b, residual=c.residual, total=t["total"], mean=t["mean"], rstd=t["rstd"], p=0.3,
                         rng=rng, offset=5)
        m.moe_layer_norm_backward(t["total"], c.w, t["rstd"], dy, t["dx"], t["dw"], ws, dbias=t["db"], mean=t["mean"], dtotal=dy,
                                  dresidual=t["dres"], p=0.3, rng=rng, offset=5)

    held = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(held)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(held)
    masks = []
    for rep in range(3):
        rng[1] = 100 * rep
        for t in held.values():
            t.view(torch.uint8).fill_(0x5A)
        g.replay()
        want = buffers()
        call(want)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(held[k], want[k]), (rep, k)
        masks.append(held["dx"] == 0)
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[1], masks[2])
