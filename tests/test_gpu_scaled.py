"""The 8-bit path on the GPU: quantisers and the scaled grouped GEMM against float64."""
import numpy as np
import pytest
import torch

from oracle import scaled_ref as ref
from scaled_common import FP8, TORCH, Operands, bf16, bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


# ---- rows ------------------------------------------------------------------------------------

def run_rows(m, x, fmt, dtype, gather=None, div=1, row_scale=None, copy=False):
    rows = len(x) if gather is None else len(gather)
    xt = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TORCH[dtype]).cuda()
    q = torch.full((rows, x.shape[1]), 3.0, device="cuda").to(FP8[fmt])
    s = torch.full((rows, m.scale_row_bytes(x.shape[1])), 9, dtype=torch.uint8, device="cuda")
    c = torch.full((rows, x.shape[1]), 7.0, dtype=TORCH[dtype], device="cuda") if copy else None
    dev = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, t)).cuda()  # noqa: E731
    m.moe_quant_rows(xt, q, s, gather=dev(gather, np.int32), gather_div=div,
                     row_scale=dev(row_scale, np.float32), copy=c)
    torch.cuda.synchronize()
    return q, s, c


def same(q, want):
    assert np.array_equal(np.isnan(q), np.isnan(want))
    assert np.array_equal(np.nan_to_num(q, nan=0.0, posinf=1e30, neginf=-1e30),
                          np.nan_to_num(want, nan=0.0, posinf=1e30, neginf=-1e30))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", [(1, 16), (3, 128), (5, 144), (2, 1408), (7, 2048), (2, 2064), (1, 20496)])
def test_quant_rows(m, fmt, dtype, rows, width):
    rng = np.random.default_rng(rows * 7 + width)
    x = rng.standard_normal((rows, width)) * 2.0 ** rng.integers(-40, 40, (rows, width))
    x = bf16(x) if dtype == "bf16" else x.astype(np.float32)
    q, s, _ = run_rows(m, x, fmt, dtype)
    wq, ws, _ = ref.quant_rows(x, fmt)
    assert np.array_equal(s.cpu().numpy(), ws)
    same(host(q), wq)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quant_rows_every_bf16_value(m, fmt):
    """Each bf16 bit pattern beside a few others: zeros, subnormals, infinities and NaN."""
    bits = np.arange(65536, dtype=np.uint32) << 16
    x = bits.view(np.float32).reshape(512, 128)
    q, s, _ = run_rows(m, x, fmt, "f32")
    wq, ws, _ = ref.quant_rows(x, fmt)
    assert np.array_equal(s.cpu().numpy(), ws)
    same(host(q), wq)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quant_rows_borders(m, fmt):
    """Block maxima at and next to the format's largest value times a power of two, ties of every
    kind, signed zeros, blocks of zeros, subnormal blocks, fp32's largest value."""
    top = np.float32(ref.FORMATS[fmt][2])
    rows = []
    for e in (-126, -60, 0, 60, 100):
        for v in (np.nextafter(top, np.float32(0)), top, np.nextafter(top, np.float32(np.inf))):
            r = np.linspace(-1, 1, 128, dtype=np.float32) * top * np.float32(0.99)
            r[17] = -v
            rows.append(np.ldexp(r, e - 20 if e == 100 else e))
    step = np.arange(128, dtype=np.float32) / 16 * (top / 8)
    rows += [step, np.zeros(128), -np.zeros(128), np.full(128, 1e-45), np.full(128, 3e-39),
             np.full(128, np.finfo(np.float32).max)]
    x = np.array(rows, np.float32)
    q, s, _ = run_rows(m, x, fmt, "f32")
    wq, ws, _ = ref.quant_rows(x, fmt)
    assert np.array_equal(s.cpu().numpy(), ws)
    same(host(q), wq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [False, True])
def test_quant_rows_gather(m, dtype, weighted):
    rng = np.random.default_rng(5)
    src, width, div, rows = 37, 272, 3, 150
    x = rng.standard_normal((src, width))
    x = bf16(x) if dtype == "bf16" else x.astype(np.float32)
    gather = rng.integers(-2, src * div, rows)
    gather[:4] = [-1, src * div - 1, 0, src * div]       # none, last, first, past the source
    gather[4] = 2**31 - 1
    w = rng.standard_normal(src * div).astype(np.float32) if weighted else None
    q, s, c = run_rows(m, x, "e4m3", dtype, gather, div, w, copy=True)
    wq, ws, rowsv = ref.quant_rows(x, "e4m3", gather, div, w)
    assert np.array_equal(s.cpu().numpy(), ws)
    same(host(q), wq)
    assert np.array_equal(host(c), (bf16(rowsv) if dtype == "bf16" else rowsv).astype(np.float64))


def test_quant_rows_weighted_in_place_order(m):
    x = bf16(np.random.default_rng(1).standard_normal((9, 160)))
    w = np.linspace(-2, 2, 9).astype(np.float32)
    q, s, _ = run_rows(m, x, "e5m2", "bf16", row_scale=w)
    wq, ws, _ = ref.quant_rows(x, "e5m2", row_scale=w)
    assert np.array_equal(s.cpu().numpy(), ws)
    same(host(q), wq)


# ---- weights -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,K,N", [(1, 16, 16), (2, 128, 128), (3, 144, 272), (1, 400, 2064), (1, 2064, 48)])
def test_quant_weight(m, dtype, G, K, N):
    rng = np.random.default_rng(G * K + N)
    w = rng.standard_normal((G, K, N)) * 2.0 ** rng.integers(-8, 8, (G, K, 1))
    w[0, :16, :16] = 0.0
    w = bf16(w) if dtype == "bf16" else w.astype(np.float32)
    w[-1, K // 2, N // 2] = np.nan
    w[0, 0, N - 1] = np.inf
    wt = torch.from_numpy(w).to(TORCH[dtype]).cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    q = torch.full((G, K, N), 1, **u8).view(FP8["e4m3"])
    qt = torch.full((G, N, K), 1, **u8).view(FP8["e4m3"])
    qs = torch.full((G, -(-K // 128), m.scale_row_bytes(N)), 5, **u8)
    ts = torch.full((G, -(-N // 128), m.scale_row_bytes(K)), 5, **u8)
    m.moe_quant_weight(wt, q, qs, qt, ts)
    wq, wqs, wqt, wts = ref.quant_weight(w)
    same(host(q), wq)
    same(host(qt), wqt)
    assert np.array_equal(qs.cpu().numpy(), wqs)
    assert np.array_equal(ts.cpu().numpy(), wts)
    # either pair alone
    q2, t2 = torch.zeros_like(q.view(torch.uint8)).view(FP8["e4m3"]), torch.zeros_like(qt.view(torch.uint8)).view(FP8["e4m3"])
    qs2, ts2 = torch.zeros_like(qs), torch.zeros_like(ts)
    m.moe_quant_weight(wt, q2, qs2)
    m.moe_quant_weight(wt, qt=t2, qt_scale=ts2)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(qs2, qs)
    assert torch.equal(t2.view(torch.uint8), qt.view(torch.uint8)) and torch.equal(ts2, ts)


# ---- product -------------------------------------------------------------------------------------

SEGMENTS = {
    "one_row": [1], "one_each": [1] * 9, "empty_ends": [0, 0, 5, 0, 17, 0], "sixteen": [16, 16, 0, 32],
    "uneven": [3, 0, 130, 1, 64, 0, 65, 257], "one_expert": [0, 0, 0, 300, 0], "none": [0, 0, 0],
}


@pytest.mark.parametrize("name", list(SEGMENTS))
@pytest.mark.parametrize("K,C", [(16, 16), (128, 48), (144, 272), (1408, 128), (528, 400)])
def test_product(m, name, K, C):
    lens = SEGMENTS[name]
    ops = Operands(K + C, lens, len(lens), K, C, tail=3)
    got = host(ops.run(m))
    want, mag, top = ops.expected()
    end = int(ops.cu[-1])
    assert (np.abs(got - want) <= bound(K, want, mag, top))[:end].all()
    assert (got[end:] == -7.0).all()      # rows behind the last segment stay


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("K,C,lens", [(2048, 256, [100, 0, 29, 300]), (1040, 528, [700, 1, 40]),
                                      (2064, 2064, [5, 0, 2]), (4112, 16, [31, 33])])
def test_product_integers(m, fmt, grad, K, C, lens):
    """Integers times powers of two: every partial sum is exact (the products of a group of 8 span
    2^4, the scales 2^12), so the one rounding to bf16 is all that happens, bit for bit."""
    ops = Operands(3, lens, len(lens), K, C, fmt, ints=True, first=2)
    got = host(ops.run(m, grad))
    want = bf16(ops.expected()[0].astype(np.float32))
    assert np.array_equal(got[2:], want[2:])
    assert (got[:2] == -7.0).all()        # rows ahead of the first segment stay


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_product_scale_range(m, fmt):
    """Scales from the smallest to large ones, one block far above the others."""
    ops = Operands(11, [20, 7], 2, 640, 144, fmt)
    ops.a_scale[:, :5] = [0, 60, 127, 190, 20]
    ops.b_scale[:, :, :5] = [130, 127, 127, 100, 254]
    got = host(ops.run(m))
    want, mag, top = ops.expected()
    assert (np.abs(got - want) <= bound(640, want, mag, top)).all()


def test_product_nan_stays_in_its_row(m):
    """A NaN in one row of a (or an infinity in e5m2) reaches that row's results only, a NaN weight
    its column's only."""
    for fmt, byte in (("e4m3", 0x7F), ("e5m2", 0x7C)):
        ops = Operands(12, [20, 40], 2, 272, 144, fmt)
        ops.a[25, 200] = byte
        ops.b[1, 77, 3] = 0x7F
        got = host(ops.run(m))
        bad = ~np.isfinite(got)
        want = np.zeros_like(bad)
        want[25] = True
        want[20:, 77] = True
        assert np.array_equal(bad, want)


def test_product_bad_cu(m):
    """cu_seqlens outside the rows is cut to them; nothing outside out is written."""
    ops = Operands(13, [16, 16, 16], 3, 256, 64)
    want, mag, top = ops.expected()
    ops.cu = np.array([-5, 16, 32, 999], np.int32)
    got = host(ops.run(m))
    assert (np.abs(got - want) <= bound(256, want, mag, top)).all()


def test_product_strided_stream(m):
    """A call on a side stream, ordered by events."""
    ops = Operands(14, [50, 3], 2, 384, 96)
    side = torch.cuda.Stream()
    a, sa, b, sb, cu = ops.on_gpu()
    o = torch.zeros((ops.M, ops.C), dtype=torch.bfloat16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    m.moe_group_gemm_scaled(m.GEMM_FWD, a, sa, b, sb, cu, o, ops.K, ops.C, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want, mag, top = ops.expected()
    assert (np.abs(host(o) - want) <= bound(384, want, mag, top)).all()


# sizes that reach each kernel (see launch_scaled): segments, contraction, columns
KERNELS = {
    "few_rows": ([3, 0, 5, 1, 0, 2], 1296, 272), "few_rows_long": ([16], 7184, 1040),
    "tiles_64x64": ([40, 0, 65, 0], 2176, 528), "tiles_64x128": ([200, 33, 0, 90], 640, 4112),
    "tiles_64x128_short": ([130, 500], 16, 2064),
    "tiles_128x256": ([300, 0, 129, 127, 511], 1424, 8192), "tiles_128x256_short": ([700, 300], 272, 8208),
    "tiles_256x256": ([1500, 1700], 2176, 4112), "tiles_256x256_short": ([1025], 112, 16400),
    "tiles_256x256_many": ([5000], 528, 8208),
    # several tiles a workgroup and a last piece of scales (16 blocks of the contraction) of 1 to 7 blocks
    "stream_64x64": ([576], 2176, 2048), "stream_64x128": ([60] * 40, 2064, 2064),
    "stream_64x128_3": ([60] * 40, 2352, 2064), "stream_64x128_6": ([60] * 40, 2800, 2064),
    "stream_128x256": ([300] * 12, 2176, 8208), "stream_128x256_2": ([300] * 12, 2304, 8208),
    # several tiles a workgroup of one or two blocks of the contraction each
    "blocks_256x256_1": ([5000], 96, 16400), "blocks_256x256_2": ([9000], 256, 8208),
    "stream_256x256": ([5000], 2064, 8208), "stream_256x256_2": ([5000], 4352, 8208),
}


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("name", list(KERNELS))
def test_product_kernels(m, name, fmt, grad):
    """Every kernel, on integers times powers of two (scales within 2^6, so that sums over the whole
    contraction stay exact in fp32): equal to the float64 product rounded once."""
    lens, K, C = KERNELS[name]
    gen = torch.Generator(device="cuda").manual_seed(K + C)
    M, G, tail = sum(lens) + 5, len(lens), 3
    ints = lambda *s: torch.randint(-1, 2, s, device="cuda", generator=gen).float()  # noqa: E731
    a, b = ints(M + tail, K).to(FP8[fmt]), ints(G, C, K).to(FP8["e4m3"])

    def scales(*rows):
        s = torch.full(rows + (m.scale_row_bytes(K),), 255, dtype=torch.uint8, device="cuda")
        s[..., :-(-K // 128)] = torch.randint(126, 129, rows + (-(-K // 128),), device="cuda", generator=gen).byte()
        return s

    sa, sb = scales(M + tail), scales(G, -(-C // 128))
    cu = torch.tensor(np.concatenate([[5], 5 + np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out = torch.full((M + tail, C), -7.0, dtype=torch.bfloat16, device="cuda")
    op, kd, n = (m.GEMM_DGRAD, C, K) if grad else (m.GEMM_FWD, K, C)
    m.moe_group_gemm_scaled(op, a, sa, b, sb, cu, out, kd, n)
    want = torch.full_like(out, -7.0)
    kb = torch.arange(K, device="cuda") // 128
    two = lambda s: torch.exp2((s.double() - 127))[..., kb]  # noqa: E731
    at = 5
    for g, n_rows in enumerate(lens):
        rows = slice(at, at + n_rows)
        w = b[g].double() * two(sb[g]).repeat_interleave(128, 0)[:C]
        want[rows] = (a[rows].double() * two(sa[rows])).mm(w.t().contiguous()).bfloat16()
        at += n_rows
    assert torch.equal(out, want)


def test_over_32_bits(m):
    """Operands of more than 2^32 bytes, results in their last rows: the same bits as from small ones."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, G, K, C, n = 600000, 270, 8192, 2048, 100
    last_a = torch.randint(-1, 2, (n, K), device="cuda", generator=gen).float().to(FP8["e4m3"])
    last_b = torch.randint(-1, 2, (C, K), device="cuda", generator=gen).float().to(FP8["e4m3"])
    want = (last_a.double() @ last_b.double().t().contiguous()).bfloat16()
    a = torch.zeros((M, K), dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    b = torch.zeros((G, C, K), dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    a.view(torch.uint8)[M - n:] = last_a.view(torch.uint8)
    b.view(torch.uint8)[G - 1] = last_b.view(torch.uint8)
    sa = torch.full((M, m.scale_row_bytes(K)), 127, dtype=torch.uint8, device="cuda")
    sb = torch.full((G, C // 128, m.scale_row_bytes(K)), 127, dtype=torch.uint8, device="cuda")
    cu = torch.full((G + 1,), M - n, dtype=torch.int32, device="cuda")
    cu[G] = M
    out = torch.full((M, C), -7.0, dtype=torch.bfloat16, device="cuda")
    m.moe_group_gemm_scaled(m.GEMM_FWD, a, sa, b, sb, cu, out, K, C)
    assert torch.equal(out[M - n:], want) and (out[M - n - 1] == -7.0).all()
    # the few-rows kernel: as many segments as make the rows few
    few = torch.full((8, C), -7.0, dtype=torch.bfloat16, device="cuda")
    cu8 = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    cu8[G] = 8
    m.moe_group_gemm_scaled(m.GEMM_FWD, a[M - n:M - n + 8].contiguous(), sa[:8], b, sb, cu8, few, K, C)
    assert torch.equal(few, want[:8])
    del a, b, out
    x = torch.zeros((M, 4096), dtype=torch.bfloat16, device="cuda")
    x[M - 1] = torch.randn(4096, device="cuda", generator=gen).bfloat16()
    q = torch.full((M, 4096), 1, dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    s = torch.full((M, m.scale_row_bytes(4096)), 9, dtype=torch.uint8, device="cuda")
    copy = torch.empty_like(x)
    m.moe_quant_rows(x, q, s, copy=copy)
    wq, ws, _ = ref.quant_rows(host(x[M - 1:]), "e4m3")
    assert np.array_equal(host(q[M - 1:]), wq) and np.array_equal(s[M - 1:].cpu().numpy(), ws)
    assert torch.equal(copy[M - 1], x[M - 1]) and (q[M - 2].view(torch.uint8) == 0).all()
    g = torch.tensor([(M - 1) * 3 + 2, -1], dtype=torch.int32, device="cuda")
    m.moe_quant_rows(x, q[:2], s[:2], gather=g, gather_div=3)
    assert np.array_equal(host(q[:1]), wq) and (q[1].view(torch.uint8) == 0).all()


def test_weights_over_32_bits(m):
    """moe_quant_weight past 2^32 bytes: the last expert as quantised alone."""
    G, K, N = 130, 4096, 4112
    w = torch.zeros((G, K, N), dtype=torch.bfloat16, device="cuda")
    w[G - 1] = torch.randn((K, N), device="cuda").bfloat16()
    u8 = dict(dtype=torch.uint8, device="cuda")

    def quantise(w):
        g = w.shape[0]
        out = (torch.full((g, K, N), 1, **u8).view(FP8["e4m3"]), torch.full((g, K // 128, m.scale_row_bytes(N)), 5, **u8),
               torch.full((g, N, K), 1, **u8).view(FP8["e4m3"]), torch.full((g, -(-N // 128), m.scale_row_bytes(K)), 5, **u8))
        m.moe_quant_weight(w, *out)
        return out

    for big, alone in zip(quantise(w), quantise(w[G - 1:])):
        assert torch.equal(big.view(torch.uint8)[G - 1:], alone.view(torch.uint8))


def test_sizes_past_32_bits_are_refused(m):
    """A size that would wrap around in a 32-bit argument: an error, nothing written."""
    x = torch.randn(4, 64, device="cuda")
    g = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.full((4, 64), 7, dtype=torch.uint8, device="cuda")
    s = torch.full((4, 16), 9, dtype=torch.uint8, device="cuda")
    with pytest.raises(m.MoeError, match="sizes"):
        m.moe_quant_rows(x, q.view(FP8["e4m3"]), s, gather=g, gather_div=(1 << 32) + 1)
    a = torch.empty((0, 64), dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    with pytest.raises(m.MoeError):
        m.moe_group_gemm_scaled(m.GEMM_FWD, a, s[:0], q.view(FP8["e4m3"]), s, g[:2],
                                torch.empty((0, 4), dtype=torch.bfloat16, device="cuda"), (1 << 32) + 64, 4)
    assert (q == 7).all() and (s == 9).all()


def test_no_rows_and_no_source(m):
    e = torch.empty((0, 64), device="cuda")
    m.moe_quant_rows(e, e.to(FP8["e4m3"]), torch.empty((0, 16), dtype=torch.uint8, device="cuda"))
