"""The 8-bit path and the clipping where their other tests do not go: packed bf16 rows with every bit pattern, the kernel
for few rows over several passes of its grid."""
import numpy as np
import pytest
import torch

from oracle import scaled_ref as ref
from scaled_common import FP8, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def quantise_bf16(m, x, fmt):
    """(q as float64, scale bytes, copy) of bf16 rows without weights: the path that keeps them packed."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().cuda()
    q = torch.full(t.shape, 3, dtype=torch.uint8, device="cuda").view(FP8[fmt])
    s = torch.full((t.shape[0], m.scale_row_bytes(t.shape[1])), 9, dtype=torch.uint8, device="cuda")
    copy = torch.full_like(t, 7.0)
    m.moe_quant_rows(t, q, s, copy=copy)
    assert torch.equal(copy.view(torch.int16), t.view(torch.int16))
    return q.float().cpu().numpy().astype(np.float64), s.cpu().numpy()


def exactly(m, x, fmt):
    q, s = quantise_bf16(m, x, fmt)
    wq, ws, _ = ref.quant_rows(x, fmt)
    assert np.array_equal(s, ws)
    assert np.array_equal(q, wq, equal_nan=True)
    return ws


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_bf16_rows_of_every_value(m, fmt):
    """Each bf16 bit pattern beside its neighbours, and all of them shuffled, so that every block holds
    ordinary values, infinities or NaN and tiny ones together."""
    bits = np.arange(65536, dtype=np.uint32) << 16
    x = bits.view(np.float32).reshape(512, 128)
    ws = exactly(m, x, fmt)
    assert (ws[:, 0] == 0).any()        # blocks held at the smallest scale
    exactly(m, np.random.default_rng(0).permutation(bits).view(np.float32).reshape(64, 1024), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_bf16_rows_with_one_not_finite(m, fmt):
    """One infinity or NaN, in each place of a block, beside ordinary values: it does not count for the
    block's scale, and the others round as without it."""
    rng = np.random.default_rng(1)
    base = bf16(rng.standard_normal((128, 272)) * 2.0 ** rng.integers(-3, 4, (128, 272)))
    for v in (np.inf, -np.inf, np.nan):
        x = base.copy()
        x[np.arange(128), np.arange(128)] = v
        x[:, 256 + 5] = v
        exactly(m, x, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_bf16_rows_borders(m, fmt):
    """Block maxima at and next to the format's largest value times a power of two, signed zeros, blocks of
    zeros, of subnormals, of bf16's largest and smallest values, ties of every kind."""
    top = ref.FORMATS[fmt][2]
    rows = []
    for e in (-126, -60, 0, 60, 100):
        for f in (1.0 - 2.0 ** -8, 1.0, 1.0 + 2.0 ** -6 / 1.75):   # 0.875 2^n less half a step, itself, the value above
            r = np.linspace(-1, 1, 128) * top * 0.99
            r[17] = -top * f
            rows.append(np.ldexp(r, e - 20 if e == 100 else e))
    rows += [np.arange(128) / 16 * (top / 8), np.zeros(128), -np.zeros(128), np.full(128, 2.0 ** -133),
             np.full(128, 3e-39), np.arange(128) * 2.0 ** -133, np.full(128, 2.0 ** -126),
             np.full(128, float(torch.finfo(torch.bfloat16).max)),
             np.where(np.arange(128) % 2, 2.0 ** -133, 1.0)]
    exactly(m, bf16(np.array(rows)), fmt)


# Sizes that the rule for few rows takes (M_total <= 16, or <= 8 a segment): segments, contraction, columns
FEW = {
    "at_most_16": ([7], 7184, 1040), "8_a_segment": ([16, 0, 0], 7184, 1040), "16_in_one": ([0, 24, 0, 0], 2064, 528),
    # more tiles than one pass of the grid (8 workgroups a compute unit): a workgroup's second tile and on
    "second_pass": ([i % 5 for i in range(264)], 400, 1024), "third_pass": ([8] * 300 + [0], 144, 1040),
    "long_segments": ([1000] + [0] * 300 + [900, 3], 272, 1552),
}


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("name", list(FEW))
def test_few_rows(m, name, fmt, grad):
    """The kernel for few rows on integers times powers of two (scales within 2^6, so that sums over the whole
    contraction stay exact in fp32): equal to the float64 product rounded once."""
    lens, K, C = FEW[name]
    M, G = sum(lens) + 3, len(lens)      # 3 rows outside every segment
    assert M <= 16 or M <= 8 * G
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sum(-(-n // 16) for n in lens) * -(-C // 32)
    assert "pass" not in name or tiles > 8 * cus * (2 if name == "third_pass" else 1)
    gen = torch.Generator(device="cuda").manual_seed(K + C)
    ints = lambda *s: torch.randint(-1, 2, s, device="cuda", generator=gen).float()  # noqa: E731
    a, b = ints(M, K).to(FP8[fmt]), ints(G, C, K).to(FP8["e4m3"])

    def scales(*rows):
        s = torch.full(rows + (m.scale_row_bytes(K),), 255, dtype=torch.uint8, device="cuda")
        s[..., :-(-K // 128)] = torch.randint(126, 129, rows + (-(-K // 128),), device="cuda", generator=gen).byte()
        return s

    sa, sb = scales(M), scales(G, -(-C // 128))
    cu = torch.tensor(np.concatenate([[2], 2 + np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    out = torch.full((M, C), -7.0, dtype=torch.bfloat16, device="cuda")
    op, kd, n = (m.GEMM_DGRAD, C, K) if grad else (m.GEMM_FWD, K, C)
    m.moe_group_gemm_scaled(op, a, sa, b, sb, cu, out, kd, n)
    want = torch.full_like(out, -7.0)
    kb = torch.arange(K, device="cuda") // 128
    two = lambda s: torch.exp2((s.double() - 127))[..., kb]  # noqa: E731
    at = 2
    for g, n_rows in enumerate(lens):
        rows = slice(at, at + n_rows)
        w = b[g].double() * two(sb[g]).repeat_interleave(128, 0)[:C]
        want[rows] = (a[rows].double() * two(sa[rows])).mm(w.t().contiguous()).bfloat16()
        at += n_rows
    assert torch.equal(out, want)


def test_a_segment_of_nearly_2_31_rows(m):
    """More rows in one segment than 2^31 less a tile: they are all written."""
    torch.cuda.empty_cache()
    M, K = (1 << 31) - 64, 16
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of memory")
    gen = torch.Generator(device="cuda").manual_seed(2)
    ends = torch.randint(-2, 3, (600, K), device="cuda", generator=gen).float().to(FP8["e4m3"])
    b = torch.randint(-2, 3, (1, K, K), device="cuda", generator=gen).float().to(FP8["e4m3"])
    want = (ends.double() @ b[0].double().t().contiguous()).bfloat16()
    a = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    a[:300], a[M - 300:] = ends[:300].view(torch.uint8), ends[300:].view(torch.uint8)
    sa = torch.full((M, 16), 127, dtype=torch.uint8, device="cuda")
    sb = torch.full((1, 1, 16), 127, dtype=torch.uint8, device="cuda")
    out = torch.full((M, K), -7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    m.moe_group_gemm_scaled(m.GEMM_FWD, a.view(FP8["e4m3"]), sa, b, sb, cu, out, K, K)
    assert torch.equal(out[:300], want[:300]) and torch.equal(out[M - 300:], want[300:])
    for lo in range(300, M - 300, 1 << 27):
        assert not out[lo:min(lo + (1 << 27), M - 300)].any()
    del a, sa, out
    torch.cuda.empty_cache()


def layer_step(**kw):
    """A small layer with filled inputs."""
    import synth
    from balanced_token_dispatch_amd.layer import LayerStep, Shape
    s = Shape(R=4, S=96, K=2, E=16, B=2, H=272, Hp=144)
    L = LayerStep(s, rank=1, **kw)
    idx, w = synth.routing(synth.Dims(R=s.R, S=s.S, K=s.K, E=s.E, B=s.B, H=s.H, Hp=s.Hp), 1.0, 31)
    synth.fill_normal_(L.x_all, 1.0, 311)
    synth.fill_normal_(L.w_up, 0.1, 312)
    synth.fill_normal_(L.w_down, 0.1, 313)
    L.topk_idx.copy_(torch.from_numpy(idx))
    L.topk_w.copy_(torch.from_numpy(w))
    return L


def test_a_kept_norm_stays(m):
    """The norm that clip_gradients returned, after further calls and replays of a captured one."""
    L = layer_step()
    kept = []
    for n in (1.0, 2.0):
        L.dw_up.fill_(n)
        kept.append(L.clip_gradients(1e9))
    L.dw_up.fill_(1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.clip_gradients(1e9)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = L.clip_gradients(1e9)
    one = (16 * 272 * 144) ** 0.5
    for n in (3.0, 4.0, 5.0):
        L.dw_up.fill_(n)
        g.replay()
        assert captured.item() == pytest.approx(n * one, rel=1e-6) and L.grad_norm.item() == captured.item()
        L.dw_up.fill_(2 * n)
        kept.append(L.clip_gradients(1e9))
        assert captured.item() == pytest.approx(n * one, rel=1e-6)
    assert [k.item() for k in kept] == pytest.approx([n * one for n in (1.0, 2.0, 6.0, 8.0, 10.0)], rel=1e-6)


def test_forward_only_layer(m):
    """A layer without a backward holds the weights in the order FWD reads, and gives the same results."""
    both, one = (layer_step(gemm="scaled", backward=b) for b in (True, False))
    for L in (both, one):
        L.y_all.zero_()
        L.quantise_weights()
        L.forward()
    assert one.q_up.q is None and one.q_down.q_scale is None
    assert both.q_up.q is not None
    for k in ("z", "y", "out"):
        assert torch.equal(getattr(one, k), getattr(both, k))
    one.w_up.mul_(2.0)
    with pytest.raises(ValueError, match="quantise_weights"):
        one.forward()
    one.quantise_weights()
    one.step()
    assert torch.equal(one.z, 2 * both.z)       # a scale one step up, the same 8-bit values


def test_8_bit_layer_without_the_16_bit_scratch(m):
    """Its products take no workspace and its weight gradients neither: none is allocated."""
    L = layer_step(gemm="scaled")
    assert L.gemm_ws is None and layer_step().gemm_ws is not None
    for k in ("y_all", "dout_all", "dxp_all"):
        getattr(L, k).normal_()
    L.quantise_weights()
    L.step()
    assert L.dw_up.isfinite().all() and L.dw_up.any()
