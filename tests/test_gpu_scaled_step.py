"""The 8-bit layer step with its router and clipping, run together as a training step runs them: every
stage against float64 from what the stage before it wrote, the step in a graph and with its second
stream, and the weight gradients against the 16-bit step's."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import scaled_ref as ref
from scaled_common import bf16, bound

pytestmark = pytest.mark.gpu

R, S, K, E, B, H, Hp, RANK = 4, 96, 2, 16, 2, 272, 144, 1


def make(overlap=None, grad_format=torch.float8_e4m3fn, **kw):
    from balanced_token_dispatch_amd.layer import LayerStep, Shape
    L = LayerStep(Shape(R, S, K, E, B, H, Hp), rank=RANK, gemm="scaled", overlap=overlap,
                  grad_format=grad_format, **kw)
    idx, w = synth.routing(synth.Dims(R=R, S=S, K=K, E=E, B=B, H=H, Hp=Hp), 1.0, 31)
    for t, sd in ((L.x_all, 311), (L.y_all, 314), (L.dout_all, 315), (L.dxp_all, 316)):
        synth.fill_normal_(t, 1.0, sd)
    synth.fill_normal_(L.w_up, 0.1, 312)
    synth.fill_normal_(L.w_down, 0.1, 313)
    L.topk_idx.copy_(torch.from_numpy(idx))
    L.topk_w.copy_(torch.from_numpy(w))
    gen = torch.Generator().manual_seed(9)
    logits = torch.randn(S, E, generator=gen).cuda()
    return L, logits


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def run(L, logits, limit=0.5):
    dlogits = torch.full_like(logits, 7.0)
    L.dw_up.zero_()
    L.dw_down.zero_()
    L.route(logits, factor=2.0)
    L.quantise_weights()
    L.step()
    L.route_backward(logits, dlogits, factor=2.0)
    before = [L.dw_up.clone(), L.dw_down.clone(), dlogits.clone()]
    norm = L.clip_gradients(limit, others=[dlogits])
    return dlogits, before, norm


def quantised(q, s, rows, fmt="e4m3"):
    """q and s against the rows they were made of: exact."""
    wq, ws, _ = ref.quant_rows(rows, fmt)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(host(q), wq)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_step_stage_by_stage(fmt):
    L, logits = make(grad_format={"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt])
    dlogits, (dw_up, dw_down, dl), norm = run(L, logits)
    torch.cuda.synchronize()
    assert int(L.status.item()) == 0
    ids, w = ref.router_topk(host(logits), K, "softmax_topk", factor=2.0)
    assert np.array_equal(L.topk_idx[RANK].cpu().numpy(), ids)
    assert np.allclose(host(L.topk_w[RANK]), w, rtol=1e-5, atol=0)
    idx = L.topk_idx.cpu().numpy()
    pl = oracle.plan(idx, E, B)
    cu, dest, src = oracle.layout(idx, pl, RANK)
    assert np.array_equal(L.cu.cpu().numpy(), cu) and np.array_equal(L.src.cpu().numpy(), src)

    # weights: the home experts', and in the slots the rows of the experts they duplicate
    for wt, qw in ((L.w_up, L.q_up), (L.w_down, L.q_down)):
        q, qs, qt, ts = ref.quant_weight(host(wt)[:E])
        for got, want in zip(qw.tensors(), (q, qs, qt, ts)):
            got = host(got) if got.dtype != torch.uint8 else got.cpu().numpy()
            assert np.array_equal(got[:E], want)
            for j in range(B):
                e = slot_expert(pl, j)
                if e >= 0:
                    assert np.array_equal(got[E + j], want[e])

    # forward
    x, tw = host(L.x_all), L.topk_w.view(-1).cpu().numpy()
    q, s, rows = ref.quant_rows(x, "e4m3", src, K)
    assert np.array_equal(host(L.xq.q), q) and np.array_equal(L.xq.scale.cpu().numpy(), s)
    assert np.array_equal(host(L.xp), rows)
    product(L.z, L.xq, L.q_up.qt, L.q_up.qt_scale, cu)
    quantised(L.zq.q, L.zq.scale, host(L.z))
    product(L.y, L.zq, L.q_down.qt, L.q_down.qt_scale, cu)

    # backward
    q, s, rows = ref.quant_rows(host(L.dout_all), fmt, src, K, tw)
    assert np.array_equal(host(L.dyq.q), q) and np.array_equal(L.dyq.scale.cpu().numpy(), s)
    assert np.array_equal(host(L.dy), bf16(rows))
    product(L.dz, L.dyq, L.q_down.q, L.q_down.q_scale, cu)
    quantised(L.dzq.q, L.dzq.scale, host(L.dz), fmt)
    product(L.dxp, L.dzq, L.q_up.q, L.q_up.q_scale, cu)
    for dw, a, b in ((dw_up, L.xp, L.dz), (dw_down, L.z, L.dy)):  # contraction over a segment's rows in fp32
        a, b = host(a), host(b)
        want, mag = np.zeros(dw.shape), np.zeros(dw.shape)
        for g in range(E + B):
            home = g if g < E else slot_expert(pl, g - E)
            rows_g = slice(cu[g], cu[g + 1])
            if home >= 0:
                want[home] += a[rows_g].T @ b[rows_g]
                mag[home] += np.abs(a[rows_g]).T @ np.abs(b[rows_g])
        assert (np.abs(host(dw) - want) <= (S * K + 8) * 2.0 ** -23 * mag).all()
    dtw = host(L.dtopk_w).reshape(S, K)
    want = ref.router_backward(host(logits), ids, dtw, "softmax_topk", 2.0)
    assert (np.abs(host(dl) - want) <= 1e-5 * np.abs(dtw).sum(1, keepdims=True)).all()

    # clipping, over the experts' and the gate's gradients
    n, coef = ref.grad_clip([host(dw_up), host(dw_down), host(dl)], 0.5)
    assert coef < 1.0 and abs(norm.item() - n) <= 2.0 ** -23 * n
    for got, was in ((L.dw_up, dw_up), (L.dw_down, dw_down), (dlogits, dl)):
        assert (np.abs(host(got) - coef * host(was)) <= 2.0 ** -22 * np.abs(host(was))).all()


def slot_expert(pl, j):
    """Expert of slot j of this rank (-1: empty), from the plan's blob."""
    blob = pl.to_blob()
    off = 8 + 4 * E + 5 * (E + R)
    return int(blob[off + RANK * B + j])


def product(out, rows, b, b_scale, cu):
    fmt = "e4m3" if rows.q.dtype == torch.float8_e4m3fn else "e5m2"
    want, mag, top = ref.group_gemm_scaled(ref.table(fmt)[rows.q.view(torch.uint8).cpu().numpy()],
                                           rows.scale.cpu().numpy(),
                                           ref.table("e4m3")[b.view(torch.uint8).cpu().numpy()],
                                           b_scale.cpu().numpy(), cu)
    end = cu[-1]
    assert (np.abs(host(out) - want) <= bound(rows.q.shape[1], want, mag, top))[:end].all()


NAMES = ("topk_idx", "topk_w", "cu", "src", "xp", "z", "y", "out", "dy", "dz", "dxp", "dx", "dtopk_w",
         "dw_up", "dw_down", "grad_norm")


def outputs(L, dlogits):
    return {**{k: getattr(L, k).clone() for k in NAMES}, "dlogits": dlogits.clone()}


def same(a, b, what):
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), f"{what}: {k}"


def test_step_in_a_graph():
    """Captured and replayed, with eager steps and overwritten buffers between the replays."""
    L, logits = make()
    dlogits, _, _ = run(L, logits)
    want = outputs(L, dlogits)
    out = torch.full_like(logits, 7.0)

    def step():
        L.dw_up.zero_()
        L.dw_down.zero_()
        L.route(logits, factor=2.0)
        L.quantise_weights()
        L.step()
        L.route_backward(logits, out, factor=2.0)
        L.clip_gradients(0.5, others=[out])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(3):
        for k in ("xp", "z", "y", "out", "dy", "dz", "dx", "dtopk_w", "dw_up", "dw_down", "sumsq", "clip_ws"):
            getattr(L, k).view(torch.uint8).fill_(0x5A)
        for rows in (L.xq, L.zq, L.dyq, L.dzq):
            rows.q.view(torch.uint8).fill_(0x5A)
            rows.scale.fill_(0x5A)
        for qw in (L.q_up, L.q_down):
            for t in qw.tensors():
                t.view(torch.uint8).fill_(0x33)
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        same(outputs(L, out), want, f"replay {rep}")
        dlogits, _, _ = run(L, logits)
        torch.cuda.synchronize()
        same(outputs(L, dlogits), want, f"eager after replay {rep}")


def test_step_second_stream():
    L, logits = make(overlap=False)
    dlogits, _, _ = run(L, logits)
    want = outputs(L, dlogits)
    L.overlap = True
    for _ in range(3):
        dlogits, _, _ = run(L, logits)
        torch.cuda.synchronize()
        same(outputs(L, dlogits), want, "second stream")


def test_weight_gradients_near_the_16_bit_step():
    """The operands' rounding to e4m3 (half a step: 2^-4 of a value, in each of z's and dz's products) keeps
    the weight gradients within 2^-4 + 2^-4 of the 16-bit step's, plus cross terms and bf16 roundings,
    in the 2-norm: below 0.15."""
    from balanced_token_dispatch_amd.layer import LayerStep, Shape
    L, logits = make()
    run(L, logits, limit=1e30)
    P = LayerStep(Shape(R, S, K, E, B, H, Hp), rank=RANK)
    for k in ("x_all", "w_up", "w_down", "y_all", "dout_all", "dxp_all", "topk_idx", "topk_w"):
        getattr(P, k).copy_(getattr(L, k))
    P.step()
    for k in ("dw_up", "dw_down", "out", "dx"):
        a, b = host(getattr(L, k)), host(getattr(P, k))
        assert np.linalg.norm(a - b) <= 0.15 * np.linalg.norm(b), k


def test_refusals():
    from balanced_token_dispatch_amd.layer import LayerStep, Shape
    for kw in (dict(activation="swiglu"), dict(fused_gather=True), dict(dtype=torch.float32),
               dict(grad_format=torch.bfloat16)):
        with pytest.raises(ValueError):
            LayerStep(Shape(R, S, K, E, B, H, Hp), gemm="scaled", **kw)
    with pytest.raises(ValueError):
        LayerStep(Shape(R, S, K, E, B, H, Hp), gemm="int4")
    with pytest.raises(ValueError):
        LayerStep(Shape(R, S, K, E, B, 264, Hp), gemm="scaled")
    L, logits = make()
    import balanced_token_dispatch_amd as m
    with pytest.raises(m.MoeError):
        L.route(logits[: S - 1])
    with pytest.raises(m.MoeError):
        m.moe_quant_rows(L.x_all[:, ::2], L.xq.q, L.xq.scale)
    with pytest.raises(m.MoeError):
        m.moe_quant_rows(L.x_all, L.zq.q, L.xq.scale)
    with pytest.raises(m.MoeError):
        m.moe_group_gemm_scaled(m.GEMM_WGRAD, L.xq.q, L.xq.scale, L.q_up.qt, L.q_up.qt_scale, L.cu, L.z, H, Hp)


def test_refuses_weights_not_quantised():
    from balanced_token_dispatch_amd.layer import LayerStep, Shape
    L = LayerStep(Shape(R, S, K, E, B, H, Hp), rank=RANK, gemm="scaled")
    with pytest.raises(ValueError, match="quantise_weights"):
        L.forward()
    with pytest.raises(ValueError, match="8 bits"):
        LayerStep(Shape(R, S, K, E, B, H, Hp), rank=RANK).quantise_weights()
