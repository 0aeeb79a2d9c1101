"""A transformer block around the layer, run as a training step runs it: into the layer through the norm, the gate with its
losses, the layer, out through the dropout, and all of it back; every stage against float64 from what the stage before it
wrote, and the whole in a graph."""
import numpy as np
import pytest
import torch

import synth
from block_common import BF16, F32, U, balance_bound, exactly, norm_backward_bound, norm_bound, rng_of, rounding
from oracle import block_ref, scaled_ref

pytestmark = pytest.mark.gpu

R, S, K, E, B, H, Hp, RANK = 4, 96, 2, 16, 2, 272, 144, 1
CU = [0, 40, 40, 90]  # three sequences, one empty, and tokens behind the last
P_IN, P_OUT = 0.25, 0.125
SEED = 77


class Block:
    def __init__(self, norm, score, **kw):
        from balanced_token_dispatch_amd.layer import LayerStep, Shape
        self.norm, self.score = norm, score
        self.L = L = LayerStep(Shape(R, S, K, E, B, H, Hp), rank=RANK, norm=norm, sequences=len(CU) - 1, **kw)
        idx, w = synth.routing(synth.Dims(R=R, S=S, K=K, E=E, B=B, H=H, Hp=Hp), 1.0, 31)
        for t, sd in ((L.x_all, 311), (L.y_all, 314), (L.dout_all, 315), (L.dxp_all, 316)):
            synth.fill_normal_(t, 1.0, sd)
        synth.fill_normal_(L.w_up, 0.1, 312)
        synth.fill_normal_(L.w_down, 0.1, 313)
        L.topk_idx.copy_(torch.from_numpy(idx))
        L.topk_w.copy_(torch.from_numpy(w))
        g = torch.Generator().manual_seed(5)
        rows = lambda scale=1.0: (torch.randn(S, H, generator=g) * scale).bfloat16().cuda()  # noqa: E731
        self.x, self.residual, self.dout = rows(), rows(2.0), rows()
        self.w = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
        self.b = (0.1 * torch.randn(H, generator=g)).cuda() if norm == "layer" else None
        self.gate = (torch.randn(H, E, generator=g) * 0.1).cuda()
        self.cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
        self.rng = rng_of(SEED, 1000)
        self.dbalance, self.dz = torch.rand(3, generator=g).cuda(), torch.rand(3, generator=g).cuda()
        f32 = dict(dtype=F32, device="cuda")
        self.o = dict(out=torch.empty_like(self.x), logits=torch.empty(S, E, **f32), balance=torch.empty(3, **f32),
                      z=torch.empty(3, **f32), dlogits=torch.empty(S, E, **f32), droute=torch.empty(S, E, **f32),
                      dy=torch.empty_like(self.x), dx=torch.empty_like(self.x), dresidual=torch.empty_like(self.x),
                      dw=torch.empty(H, **f32), db=torch.empty(H, **f32))

    def step(self):
        L, o, score = self.L, self.o, self.score
        L.dw_up.zero_()
        L.dw_down.zero_()
        L.enter(self.x, self.w, self.b, self.residual, p=P_IN, rng=self.rng, offset=0)
        torch.mm(L.tokens.float(), self.gate, out=o["logits"])
        L.route(o["logits"], score)
        L.count_experts(self.cu)
        L.balance_loss(o["logits"], o["balance"], o["z"], score, self.cu)
        if L.scaled:
            L.quantise_weights()
        L.forward()
        L.leave(o["out"], P_OUT, self.rng, offset=1)
        L.leave_backward(self.dout, P_OUT, self.rng, offset=1)
        L.backward()
        L.route_backward(o["logits"], o["dlogits"], score)
        o["droute"].copy_(o["dlogits"])
        L.balance_loss_backward(o["logits"], o["dlogits"], self.dbalance, self.dz, score, self.cu, add=o["dlogits"])
        o["dy"].copy_(L.dx.float() + o["dlogits"] @ self.gate.t())
        L.enter_backward(o["dy"], self.w, o["dx"], o["dw"], o["db"] if self.b is not None else None, dtotal=self.dout,
                         dresidual=o["dresidual"], p=P_IN, rng=self.rng, offset=0)


def near(got, want, bound):
    assert (np.abs(exactly(got) - want) <= bound).all()


@pytest.mark.parametrize("norm,score,gemm", [("layer", "softmax_topk", "bf16"), ("rms", "sigmoid", "scaled"), ("rms", "softmax", "bf16")])
def test_block_stage_by_stage(norm, score, gemm):
    k = Block(norm, score, gemm=gemm)
    k.step()
    torch.cuda.synchronize()
    L, o = k.L, k.o
    assert int(L.status.item()) == 0
    half = rounding(BF16)

    # in: total = residual + drop(x), normalised
    xs = block_ref.drop(exactly(k.x), P_IN, SEED, 1000)
    h = xs + exactly(k.residual)
    eh = U * (2 * np.abs(xs) + np.abs(h))
    near(L.total, h, eh + half * (np.abs(h) + eh))
    w, b = exactly(k.w), None if k.b is None else exactly(k.b)
    y, mean, rstd = block_ref.layer_norm(h, w, b, 1e-5, norm)
    by, bm, br = norm_bound(h, eh, y, mean, rstd, w, 1e-5, norm, BF16)
    near(L.tokens, y, by)
    near(L.norm_rstd, rstd, br)

    # the gate and its losses
    logits = exactly(o["logits"])
    ids, tw = scaled_ref.router_topk(logits, K, score)
    assert np.array_equal(L.topk_idx[RANK].cpu().numpy(), ids)
    counts = block_ref.expert_counts(ids, E, CU)
    assert np.array_equal(L.seq_counts.cpu().numpy(), counts)
    balance, z = block_ref.balance_loss(logits, counts, CU, score)
    rel = balance_bound(logits, E) + 80 * U
    near(o["balance"], balance, rel * balance)
    assert (np.abs(exactly(o["z"]) - z) <= 3 * rel * (z + np.sqrt(z) + 1)).all()

    # out: total + drop(the layer's output), and the layer's output gradient
    ys = block_ref.drop(exactly(L.out), P_OUT, SEED, 1001)
    want = exactly(L.total) + ys
    e = U * (2 * np.abs(ys) + np.abs(want))
    near(o["out"], want, e + half * (np.abs(want) + e))
    d = block_ref.drop(exactly(k.dout), P_OUT, SEED, 1001)
    near(L.dout_all[RANK * S:(RANK + 1) * S], d, (half + 3 * U) * np.abs(d))

    # the logits' gradient: the router's and the losses'; tokens behind the last sequence have the router's alone
    g = block_ref.balance_loss_backward(logits, counts, CU, exactly(k.dbalance), exactly(k.dz), score)
    want = exactly(o["droute"]) + g
    lens = np.maximum(np.diff(CU), 1)
    f = E * counts.max(1) / np.maximum(counts.sum(1), 1)
    most = np.zeros(S)
    for i in range(3):
        most[CU[i]:CU[i + 1]] = (2 * rel * 2 * f[i] * exactly(k.dbalance)[i] + 4 * rel * (np.sqrt(z[i]) * 3 + 3) * exactly(k.dz)[i]) / lens[i]
    near(o["dlogits"], want, most[:, None] + U * np.abs(want))
    assert torch.equal(o["dlogits"][CU[-1]:], o["droute"][CU[-1]:]) and (np.abs(g[:CU[-1]]).max(1) > 0).all()

    # back through the norm, from what the stages wrote
    hd = exactly(L.total)
    m_, r_ = exactly(L.norm_mean) if norm == "layer" else None, exactly(L.norm_rstd)
    dh, dw, db = block_ref.layer_norm_backward(hd, w, m_, r_, exactly(o["dy"]), norm)
    dh = dh + exactly(k.dout)
    bh, bw, bb = norm_backward_bound(hd, w, m_, r_, exactly(o["dy"]), exactly(k.dout), dh, norm, BF16)
    near(o["dresidual"], dh, bh)
    dx = block_ref.drop(dh, P_IN, SEED, 1000)
    near(o["dx"], dx, bh / (1 - P_IN) + 3 * U * np.abs(dx))
    near(o["dw"], dw, bw + U * np.abs(dw))
    if norm == "layer":
        near(o["db"], db, bb + U * np.abs(db))


@pytest.mark.parametrize("norm,score,overlap", [("layer", "softmax_topk", False), ("rms", "sigmoid", True)])
def test_block_in_a_graph(norm, score, overlap):
    """Every replay equals the eager step with the same seed and offset, bit for bit; a moved offset draws other masks."""
    k = Block(norm, score, overlap=overlap)

    def outputs():
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in dict(k.o, dtopk=k.L.dtopk_w, dw_up=k.L.dw_up, total=k.L.total, tokens=k.L.tokens).items()
                if n != "db" or k.b is not None}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        k.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k.step()
    seen = []
    for rep in range(3):
        k.rng[1] = 1000 + 10 * rep
        for t in k.o.values():
            t.view(torch.uint8).fill_(0x5A)
        g.replay()
        got = outputs()
        k.step()
        want = outputs()
        for n in want:
            assert torch.equal(got[n], want[n]), (rep, n)
        seen.append(got["out"])
    assert not torch.equal(seen[0], seen[1])


def test_without_dropout_the_stream_passes_through():
    """p = 0 and a layer whose output is 0: leave() gives back what came in, and its gradient is the one behind it."""
    k = Block("rms", "softmax_topk")
    L = k.L
    L.enter(k.x, k.w, residual=None)
    assert torch.equal(L.total, k.x)
    L.out.zero_()
    L.leave(k.o["out"])
    assert torch.equal(k.o["out"], k.x)
    L.leave_backward(k.dout)
    assert torch.equal(L.dout_all[RANK * S:(RANK + 1) * S], k.dout)
