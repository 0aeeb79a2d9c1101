"""Expert counts, balance loss, z loss and their gradient on the GPU against float64."""
import numpy as np
import pytest
import torch

from block_common import BF16, F32, U, balance_bound, exactly, rounding, tensor
from oracle import block_ref as ref

pytestmark = pytest.mark.gpu
# tokens, experts, K, bounds of the sequences (None: one)
CASES = [(1, 1, 1, None), (1, 64, 6, None), (5, 7, 3, [0, 5]), (33, 64, 6, [0, 0, 33]), (40, 65, 8, [3, 10, 10, 11, 38]),
         (130, 256, 8, None), (131, 257, 8, [0, 16, 32, 131]), (70, 384, 8, [1, 2, 3, 4, 70]), (50, 1000, 16, [0, 49, 50]),
         (20, 1024, 16, None), (0, 64, 2, [0, 0, 0]), (300, 128, 2, list(range(0, 301, 3))),
         # the borders of the calls that one workgroup does by itself
         (192, 9, 3, None), (193, 9, 3, None), (48, 600, 4, [0, 7, 48]), (49, 600, 4, [0, 7, 49]),
         (90, 20, 2, sorted(i % 91 for i in range(0, 91 * 7, 7))[:64] + [90]),
         (90, 20, 2, sorted(i % 91 for i in range(0, 91 * 7, 7))[:65] + [90])]


@pytest.fixture(scope="module")
def m():
    import balanced_token_dispatch_amd as m
    return m


def inputs(seed, T, E, K, dtype, bad_ids=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, E)) * 2 - 0.3 * np.log1p(np.arange(E))
    idx = np.argsort(-x, 1, kind="stable")[:, :K].astype(np.int32) if T else np.zeros((0, K), np.int32)
    if bad_ids and T > 3:
        idx[2, 0], idx[3, 0] = -1, E
    return tensor(x, dtype), torch.from_numpy(np.ascontiguousarray(idx)).cuda()


def on_gpu(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def counts_of(m, idx, E, cu):
    n = 1 if cu is None else len(cu) - 1
    out = torch.full((n, E), -5, dtype=torch.int32, device="cuda")
    m.moe_expert_counts(idx, out, cu_tokens=on_gpu(cu))
    return out


def losses(m, x, counts, cu, score, z=True):
    n = counts.shape[0]
    b, zl = torch.full((n,), -9.0, device="cuda"), torch.full((n,), -9.0, device="cuda")
    ws = torch.full((m.balance_loss_workspace_bytes(x.shape[0], n),), 0xFF, dtype=torch.uint8, device="cuda")
    m.moe_balance_loss(x, counts, b, ws, zloss=zl if z else None, score=score, cu_tokens=on_gpu(cu))
    return b, zl


def bounds(cu, T):
    return np.array([0, T] if cu is None else cu)


@pytest.mark.parametrize("T,E,K,cu", CASES)
def test_counts(m, T, E, K, cu):
    _, idx = inputs(T + E, T, E, K, F32)
    assert np.array_equal(counts_of(m, idx, E, cu).cpu().numpy(), ref.expert_counts(idx.cpu().numpy(), E, bounds(cu, T)))


@pytest.mark.parametrize("T,E,K,n", [(9000, 256, 8, 1), (9000, 8, 2, 40), (70001, 384, 8, 5), (4097, 64, 6, 4000)])
def test_counts_of_many_tokens(m, T, E, K, n):
    r = np.random.default_rng(n)
    idx = r.integers(-1, E + 1, (T, K)).astype(np.int32)
    cu = np.concatenate([[0], np.sort(r.integers(0, T + 1, n - 1)), [T]]).astype(np.int32)
    which = np.repeat(np.arange(n), np.diff(cu))
    flat = (which[:, None] * E + idx)[(idx >= 0) & (idx < E)]
    want = np.bincount(flat, minlength=n * E).reshape(n, E)
    got = counts_of(m, torch.from_numpy(idx).cuda(), E, list(cu) if n > 1 else None)
    assert np.array_equal(got.cpu().numpy(), want)


def check_losses(x, counts, cu, score, b, z):
    T, E = x.shape
    xd, at = exactly(x), bounds(cu, T)
    wb, wz = ref.balance_loss(xd, exactly(counts), at, score)
    rel = balance_bound(xd, E) + 80 * U  # and the tokens' sum
    assert (np.abs(exactly(b) - wb) <= rel * wb).all()
    # a logarithm of a sum that is off by `rel`, an addition, the square
    for i in range(len(wz)):
        lse = np.array([ref.logsumexp(v) for v in xd[at[i]:at[i + 1]]])
        e = rel + 4 * U * (np.abs(lse) + np.abs(xd).max(initial=0.0))
        assert abs(exactly(z)[i] - wz[i]) <= (2 * np.abs(lse) * e + e * e).mean() + 80 * U * wz[i] if len(lse) else exactly(z)[i] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,K,cu", CASES)
def test_losses(m, T, E, K, cu, dtype, score):
    x, idx = inputs(T * E, T, E, K, dtype)
    counts = counts_of(m, idx, E, cu)
    b, z = losses(m, x, counts, cu, score)
    check_losses(x, counts, cu, score, b, z)
    assert torch.equal(losses(m, x, counts, cu, score, z=False)[0], b)
    if score == "softmax":
        again = losses(m, x, counts, cu, "softmax_topk")
        assert torch.equal(again[0], b) and torch.equal(again[1], z)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_losses_of_many_tokens(m, score):
    T, E = 20011, 32
    x, idx = inputs(1, T, E, 2, BF16)
    cu = [5, 9000, 9000, 9016, 20000]
    counts = counts_of(m, idx, E, cu)
    check_losses(x, counts, cu, score, *losses(m, x, counts, cu, score))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,cu", [(150001, 12, [0, 70000, 70001, 150000]), (20011, 1000, [3, 20011]), (40003, 300, None),
                                    (150000, 64, list(range(0, 150001, 1000)))])
def test_chunks_of_many_tokens(m, T, E, cu, score):
    """Tokens enough for several of them a group of lanes: chunks inside a sequence and over its borders, against torch in
    float64."""
    x, idx = inputs(T, T, E, 2, F32)
    counts = counts_of(m, idx, E, cu)
    n, at = counts.shape[0], torch.from_numpy(bounds(cu, T)).cuda()
    b, z = losses(m, x, counts, cu, score)
    g = torch.Generator().manual_seed(1)
    db, dz = torch.rand(n, generator=g).cuda(), torch.rand(n, generator=g).cuda()
    got = gradient(m, x, counts, cu, db, dz, score).double()

    which = torch.searchsorted(at[1:], torch.arange(T, device="cuda"), right=True)
    inside = (torch.arange(T, device="cuda") >= at[0]) & (which < n)
    which = which.clamp(max=n - 1)
    xd, lens = x.double(), at.diff().clamp(min=1)
    logs = xd if score == "softmax" else torch.nn.functional.logsigmoid(xd)
    p, soft, lse = torch.softmax(logs, 1), torch.softmax(xd, 1), torch.logsumexp(xd, 1)
    c = counts.double()
    f = (E * c / c.sum(1, keepdim=True).clamp(min=1))[which]
    d = (f * p).sum(1)
    sums = torch.zeros(n, 2, dtype=torch.float64, device="cuda").index_add(0, which[inside], torch.stack([d, lse ** 2], 1)[inside])
    rel = balance_bound(exactly(x), E) + 80 * U
    wb, wz = (sums / lens[:, None]).unbind(1)
    assert ((b - wb).abs() <= rel * wb).all() and ((z - wz).abs() <= 3 * rel * (wz + wz.sqrt() + 1)).all()
    k = (1.0 / lens)[which][:, None]
    want = p * (f - d[:, None])
    if score == "sigmoid":
        want = want * torch.sigmoid(-xd)
    want = k * (db[which][:, None] * want + 2 * dz[which][:, None] * lse[:, None] * soft)
    e = k * (db[which][:, None] * p * 2 * rel * (f + d[:, None]) + 2 * dz[which][:, None] * soft * (
        2 * rel * (lse.abs()[:, None] + 1) + 4 * U * xd.abs().amax(1, keepdim=True))) + 2 * U * want.abs() + 1e-38
    assert ((got - want).abs() <= e)[inside].all() and (got[~inside] == 7.0).all()


def gradient(m, x, counts, cu, db, dz, score, add=None, out=None):
    out = torch.full_like(x, 7.0) if out is None else out
    m.moe_balance_loss_backward(x, counts, out, dbalance=db, dzloss=dz, score=score, cu_tokens=on_gpu(cu), add=add)
    return out


def check_gradient(x, counts, cu, db, dz, score, add, got, rows):
    T, E = x.shape
    xd, c, at = exactly(x), exactly(counts), bounds(cu, T)
    n = len(at) - 1
    b, z = (np.zeros(n) if t is None else exactly(t) for t in (db, dz))
    want = ref.balance_loss_backward(xd, c, at, b, z, score)
    e = np.zeros_like(want)
    rel = balance_bound(xd, E) + 16 * U
    for i in range(n):
        f = E * c[i] / max(c[i].sum(), 1)
        for t in range(at[i], at[i + 1]):
            p, s = ref.probabilities(xd[t], score), ref.probabilities(xd[t], "softmax")
            lse = abs(ref.logsumexp(xd[t]))
            k = 1.0 / (at[i + 1] - at[i])
            # P (f - D): P by rel, D = sum f P by rel of itself; then the z term
            e[t] = k * abs(b[i]) * p * (2 * rel * (f + (f * p).sum())) + 2 * k * abs(z[i]) * s * (
                2 * rel * (lse + 1) + 4 * U * np.abs(xd[t]).max())
    if add is not None:
        want = want + exactly(add)
        e = e + U * np.abs(want)
    e = e + rounding(x.dtype) * (np.abs(want) + e) + 1e-38
    assert (np.abs(exactly(got) - want) <= e)[rows].all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,K,cu", CASES)
def test_gradient(m, T, E, K, cu, dtype, score):
    x, idx = inputs(T + 3 * E, T, E, K, dtype)
    counts = counts_of(m, idx, E, cu)
    r = np.random.default_rng(T)
    db, dz = (tensor(r.standard_normal(counts.shape[0]), F32) for _ in range(2))
    add = tensor(r.standard_normal((T, E)) * 0.01, dtype)
    at = bounds(cu, T)
    inside = np.arange(at[0], at[-1])
    out = gradient(m, x, counts, cu, db, dz, score)
    check_gradient(x, counts, cu, db, dz, score, None, out, inside)
    outside = np.setdiff1d(np.arange(T), inside)
    assert (exactly(out)[outside] == 7.0).all()  # left as they were
    check_gradient(x, counts, cu, db, None, score, None, gradient(m, x, counts, cu, db, None, score), inside)
    check_gradient(x, counts, cu, None, dz, score, None, gradient(m, x, counts, cu, None, dz, score), inside)
    added = gradient(m, x, counts, cu, db, dz, score, add=add)
    check_gradient(x, counts, cu, db, dz, score, add, added, inside)
    in_place = gradient(m, x, counts, cu, db, dz, score, add=add, out=add)
    assert torch.equal(in_place[inside], added[inside])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(m, score):
    """The losses moved along a direction, worked out in fp32 by the loss kernels."""
    T, E = 24, 40
    x, idx = inputs(5, T, E, 4, F32)
    cu = [0, 9, 24]
    counts = counts_of(m, idx, E, cu)
    r = np.random.default_rng(1)
    db, dz = (tensor(r.standard_normal(2), F32) for _ in range(2))
    v = tensor(r.standard_normal((T, E)), F32)
    step = 2.0 ** -6

    def loss(x):
        b, z = losses(m, x, counts, cu, score)
        return float((b.double() * db.double()).sum() + (z.double() * dz.double()).sum())

    got = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
    want = float((gradient(m, x, counts, cu, db, dz, score).double() * v.double()).sum())
    size = float(losses(m, x, counts, cu, score)[0].abs().sum() + losses(m, x, counts, cu, score)[1].abs().sum()) * 3
    # step^2 / 6 of a third derivative (of order |v|^3 times the loss), and the losses' rounding over the step
    assert abs(got - want) <= step ** 2 / 6 * 30 * size + 100 * U * size / step


def test_masked_and_odd_logits(m):
    """-inf has no probability and no gradient; a token of -inf alone adds nothing; the type's lowest value is a number."""
    low = torch.finfo(F32).min
    for score in ("softmax", "sigmoid"):
        x = torch.randn(4, 12, device="cuda")
        x[0, 3:] = -float("inf")
        x[1] = -float("inf")
        x[2, :11] = low
        counts = torch.arange(12, dtype=torch.int32, device="cuda").view(1, 12)
        b, z = losses(m, x, counts, None, score)
        wb, wz = ref.balance_loss(exactly(x), exactly(counts), np.array([0, 4]), score)
        assert abs(b.item() - wb[0]) <= 64 * U * wb[0] and abs(z.item() - wz[0]) <= 64 * U * wz[0]
        db, dz = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
        g = gradient(m, x, counts, None, db, dz, score)
        assert torch.isfinite(g).all() and (g[1] == 0).all() and (g[0, 3:] == 0).all() and (g[2, :11] == 0).all()
        want = ref.balance_loss_backward(exactly(x), exactly(counts), np.array([0, 4]), np.ones(1), np.ones(1), score)
        assert (np.abs(exactly(g) - want) <= 64 * U * 12).all()
        x[3, 5] = float("nan")
        b, z = losses(m, x, counts, None, score)
        assert torch.isnan(b).all() and torch.isnan(z).all()
        again = gradient(m, x, counts, None, db, dz, score)
        assert torch.isnan(again[3]).all() and torch.equal(again[:3], g[:3])


def test_far_logistic(m):
    """Logits far below 0, where the logistic itself is 0 in fp32: the ratios hold."""
    x = torch.tensor([[-200.0, -201.0, -203.0], [90.0, -90.0, 300.0]], device="cuda")
    counts = torch.tensor([[5, 1, 2]], dtype=torch.int32, device="cuda")
    b, _ = losses(m, x, counts, None, "sigmoid")
    wb, _ = ref.balance_loss(exactly(x), exactly(counts), np.array([0, 2]), "sigmoid")
    assert abs(b.item() - wb[0]) <= (300 + 19) * 2.0 ** -23 * wb[0]
    db = torch.ones(1, device="cuda")
    check_gradient(x, counts, None, db, None, "sigmoid", None, gradient(m, x, counts, None, db, None, "sigmoid"), [0, 1])


def test_without_counts(m):
    """No copy counted: no balance loss and no gradient from it; the z loss stays."""
    x, _ = inputs(1, 8, 16, 2, F32)
    counts = torch.zeros(1, 16, dtype=torch.int32, device="cuda")
    b, z = losses(m, x, counts, None, "softmax")
    assert b.item() == 0 and z.item() > 0
    assert (gradient(m, x, counts, None, torch.ones(1, device="cuda"), None, "softmax") == 0).all()


def test_counts_of_many_ranks(m):
    """Counts added up over ranks, near 2^31 each: only their shares matter."""
    x, _ = inputs(1, 40, 16, 2, F32)
    small = torch.randint(1, 9, (1, 16), dtype=torch.int32, device="cuda")
    large = small * (1 << 27)
    a, b = losses(m, x, small, None, "softmax")[0], losses(m, x, large, None, "softmax")[0]
    assert abs(a.item() - b.item()) <= 40 * U * a.item()
    one = torch.ones(1, device="cuda")
    ga, gb = (gradient(m, x, c, None, one, None, "softmax") for c in (small, large))
    assert ((ga - gb).abs() <= 80 * U * 16 / 40).all()


def test_bounds_out_of_range(m):
    """Bounds that fall or leave the tokens: every access stays inside, the other outputs are untouched."""
    x, idx = inputs(2, 50, 32, 2, F32)
    guard = torch.full((3 * 32 + 64,), -5, dtype=torch.int32, device="cuda")
    for cu in ([-7, 10, 1000, 60], [40, 30, 20, 10], [60, 70, 80, 90], [-9, -8, -7, -6], [0, 60, 5, 50]):
        counts = guard[32:32 + 96].view(3, 32)
        m.moe_expert_counts(idx, counts, cu_tokens=on_gpu(cu))
        losses(m, x, counts, cu, "softmax")
        gradient(m, x, counts, cu, torch.ones(3, device="cuda"), None, "softmax")
        torch.cuda.synchronize()
        assert (guard[:32] == -5).all() and (guard[128:] == -5).all()


def test_same_bits_again_and_on_other_streams(m):
    x, idx = inputs(3, 5000, 256, 8, BF16)
    cu = [0, 100, 3000, 5000]
    counts = counts_of(m, idx, 256, cu)
    b, z = losses(m, x, counts, cu, "sigmoid")
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            c = counts_of(m, idx, 256, cu)
            got.append((c, *losses(m, x, c, cu, "sigmoid")))
    torch.cuda.synchronize()
    for c, v, w in got:
        assert torch.equal(c, counts) and torch.equal(v, b) and torch.equal(w, z)


def test_captured_and_replayed(m):
    x, idx = inputs(4, 3000, 64, 6, F32)
    cu, add = on_gpu([0, 1000, 3000]), torch.randn(3000, 64, device="cuda")
    ws = torch.empty(m.balance_loss_workspace_bytes(3000, 2), dtype=torch.uint8, device="cuda")
    one = torch.ones(2, device="cuda")

    def buffers():
        return dict(c=torch.empty(2, 64, dtype=torch.int32, device="cuda"), b=torch.empty(2, device="cuda"),
                    z=torch.empty(2, device="cuda"), g=torch.empty_like(x))

    def call(t):
        m.moe_expert_counts(idx, t["c"], cu_tokens=cu)
        m.moe_balance_loss(x, t["c"], t["b"], ws, zloss=t["z"], cu_tokens=cu)
        m.moe_balance_loss_backward(x, t["c"], t["g"], dbalance=one, dzloss=one, cu_tokens=cu, add=add)

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
    for rep in range(3):
        idx.copy_((idx + 1) % 64)
        x.mul_(0.9)
        cu[1] = 500 * (rep + 1)
        for t in held.values():
            t.view(torch.uint8).fill_(0x5A)
        g.replay()
        want = buffers()
        call(want)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(held[k], want[k]), (rep, k)


def test_refused(m):
    x, idx = inputs(1, 8, 16, 2, F32)
    c, f = torch.zeros(1, 16, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
    ws, g = torch.zeros(64, dtype=torch.uint8, device="cuda"), torch.zeros_like(x)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for call in (lambda: m.moe_expert_counts(idx.long(), c), lambda: m.moe_expert_counts(idx, c, cu_tokens=cu),
                 lambda: m.moe_expert_counts(idx.view(-1), c), lambda: m.moe_expert_counts(idx, c, cu_tokens=cu[:1]),
                 lambda: m.moe_expert_counts(idx, c, cu_tokens=cu.long()), lambda: m.moe_expert_counts(idx, idx),
                 lambda: m.moe_balance_loss(x, c, f, ws[:8]), lambda: m.moe_balance_loss(x, c[:, :15], f, ws),
                 lambda: m.moe_balance_loss(x, c, f, ws, score="max"), lambda: m.moe_balance_loss(x, c, f, ws, zloss=f),
                 lambda: m.moe_balance_loss(x.half(), c, f, ws), lambda: m.moe_balance_loss(x, c, f.double(), ws),
                 lambda: m.moe_balance_loss_backward(x, c, x), lambda: m.moe_balance_loss_backward(x, c, g[:7]),
                 lambda: m.moe_balance_loss_backward(x, c, g, add=g.bfloat16()),
                 lambda: m.moe_balance_loss_backward(x, c, g, dbalance=torch.zeros(2, device="cuda")),
                 lambda: m.moe_balance_loss_backward(x, c, g, cu_tokens=cu)):
        with pytest.raises(m.MoeError):
            call()
    m.moe_balance_loss_backward(x, c, g)
    assert (g == 0).all()
