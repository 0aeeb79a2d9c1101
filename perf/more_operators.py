"""What stands around the expert layer in a transformer block, as cases that can be timed and compared.

`run` computes one operator in its plain form (elementary torch operations), or, where `own` is
true, through the package's entry points:

  norm              y = (h - mean) rstd w + b per row, h = residual + dropout(x) (layer norm, or without the
                    mean: rms): moe_layer_norm
  norm_backward     the gradients of x, residual, w and b: moe_layer_norm_backward
  dropout           out = residual + dropout(x), the mask from a counter: moe_dropout
  balance           per-expert counts of each sequence, its balance loss and its z loss:
                    moe_expert_counts, moe_balance_loss
  balance_backward  the logits' gradient of both losses, added to the router's:
                    moe_balance_loss_backward

Dropout: element i (row-major) of a tensor takes 16 bits of Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
"Parallel random numbers: as easy as 1, 2, 3", 2011): counter (i // 8, offset), key seed, half i % 8 of its
four words, low halves first.  It is dropped where these are below t = floor(65536 p + 1/2), else scaled by
65536 / (65536 - t).

Balance loss of a sequence with counts c: E / sum(c) * mean over its tokens of sum_e c_e P_e, with P the
softmax of the token's logits (or their logistic over its sum).  z loss: the mean of logsumexp squared.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token entering the layer while serving: latency
        dict(name="norm_one_token", op="norm", rows=1, width=7168, kind="layer", dtype="bf16", weight="bf16",
             residual=True, p=0.0, stats=False),
        # the way into the layer in a training step: the branch before it dropped out and added
        dict(name="norm_train", op="norm", rows=4096, width=7168, kind="layer", dtype="bf16", weight="f32",
             residual=True, p=0.1, stats=True),
        # prefill of many sequences, without the mean
        dict(name="norm_prefill", op="norm", rows=32768, width=7168, kind="rms", dtype="bf16", weight="bf16",
             residual=True, p=0.0, stats=False),
        # rows that no vector load fits
        dict(name="norm_odd", op="norm", rows=5003, width=1001, kind="layer", dtype="f32", weight="f32",
             residual=False, p=0.0, stats=True),
        # the gradient at the longest step, with the residual's own gradient and the dropout undone
        dict(name="norm_grad", op="norm_backward", rows=8192, width=7168, kind="layer", dtype="bf16", weight="f32",
             residual=True, p=0.1),
        # a short micro-batch of a narrow model, odd in both directions
        dict(name="norm_grad_odd", op="norm_backward", rows=257, width=1409, kind="rms", dtype="f32", weight="f32",
             residual=False, p=0.0),
        # the hidden rows of one token's copies
        dict(name="dropout_few", op="dropout", rows=6, width=1408, dtype="bf16", residual=False, p=0.1),
        # the way out of the layer at the longest step
        dict(name="dropout_train", op="dropout", rows=8192, width=7168, dtype="bf16", residual=True, p=0.1),
        # the losses of a small micro-batch
        dict(name="balance_few", op="balance", tokens=64, experts=64, k=6, sequences=1, score="softmax", dtype="f32"),
        # a rank's tokens at the widest gate, losses by sequence
        dict(name="balance_train", op="balance", tokens=8192, experts=384, k=8, sequences=4, score="softmax", dtype="f32"),
        # its gradient for a few tokens
        dict(name="balance_grad_few", op="balance_backward", tokens=131, experts=64, k=6, sequences=3, score="softmax",
             dtype="f32", add=False),
        # a long step of short sequences, logistic scores, 16-bit logits, added to the router's gradient
        dict(name="balance_grad", op="balance_backward", tokens=32768, experts=256, k=8, sequences=61, score="sigmoid",
             dtype="bf16", add=True),
    ]


def _log(rng, lo, hi):
    """A size in [lo, hi], spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "dropout", "balance", "balance_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward", "dropout"):
        width = _log(rng, 16, 16384)
        if rng.random() < 0.6:  # most widths are whole vectors
            width = -(-width // 64) * 64
        most = 8192 * 7168 if op == "norm_backward" or dtype == "f32" else 32768 * 7168
        c = dict(op=op, rows=_log(rng, 1, min(32768, most // width)), width=width, dtype=dtype,
                 residual=rng.random() < 0.6, p=rng.choice([0.0, 0.0, 0.1, 0.3, 0.5]))
        if op == "dropout":
            c["p"] = rng.choice([0.05, 0.1, 0.3, 0.5])
            return c
        c = dict(c, kind=rng.choice(["layer", "rms"]), weight=rng.choice(["f32", dtype]))
        return dict(c, stats=rng.random() < 0.5) if op == "norm" else c
    e = _log(rng, 2, 1024)
    c = dict(op=op, tokens=_log(rng, 1, 65536), experts=e, k=rng.randint(1, min(e, 16)), sequences=_log(rng, 1, 128),
             score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["f32", "bf16"]))
    return c if op == "balance" else dict(c, add=rng.random() < 0.5)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)

    def hidden(rows, width, dtype):
        """Rows of a residual stream: a few columns far larger than the rest, a small mean."""
        v = normal(rows, width, dtype=dtype)
        size = torch.ones(width, device="cuda")
        size[torch.randint(0, width, (width // 500 + 1,), device="cuda", generator=gen)] = 16.0
        return v.mul_(size.to(dtype)).add_(0.1)

    if op in ("norm", "norm_backward", "dropout"):
        rows, width, dtype = case["rows"], case["width"], DTYPE[case["dtype"]]
        # the seed and the offset that a program's generator has reached
        st["rng"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=gen)
        if op != "norm_backward":
            st["x"] = normal(rows, width, dtype=dtype)
            st["residual"] = hidden(rows, width, dtype) if case["residual"] else None
        if op != "dropout":
            wt = DTYPE[case["weight"]]
            st["w"] = normal(width).mul_(0.1).add_(1.0).to(wt)
            st["b"] = normal(width).mul_(0.1).to(wt) if case["kind"] == "layer" else None
        if op == "norm_backward":  # what the forward pass left, and the gradients that arrive
            st["total"] = hidden(rows, width, dtype)
            h = st["total"].double()
            st["mean"] = h.mean(1).float() if case["kind"] == "layer" else None
            mean = h.mean(1, keepdim=True) if case["kind"] == "layer" else 0.0
            st["rstd"] = ((h - mean).square().mean(1) + EPS).rsqrt().float()
            st["dy"] = normal(rows, width, dtype=dtype).mul_(2.0 ** -10)
            st["dtotal"] = normal(rows, width, dtype=dtype).mul_(2.0 ** -10) if case["residual"] else None
    else:
        t, e, n = case["tokens"], case["experts"], case["sequences"]
        popular = -0.3 * torch.log1p(torch.randperm(e, device="cuda", generator=gen).float())
        st["logits"] = (normal(t, e) + popular).to(DTYPE[case["dtype"]])
        st["idx"] = torch.topk(st["logits"].float(), case["k"], dim=1)[1].int().contiguous()
        # packed sequences of uneven lengths, some of them empty where there are many
        cut = np.sort(np.random.default_rng([seed, 7]).integers(0, t + 1, n - 1))
        st["cu"] = torch.from_numpy(np.concatenate([[0], cut, [t]]).astype(np.int32)).cuda()
        st["lengths"] = st["cu"].long().diff()
        if op == "balance_backward":  # the weight of each loss, over the sequences
            st["dbalance"] = torch.rand(n, device="cuda", generator=gen).add_(0.5).mul_(0.01 / n)
            st["dz"] = torch.rand(n, device="cuda", generator=gen).add_(0.5).mul_(0.001 / n)
            which = torch.repeat_interleave(torch.arange(n, device="cuda"), st["lengths"])
            flat = (which[:, None] * e + st["idx"].long()).view(-1)
            st["counts"] = torch.bincount(flat, minlength=n * e).view(n, e).int()
            st["add"] = normal(t, e).mul_(1e-6).to(st["logits"].dtype) if case["add"] else None
    return st


# ---- plain forms ---------------------------------------------------------------------------

_LOW = 0xFFFFFFFF


def _philox(block, rng):
    """Eight 16-bit numbers for each of the counters `block` (int64): [.., 8]."""
    c0, c1 = block & _LOW, block >> 32
    k0, k1 = rng[0] & _LOW, (rng[0] >> 32) & _LOW
    c2, c3 = (rng[1] & _LOW).expand_as(c0), ((rng[1] >> 32) & _LOW).expand_as(c0)
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64: the low and high words are right
        c0, c1, c2, c3 = ((p1 >> 32) & _LOW) ^ c1 ^ k0, p1 & _LOW, ((p0 >> 32) & _LOW) ^ c3 ^ k1, p0 & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    w = torch.stack([c0, c1, c2, c3], -1)
    return torch.stack([w & 0xFFFF, w >> 16], -1).flatten(-2)


def _below(p):
    return int(math.floor(65536 * p + 0.5))


def _plain_drop(x, p, rng):
    """x (fp32) with a share p of it 0 and the rest scaled."""
    if p == 0.0:
        return x
    n, t = x.numel(), _below(p)
    u = _philox(torch.arange(-(-n // 8), device=x.device), rng).view(-1)[:n].view(x.shape)
    return torch.where(u >= t, x * (65536.0 / (65536 - t)), torch.zeros((), device=x.device))


def _plain_total(st):
    h = _plain_drop(st["x"].float(), st["p"], st["rng"])
    return h if st["residual"] is None else st["residual"].float() + h


def _plain_norm(st):
    h, dtype = _plain_total(st), DTYPE[st["dtype"]]
    mean = h.mean(1, keepdim=True) if st["kind"] == "layer" else torch.zeros((), device=h.device)
    c = h - mean
    rstd = 1.0 / torch.sqrt(c.square().mean(1, keepdim=True) + EPS)
    y = c * rstd * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    out = {"y": y.to(dtype)}
    if st["residual"] is not None or st["p"] > 0:
        out["total"] = h.to(dtype)
    if st["stats"]:
        out["rstd"] = rstd.view(-1)
        if st["kind"] == "layer":
            out["mean"] = mean.view(-1)
    return out


def _plain_norm_backward(st):
    dtype, rstd = DTYPE[st["dtype"]], st["rstd"][:, None]
    h, dy = st["total"].float(), st["dy"].float()
    xh = (h if st["mean"] is None else h - st["mean"][:, None]) * rstd
    g = dy * st["w"].float()
    d = g - xh * (g * xh).mean(1, keepdim=True)
    if st["mean"] is not None:
        d = d - g.mean(1, keepdim=True)
    d = d * rstd
    if st["dtotal"] is not None:
        d = d + st["dtotal"].float()
    out = {"dx": _plain_drop(d, st["p"], st["rng"]).to(dtype), "dw": (dy * xh).sum(0)}
    if st["p"] > 0:
        out["dresidual"] = d.to(dtype)
    if st["b"] is not None:
        out["db"] = dy.sum(0)
    return out


def _plain_dropout(st):
    return _plain_total(st).to(DTYPE[st["dtype"]])


def _sequence(st):
    """The sequence of each token."""
    return torch.repeat_interleave(torch.arange(st["sequences"], device="cuda"), st["lengths"], output_size=st["tokens"])


def _log_scores(x, score):
    """Logarithm of what P is proportional to."""
    return x if score == "softmax" else x.clamp(max=0.0) - torch.log1p(torch.exp(-x.abs()))


def _normalised(x):
    """exp(x) over its row's sum, and the logarithm of that sum."""
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - top)
    s = p.sum(1, keepdim=True)
    return p / s, top + torch.log(s)


def _plain_balance(st):
    x, n, e = st["logits"].float(), st["sequences"], st["experts"]
    which = _sequence(st)
    counts = torch.zeros(n * e, dtype=torch.int32, device=x.device)
    flat = (which[:, None] * e + st["idx"].long()).view(-1)
    counts = counts.index_add(0, flat, torch.ones_like(flat, dtype=torch.int32)).view(n, e)
    p, _ = _normalised(_log_scores(x, st["score"]))
    lse = _normalised(x)[1]
    f = counts.float() * (e / counts.sum(1, keepdim=True).clamp(min=1).float())
    rows = torch.stack([(f[which] * p).sum(1), lse.view(-1).square()], 1)
    # one long sum a sequence: in 64 bits
    sums = torch.zeros(n, 2, dtype=torch.float64, device=x.device).index_add(0, which, rows.double())
    means = (sums / st["lengths"].clamp(min=1)[:, None]).float()
    return {"counts": counts, "balance": means[:, 0].contiguous(), "z": means[:, 1].contiguous()}


def _plain_balance_backward(st):
    x, counts = st["logits"].float(), st["counts"]
    which = _sequence(st)
    p, _ = _normalised(_log_scores(x, st["score"]))
    soft, lse = _normalised(x)
    f = (counts.float() * (st["experts"] / counts.sum(1, keepdim=True).clamp(min=1).float()))[which]
    n = st["lengths"].clamp(min=1).float()
    d = (st["dbalance"] / n)[which][:, None] * p * (f - (f * p).sum(1, keepdim=True))
    if st["score"] == "sigmoid":
        d = d / (1.0 + torch.exp(x))
    d = d + (2.0 * st["dz"] / n)[which][:, None] * lse * soft
    if st["add"] is not None:
        d = st["add"].float() + d
    return d.to(st["logits"].dtype)


# ---- the package's own -----------------------------------------------------------------------

def _own(st):
    import balanced_token_dispatch_amd as m

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    op = st["op"]
    if op == "dropout":
        out = torch.empty_like(st["x"])
        m.moe_dropout(st["x"], out, st["p"], st["rng"], residual=st["residual"])
        return out
    if op == "norm":
        x, rows = st["x"], st["rows"]
        out = {"y": torch.empty_like(x)}
        if st["residual"] is not None or st["p"] > 0:
            out["total"] = torch.empty_like(x)
        if st["stats"]:
            out["rstd"] = empty(rows, dtype=torch.float32)
            if st["kind"] == "layer":
                out["mean"] = empty(rows, dtype=torch.float32)
        m.moe_layer_norm(x, st["w"], out["y"], bias=st["b"], eps=EPS, kind=st["kind"], residual=st["residual"],
                         total=out.get("total"), mean=out.get("mean"), rstd=out.get("rstd"), p=st["p"], rng=st["rng"])
        return out
    if op == "norm_backward":
        width = st["width"]
        out = {"dx": torch.empty_like(st["dy"]), "dw": empty(width, dtype=torch.float32)}
        if st["p"] > 0:
            out["dresidual"] = torch.empty_like(st["dy"])
        if st["b"] is not None:
            out["db"] = empty(width, dtype=torch.float32)
        ws = empty(m.layer_norm_backward_workspace_bytes(st["rows"], width), dtype=torch.uint8)
        m.moe_layer_norm_backward(st["total"], st["w"], st["rstd"], st["dy"], out["dx"], out["dw"], ws,
                                  dbias=out.get("db"), mean=st["mean"], kind=st["kind"], dtotal=st["dtotal"],
                                  dresidual=out.get("dresidual"), p=st["p"], rng=st["rng"])
        return out
    n = st["sequences"]
    if op == "balance":
        out = {"counts": empty(n, st["experts"], dtype=torch.int32), "balance": empty(n, dtype=torch.float32),
               "z": empty(n, dtype=torch.float32)}
        ws = empty(m.balance_loss_workspace_bytes(st["tokens"], n), dtype=torch.uint8)
        m.moe_expert_counts(st["idx"], out["counts"], cu_tokens=st["cu"])
        m.moe_balance_loss(st["logits"], out["counts"], out["balance"], ws, zloss=out["z"], score=st["score"],
                           cu_tokens=st["cu"])
        return out
    out = torch.empty_like(st["logits"])
    m.moe_balance_loss_backward(st["logits"], st["counts"], out, dbalance=st["dbalance"], dzloss=st["dz"],
                                score=st["score"], cu_tokens=st["cu"], add=st["add"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "dropout": _plain_dropout,
            "balance": _plain_balance, "balance_backward": _plain_balance_backward}[state["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}[case["dtype"]]
    if op in ("norm", "norm_backward", "dropout"):
        n, width = case["rows"] * case["width"], case["width"]
        res, drop = case["residual"], case["p"] > 0
        if op == "dropout":
            return {"bytes": n * size * (2 + res), "flops": 2.0 * n}
        params = width * {"f32": 4, "bf16": 2}[case["weight"]] * (2 if case["kind"] == "layer" else 1)
        if op == "norm":
            stats = 4 * case["rows"] * (2 if case["kind"] == "layer" else 1) if case["stats"] else 0
            return {"bytes": n * size * (2 + res + (res or drop)) + params + stats, "flops": 8.0 * n}
        rows = 4 * case["rows"] * (2 if case["kind"] == "layer" else 1)
        return {"bytes": n * size * (3 + res + drop) + params + 8 * width + rows, "flops": 14.0 * n}
    n, s = case["tokens"] * case["experts"], case["sequences"]
    if op == "balance":
        return {"bytes": n * size + case["tokens"] * case["k"] * 4 + s * (case["experts"] * 4 + 12), "flops": 8.0 * n}
    return {"bytes": n * size * (2 + case["add"]) + s * (case["experts"] * 4 + 12), "flops": 16.0 * n}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _product(a, b):
    """High and low 32 bits of the product of a (32-bit values) and the number b, by 16-bit limbs."""
    a0, a1, b0, b1 = a % 65536, a // 65536, b % 65536, b // 65536
    low, mid = a0 * b0, a1 * b0
    mid = mid + low // 65536
    top = a0 * b1 + mid % 65536
    return a1 * b1 + mid // 65536 + top // 65536, top % 65536 * 65536 + low % 65536


def _exact_kept(n, p, rng):
    """Which of n elements are kept."""
    seed, offset = (int(v) for v in rng.tolist())
    mask = (1 << 32) - 1
    kept = torch.empty(n, dtype=torch.bool, device="cuda")
    step = 1 << 25
    for lo in range(0, n, step):
        i = torch.arange(lo, min(n, lo + step), device="cuda")[::8] // 8
        c = [i % (1 << 32), i // (1 << 32), torch.full_like(i, offset & mask), torch.full_like(i, offset >> 32)]
        for r in range(10):
            k0, k1 = ((seed & mask) + r * 0x9E3779B9) & mask, ((seed >> 32) + r * 0xBB67AE85) & mask
            h0, l0 = _product(c[0], 0xD2511F53)
            h1, l1 = _product(c[2], 0xCD9E8D57)
            c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        for j in range(8):
            at = kept[lo + j:min(n, lo + step):8]
            at.copy_((c[j // 2] // (65536 if j % 2 else 1) % 65536 >= _below(p))[:at.numel()])
    return kept


def _exact_drop(v, p, rng):
    if p == 0.0:
        return v
    kept = _exact_kept(v.numel(), p, rng).view(v.shape)
    return torch.where(kept, v / (1.0 - _below(p) / 65536), 0.0)


def _exact_scores(x, score):
    return torch.softmax(x if score == "softmax" else torch.nn.functional.logsigmoid(x), 1)


def _exact_losses(x, counts, lengths, score):
    """Balance and z loss of each sequence, from their definitions."""
    balance, z = [], []
    for rows, c in zip(torch.split(x, lengths.tolist()), counts.double()):
        f = c / c.sum().clamp(min=1) * x.shape[1]
        empty = rows.shape[0] == 0
        balance.append(x.sum() * 0 if empty else (_exact_scores(rows, score).mean(0) * f).sum())
        z.append(x.sum() * 0 if empty else torch.logsumexp(rows, 1).square().mean())
    return torch.stack(balance), torch.stack(z)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "dropout"):
        h = _exact_drop(st["x"].double(), case["p"], st["rng"])
        if st["residual"] is not None:
            h = h + st["residual"].double()
        if op == "dropout":
            return h
        out = {}
        var, mean = torch.var_mean(h, 1, correction=0)
        if case["kind"] == "rms":
            var, mean = h.pow(2).mean(1), torch.zeros_like(mean)
        out["y"] = (h - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * st["w"].double()
        if st["b"] is not None:
            out["y"] += st["b"].double()
        if st["residual"] is not None or case["p"] > 0:
            out["total"] = h
        if case["stats"]:
            out["rstd"] = (var + EPS).pow(-0.5)
            if case["kind"] == "layer":
                out["mean"] = mean
        return out
    if op == "norm_backward":  # the derivative of the definition, by automatic differentiation
        h = st["total"].double().requires_grad_(True)
        w = st["w"].double().requires_grad_(True)
        b = torch.zeros(case["width"], dtype=torch.float64, device="cuda", requires_grad=True)
        if case["kind"] == "layer":
            c = h - h.mean(1, keepdim=True)
        else:
            c = h
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * w + b
        dh, dw, db = torch.autograd.grad(y, (h, w, b), st["dy"].double())
        if st["dtotal"] is not None:
            dh = dh + st["dtotal"].double()
        out = {"dx": _exact_drop(dh, case["p"], st["rng"]), "dw": dw}
        if case["p"] > 0:
            out["dresidual"] = dh
        if st["b"] is not None:
            out["db"] = db
        return out
    x = st["logits"].double()
    if op == "balance":
        which = torch.searchsorted(st["cu"][1:].long(), torch.arange(case["tokens"], device="cuda"), right=True)
        flat = which[:, None] * case["experts"] + st["idx"].long()
        counts = torch.bincount(flat.view(-1), minlength=case["sequences"] * case["experts"])
        counts = counts.view(case["sequences"], case["experts"])
        balance, z = _exact_losses(x, counts, st["lengths"], case["score"])
        return {"counts": None, "balance": balance, "z": z}
    x.requires_grad_(True)
    balance, z = _exact_losses(x, st["counts"], st["lengths"], case["score"])
    d = torch.autograd.grad((balance * st["dbalance"].double()).sum() + (z * st["dz"].double()).sum(), x)[0]
    return d if st["add"] is None else d + st["add"].double()
