"""The 8-bit expert path, the router and the gradient clipping as cases that can be timed and compared.

`run` computes one operator in its plain form (elementary torch operations), or, where `own` is
true, through the package's entry points:

  product          out[seg] = a[seg] @ b[g]^T per segment, both operands in 8 bits with a power-of-two
                   scale for each block of 128 (rows: 1 x 128, weights: 128 x 128), the contraction
                   contiguous in both: moe_group_gemm_scaled
  quantise_rows    token rows gathered, weighted and put into 8 bits: moe_quant_rows
  quantise_weights the experts' weights in 8 bits, in both layouts: moe_quant_weight
  router           top-K experts of each token and their weights: moe_router_topk
  router_backward  the logits' gradient from the weights': moe_router_backward
  clip             the global norm of many gradients, and the gradients scaled to it:
                   moe_grad_sumsq, moe_grad_clip

Scales are bytes: byte s stands for 2^(s - 127).  A row's scales fill 16 bytes for each 2048
columns begun; bytes past its last block hold 127.
"""
import math

import numpy as np
import torch

own = False

FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
# the largest value v = 0.875 * 2^TOP of each format
TOP = {"e4m3": 9, "e5m2": 16}


def listed():
    return [
        # one token's copies on the experts it chose: latency, the weights of a few experts
        dict(name="product_one_token", op="product", rows=6, groups=68, contraction=2048, columns=1408,
             skew=0.3, fmt="e4m3", grad=False),
        # a decode batch of 64 tokens with 8 experts each: every expert's weights are read for a few rows
        dict(name="product_decode_batch", op="product", rows=512, groups=264, contraction=7168, columns=2048,
             skew=0.3, fmt="e4m3", grad=False),
        # a small step with very uneven and empty segments
        dict(name="product_ragged", op="product", rows=5003, groups=18, contraction=1408, columns=2064,
             skew=1.5, fmt="e4m3", grad=False),
        # the up projection of a training or prefill step at the largest layer
        dict(name="product_up_large", op="product", rows=32768, groups=264, contraction=7168, columns=2048,
             skew=0.3, fmt="e4m3", grad=False),
        # the input gradient of the up projection at the middle layer, gradients in e5m2
        dict(name="product_grad", op="product", rows=24576, groups=68, contraction=1408, columns=2048,
             skew=0.3, fmt="e5m2", grad=True),
        # one token's hidden rows between the projections
        dict(name="quantise_few_rows", op="quantise_rows", rows=6, source=6, width=1408, div=1, dtype="bf16",
             fmt="e4m3", weighted=False, copy=False),
        # the dispatch of a training step: rows gathered in expert order, the 16-bit rows kept for the weights' gradient
        dict(name="quantise_dispatch", op="quantise_rows", rows=32768, source=16384, width=7168, div=8,
             dtype="bf16", fmt="e4m3", weighted=False, copy=True),
        # the weights of one projection after an optimizer step, for the forward and the input gradient
        dict(name="quantise_weights", op="quantise_weights", groups=68, rows=2048, columns=1408, dtype="bf16"),
        # the gate of one rank's tokens
        dict(name="router", op="router", tokens=4096, experts=256, k=8, score="softmax_topk", bias=False, dtype="f32"),
        # its gradient at the widest gate, 16-bit logits
        dict(name="router_grad", op="router_backward", tokens=8192, experts=384, k=8, score="sigmoid", dtype="bf16"),
        # the small parameters of a model: many short gradients of odd sizes and both types
        dict(name="clip_many", op="clip", tensors=61, elements=3000, dtype="mixed", limit=1.0),
        # the gradients of both projections of the middle layer
        dict(name="clip_experts", op="clip", tensors=2, elements=68 * 2048 * 1408, dtype="f32", limit=1.0),
    ]


def _log(rng, lo, hi, step=1):
    """A size in [lo, hi], spread over the logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["product"] * 4 + ["quantise_rows"] * 2 + ["quantise_weights", "router", "router_backward", "clip"])
    if op == "product":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 32768), groups=_log(rng, 1, 264), contraction=_log(rng, 128, 7168, 16),
                     columns=_log(rng, 128, 7168, 16), skew=rng.choice([0.0, 0.3, 0.8, 1.5]),
                     fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), grad=rng.random() < 0.4)
            mat = c["contraction"] * c["columns"]
            if c["rows"] * mat <= 32768 * 7168 * 2048 and c["groups"] * mat <= 264 * 7168 * 2048:
                return c
    if op == "quantise_rows":
        div = rng.choice([1, 2, 6, 8])
        return dict(op=op, rows=_log(rng, 1, 32768), source=_log(rng, 1, 16384), width=_log(rng, 128, 7168, 16),
                    div=div, dtype=rng.choice(["bf16", "bf16", "f32"]), fmt=rng.choice(["e4m3", "e5m2"]),
                    weighted=rng.random() < 0.5, copy=rng.random() < 0.5)
    if op == "quantise_weights":
        return dict(op=op, groups=_log(rng, 1, 68), rows=_log(rng, 128, 4096, 16), columns=_log(rng, 128, 4096, 16),
                    dtype=rng.choice(["bf16", "f32"]))
    if op in ("router", "router_backward"):
        e = _log(rng, 2, 1024)
        c = dict(op=op, tokens=_log(rng, 1, 65536), experts=e, k=rng.randint(1, min(e, 16)),
                 score=rng.choice(["softmax_topk", "softmax", "sigmoid"]), dtype=rng.choice(["f32", "bf16"]))
        return dict(c, bias=rng.random() < 0.3) if op == "router" else c
    n = _log(rng, 1, 60)
    return dict(op=op, tensors=n, elements=_log(rng, 1, 200000000 // n), dtype=rng.choice(["f32", "bf16", "mixed"]),
                limit=rng.choice([1.0, 1e9]))


def _pitch(n):
    return -(-n // 2048) * 16


def _lengths(case, seed):
    """Rows of each segment: popularity falls by rank, ranks fall on random experts."""
    r = np.random.default_rng([seed, 7])
    p = (1.0 + np.arange(case["groups"])) ** -case["skew"]
    return r.multinomial(case["rows"], r.permutation(p / p.sum()))


def _eight_bits(shape, fmt, gen):
    """What normal rows look like in 8 bits: the largest of a block near the format's largest value."""
    v = torch.randn(shape, dtype=torch.bfloat16, device="cuda", generator=gen)
    top = 0.875 * 2.0 ** TOP[fmt]
    return v.mul_(0.25 * top).clamp_(-top, top).to(FMT[fmt])


def _scale_bytes(rows, n, around, gen):
    """[rows, pitch] scale bytes of n columns, within a factor of two of 2^around."""
    s = torch.randint(around + 126, around + 129, (rows, _pitch(n)), device="cuda", generator=gen, dtype=torch.uint8)
    s[:, -(-n // 128):] = 127
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, dtype=dtype, device="cuda", generator=gen)

    if op == "product":
        lens = _lengths(case, seed)
        cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        m, g, k, n = case["rows"], case["groups"], case["contraction"], case["columns"]
        st["a"] = _eight_bits((m, k), case["fmt"], gen)
        st["a_scale"] = _scale_bytes(m, k, -TOP[case["fmt"]] + 2, gen)
        st["b"] = torch.empty((g, n, k), dtype=torch.float8_e4m3fn, device="cuda")
        for i in range(0, g, 32):
            st["b"][i:i + 32] = _eight_bits((min(32, g - i), n, k), "e4m3", gen)
        st["b_scale"] = _scale_bytes(g * -(-n // 128), k, -13, gen).view(g, -(-n // 128), _pitch(k))
        st["cu"] = torch.from_numpy(cu).cuda()
        st["segments"] = [(i, int(cu[i]), int(cu[i + 1])) for i in range(g) if cu[i + 1] > cu[i]]
    elif op == "quantise_rows":
        src, rows, div = case["source"], case["rows"], case["div"]
        st["x"] = normal(src, case["width"], dtype=DTYPE[case["dtype"]])
        st["gather"] = None
        if rows != src or div != 1:  # copy ids, a few rows with none
            st["gather"] = torch.randint(0, src * div, (rows,), device="cuda", generator=gen, dtype=torch.int32)
            st["gather"][::97] = -1
        st["row_scale"] = torch.rand(src * div, device="cuda", generator=gen) if case["weighted"] else None
    elif op == "quantise_weights":
        st["w"] = normal(case["groups"], case["rows"], case["columns"], dtype=DTYPE[case["dtype"]]).mul_(0.02)
    elif op == "router":
        st["logits"] = normal(case["tokens"], case["experts"]).to(DTYPE[case["dtype"]])
        st["bias_row"] = normal(case["experts"]).mul_(0.1) if case["bias"] else None
    elif op == "router_backward":
        t, e = case["tokens"], case["experts"]
        st["logits"] = normal(t, e).to(DTYPE[case["dtype"]])
        st["idx"] = torch.sort(st["logits"].float(), dim=1, descending=True, stable=True)[1][:, :case["k"]].int().contiguous()
        st["dw"] = normal(t, case["k"])
    else:
        r = np.random.default_rng([case["tensors"], case["elements"]])  # a model's shapes stay
        sizes = [max(1, int(case["elements"] * f)) for f in r.uniform(0.5, 1.0, case["tensors"])]
        kinds = {"f32": [torch.float32], "bf16": [torch.bfloat16], "mixed": [torch.float32, torch.bfloat16]}[case["dtype"]]
        st["grads"] = [normal(n, dtype=kinds[i % len(kinds)]) for i, n in enumerate(sizes)]
        st["outs"] = [torch.empty_like(g) for g in st["grads"]]  # what the optimizer reads
    return st


# ---- plain forms ---------------------------------------------------------------------------

def _values(s):
    """What scale bytes stand for, in fp32."""
    return s.view(torch.float8_e8m0fnu).float()


def _spread(s, n):
    """Block values of the last axis repeated over its n columns."""
    return s.repeat_interleave(128, dim=-1)[..., :n]


def _plain_product(st):
    k, n = st["contraction"], st["columns"]
    a = st["a"].float() * _spread(_values(st["a_scale"]), k)

    def weight(g):
        s = _spread(_values(st["b_scale"][g]), k).repeat_interleave(128, dim=0)[:n]
        return st["b"][g].float() * s

    return torch.cat([a[lo:hi] @ weight(g).t() for g, lo, hi in st["segments"]]).bfloat16()


def _block_exponent(top, fmt):
    """The least e with top <= (largest value of the format) * 2^e; 0 for a block of zeros."""
    m, ex = torch.frexp(top)
    e = (ex - TOP[fmt] + (m > 0.875).to(ex.dtype)).clamp(-127, 127)
    return torch.where(top > 0, e, torch.zeros_like(e))


def _scale_rows(e, n):
    """Exponents [.., blocks] as scale bytes [.., pitch]."""
    s = torch.full(e.shape[:-1] + (_pitch(n),), 127, dtype=torch.uint8, device=e.device)
    s[..., :e.shape[-1]] = (e + 127).to(torch.uint8)
    return s


def _plain_quantise_rows(st):
    fmt, width = st["fmt"], st["width"]
    v = st["x"].float()
    if st["gather"] is not None:
        src = st["gather"].long()
        v = torch.where((src >= 0)[:, None], v[src.clamp(min=0) // st["div"]], torch.zeros((), device=v.device))
        if st["row_scale"] is not None:
            v = v * st["row_scale"][src.clamp(min=0)][:, None]
    elif st["row_scale"] is not None:
        v = v * st["row_scale"][:, None]
    blocks = torch.nn.functional.pad(v, (0, -width % 128)).view(v.shape[0], -1, 128)
    e = _block_exponent(blocks.abs().amax(-1), fmt)
    q = (v * _spread(_values((127 - e).to(torch.uint8)), width)).to(FMT[fmt])
    out = {"q": q, "scale": _scale_rows(e, width)}
    if st["copy"]:
        out["copy"] = v.to(st["x"].dtype)
    return out


def _plain_quantise_weights(st):
    w = st["w"].float()
    g, k, n = w.shape
    pad = torch.nn.functional.pad(w.abs(), (0, -n % 128, 0, -k % 128))
    e = _block_exponent(pad.view(g, -(-k // 128), 128, -(-n // 128), 128).amax((2, 4)), "e4m3")
    s = _spread(_values((127 - e).to(torch.uint8)), n).repeat_interleave(128, dim=1)[:, :k]
    q = (w * s).to(torch.float8_e4m3fn)
    qt = q.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
    return {"q": q, "q_scale": _scale_rows(e, n), "qt": qt, "qt_scale": _scale_rows(e.transpose(1, 2), k)}


def _scores(chosen, logits, score):
    """The router weights of the chosen logits."""
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-chosen))
        return s / s.sum(-1, keepdim=True)
    whole = chosen if score == "softmax_topk" else logits
    top = whole.amax(-1, keepdim=True)
    p, whole = torch.exp(chosen - top), torch.exp(whole - top)
    return p / whole.sum(-1, keepdim=True)


def _plain_router(st):
    logits = st["logits"].float()
    rank = logits
    if st["bias_row"] is not None:  # selection next to a border: in 64 bits
        rank = logits.double()
        if st["score"] == "sigmoid":
            rank = 1.0 / (1.0 + torch.exp(-rank))
        elif st["score"] == "softmax":
            rank = torch.exp(rank - rank.amax(-1, keepdim=True))
            rank = rank / rank.sum(-1, keepdim=True)
        rank = rank + st["bias_row"].double()
    idx = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :st["k"]]
    return {"idx": idx.int(), "w": _scores(logits.gather(1, idx), logits, st["score"])}


def _plain_router_backward(st):
    logits, dw = st["logits"].float(), st["dw"]
    idx = st["idx"].long()
    chosen = logits.gather(1, idx)
    w = _scores(chosen, logits, st["score"])
    inner = (dw * w).sum(-1, keepdim=True)
    if st["score"] == "softmax":
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - top)
        d = -inner * p / p.sum(-1, keepdim=True)
        d = d.scatter_add(1, idx, dw * w)
    else:
        g = w * (dw - inner)
        if st["score"] == "sigmoid":
            g = g / (1.0 + torch.exp(chosen))  # w (dw - inner) (1 - s)
        d = torch.zeros_like(logits).scatter_add(1, idx, g)
    return d.to(st["logits"].dtype)


def _plain_clip(st):
    sumsq = torch.stack([g.double().square().sum() for g in st["grads"]]).sum()
    norm = sumsq.sqrt()
    coef = (st["limit"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float(), "grads": [(g.float() * coef).to(g.dtype) for g in st["grads"]]}


# ---- the package's own -----------------------------------------------------------------------

def _own(st):
    import balanced_token_dispatch_amd as m

    def empty(*shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    op = st["op"]
    if op == "product":
        out = empty(st["rows"], st["columns"], dtype=torch.bfloat16)
        # the input gradient contracts the weights' columns: [Kd, N] rows of N, out Kd wide
        kind = m.GEMM_DGRAD if st["grad"] else m.GEMM_FWD
        kd, n = (st["columns"], st["contraction"]) if st["grad"] else (st["contraction"], st["columns"])
        m.moe_group_gemm_scaled(kind, st["a"], st["a_scale"], st["b"], st["b_scale"], st["cu"], out, kd, n)
        return out
    if op == "quantise_rows":
        rows, width = st["rows"] if st["gather"] is not None else st["source"], st["width"]
        out = {"q": empty(rows, width, dtype=FMT[st["fmt"]]), "scale": empty(rows, _pitch(width), dtype=torch.uint8)}
        if st["copy"]:
            out["copy"] = empty(rows, width, dtype=st["x"].dtype)
        m.moe_quant_rows(st["x"], out["q"], out["scale"], gather=st["gather"], gather_div=st["div"],
                         row_scale=st["row_scale"], copy=out.get("copy"))
        return out
    if op == "quantise_weights":
        g, k, n = st["w"].shape
        out = {"q": empty(g, k, n, dtype=torch.float8_e4m3fn),
               "q_scale": empty(g, -(-k // 128), _pitch(n), dtype=torch.uint8),
               "qt": empty(g, n, k, dtype=torch.float8_e4m3fn),
               "qt_scale": empty(g, -(-n // 128), _pitch(k), dtype=torch.uint8)}
        m.moe_quant_weight(st["w"], out["q"], out["q_scale"], out["qt"], out["qt_scale"])
        return out
    if op == "router":
        out = {"idx": empty(st["tokens"], st["k"], dtype=torch.int32), "w": empty(st["tokens"], st["k"], dtype=torch.float32)}
        m.moe_router_topk(st["logits"], out["idx"], out["w"], score=st["score"], bias=st["bias_row"])
        return out
    if op == "router_backward":
        out = torch.empty_like(st["logits"])
        m.moe_router_backward(st["logits"], st["idx"], st["dw"], out, score=st["score"])
        return out
    grads, outs = st["grads"], st["outs"]
    sumsq, norm = empty(1, dtype=torch.float64), empty(1, dtype=torch.float32)
    ws = empty(m.grad_sumsq_workspace_bytes(), dtype=torch.uint8)
    m.moe_grad_sumsq(grads, sumsq, ws)
    m.moe_grad_clip(grads, sumsq, st["limit"], norm, out=outs)
    return {"norm": norm[0], "grads": outs}


def run(state):
    if own:
        return _own(state)
    return {"product": _plain_product, "quantise_rows": _plain_quantise_rows,
            "quantise_weights": _plain_quantise_weights, "router": _plain_router,
            "router_backward": _plain_router_backward, "clip": _plain_clip}[state["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "mixed": 3}
    if op == "product":
        m, g, k, n = case["rows"], case["groups"], case["contraction"], case["columns"]
        p = (1.0 + np.arange(g)) ** -case["skew"]
        used = float((1.0 - (1.0 - p / p.sum()) ** m).sum())  # experts with a row
        return {"bytes": m * (k + k / 128) + used * (n * k + n * k / 16384) + m * n * 2,
                "flops": 2.0 * m * k * n}
    if op == "quantise_rows":
        rows, width, s = case["rows"], case["width"], size[case["dtype"]]
        read = rows if rows == case["source"] and case["div"] == 1 else case["source"] * -math.expm1(-rows / case["source"])
        return {"bytes": read * width * s + rows * width * (1 + 1 / 128 + (s if case["copy"] else 0)),
                "flops": 2.0 * rows * width}
    if op == "quantise_weights":
        n = case["groups"] * case["rows"] * case["columns"]
        return {"bytes": n * (size[case["dtype"]] + 2 + 2 / 16384), "flops": 2.0 * n}
    if op in ("router", "router_backward"):
        n, s = case["tokens"] * case["experts"], size[case["dtype"]]
        dense = op == "router" or case["score"] == "softmax"
        return {"bytes": (n * s if dense else 0) + (n * s if op != "router" else 0) + case["tokens"] * case["k"] * 8,
                "flops": 4.0 * n}
    n = 0.75 * case["tensors"] * case["elements"]
    return {"bytes": 3 * n * size[case["dtype"]], "flops": 3.0 * n}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _table(fmt):
    """The 256 values of an 8-bit format: sign, exponent, fraction."""
    man, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    vals = []
    for b in range(256):
        e, f = (b & 127) >> man, b & ((1 << man) - 1)
        v = math.ldexp(f, 1 - bias - man) if e == 0 else math.ldexp(f + (1 << man), e - bias - man)
        if fmt == "e4m3" and b & 127 == 127:
            v = math.nan
        if fmt == "e5m2" and e == 31:
            v = math.inf if f == 0 else math.nan
        vals.append(-v if b & 128 else v)
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _exact_round(v, fmt):
    """v (64 bits, within the format's range) to the nearest value of the format, ties to even."""
    man, low = (3, -6) if fmt == "e4m3" else (2, -14)
    ex = torch.frexp(v)[1] - 1
    step = _two(ex.clamp(min=low) - man)
    return torch.round(v / step) * step


def _exact_exponent(top, fmt):
    """ceil(log2(top / largest)), counted from exact comparisons with the powers of two."""
    powers = torch.tensor([0.875 * 2.0 ** (TOP[fmt] + e) for e in range(-127, 128)], dtype=torch.float64, device=top.device)
    e = torch.searchsorted(powers, top.contiguous()) - 127
    return torch.where(top > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _two(e):
    """2^e in 64 bits, exactly."""
    return torch.tensor([2.0 ** i for i in range(-300, 301)], dtype=torch.float64, device=e.device)[e.long() + 300]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "product":
        k, n = case["contraction"], case["columns"]
        ta, tb = _table(case["fmt"]), _table("e4m3")
        kb, nb = torch.arange(k, device="cuda") // 128, torch.arange(n, device="cuda") // 128
        out = torch.zeros((case["rows"], n), dtype=torch.float64, device="cuda")
        for g, lo, hi in st["segments"]:
            a = ta[st["a"][lo:hi].view(torch.uint8).int()] * _two(st["a_scale"][lo:hi].int() - 127)[:, kb]
            b = tb[st["b"][g].view(torch.uint8).int()] * _two(st["b_scale"][g].int() - 127)[nb][:, kb]
            out[lo:hi] = torch.mm(a, b.t().contiguous())
        return out
    if op == "quantise_rows":
        x = st["x"].double()
        rows = case["rows"] if st["gather"] is not None else case["source"]
        v = torch.zeros((rows, case["width"]), dtype=torch.float64, device="cuda")
        src = st["gather"].long() if st["gather"] is not None else torch.arange(rows, device="cuda")
        real = src >= 0
        v[real] = x[src[real] // case["div"]]
        if st["row_scale"] is not None:
            v[real] *= st["row_scale"].double()[src[real]][:, None]
        copy = v
        if st["row_scale"] is not None:  # the product is rounded to 32 bits before its block is scaled
            v = v.float().double()
        q = torch.empty_like(v)
        for c in range(0, case["width"], 128):
            e = _exact_exponent(v[:, c:c + 128].abs().amax(1), case["fmt"])
            q[:, c:c + 128] = _exact_round(v[:, c:c + 128] / _two(e)[:, None], case["fmt"])
        return {"q": q, "scale": None, **({"copy": copy} if case["copy"] else {})}
    if op == "quantise_weights":
        q = torch.empty(st["w"].shape, dtype=torch.float64, device="cuda")
        for k in range(0, q.shape[1], 128):
            for n in range(0, q.shape[2], 128):
                w = st["w"][:, k:k + 128, n:n + 128].double()
                e = _exact_exponent(w.abs().amax((1, 2)), "e4m3")
                q[:, k:k + 128, n:n + 128] = _exact_round(w / _two(e)[:, None, None], "e4m3")
        return {"q": q, "q_scale": None, "qt": q.transpose(1, 2).contiguous(), "qt_scale": None}
    if op == "router":
        x = st["logits"].double()
        rank = x
        if st["bias_row"] is not None:
            rank = {"sigmoid": torch.sigmoid, "softmax": lambda v: torch.softmax(v, 1), "softmax_topk": lambda v: v}[case["score"]](x)
            rank = rank + st["bias_row"].double()
        idx = torch.argsort(-rank, dim=1, stable=True)[:, :case["k"]]
        c = x.gather(1, idx)
        w = {"softmax_topk": lambda: torch.softmax(c, 1), "softmax": lambda: torch.softmax(x, 1).gather(1, idx),
             "sigmoid": lambda: torch.sigmoid(c) / torch.sigmoid(c).sum(1, keepdim=True)}[case["score"]]()
        return {"idx": None, "w": w}
    if op == "router_backward":  # the derivative of the definition, by automatic differentiation in 64 bits
        x = st["logits"].double().requires_grad_(True)
        c = x.gather(1, st["idx"].long())
        w = {"softmax_topk": lambda: torch.softmax(c, 1), "softmax": lambda: torch.softmax(x, 1).gather(1, st["idx"].long()),
             "sigmoid": lambda: torch.sigmoid(c) / torch.sigmoid(c).sum(1, keepdim=True)}[case["score"]]()
        return torch.autograd.grad((w * st["dw"].double()).sum(), x)[0]
    total = math.sqrt(math.fsum(float(torch.dot(g.double().view(-1), g.double().view(-1))) for g in st["grads"]))
    coef = min(1.0, case["limit"] / (total + 1e-6))
    return {"norm": torch.tensor(total, dtype=torch.float64, device="cuda"),
            "grads": [g.double() * coef for g in st["grads"]]}
