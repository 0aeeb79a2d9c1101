"""8-bit block-scaled operands, the router and gradient clipping in float64 (numpy loops over
blocks, entries and tokens; small sizes)."""
import math

import numpy as np

# format: fraction bits, exponent bias, largest value
FORMATS = {"e4m3": (3, 7, 448.0), "e5m2": (2, 15, 57344.0)}


def decode(byte, fmt):
    """The value of one byte."""
    man, bias, _ = FORMATS[fmt]
    e, f = (byte & 127) >> man, byte & ((1 << man) - 1)
    v = math.ldexp(f, 1 - bias - man) if e == 0 else math.ldexp(f + (1 << man), e - bias - man)
    if fmt == "e4m3" and byte & 127 == 127:
        v = math.nan
    if fmt == "e5m2" and e == 31:
        v = math.nan if f else math.inf
    return -v if byte & 128 else v


def table(fmt):
    return np.array([decode(b, fmt) for b in range(256)])


def round_to(v, fmt):
    """float64 values (within the format's range, or not finite) to the nearest of the format's
    values, ties to even."""
    man, bias, _ = FORMATS[fmt]
    v = np.asarray(v, np.float64)
    ok = np.isfinite(v)
    ex = np.frexp(np.where(ok, v, 1.0))[1] - 1
    step = np.ldexp(1.0, np.maximum(ex, 1 - bias) - man)
    r = np.rint(np.where(ok, v, 0.0) / step) * step
    bad = np.where(np.isnan(v) | (fmt == "e4m3"), np.nan, v)  # e4m3 has no infinities
    return np.where(ok, r, bad)


def block_exponent(block, fmt):
    """Least e >= -127 with every finite |value| <= largest * 2^e; 0 for a block of zeros."""
    mag = np.abs(np.asarray(block, np.float64))
    top = float(np.max(np.where(np.isfinite(mag), mag, 0.0), initial=0.0))
    if top == 0.0:
        return 0
    e = -127
    while top > FORMATS[fmt][2] * 2.0 ** e:
        e += 1
    return e


def scale_row_bytes(n):
    return -(-n // 2048) * 16


def quant_rows(x, fmt, gather=None, div=1, row_scale=None):
    """(values of q before scaling, scale bytes, rows) of the fp32 rows x."""
    x = np.asarray(x, np.float32)
    if gather is None:
        v = x.copy()
        if row_scale is not None:
            v = v * np.asarray(row_scale, np.float32)[:len(v), None]
    else:
        v = np.zeros((len(gather), x.shape[1]), np.float32)
        for i, c in enumerate(gather):
            if c >= 0 and c // div < len(x):
                v[i] = x[c // div]
                if row_scale is not None:
                    v[i] = v[i] * np.float32(row_scale[c])
    q = np.zeros(v.shape)
    s = np.full((len(v), scale_row_bytes(v.shape[1])), 127, np.uint8)
    for i in range(len(v)):
        for b in range(-(-v.shape[1] // 128)):
            blk = v[i, b * 128:(b + 1) * 128].astype(np.float64)
            e = block_exponent(blk, fmt)
            s[i, b] = e + 127
            q[i, b * 128:(b + 1) * 128] = round_to(blk * 2.0 ** -e, fmt)
    return q, s, v


def quant_weight(w):
    """(q, q_scale, qt, qt_scale) of w [G, Kd, N], q as values before scaling."""
    w = np.asarray(w, np.float64)
    G, K, N = w.shape
    q = np.zeros(w.shape)
    qs = np.full((G, -(-K // 128), scale_row_bytes(N)), 127, np.uint8)
    ts = np.full((G, -(-N // 128), scale_row_bytes(K)), 127, np.uint8)
    for g in range(G):
        for k in range(0, K, 128):
            for n in range(0, N, 128):
                blk = w[g, k:k + 128, n:n + 128]
                e = block_exponent(blk, "e4m3")
                qs[g, k // 128, n // 128] = ts[g, n // 128, k // 128] = e + 127
                q[g, k:k + 128, n:n + 128] = round_to(blk * 2.0 ** -e, "e4m3")
    return q, qs, q.transpose(0, 2, 1), ts


def scaled(q, s):
    """q [.., rows, n] times its 1 x 128 scales [.., rows, bytes]."""
    kb = np.arange(q.shape[-1]) // 128
    return q * 2.0 ** (s.astype(np.float64) - 127)[..., kb]


def group_gemm_scaled(a, a_scale, b, b_scale, cu):
    """(out, sum of |products|, sum over groups of 8 along the contraction of the group's largest
    |product|) in float64: a [M, K] and b [G, C, K] as values before scaling; rows outside every
    segment are zero."""
    av = scaled(a, a_scale)
    out = np.zeros((len(a), b.shape[1]))
    mag, top = np.zeros_like(out), np.zeros_like(out)
    for g in range(len(cu) - 1):
        lo, hi = cu[g], cu[g + 1]
        if hi > lo:
            bv = scaled(b[g], np.repeat(b_scale[g], 128, axis=0)[:b.shape[1]])
            out[lo:hi] = av[lo:hi] @ bv.T
            aa, ab = np.abs(av[lo:hi]), np.abs(bv)
            mag[lo:hi] = aa @ ab.T
            for k in range(0, a.shape[1], 8):
                top[lo:hi] += (aa[:, None, k:k + 8] * ab[None, :, k:k + 8]).max(-1)
    return out, mag, top


def _logistic(x):
    return 1.0 / (1.0 + np.exp(-x))


def router_topk(logits, K, score, bias=None, factor=1.0):
    """(ids, weights) of each token; logits float64, ties to the lower id."""
    logits = np.asarray(logits, np.float64)
    ids, ws = [], []
    for x in logits:
        rank = x
        if bias is not None:
            if score == "sigmoid":
                rank = _logistic(x)
            elif score == "softmax":
                rank = router_weights(x, range(len(x)), "softmax")
            rank = rank + np.asarray(bias, np.float64)
        order = sorted(range(len(x)), key=lambda e: (-(np.inf if np.isnan(rank[e]) else rank[e]),
                                                     not np.isnan(rank[e]), e))[:K]
        ids.append(order)
        ws.append(factor * router_weights(x, order, score))
    return np.array(ids, np.int32), np.array(ws)


def router_weights(x, order, score):
    """Weights of the chosen entries of one token's logits."""
    c = x[list(order)]
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            # over exp(the largest, at most 0), which leaves the ratios: the logistic itself is 0 in
            # float64 below -745
            m = min(np.fmax.reduce(c, initial=-np.inf), 0.0)
            s = np.where(c == -np.inf, 0.0, np.exp(np.minimum(c, 0.0) - m) / (1.0 + np.exp(-np.abs(c))))
            total = s.sum()
        else:
            whole = c if score == "softmax_topk" else x
            m = whole.max()
            s = np.where(c == -np.inf, 0.0, np.exp(c - m))
            total = np.where(whole == -np.inf, 0.0, np.exp(whole - m)).sum()
    return np.zeros(len(c)) if total == 0 else s / total


def router_backward(logits, idx, dw, score, factor=1.0):
    """dlogits in float64; ids outside [0, E) take no part."""
    logits = np.asarray(logits, np.float64)
    out = np.zeros(logits.shape)
    for t, x in enumerate(logits):
        keep = [k for k, e in enumerate(idx[t]) if 0 <= e < len(x)]
        if not keep:
            continue
        order = [int(idx[t][k]) for k in keep]
        d = factor * np.asarray(dw[t], np.float64)[keep]
        w = router_weights(x, order, score)
        inner = float((d * w).sum())
        if score == "softmax":
            out[t] = -inner * router_weights(x, range(len(x)), "softmax")
        for e, wk, dk in zip(order, w, d):
            g = wk * dk if score == "softmax" else wk * (dk - inner)
            if score == "sigmoid":
                g *= 1.0 - _logistic(x[e])
            out[t, e] += g
    return out


def grad_clip(grads, max_norm):
    """(norm, factor) of a list of float64 arrays."""
    norm = math.sqrt(math.fsum(float((g * g).sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))
