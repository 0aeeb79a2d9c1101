"""Norm, dropout and balance loss in float64 (numpy; small sizes)."""
import math

import numpy as np


def philox(block, seed, offset):
    """The four 32-bit words of Philox4x32-10 for counters (block, offset): [.., 4] uint64.  Constants of
    Salmon, Moraes, Dror and Shaw, 2011."""
    u = np.uint64
    low, s32 = u(0xFFFFFFFF), u(32)
    block = np.asarray(block, np.uint64)
    off, key = u(offset % 2 ** 64), u(seed % 2 ** 64)
    c = [block & low, block >> s32, np.full_like(block, off & low), np.full_like(block, off >> s32)]
    k = [int(key & low), int(key >> s32)]
    for _ in range(10):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> s32) ^ c[1] ^ u(k[0]), q & low, (p >> s32) ^ c[3] ^ u(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, -1)


def below(p):
    return int(math.floor(65536 * p + 0.5))


def kept(n, p, seed, offset, first=0):
    """Which of the n elements from `first` on are kept."""
    i = np.arange(first, first + n, dtype=np.uint64)
    lo, hi = first // 8, -(-(first + n) // 8)
    words = philox(np.arange(lo, hi, dtype=np.uint64), seed, offset)
    halves = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], -1).reshape(-1)
    return halves[(i - np.uint64(8 * lo)).astype(np.int64)] >= below(p)


def drop(x, p, seed, offset):
    """x with a share p of it 0 and the rest scaled."""
    x = np.asarray(x, np.float64)
    if below(p) == 0:
        return x.copy()
    scale = 65536.0 / (65536 - below(p)) if below(p) < 65536 else 0.0
    return np.where(kept(x.size, p, seed, offset).reshape(x.shape), x * scale, 0.0)


def layer_norm(h, weight, bias, eps, kind):
    """(y, mean, rstd) of the rows h."""
    mean = h.mean(1) if kind == "layer" else np.zeros(len(h))
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(h, weight, mean, rstd, dy, kind):
    """(dh, dweight, dbias); mean and rstd as the forward left them."""
    xh = (h - (mean[:, None] if kind == "layer" else 0.0)) * rstd[:, None]
    g = dy * weight
    dh = g - xh * (g * xh).mean(1, keepdims=True)
    if kind == "layer":
        dh = dh - g.mean(1, keepdims=True)
    return dh * rstd[:, None], (dy * xh).sum(0), dy.sum(0)


def expert_counts(idx, E, cu):
    counts = np.zeros((len(cu) - 1, E), np.int64)
    for b in range(len(cu) - 1):
        for e in idx[cu[b]:cu[b + 1]].reshape(-1):
            if 0 <= e < E:
                counts[b, e] += 1
    return counts


def probabilities(x, score):
    """P of one token's logits: their softmax, or their logistic over its sum; 0 where all are -inf."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        logs = x if score != "sigmoid" else np.minimum(x, 0.0) - np.log1p(np.exp(-np.abs(x)))
        m = logs.max()
        p = np.where(logs == -np.inf, 0.0, np.exp(logs - m))
    return p / p.sum() if m > -np.inf or np.isnan(m) else np.zeros(len(x))


def logsumexp(x):
    """0 where all are -inf."""
    m = x.max()
    return 0.0 if m == -np.inf else m + math.log(np.exp(x - m).sum())


def balance_loss(logits, counts, cu, score):
    """(balance, z) of each sequence."""
    E = logits.shape[1]
    balance, z = np.zeros(len(cu) - 1), np.zeros(len(cu) - 1)
    for b in range(len(cu) - 1):
        rows = logits[cu[b]:cu[b + 1]]
        if len(rows) == 0:
            continue
        c = counts[b].astype(np.float64)
        if c.sum():
            balance[b] = E / c.sum() * np.mean([float((c * probabilities(x, score)).sum()) for x in rows])
        z[b] = np.mean([logsumexp(x) ** 2 for x in rows])
    return balance, z


def balance_loss_backward(logits, counts, cu, dbalance, dz, score):
    """The gradient of sum dbalance balance + dz z in the logits; 0 in rows of no sequence."""
    E = logits.shape[1]
    out = np.zeros(logits.shape)
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        c = counts[b].astype(np.float64)
        f = E * c / c.sum() if c.sum() else 0.0 * c
        for t in range(cu[b], cu[b + 1]):
            x = logits[t]
            p = probabilities(x, score)
            g = p * (f - (f * p).sum())
            if score == "sigmoid":
                with np.errstate(over="ignore"):
                    g = g / (1.0 + np.exp(x))
            out[t] = dbalance[b] / n * g + 2.0 * dz[b] / n * logsumexp(x) * probabilities(x, "softmax")
    return out
