"""Helpers of the tests of norm, dropout and balance loss: inputs, calls and bounds.

u = 2^-24 is half a step of fp32, the most that one operation loses of its result; a sum of n terms in some
order with at most D additions on any term's way loses at most D u of the sum of magnitudes."""
import numpy as np
import torch

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def rounding(dtype):
    """Half a step of the result's type, relative."""
    return 2.0 ** -8 if dtype == BF16 else U


def additions(width):
    """More than the additions on any term's way in a row's sum: at most 32 in a thread (or the eighth of a row wider
    than that over 1024 threads), and as many again over lanes and waves."""
    return 64 + width // 1024


def tensor(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype).cuda()


def exactly(t):
    return t.double().cpu().numpy()


def rng_of(seed, offset):
    wrap = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda")


def norm_bound(h, eh, y, mean, rstd, weight, eps, kind, dtype):
    """(bound of y, of mean, of rstd): h is off by eh already."""
    D = additions(h.shape[1])
    d = np.abs(h - mean[:, None])
    em = (D + 2) * U * np.abs(h).mean(1) + eh.mean(1) + U * np.abs(mean) if kind == "layer" else np.zeros(len(h))
    ed = eh + em[:, None] + (U * d if kind == "layer" else 0)
    var = (d * d).mean(1)
    evar = (2 * d * ed + ed * ed).mean(1) + (D + 3) * U * var
    whole = rstd ** -2.0  # var + eps
    rel = 0.55 * (evar / whole + 2 * U) + 3 * U  # of 1 / sqrt: half, and its second order while evar is under a tenth
    assert (evar < 0.1 * whole).all()
    ey = np.abs(weight) * rstd[:, None] * ed * (1 + rel[:, None]) + np.abs(weight) * d * rstd[:, None] * (rel[:, None] + 4 * U)
    ey = ey + U * np.abs(y)
    return ey + rounding(dtype) * (np.abs(y) + ey), em, rel * rstd


def norm_backward_bound(h, weight, mean, rstd, dy, dtotal, out, kind, dtype):
    """(bound of dh, of dweight, of dbias)."""
    D = additions(h.shape[1])
    xh = np.abs(h - (mean[:, None] if kind == "layer" else 0.0)) * rstd[:, None]
    g = np.abs(dy * weight)
    e1 = (D + 2) * U * g.mean(1, keepdims=True) if kind == "layer" else 0.0
    s1 = g.mean(1, keepdims=True) if kind == "layer" else 0.0
    e2 = (D + 6) * U * (g * xh).mean(1, keepdims=True)
    s2 = (g * xh).mean(1, keepdims=True)
    e = rstd[:, None] * (e1 + xh * e2 + 6 * U * (g + s1 + xh * s2))
    if dtotal is not None:
        e = e + U * np.abs(out)
    rows = len(h)
    sums = min(rows, 64 + rows // 64) + 8  # additions: rows of a part, then parts
    return e + rounding(dtype) * (np.abs(out) + e), sums * U * (np.abs(dy) * xh).sum(0), sums * U * np.abs(dy).sum(0)


def balance_bound(x, spread_of):
    """Relative error of a token's probabilities: the exponent's argument is rounded once (2^-24 of the spread of the
    logits, or of their size for the logistic), exp and the divisions lose at most two steps (2^-23) each, the sum one
    rounding a term."""
    x = x[np.isfinite(x)]
    spread = max(float(np.ptp(x)), float(np.abs(x).max())) if x.size else 0.0
    return (spread + spread_of + 16) * 2.0 ** -23
