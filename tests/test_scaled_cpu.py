"""The definitions of the 8-bit path, the router and the clipping checked on the CPU, and what the
library and the binding refuse (no test here launches anything)."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import scaled_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "balanced_token_dispatch_amd", "libmoe.so")


@pytest.fixture(scope="module")
def mod():
    if not os.path.exists(LIB):
        pytest.skip("libmoe.so not built")
    import balanced_token_dispatch_amd as m
    return m


@pytest.mark.parametrize("fmt,t", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_formats(fmt, t):
    """Table and rounding against torch's types."""
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(t).float().numpy()
    got = ref.table(fmt).astype(np.float32)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    top = ref.FORMATS[fmt][2]
    v = np.random.default_rng(0).uniform(-top, top, 5000) * 2.0 ** -np.random.default_rng(1).integers(0, 24, 5000)
    v = v.astype(np.float32)
    assert np.array_equal(ref.round_to(v, fmt).astype(np.float32), torch.from_numpy(v).to(t).float().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantised_rows_are_close(fmt):
    """Each value is off by at most half a step of its binade, or of the smallest normal one."""
    x = np.random.default_rng(2).standard_normal((4, 300)).astype(np.float32)
    q, s, _ = ref.quant_rows(x, fmt)
    back = ref.scaled(q, s)
    man, bias, top = ref.FORMATS[fmt]
    unit = 2.0 ** (s.astype(float) - 127)[:, np.arange(300) // 128]
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -(man + 1), unit * 2.0 ** (-bias - man))).all()
    assert (np.abs(q).reshape(4, -1)[:, :128].max(1) > top / 2 * (1 - 2.0 ** -man)).all()


@pytest.mark.parametrize("score", ["softmax_topk", "softmax", "sigmoid"])
def test_router_gradient_by_differences(score):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 9))
    dw = rng.standard_normal((3, 4))
    idx, _ = ref.router_topk(x, 4, score)
    d = ref.router_backward(x, idx, dw, score, 1.7)
    h = 1e-5
    for t in range(3):
        for e in range(9):
            up, dn = x[t].copy(), x[t].copy()
            up[e] += h
            dn[e] -= h
            diff = 1.7 * (dw[t] * (ref.router_weights(up, idx[t], score) - ref.router_weights(dn, idx[t], score))).sum() / (2 * h)
            assert abs(diff - d[t, e]) <= 1e-8


def test_router_matches_torch():
    x = np.random.default_rng(6).standard_normal((5, 12))
    t = torch.from_numpy(x)
    v, i = t.topk(4, dim=1)
    for score, w in (("softmax_topk", torch.softmax(v, 1)), ("softmax", torch.softmax(t, 1).gather(1, i)),
                     ("sigmoid", torch.sigmoid(v) / torch.sigmoid(v).sum(1, keepdim=True))):
        idx, got = ref.router_topk(x, 4, score)
        assert np.array_equal(idx, i.numpy()) and np.allclose(got, w.numpy(), rtol=1e-12)


def test_clip_matches_torch():
    p = [torch.nn.Parameter(torch.zeros(7)), torch.nn.Parameter(torch.zeros(3, 5))]
    for i, q in enumerate(p):
        q.grad = torch.randn(q.shape, generator=torch.Generator().manual_seed(i))
    g = [q.grad.double().numpy().copy() for q in p]
    norm, coef = ref.grad_clip(g, 0.7)
    got = torch.nn.utils.clip_grad_norm_(p, 0.7)
    assert abs(got.item() - norm) <= 1e-6 * norm
    assert all(np.allclose(q.grad.numpy(), b * coef, rtol=1e-5) for q, b in zip(p, g))


def test_scale_row_bytes(mod):
    lib = mod.library()
    for n in (1, 16, 128, 2047, 2048, 2049, 4096, 7168, 1 << 22):
        assert lib.moe_scale_row_bytes(n) == mod.scale_row_bytes(n) == ref.scale_row_bytes(n)
    assert lib.moe_scale_row_bytes(0) == 0


P = ctypes.c_void_p(16)   # never dereferenced: every call below is refused before anything is launched
ODD, BYTE = ctypes.c_void_p(24), ctypes.c_void_p(17)


def refused(fn, ok, **kw):
    a = list(ok)
    for k, v in kw.items():
        a[int(k[1:])] = v
    return fn(*a)


def test_quant_rows_refuses(mod):
    fn, bad = mod.library().moe_quant_rows, mod.MOE_EINVAL
    ok = (mod.BF16, mod.E4M3, 8, 256, P, 8, None, 1, None, P, P, None, None)
    for kw in (dict(a0=2), dict(a1=2), dict(a2=-1), dict(a2=1 << 31), dict(a3=0), dict(a3=24), dict(a3=(1 << 22) + 16),
               dict(a4=None), dict(a4=ODD), dict(a5=0), dict(a5=1 << 31), dict(a5=7), dict(a7=0), dict(a9=None),
               dict(a9=ODD), dict(a10=None), dict(a10=ODD), dict(a11=ODD), dict(a6=BYTE),
               dict(a8=BYTE)):
        assert refused(fn, ok, **kw) == bad, kw
    assert refused(fn, ok, a2=0) == mod.MOE_OK
    assert refused(fn, ok, a2=0, a4=None, a5=0) == mod.MOE_OK   # a rank without tokens


def test_quant_weight_refuses(mod):
    fn, bad = mod.library().moe_quant_weight, mod.MOE_EINVAL
    ok = (mod.BF16, 2, 128, 256, P, P, P, P, P, None)
    for kw in (dict(a0=5), dict(a1=0), dict(a2=24), dict(a2=0), dict(a3=8), dict(a3=(1 << 22) + 16), dict(a4=None),
               dict(a4=ODD), dict(a5=None), dict(a6=None), dict(a7=None), dict(a8=None), dict(a5=ODD), dict(a8=ODD),
               dict(a5=None, a6=None, a7=None, a8=None)):
        assert refused(fn, ok, **kw) == bad, kw


def test_scaled_gemm_refuses(mod):
    fn, bad = mod.library().moe_group_gemm_scaled, mod.MOE_EINVAL
    ok = (mod.GEMM_FWD, mod.E4M3, 4, 64, 128, 256, P, P, P, P, P, P, None)
    for kw in (dict(a0=mod.GEMM_WGRAD), dict(a0=9), dict(a1=2), dict(a2=0), dict(a2=1089), dict(a3=-1), dict(a4=0),
               dict(a4=24), dict(a4=(1 << 21) + 16), dict(a5=8), dict(a5=(1 << 21) + 16), dict(a6=None), dict(a7=None),
               dict(a8=None), dict(a9=None), dict(a10=None), dict(a11=None), dict(a6=ODD), dict(a7=ODD), dict(a8=ODD),
               dict(a9=ODD), dict(a11=ODD), dict(a10=ctypes.c_void_p(18)), dict(a3=(1 << 31) - 1, a5=1 << 14)):
        assert refused(fn, ok, **kw) == bad, kw
    assert refused(fn, ok, a3=0) == mod.MOE_OK


def test_router_refuses(mod):
    lib, bad = mod.library(), mod.MOE_EINVAL
    ok = (mod.F32, 0, 4, 64, 8, P, None, 1.0, P, P, None)
    for kw in (dict(a0=2), dict(a1=3), dict(a1=-1), dict(a2=-1), dict(a2=1 << 31), dict(a3=0), dict(a3=1025), dict(a4=0),
               dict(a4=65), dict(a5=None), dict(a7=float("nan")), dict(a7=float("inf")), dict(a8=None), dict(a9=None),
               dict(a5=BYTE), dict(a6=BYTE), dict(a8=BYTE), dict(a9=BYTE)):
        assert refused(lib.moe_router_topk, ok, **kw) == bad, kw
    assert refused(lib.moe_router_topk, ok, a2=0) == mod.MOE_OK
    ok = (mod.F32, 0, 4, 64, 8, P, P, P, 1.0, ODD, None)
    for kw in (dict(a0=2), dict(a1=3), dict(a2=-1), dict(a3=1025), dict(a4=0), dict(a5=None), dict(a6=None), dict(a7=None),
               dict(a8=float("inf")), dict(a9=None), dict(a9=P), dict(a5=BYTE), dict(a6=BYTE), dict(a7=BYTE), dict(a9=BYTE)):
        assert refused(lib.moe_router_backward, ok, **kw) == bad, kw
    assert refused(lib.moe_router_backward, ok, a2=0) == mod.MOE_OK


def test_grads_refuse(mod):
    lib, bad = mod.library(), mod.MOE_EINVAL
    ptr = lambda *v: (ctypes.c_void_p * len(v))(*v)            # noqa: E731
    num = lambda *v: (ctypes.c_int64 * len(v))(*v)             # noqa: E731
    typ = lambda *v: (ctypes.c_int * len(v))(*v)               # noqa: E731
    need = mod.grad_sumsq_workspace_bytes()
    ok = (2, ptr(16, 32), num(5, 6), typ(0, 1), P, P, need, None)
    for kw in (dict(a0=-1), dict(a1=None), dict(a2=None), dict(a3=None), dict(a4=None), dict(a5=None),
               dict(a4=ctypes.c_void_p(20)), dict(a5=ctypes.c_void_p(20)), dict(a1=ptr(16, None)), dict(a1=ptr(18, 32)),
               dict(a1=ptr(16, 33)), dict(a2=num(5, -1)), dict(a2=num(5, 1 << 40)), dict(a3=typ(0, 2))):
        assert refused(lib.moe_grad_sumsq, ok, **kw) == bad, kw
    assert refused(lib.moe_grad_sumsq, ok, a6=need - 1) == mod.MOE_ENOSPACE
    ok = (2, ptr(16, 32), num(5, 6), typ(0, 1), P, 1.0, P, ptr(16, 32), None)
    for kw in (dict(a0=-1), dict(a1=None), dict(a4=None), dict(a5=-1.0), dict(a5=float("nan")), dict(a6=ctypes.c_void_p(18)),
               dict(a7=None), dict(a7=ptr(16, None)), dict(a7=ptr(16, 33)), dict(a7=ptr(18, 32))):
        assert refused(lib.moe_grad_clip, ok, **kw) == bad, kw


def test_binding_refuses_host_tensors(mod):
    """Tensors that are not on the GPU are refused by name, before their addresses go anywhere."""
    x, q = torch.zeros(4, 128), torch.zeros(4, 128).to(torch.float8_e4m3fn)
    u = torch.zeros(4, 16, dtype=torch.uint8)
    i, f = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    cu = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: mod.moe_quant_rows(x, q, u), lambda: mod.moe_quant_weight(x[None], q[None], u[None]),
                 lambda: mod.moe_group_gemm_scaled(mod.GEMM_FWD, q, u, q, u, cu, x, 128, 128),
                 lambda: mod.moe_router_topk(x, i, f), lambda: mod.moe_router_backward(x, i, f, x.clone()),
                 lambda: mod.moe_grad_sumsq([x], torch.zeros(1, dtype=torch.float64), u),
                 lambda: mod.moe_grad_clip([x], torch.zeros(1, dtype=torch.float64), 1.0)):
        with pytest.raises(mod.MoeError):
            call()
    with pytest.raises(mod.MoeError):
        mod.moe_router_topk(x, i, f, score="tanh")
