"""Norm, dropout and balance loss: the float64 definitions against published vectors and differences, and
the calls that the library and the binding refuse before anything reaches a GPU."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    if not os.path.exists(os.path.join(ROOT, "balanced_token_dispatch_amd", "libmoe.so")):
        pytest.skip("libmoe.so not built")
    import balanced_token_dispatch_amd as m
    return m


@pytest.mark.parametrize("counter,key,words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_philox_published_vectors(counter, key, words):
    got = ref.philox(counter[0] | counter[1] << 32, key[0] | key[1] << 32, counter[2] | counter[3] << 32)
    assert tuple(int(v) for v in got) == words


def test_mask_share_and_mean():
    """A share p is dropped (5 standard deviations of a binomial), the scale belongs to the p that is met."""
    n = 1 << 18
    for p in (0.1, 0.5, 0.9):
        k = ref.kept(n, p, 1234, 5)
        met = ref.below(p) / 65536
        assert abs(met - p) <= 2.0 ** -17
        assert abs((~k).sum() - n * met) <= 5 * np.sqrt(n * met * (1 - met))
        assert np.isclose(ref.drop(np.ones(n), p, 1234, 5).max(), 1 / (1 - met), rtol=1e-15)
    assert ref.kept(64, 0.3, 1, 2, first=13).tolist() == ref.kept(77, 0.3, 1, 2)[13:].tolist()
    assert (ref.drop(np.ones(99), 1.0, 1, 2) == 0).all() and (ref.drop(np.ones(99), 0.0, 1, 2) == 1).all()


def numeric(f, x, h=1e-6):
    """Central differences of the number f(x) in every entry of x."""
    g = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        y = x.copy()
        y[i] += h
        up = f(y)
        y[i] -= 2 * h
        g[i] = (up - f(y)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_is_the_derivative(kind):
    r = np.random.default_rng(1)
    h, w, b, dy = r.standard_normal((3, 11)) + 0.5, r.standard_normal(11), r.standard_normal(11), r.standard_normal((3, 11))
    _, mean, rstd = ref.layer_norm(h, w, b, 1e-3, kind)
    dh, dw, db = ref.layer_norm_backward(h, w, mean, rstd, dy, kind)
    loss = lambda h, w, b: float((ref.layer_norm(h, w, b, 1e-3, kind)[0] * dy).sum())  # noqa: E731
    # central differences: h^2 times a third derivative of order 10, and rounding / h
    for got, want in ((dh, numeric(lambda v: loss(v, w, b), h)), (dw, numeric(lambda v: loss(h, v, b), w)),
                      (db, numeric(lambda v: loss(h, w, v), b))):
        assert np.allclose(got, want, rtol=0, atol=1e-8 * 10 + 1e-15 / 1e-6 * 100)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_the_derivative(score):
    r = np.random.default_rng(2)
    cu = np.array([1, 4, 4, 7])
    x = r.standard_normal((8, 6)) * 2
    counts = r.integers(0, 9, (3, 6))
    db, dz = r.standard_normal(3), r.standard_normal(3)

    def loss(x):
        b, z = ref.balance_loss(x, counts, cu, score)
        return float((b * db).sum() + (z * dz).sum())

    got = ref.balance_loss_backward(x, counts, cu, db, dz, score)
    assert np.allclose(got, numeric(loss, x), rtol=0, atol=1e-7)
    assert (got[[0, 7]] == 0).all()


def test_balance_of_even_tokens_is_one():
    x = np.zeros((5, 8))
    for score in ("softmax", "sigmoid"):
        b, z = ref.balance_loss(x, np.full((1, 8), 3), np.array([0, 5]), score)
        assert np.allclose(b, 1.0) and np.allclose(z, np.log(8) ** 2)


P = ctypes.c_void_p(4096)  # never dereferenced: every call below is refused first
Q = ctypes.c_void_p(1 << 30)
R_ = ctypes.c_void_p(1 << 32)


def test_dropout_refusals(m):
    f = m.library().moe_dropout
    ok = [m.F32, 8, P, None, 0.5, R_, 0, Q, None]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    V = ctypes.c_void_p
    for bad in (dict(a0=2), dict(a1=-1), dict(a1=1 << 48), dict(a2=None), dict(a7=None), dict(a4=-0.1), dict(a4=1.5),
                dict(a4=float("nan")), dict(a5=None), dict(a5=V(4100)), dict(a2=V(4098)), dict(a7=V((1 << 30) + 2)),
                dict(a7=V(4096 + 16)), dict(a7=V(4096 - 31)), dict(a3=V((1 << 30) + 4)), dict(a7=V((1 << 32) + 8))):
        assert call(**bad) == m.MOE_EINVAL, bad
    assert call(a1=0, a2=None, a7=None) == m.MOE_OK


def test_norm_refusals(m):
    lib = m.library()
    V = ctypes.c_void_p
    at = lambda i: V((i + 1) << 24)  # noqa: E731
    fwd = [m.BF16, 0, m.F32, 4, 64, at(0), at(1), at(2), at(3), 1e-5, 0.1, at(4), 0, at(5), at(6), at(7), at(8), None]
    bwd = [m.BF16, 0, m.F32, 4, 64, at(0), at(1), at(2), at(3), at(4), at(5), 0.1, at(6), 0, at(7), at(8), at(9), at(10), 0,
           at(11), 1 << 20, None]

    def call(f, ok, kw):
        a = list(ok)
        for i, v in kw.items():
            a[i] = v
        return f(*a)

    odd = V((1 << 24) + 1)
    for kw in ({0: 2}, {1: 2}, {2: 5}, {3: -1}, {3: 1 << 31}, {4: 0}, {4: (1 << 22) + 1}, {5: None}, {7: None}, {14: None},
               {13: None}, {9: -1e-5}, {9: float("nan")}, {9: float("inf")}, {10: 1.1}, {11: None}, {5: odd}, {7: V((3 << 24) + 2)},
               {16: V((9 << 24) + 2)}, {1: 1},                       # a mean without one
               {14: at(5)}, {13: V((1 << 24) + 256)}, {14: V((2 << 24) + 2)}, {14: at(2)}, {13: at(4)}, {15: at(8)},
               {16: at(6)}, {15: at(0)}, {3: 2, 4: 2, 0: 1, 15: at(0)}):
        assert call(lib.moe_layer_norm, fwd, kw) == m.MOE_EINVAL, kw
    assert call(lib.moe_layer_norm, fwd, {3: 0, 5: None}) == m.MOE_OK
    for kw in ({0: 2}, {1: 2}, {2: 5}, {3: -1}, {4: 0}, {5: None}, {6: None}, {7: None}, {8: None}, {9: None}, {14: None},
               {18: 2}, {19: None}, {19: V((12 << 24) + 8)}, {11: -1.0}, {12: None}, {1: 1},
               {14: at(8)}, {14: at(0)}, {15: at(0)}, {14: V((5 << 24) + 2)}, {16: at(10)}, {16: at(4)}, {19: at(4)},
               {14: at(11)}, {16: V((11 << 24) + 4)}, {17: at(1)}):
        assert call(lib.moe_layer_norm_backward, bwd, kw) == m.MOE_EINVAL, kw
    need = m.layer_norm_backward_workspace_bytes(4, 64)
    assert need > 0 and call(lib.moe_layer_norm_backward, bwd, {20: need - 1}) == m.MOE_ENOSPACE
    for bad in ((-1, 64), (4, 0), (4, 1 << 23), (1 << 31, 64)):
        assert m.layer_norm_backward_workspace_bytes(*bad) == 0
    assert call(lib.moe_layer_norm_backward, bwd, {3: 0, 16: None, 17: None}) == m.MOE_OK


def test_balance_refusals(m):
    lib = m.library()
    V = ctypes.c_void_p
    at = lambda i: V((i + 1) << 24)  # noqa: E731
    counts = [100, 8, 2, at(0), 3, at(1), at(2), None]
    loss = [m.F32, 1, 100, 8, at(0), 3, at(1), at(2), at(3), at(4), at(5), 1 << 20, None]
    bwd = [m.F32, 1, 100, 8, at(0), 3, at(1), at(2), at(3), at(4), at(5), at(6), None]

    def call(f, ok, kw):
        a = list(ok)
        for i, v in kw.items():
            a[i] = v
        return f(*a)

    for kw in ({0: -1}, {0: 1 << 31}, {0: 1 << 30}, {1: 0}, {1: 1025}, {2: 0}, {2: 9}, {3: None}, {4: 0}, {4: (1 << 20) + 1},
               {5: None}, {6: None}, {6: at(0)}, {6: V((2 << 24) + 4)}, {3: V(4098)}):
        assert call(lib.moe_expert_counts, counts, kw) == m.MOE_EINVAL, kw
    for kw in ({0: 2}, {1: 3}, {2: -1}, {3: 0}, {3: 1025}, {4: None}, {5: 0}, {6: None}, {7: None}, {8: None}, {10: None},
               {10: V(4100)}, {4: V(4098)}, {9: at(3)}, {8: at(2)}, {10: at(0)}, {8: at(5)}):
        assert call(lib.moe_balance_loss, loss, kw) == m.MOE_EINVAL, kw
    need = m.balance_loss_workspace_bytes(100, 3)
    assert need > 0 and call(lib.moe_balance_loss, loss, {11: need - 1}) == m.MOE_ENOSPACE
    assert m.library().moe_balance_loss_workspace_bytes(-1, 3) == 0
    assert m.library().moe_balance_loss_workspace_bytes(5, 0) == 0
    for kw in ({0: 2}, {1: 3}, {2: 1 << 31}, {3: 0}, {4: None}, {5: 0}, {6: None}, {7: None}, {11: None}, {11: at(0)},
               {11: V((6 << 24) + 4)}, {11: at(2)}, {10: V((6 << 24) + 2)}, {8: V(4098)}):
        assert call(lib.moe_balance_loss_backward, bwd, kw) == m.MOE_EINVAL, kw
    assert call(lib.moe_balance_loss_backward, bwd, {2: 0}) == m.MOE_OK


def test_binding_refuses_tensors_off_the_gpu(m):
    x, f = torch.zeros(4, 8), torch.zeros(4)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: m.moe_dropout(x, x, 0.1, i), lambda: m.moe_layer_norm(x, f, x),
                 lambda: m.moe_layer_norm_backward(x, f, f, x, x), lambda: m.moe_expert_counts(i, i),
                 lambda: m.moe_balance_loss(x, i, f, f), lambda: m.moe_balance_loss_backward(x, i, x)):
        with pytest.raises(m.MoeError, match="not on the current GPU"):
            call()
    with pytest.raises(m.MoeError, match="p 1.5"):
        m._drop_args(0, 1.5, i, 0)
    with pytest.raises(m.MoeError, match="without rng"):
        m._drop_args(0, 0.5, None, 0)
    with pytest.raises(m.MoeError, match="kind"):
        m._kind("batch")
    with pytest.raises(m.MoeError, match="64-bit"):
        m._drop_args(0, 0.5, torch.zeros(2, dtype=torch.int64), 1 << 63)
