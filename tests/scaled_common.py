"""Helpers of the tests of the 8-bit path: operands made on the host, and their bounds."""
import numpy as np
import torch

from oracle import scaled_ref as ref

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def bf16(a):
    """float array -> bf16 values (float32 array holding them)."""
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16().float().numpy()


def random_bytes(rng, shape, fmt, ints=False):
    """Bytes of finite values: all of them, or the integers -2 .. 2."""
    t = ref.table(fmt)
    if ints:
        pool = np.array([i for i in range(256) if t[i] in (-2.0, -1.0, 0.0, 1.0, 2.0)], np.uint8)
    else:  # magnitudes within 2^8 of each other, so that many values matter in a sum
        top = ref.FORMATS[fmt][2]
        pool = np.array([i for i in range(256) if np.isfinite(t[i]) and top / 256 < abs(t[i])], np.uint8)
    return rng.choice(pool, shape)


def scale_bytes(rng, shape_rows, n, lo, hi):
    s = np.full(shape_rows + (ref.scale_row_bytes(n),), 127, np.uint8)
    nb = -(-n // 128)
    s[..., :nb] = rng.integers(lo, hi + 1, shape_rows + (nb,))
    return s


class Operands:
    """Operands of one scaled product: bytes, scales and segments on the host."""

    def __init__(self, seed, lens, G, K, C, fmt="e4m3", ints=False, tail=0, first=0):
        rng = np.random.default_rng(seed)
        self.G, self.K, self.C, self.fmt = G, K, C, fmt
        self.cu = (first + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        self.M = int(self.cu[-1]) + tail
        self.a = random_bytes(rng, (self.M, K), fmt, ints)
        self.b = random_bytes(rng, (G, C, K), "e4m3", ints)
        self.a_scale = scale_bytes(rng, (self.M,), K, 124, 130)
        self.b_scale = scale_bytes(rng, (G, -(-C // 128)), K, 124, 130)

    def expected(self):
        return ref.group_gemm_scaled(ref.table(self.fmt)[self.a], self.a_scale,
                                     ref.table("e4m3")[self.b], self.b_scale, self.cu)

    def on_gpu(self):
        dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
        return (dev(self.a).view(FP8[self.fmt]), dev(self.a_scale), dev(self.b).view(FP8["e4m3"]),
                dev(self.b_scale), dev(self.cu))

    def run(self, m, grad=False, poison=-7.0):
        a, sa, b, sb, cu = self.on_gpu()
        o = torch.full((self.M, self.C), poison, dtype=torch.bfloat16, device="cuda")
        op, kd, n = (m.GEMM_DGRAD, self.C, self.K) if grad else (m.GEMM_FWD, self.K, self.C)
        m.moe_group_gemm_scaled(op, a, sa, b, sb, cu, o, kd, n)
        return o


def bound(K, value, mag, top):
    """How far a result may be from `value`.  Of 8 neighbouring products with the largest exponent E
    the other 7 are cut off below 2^(E - 13), and 2^E is no larger than the group's largest product:
    7 * 2^-13 of the sum `top` of the groups' largest.  The at most K further additions are off by one
    step (2^-23) each of a partial sum no larger than the sum of magnitudes `mag`.  Then one rounding
    to bf16, half a step: 2^-8 of the value."""
    b = 7 * 2.0 ** -13 * top + (K + 16) * 2.0 ** -23 * mag
    return b + 2.0 ** -8 * (np.abs(value) + b)

