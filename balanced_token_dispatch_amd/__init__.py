"""Python binding of libmoe.so: the one-rank hot path of a redundant-expert MoE layer.

Argument marshalling only.  Every step runs in the HIP kernels of
libmoe.so (see include/moe.h for each call's contract); this module turns
torch tensors into device pointers and torch's current stream into a
hipStream_t.  Importing it fails loudly when the library is not built.
"""
import ctypes
import os
from array import array
from operator import attrgetter

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is not built; build it with `python balanced_token_dispatch_amd/_build.py`")

_lib = ctypes.CDLL(_LIB_PATH)

MOE_OK, MOE_EINVAL, MOE_ENOSPACE, MOE_EHIP = 0, 1, 2, 3
DEV_BAD_EXPERT_ID, DEV_SLOT_OVERFLOW = 1, 2
F32, BF16 = 0, 1
GEMM_FWD, GEMM_DGRAD, GEMM_WGRAD = 0, 1, 2
E4M3, E5M2 = 0, 1
SCORES = {"softmax_topk": 0, "softmax": 1, "sigmoid": 2}   # moe_score
NORMS = {"layer": 0, "rms": 1}                             # moe_norm_kind

EXPORTS = ("moe_status_string", "moe_plan_words", "moe_plan_workspace_bytes", "moe_plan",
           "moe_dispatch_layout_workspace_bytes", "moe_dispatch_layout", "moe_prefetch",
           "moe_permute", "moe_group_gemm", "moe_combine", "moe_replica_grad_fold",
           "moe_unpermute_reduce", "moe_combine_weight_grad", "moe_group_gemm_swiglu",
           "moe_swiglu_backward", "moe_group_gemm_workspace_bytes", "moe_plan_noalloc",
           "moe_group_gemm_gather", "moe_scale_row_bytes", "moe_quant_rows", "moe_quant_weight",
           "moe_group_gemm_scaled", "moe_router_topk",
           "moe_router_backward", "moe_grad_sumsq_workspace_bytes", "moe_grad_sumsq",
           "moe_grad_clip", "moe_dropout", "moe_layer_norm", "moe_layer_norm_backward_workspace_bytes",
           "moe_layer_norm_backward", "moe_expert_counts", "moe_balance_loss_workspace_bytes",
           "moe_balance_loss", "moe_balance_loss_backward")

PLAN_NOALLOC_SCRATCH_BYTES = 4 << 20   # MOE_PLAN_NOALLOC_SCRATCH_BYTES in moe.h


class MoeDims(ctypes.Structure):
    _fields_ = [("R", ctypes.c_int32), ("S", ctypes.c_int32), ("K", ctypes.c_int32),
                ("E", ctypes.c_int32), ("B", ctypes.c_int32)]


_P = ctypes.c_void_p
_D = ctypes.POINTER(MoeDims)
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t

_lib.moe_status_string.restype = ctypes.c_char_p
_lib.moe_status_string.argtypes = [ctypes.c_int]
for _n in ("moe_plan_words", "moe_plan_workspace_bytes", "moe_dispatch_layout_workspace_bytes"):
    getattr(_lib, _n).restype = _SZ
    getattr(_lib, _n).argtypes = [_D]
_lib.moe_plan.argtypes = [_D, _P, _P, _P, _P, _P, _SZ, _P]
_lib.moe_plan_noalloc.argtypes = [_D, _P, _P, _P, _P, _P]
_lib.moe_dispatch_layout.argtypes = [_D, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]
_lib.moe_prefetch.argtypes = [_D, _I32, _P, _P, _I64, _P]
_lib.moe_permute.argtypes = [_D, ctypes.c_int, _I64, _P, _P, _P, _P, _P]
_lib.moe_group_gemm_workspace_bytes.restype = _SZ
_lib.moe_group_gemm_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
_lib.moe_group_gemm.argtypes = [ctypes.c_int, ctypes.c_int, _I32, _I32, _I32, _I32, _P, _P, _P,
                                _P, _P, _SZ, _P]
_lib.moe_group_gemm_gather.argtypes = [ctypes.c_int, ctypes.c_int, _I32, _I32, _I32, _I32, _P, _I64,
                                       _P, _I32, _P, _P, _P, _P, _SZ, _P]
_lib.moe_combine.argtypes = [_D, ctypes.c_int, _I64, _I32, _P, _P, _P, _P, _P]
_lib.moe_replica_grad_fold.argtypes = [_D, _I32, _P, _P, _I64, _P]
_lib.moe_unpermute_reduce.argtypes = [_D, ctypes.c_int, _I64, _I32, _P, _P, _P, _P]
_lib.moe_combine_weight_grad.argtypes = [_D, ctypes.c_int, _I64, _I32, _P, _P, _P, _P, _P]
_lib.moe_group_gemm_swiglu.argtypes = [ctypes.c_int, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                       _P, _SZ, _P]
_lib.moe_swiglu_backward.argtypes = [ctypes.c_int, _I64, _I64, _P, _P, _P, _P]
_lib.moe_scale_row_bytes.restype = _SZ
_lib.moe_scale_row_bytes.argtypes = [_I64]
_lib.moe_grad_sumsq_workspace_bytes.restype = _SZ
_lib.moe_grad_sumsq_workspace_bytes.argtypes = []
_lib.moe_quant_rows.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I64, _P, _I64, _P, _I32, _P, _P,
                                _P, _P, _P]
_lib.moe_quant_weight.argtypes = [ctypes.c_int, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P]
_lib.moe_group_gemm_scaled.argtypes = [ctypes.c_int, ctypes.c_int, _I32, _I32, _I32, _I32, _P, _P,
                                       _P, _P, _P, _P, _P]
_lib.moe_router_topk.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I32, _I32, _P, _P,
                                 ctypes.c_float, _P, _P, _P]
_lib.moe_router_backward.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I32, _I32, _P, _P, _P,
                                     ctypes.c_float, _P, _P]
_lib.moe_grad_sumsq.argtypes = [_I32, _P, _P, _P, _P, _P, _SZ, _P]
_lib.moe_grad_clip.argtypes = [_I32, _P, _P, _P, _P, ctypes.c_double, _P, _P, _P]
_F64 = ctypes.c_double
_lib.moe_dropout.argtypes = [ctypes.c_int, _I64, _P, _P, _F64, _P, _I64, _P, _P]
_lib.moe_layer_norm.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, _I64, _I64, _P, _P, _P, _P, _F64, _F64,
                                _P, _I64, _P, _P, _P, _P, _P]
_lib.moe_layer_norm_backward_workspace_bytes.restype = _SZ
_lib.moe_layer_norm_backward_workspace_bytes.argtypes = [_I64, _I64]
_lib.moe_layer_norm_backward.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, _I64, _I64, _P, _P, _P, _P, _P,
                                         _P, _F64, _P, _I64, _P, _P, _P, _P, _I32, _P, _SZ, _P]
_lib.moe_expert_counts.argtypes = [_I64, _I32, _I32, _P, _I32, _P, _P, _P]
_lib.moe_balance_loss_workspace_bytes.restype = _SZ
_lib.moe_balance_loss_workspace_bytes.argtypes = [_I64, _I32]
_lib.moe_balance_loss.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _SZ, _P]
_lib.moe_balance_loss_backward.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I32, _P, _I32, _P, _P, _P, _P, _P, _P,
                                           _P]
for _n in EXPORTS[3:]:
    if _n.endswith("_bytes"):
        continue
    getattr(_lib, _n).restype = ctypes.c_int


class MoeError(RuntimeError):
    pass


def library():
    """The loaded ctypes library (for tests that call the C ABI directly)."""
    return _lib


def dims(R, S, K, E, B):
    return MoeDims(R, S, K, E, B)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:  # the current stream's handle, without building a Stream object (3 us a call)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc, name):
    if rc != MOE_OK:
        raise MoeError(f"{name}: {_lib.moe_status_string(rc).decode()} (status {rc})")


def _dtype(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise MoeError(f"unsupported dtype {t.dtype}")


def plan_words(d):
    return int(_lib.moe_plan_words(ctypes.byref(d)))


def plan_workspace_bytes(d):
    return int(_lib.moe_plan_workspace_bytes(ctypes.byref(d)))


def dispatch_layout_workspace_bytes(d):
    return int(_lib.moe_dispatch_layout_workspace_bytes(ctypes.byref(d)))


def moe_plan(d, topk_idx, counts, plan, dev_status, ws, stream=None):
    _check(_lib.moe_plan(ctypes.byref(d), _ptr(topk_idx), _ptr(counts), _ptr(plan),
                         _ptr(dev_status), _ptr(ws), ws.numel() * ws.element_size(),
                         _stream(stream)), "moe_plan")


def moe_plan_noalloc(d, topk_idx, counts, plan, dev_status, stream=None):
    """moe_plan without a workspace: the library's static per-GPU scratch (see moe.h)."""
    _check(_lib.moe_plan_noalloc(ctypes.byref(d), _ptr(topk_idx), _ptr(counts), _ptr(plan),
                                 _ptr(dev_status), _stream(stream)), "moe_plan_noalloc")


def moe_dispatch_layout(d, rank, topk_idx, plan, cu_seqlens, dest_pos, src_flat, ws, stream=None):
    _check(_lib.moe_dispatch_layout(ctypes.byref(d), rank, _ptr(topk_idx), _ptr(plan),
                                    _ptr(cu_seqlens), _ptr(dest_pos), _ptr(src_flat), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "moe_dispatch_layout")


def moe_prefetch(d, rank, plan, w, stream=None):
    row_bytes = w[0].numel() * w.element_size()
    _check(_lib.moe_prefetch(ctypes.byref(d), rank, _ptr(plan), _ptr(w), row_bytes,
                             _stream(stream)), "moe_prefetch")


def moe_permute(d, x_all, src_flat, xp, row_scale=None, stream=None):
    _check(_lib.moe_permute(ctypes.byref(d), _dtype(x_all), x_all.shape[1], _ptr(x_all),
                            _ptr(src_flat), _ptr(row_scale), _ptr(xp), _stream(stream)),
           "moe_permute")


def group_gemm_workspace_bytes(op, dtype=BF16):
    return _lib.moe_group_gemm_workspace_bytes(op, dtype)


def _ws(ws):
    return (None, 0) if ws is None else (_ptr(ws), ws.numel() * ws.element_size())


def moe_group_gemm(op, a, b, cu_seqlens, out, Kd, N, ws=None, stream=None):
    """ws: optional scratch tensor of at least group_gemm_workspace_bytes(op) bytes."""
    G = cu_seqlens.numel() - 1
    wp, wn = _ws(ws)
    _check(_lib.moe_group_gemm(op, _dtype(a), G, a.shape[0], Kd, N, _ptr(a), _ptr(b),
                               _ptr(cu_seqlens), _ptr(out), wp, wn, _stream(stream)),
           "moe_group_gemm")


def moe_group_gemm_gather(op, x_src, gather, gather_div, b, cu_seqlens, out, Kd, N, ws=None,
                          stream=None):
    """moe_group_gemm (FWD or WGRAD) with row m of the row operand read from token row
    x_src[gather[m] // gather_div]: the permute fused into the GEMM."""
    G = cu_seqlens.numel() - 1
    wp, wn = _ws(ws)
    _check(_lib.moe_group_gemm_gather(op, _dtype(x_src), G, gather.numel(), Kd, N, _ptr(x_src),
                                      x_src.shape[0], _ptr(gather), gather_div, _ptr(b),
                                      _ptr(cu_seqlens), _ptr(out), wp, wn, _stream(stream)),
           "moe_group_gemm_gather")


def moe_group_gemm_swiglu(a, b, cu_seqlens, z, h, Kd, N, ws=None, stream=None):
    """Gated up-projection: z = silu(gate) * up over (gate, up) column pairs of W; h optional."""
    G = cu_seqlens.numel() - 1
    wp, wn = _ws(ws)
    _check(_lib.moe_group_gemm_swiglu(_dtype(a), G, a.shape[0], Kd, N, _ptr(a), _ptr(b),
                                      _ptr(cu_seqlens), _ptr(z), _ptr(h), wp, wn,
                                      _stream(stream)),
           "moe_group_gemm_swiglu")


def moe_swiglu_backward(h, dz, dh, stream=None):
    _check(_lib.moe_swiglu_backward(_dtype(h), dz.shape[0], dz.shape[1], _ptr(h), _ptr(dz),
                                    _ptr(dh), _stream(stream)), "moe_swiglu_backward")


def moe_combine(d, rank, y_all, dest_pos, topk_w, out, stream=None):
    _check(_lib.moe_combine(ctypes.byref(d), _dtype(y_all), y_all.shape[1], rank, _ptr(y_all),
                            _ptr(dest_pos), _ptr(topk_w), _ptr(out), _stream(stream)),
           "moe_combine")


def moe_unpermute_reduce(d, rank, dxp_all, dest_pos, dx, stream=None):
    _check(_lib.moe_unpermute_reduce(ctypes.byref(d), _dtype(dxp_all), dxp_all.shape[1], rank,
                                     _ptr(dxp_all), _ptr(dest_pos), _ptr(dx), _stream(stream)),
           "moe_unpermute_reduce")


def moe_combine_weight_grad(d, rank, y_all, dest_pos, dout, dw, stream=None):
    _check(_lib.moe_combine_weight_grad(ctypes.byref(d), _dtype(y_all), y_all.shape[1], rank,
                                        _ptr(y_all), _ptr(dest_pos), _ptr(dout), _ptr(dw),
                                        _stream(stream)), "moe_combine_weight_grad")


def moe_replica_grad_fold(d, rank, plan, dw, stream=None):
    _check(_lib.moe_replica_grad_fold(ctypes.byref(d), rank, _ptr(plan), _ptr(dw),
                                      dw[0].numel(), _stream(stream)), "moe_replica_grad_fold")


# ---- 8-bit operands, router, gradient clipping, norm, dropout, balance loss ---------------------
# These calls check their tensors: on the current device (as a stream given to them has to be), contiguous, of
# the right type and size.

_FP8 = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
_SCALE = (torch.uint8, torch.float8_e8m0fnu)
_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}


def _current(name, t):
    """The current device, refused unless tensor t is on it."""
    d = t.get_device()
    if d < 0 or d != torch._C._cuda_getDevice():
        raise MoeError(f"{name}: tensor on {t.device}, not on the current GPU")
    return d


def _take(dev, name, t, dtypes, numel):
    """The address of tensor t, refused unless it is on device dev, contiguous, of one of the dtypes and
    (numel not None) of that many elements."""
    if (t.get_device() == dev and t.dtype in dtypes and t.is_contiguous()
            and (numel is None or t.numel() == numel)):
        return t.data_ptr()
    if t.get_device() != dev:
        raise MoeError(f"{name}: tensor on {t.device}, not on the current GPU")
    if t.dtype not in dtypes:
        raise MoeError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if not t.is_contiguous():
        raise MoeError(f"{name}: not contiguous")
    raise MoeError(f"{name}: shape {tuple(t.shape)}, expected {numel} elements")


def _int32(*sizes):
    """Refuses sizes that the C interface's 32-bit arguments would wrap around."""
    if min(sizes) < 0 or max(sizes) >= 1 << 31:
        raise MoeError(f"sizes {sizes}, expected numbers of 0 to 2^31 - 1")


def _on(dev, stream):
    """The handle of a stream of device dev, or of its current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise MoeError(f"stream of device {stream.device_index}, tensors on device {dev}")
    return stream.cuda_stream


def scale_row_bytes(columns):
    """Bytes of one row of scales over `columns` columns."""
    return (columns + 2047) // 2048 * 16


def moe_quant_rows(x, q, scale, gather=None, gather_div=1, row_scale=None, copy=None, stream=None):
    """Rows of x (bf16 or fp32) into q (float8_e4m3fn or float8_e5m2) with a scale for each block of
    128 columns; optionally gathered (x[gather[i] // gather_div]), weighted, and kept in `copy`."""
    if x.dim() != 2:
        raise MoeError(f"moe_quant_rows: x has {x.dim()} dimensions, expected 2")
    dev = _current("x", x)
    src_rows, width = x.shape
    rows = src_rows if gather is None else gather.numel()
    xp = _take(dev, "x", x, _FLOATS, None)
    qp = _take(dev, "q", q, _FP8, rows * width)
    sp = _take(dev, "scale", scale, _SCALE, rows * scale_row_bytes(width))
    gp = None if gather is None else _take(dev, "gather", gather, (torch.int32,), None)
    wp = None
    if row_scale is not None:
        wp = _take(dev, "row_scale", row_scale, (torch.float32,), None)
        if row_scale.numel() < (rows if gather is None else src_rows * gather_div):
            raise MoeError("row_scale: fewer entries than rows (or gather entries) to weight")
    cp = None if copy is None else _take(dev, "copy", copy, (x.dtype,), rows * width)
    _int32(gather_div, rows)
    _check(_lib.moe_quant_rows(_FLOATS[x.dtype], _FP8[q.dtype], rows, width, xp, src_rows, gp,
                               gather_div, wp, qp, sp, cp, _on(dev, stream)), "moe_quant_rows")


def moe_quant_weight(w, q=None, q_scale=None, qt=None, qt_scale=None, stream=None):
    """Expert weights w [G, Kd, N] into e4m3 with 128 x 128 block scales: q in w's order (DGRAD's
    operand) and qt [G, N, Kd] (FWD's); either pair may be left out."""
    if w.dim() != 3:
        raise MoeError(f"moe_quant_weight: w has {w.dim()} dimensions, expected 3")
    dev = _current("w", w)
    G, Kd, N = w.shape
    _int32(G, Kd, N)
    e4 = (torch.float8_e4m3fn,)
    p = [None if t is None else _take(dev, n, t, d, c) for n, t, d, c in (
        ("q", q, e4, G * Kd * N), ("q_scale", q_scale, _SCALE, G * -(-Kd // 128) * scale_row_bytes(N)),
        ("qt", qt, e4, G * Kd * N), ("qt_scale", qt_scale, _SCALE, G * -(-N // 128) * scale_row_bytes(Kd)))]
    _check(_lib.moe_quant_weight(_dtype(w), G, Kd, N, _take(dev, "w", w, _FLOATS, None), *p,
                                 _on(dev, stream)), "moe_quant_weight")


def moe_group_gemm_scaled(op, a, a_scale, b, b_scale, cu_seqlens, out, Kd, N, stream=None):
    """moe_group_gemm (FWD or DGRAD) on 8-bit operands: a from moe_quant_rows, b = qt (FWD) or q
    (DGRAD) of moe_quant_weight; out bf16."""
    dev = _current("a", a)
    G, M = cu_seqlens.numel() - 1, a.shape[0]
    K, C = (Kd, N) if op == GEMM_FWD else (N, Kd)
    _int32(M, Kd, N)
    ap = _take(dev, "a", a, _FP8, M * K)
    asp = _take(dev, "a_scale", a_scale, _SCALE, M * scale_row_bytes(K))
    bp = _take(dev, "b", b, (torch.float8_e4m3fn,), G * K * C)
    bsp = _take(dev, "b_scale", b_scale, _SCALE, G * -(-C // 128) * scale_row_bytes(K))
    cp = _take(dev, "cu_seqlens", cu_seqlens, (torch.int32,), None)
    op_ = _take(dev, "out", out, (torch.bfloat16,), M * C)
    _check(_lib.moe_group_gemm_scaled(op, _FP8[a.dtype], G, M, Kd, N, ap, asp, bp, bsp, cp,
                                      op_, _on(dev, stream)),
           "moe_group_gemm_scaled")


def _score(score):
    if score not in SCORES:
        raise MoeError(f"score {score!r}, expected one of {', '.join(SCORES)}")
    return SCORES[score]


def moe_router_topk(logits, topk_idx, topk_w, score="softmax_topk", bias=None, factor=1.0,
                    stream=None):
    """The K = topk_idx.shape[-1] experts of each token and their weights, from logits [T, E]."""
    if logits.dim() != 2:
        raise MoeError(f"moe_router_topk: logits has {logits.dim()} dimensions, expected 2")
    dev = _current("logits", logits)
    T, E = logits.shape
    K = topk_idx.shape[-1]
    _int32(E, K)
    bp = None if bias is None else _take(dev, "bias", bias, (torch.float32,), E)
    _check(_lib.moe_router_topk(_dtype(logits), _score(score), T, E, K,
                                _take(dev, "logits", logits, _FLOATS, None), bp, factor,
                                _take(dev, "topk_idx", topk_idx, (torch.int32,), T * K),
                                _take(dev, "topk_w", topk_w, (torch.float32,), T * K),
                                _on(dev, stream)), "moe_router_topk")


def moe_router_backward(logits, topk_idx, dtopk_w, dlogits, score="softmax_topk", factor=1.0,
                        stream=None):
    """dlogits [T, E] from the gradient of the router weights, the choice held fixed."""
    if logits.dim() != 2:
        raise MoeError(f"moe_router_backward: logits has {logits.dim()} dimensions, expected 2")
    dev = _current("logits", logits)
    T, E = logits.shape
    K = topk_idx.shape[-1]
    _int32(E, K)
    _check(_lib.moe_router_backward(_dtype(logits), _score(score), T, E, K,
                                    _take(dev, "logits", logits, _FLOATS, None),
                                    _take(dev, "topk_idx", topk_idx, (torch.int32,), T * K),
                                    _take(dev, "dtopk_w", dtopk_w, (torch.float32,), T * K), factor,
                                    _take(dev, "dlogits", dlogits, (logits.dtype,), T * E),
                                    _on(dev, stream)), "moe_router_backward")


def grad_sumsq_workspace_bytes():
    return _lib.moe_grad_sumsq_workspace_bytes()


_dtype_of = attrgetter("dtype")


def _table(dev, grads):
    """Host tables of a list of gradients: addresses, element counts and types.  A call may bring
    hundreds of tensors, so each attribute is one map over all of them."""
    dt = array("i", [_FLOATS.get(t, -1) for t in map(_dtype_of, grads)])
    T = torch.Tensor
    if -1 in dt or not set(map(T.get_device, grads)) <= {dev} or not all(map(T.is_contiguous, grads)):
        for g in grads:  # says which
            _take(dev, "gradient", g, _FLOATS, None)
    return array("Q", map(T.data_ptr, grads)), array("q", map(T.numel, grads)), dt


def _at(table):
    return ctypes.c_void_p(table.buffer_info()[0])


def moe_grad_sumsq(grads, sumsq, ws, stream=None):
    """sumsq (one float64) = the sum of squares over a list of gradients (fp32 or bf16)."""
    dev = _current("sumsq", sumsq)
    ptr, numel, dt = _table(dev, grads)
    _check(_lib.moe_grad_sumsq(len(grads), _at(ptr), _at(numel), _at(dt),
                               _take(dev, "sumsq", sumsq, (torch.float64,), 1),
                               _take(dev, "ws", ws, (ws.dtype,), None), ws.numel() * ws.element_size(),
                               _on(dev, stream)), "moe_grad_sumsq")


def moe_grad_clip(grads, sumsq, max_norm, norm=None, out=None, stream=None):
    """Scales a list of gradients by min(1, max_norm / (sqrt(sumsq) + 1e-6)), in place or into the
    tensors of `out`; norm (one float32, optional) receives sqrt(sumsq).  No two of the tensors may share
    memory, but for a gradient and its own place in `out`: only equal addresses are found and refused."""
    dev = _current("sumsq", sumsq)
    ptr, numel, dt = _table(dev, grads)
    optr = ptr
    if out is not None:
        optr, onumel, odt = _table(dev, out)
        if onumel != numel or odt != dt:
            raise MoeError("out: not one tensor of the type and size of each gradient")
    written = [p for p, n in zip(optr, numel) if n]
    if len(set(written)) != len(written):
        raise MoeError("moe_grad_clip: a tensor is listed twice")
    np_ = None if norm is None else _take(dev, "norm", norm, (torch.float32,), 1)
    _check(_lib.moe_grad_clip(len(grads), _at(ptr), _at(numel), _at(dt),
                              _take(dev, "sumsq", sumsq, (torch.float64,), 1), max_norm, np_, _at(optr),
                              _on(dev, stream)), "moe_grad_clip")


_F32, _INT32, _INT64 = (torch.float32,), (torch.int32,), (torch.int64,)


def _maybe(dev, name, t, dtypes, numel):
    """The address of a tensor that may be left out."""
    return None if t is None else _take(dev, name, t, dtypes, numel)


def _drop_args(dev, p, rng, offset):
    """(p, address of the seed and offset, the further offset) of a dropout."""
    if p == 0.0:
        return 0.0, None, 0
    if not 0.0 <= p <= 1.0:
        raise MoeError(f"p {p}, expected 0 to 1")
    if rng is None:
        raise MoeError("dropout without rng (int64: seed, offset)")
    if not -(1 << 63) <= offset < 1 << 63:
        raise MoeError(f"offset {offset}, expected a 64-bit number")
    return p, _take(dev, "rng", rng, _INT64, 2), offset


def moe_dropout(x, out, p, rng, residual=None, offset=0, stream=None):
    """out = residual + x with a share p of its values 0 and the others scaled; the mask is a function of
    rng (two int64 on the device: seed, offset), `offset` and each value's place.  The gradient of x is the
    same call on out's gradient, without the residual."""
    dev = _current("x", x)
    p, rp, offset = _drop_args(dev, p, rng, offset)
    dt, same, n = _dtype(x), (x.dtype,), x.numel()
    _check(_lib.moe_dropout(dt, n, _take(dev, "x", x, same, n),
                            None if residual is None else _take(dev, "residual", residual, same, n), p, rp, offset,
                            _take(dev, "out", out, same, n), _on(dev, stream)), "moe_dropout")


def _kind(kind):
    if kind not in NORMS:
        raise MoeError(f"kind {kind!r}, expected one of {', '.join(NORMS)}")
    return NORMS[kind]


def _rows(name, x):
    """Rows, width and elements of x: its last dimension is a row."""
    shape, n = x.shape, x.numel()
    if not shape or shape[-1] < 1:
        raise MoeError(f"{name}: shape {tuple(shape)}, expected rows of at least one value")
    return n // shape[-1], shape[-1], n


def moe_layer_norm(x, weight, y, bias=None, eps=1e-5, kind="layer", residual=None, total=None, mean=None, rstd=None,
                   p=0.0, rng=None, offset=0, stream=None):
    """y = (h - mean) rstd weight + bias over the last dimension, h = residual + dropout(x) (see moe_dropout);
    total receives h, mean and rstd (fp32) what the backward takes.  kind "rms": mean 0."""
    dev = _current("x", x)
    rows, width, n = _rows("x", x)
    p, rp, offset = _drop_args(dev, p, rng, offset)
    dt, same = _dtype(x), (x.dtype,)
    _check(_lib.moe_layer_norm(
        dt, _kind(kind), _dtype(weight), rows, width, _take(dev, "x", x, same, n),
        None if residual is None else _take(dev, "residual", residual, same, n), _take(dev, "weight", weight, _FLOATS, width),
        None if bias is None else _take(dev, "bias", bias, (weight.dtype,), width), eps, p, rp, offset,
        None if total is None else _take(dev, "total", total, same, n), _take(dev, "y", y, same, n),
        None if mean is None else _take(dev, "mean", mean, _F32, rows),
        None if rstd is None else _take(dev, "rstd", rstd, _F32, rows), _on(dev, stream)), "moe_layer_norm")


def layer_norm_backward_workspace_bytes(rows, width):
    return _lib.moe_layer_norm_backward_workspace_bytes(rows, width)


def moe_layer_norm_backward(total, weight, rstd, dy, dx, dweight=None, ws=None, dbias=None, mean=None, kind="layer",
                            dtotal=None, dresidual=None, accumulate=False, p=0.0, rng=None, offset=0, stream=None):
    """The gradients of moe_layer_norm: dx, dresidual (of the residual; dx itself where p is 0), dweight and dbias
    (fp32, added to what they hold with accumulate).  total is h, dtotal the gradient that reaches it by other ways;
    ws: scratch of layer_norm_backward_workspace_bytes(rows, width) bytes for dweight and dbias."""
    dev = _current("total", total)
    rows, width, n = _rows("total", total)
    p, rp, offset = _drop_args(dev, p, rng, offset)
    dt, same = _dtype(total), (total.dtype,)
    _check(_lib.moe_layer_norm_backward(
        dt, _kind(kind), _dtype(weight), rows, width, _take(dev, "total", total, same, n),
        _take(dev, "weight", weight, _FLOATS, width), None if mean is None else _take(dev, "mean", mean, _F32, rows),
        _take(dev, "rstd", rstd, _F32, rows), _take(dev, "dy", dy, same, n),
        None if dtotal is None else _take(dev, "dtotal", dtotal, same, n), p, rp, offset, _take(dev, "dx", dx, same, n),
        None if dresidual is None else _take(dev, "dresidual", dresidual, same, n),
        None if dweight is None else _take(dev, "dweight", dweight, _F32, width),
        None if dbias is None else _take(dev, "dbias", dbias, _F32, width), int(bool(accumulate)),
        None if ws is None else _take(dev, "ws", ws, (ws.dtype,), None),
        0 if ws is None else ws.numel() * ws.element_size(), _on(dev, stream)), "moe_layer_norm_backward")


def _sequences(dev, cu_tokens):
    """(number of sequences, address of their bounds)."""
    if cu_tokens is None:
        return 1, None
    cp = _take(dev, "cu_tokens", cu_tokens, (torch.int32,), None)
    n = cu_tokens.numel() - 1
    if not 1 <= n <= 1 << 20:
        raise MoeError(f"cu_tokens: {n} sequences, expected 1 to 2^20")
    return n, cp


def moe_expert_counts(topk_idx, counts, cu_tokens=None, stream=None):
    """counts[b, e] = copies that the tokens of sequence b, [cu_tokens[b], cu_tokens[b + 1]), send to expert e;
    topk_idx [T, K].  Without cu_tokens all tokens are one sequence."""
    if topk_idx.dim() != 2 or counts.dim() < 1:
        raise MoeError(f"moe_expert_counts: topk_idx of shape {tuple(topk_idx.shape)}, counts {tuple(counts.shape)}, "
                       "expected [T, K] and [sequences, E]")
    dev = _current("topk_idx", topk_idx)
    (T, K), E = topk_idx.shape, counts.shape[-1]
    n, cp = _sequences(dev, cu_tokens)
    _int32(K, E)
    _check(_lib.moe_expert_counts(T, E, K, _take(dev, "topk_idx", topk_idx, _INT32, None), n, cp,
                                  _take(dev, "counts", counts, _INT32, n * E), _on(dev, stream)),
           "moe_expert_counts")


def balance_loss_workspace_bytes(tokens, sequences=1):
    _int32(sequences)
    return _lib.moe_balance_loss_workspace_bytes(tokens, sequences)


def _logits(name, logits, cu_tokens):
    """Device, T, E, number of sequences and the address of their bounds."""
    if logits.dim() != 2:
        raise MoeError(f"{name}: logits has {logits.dim()} dimensions, expected 2")
    dev = _current("logits", logits)
    T, E = logits.shape
    _int32(E)
    return (dev, T, E, *_sequences(dev, cu_tokens))


def moe_balance_loss(logits, counts, balance, ws, zloss=None, score="softmax_topk", cu_tokens=None, stream=None):
    """balance[b] = E / sum(counts[b]) * mean over the sequence's tokens of sum_e counts[b, e] P[s, e], and
    zloss[b] = mean logsumexp^2, from logits [T, E]; P: softmax, or the logistic over its sum (score "sigmoid").
    ws: scratch of balance_loss_workspace_bytes(T, sequences) bytes."""
    dev, T, E, n, cp = _logits("moe_balance_loss", logits, cu_tokens)
    _check(_lib.moe_balance_loss(_dtype(logits), _score(score), T, E, _take(dev, "logits", logits, _FLOATS, None), n, cp,
                                 _take(dev, "counts", counts, _INT32, n * E),
                                 _take(dev, "balance", balance, _F32, n), _maybe(dev, "zloss", zloss, _F32, n),
                                 _take(dev, "ws", ws, (ws.dtype,), None), ws.numel() * ws.element_size(),
                                 _on(dev, stream)), "moe_balance_loss")


def moe_balance_loss_backward(logits, counts, dlogits, dbalance=None, dzloss=None, score="softmax_topk",
                              cu_tokens=None, add=None, stream=None):
    """dlogits = add + the gradient of sum_b dbalance[b] balance[b] + dzloss[b] zloss[b], the counts held fixed; add
    may be dlogits itself.  Rows of tokens in no sequence are left as they are."""
    dev, T, E, n, cp = _logits("moe_balance_loss_backward", logits, cu_tokens)
    same = (logits.dtype,)
    _check(_lib.moe_balance_loss_backward(_dtype(logits), _score(score), T, E,
                                          _take(dev, "logits", logits, _FLOATS, None), n, cp,
                                          _take(dev, "counts", counts, _INT32, n * E),
                                          _maybe(dev, "dbalance", dbalance, _F32, n), _maybe(dev, "dzloss", dzloss, _F32, n),
                                          _maybe(dev, "add", add, same, T * E), _take(dev, "dlogits", dlogits, same, T * E),
                                          _on(dev, stream)), "moe_balance_loss_backward")
