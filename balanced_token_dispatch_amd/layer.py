"""One MoE layer step on one rank, as a sequence of libmoe.so calls.

Buffers are allocated once (static shapes: every rank receives exactly S*K
rows, so nothing here depends on the routing).  ``forward`` and
``backward`` only enqueue C-ABI calls on torch's current stream (and, with
``overlap``, the backward on a second stream joined back into it); every
number is computed by the HIP kernels.

In one stream (``overlap=False``):
Forward (rank r):  plan -> dispatch layout -> prefetch slot rows of both
projections -> permute -> up GEMM -> down GEMM (written into rank r's
slice of the all-ranks expert-output buffer) -> combine.
Backward:          weighted permute of the output gradient (combine's
adjoint for the expert outputs) -> router-weight gradient (combine's
adjoint for the weights) -> down DGRAD -> down WGRAD -> up DGRAD (into rank
r's slice of the all-ranks input-gradient buffer) -> up WGRAD -> un-permute
reduce of the input gradients to the tokens (dispatch's adjoint) -> fold the
replica rows of both weight gradients into their home experts.
With ``plan_noalloc=True`` the plan runs on the library's static scratch
(moe_plan_noalloc) instead of the workspace.
With ``fused_gather=True`` (identity activation) there is no permute and no
xp buffer: the up projection's FWD and WGRAD read their row operand straight
from the token rows through src_flat (moe_group_gemm_gather), the permute
fused into the expert GEMM.
With ``overlap=True`` the backward puts the kernels whose results no later
kernel of the step reads on a second stream, each under a GEMM of the
four-wave form (one workgroup per CU that leaves room on every CU for a row
kernel's waves): the router-weight gradient beside the down DGRAD, and both
folds beside the up DGRAD, which then comes after the up WGRAD.  Events order
them after what they read; the main stream waits for the second one before
the step ends.  The default (``overlap=None``) turns it on for steps with
S*K*H*H' >= kOverlapMinWork, where the GEMMs are long enough to hide the
kernels beside them.
The activation between the projections is the identity, or, with
``activation="swiglu"``, the gated linear unit: the up projection then has
2H' columns holding (gate, up) pairs, its GEMM writes both the pre-activation
h and z = silu(gate) * up, and the backward turns dz into dh with the gated
unit's derivative before the up projection's DGRAD and WGRAD.
With ``gemm="scaled"`` (bf16, identity) the forward and input-gradient GEMMs run on 8-bit operands
with a scale for each block of 128 (moe_group_gemm_scaled): quantise_weights() puts the home
experts' weights into 8 bits once per weight update, the prefetch copies their 8-bit rows into the
slots, the permutes write 8-bit rows beside the 16-bit ones, and z and dz are quantised between the
projections.  The weight gradients stay on the 16-bit rows.
Around the step: route() makes this rank's expert ids and weights from its gate's logits,
route_backward() the logits' gradient from the step's router-weight gradient, and clip_gradients()
scales the expert gradients (and any others given) to a largest global norm.
"""
from dataclasses import dataclass

import torch

from . import (GEMM_DGRAD, GEMM_FWD, GEMM_WGRAD, MoeError, dims as _mk_dims, dispatch_layout_workspace_bytes,
               grad_sumsq_workspace_bytes, group_gemm_workspace_bytes, moe_combine, moe_combine_weight_grad,
               moe_dispatch_layout, moe_grad_clip, moe_grad_sumsq, moe_group_gemm,
               moe_group_gemm_gather, moe_group_gemm_scaled, moe_group_gemm_swiglu,
               moe_permute, moe_plan, moe_plan_noalloc,
               moe_prefetch, moe_quant_rows, moe_quant_weight, moe_replica_grad_fold,
               moe_router_backward, moe_router_topk, moe_swiglu_backward, moe_unpermute_reduce,
               plan_words, plan_workspace_bytes, scale_row_bytes)


# S*K*H*H' from which the backward uses its second stream by default (the R32 S4096 K8 H7168
# H'2048 step has 4.8e11; its DGRADs take ~0.8 ms each)
kOverlapMinWork = 1e11


class QuantWeights:
    """One projection's weights [G, Kd, N] in 8 bits, in the order FWD contracts (qt) and, with `dgrad`, the
    order DGRAD contracts (q), each with its scales."""

    def __init__(self, w, dgrad=True):
        G, Kd, N = w.shape
        u8 = dict(dtype=torch.uint8, device=w.device)
        self.q = self.q_scale = None
        if dgrad:
            self.q = torch.zeros((G, Kd, N), **u8).view(torch.float8_e4m3fn)
            self.q_scale = torch.full((G, -(-Kd // 128), scale_row_bytes(N)), 127, **u8)
        self.qt = torch.zeros((G, N, Kd), **u8).view(torch.float8_e4m3fn)
        self.qt_scale = torch.full((G, -(-N // 128), scale_row_bytes(Kd)), 127, **u8)

    def tensors(self):
        return self.q, self.q_scale, self.qt, self.qt_scale


class QuantRows:
    """A buffer of rows in 8 bits with their scales."""

    def __init__(self, rows, width, dtype, device):
        self.q = torch.zeros((rows, width), dtype=torch.uint8, device=device).view(dtype)
        self.scale = torch.full((rows, scale_row_bytes(width)), 127, dtype=torch.uint8, device=device)


@dataclass
class Shape:
    R: int
    S: int
    K: int
    E: int
    B: int
    H: int
    Hp: int

    @property
    def SK(self):
        return self.S * self.K

    @property
    def G(self):
        return self.E + self.B


class LayerStep:
    def __init__(self, shape: Shape, rank: int = 0, dtype=torch.bfloat16, device="cuda",
                 backward: bool = True, activation: str = "identity", fused_gather: bool = False,
                 plan_noalloc: bool = False, overlap=None, gemm: str = "bf16",
                 grad_format=torch.float8_e4m3fn):
        s = shape
        if activation not in ("identity", "swiglu"):
            raise ValueError(f"activation {activation!r}")
        if fused_gather and (activation != "identity" or dtype != torch.bfloat16):
            raise ValueError("the gathered (permute-fused) up projection is bf16, identity only")
        if gemm not in ("bf16", "scaled"):
            raise ValueError(f"gemm {gemm!r}")
        if gemm == "scaled" and (activation != "identity" or dtype != torch.bfloat16 or fused_gather):
            raise ValueError("8-bit GEMMs are for bf16 layers, identity activation, unfused permute")
        if gemm == "scaled" and (s.H % 16 or s.Hp % 16):
            raise ValueError("8-bit GEMMs need H and H' to be multiples of 16")
        if grad_format not in (torch.float8_e4m3fn, torch.float8_e5m2):
            raise ValueError(f"grad_format {grad_format}")
        self.scaled = gemm == "scaled"
        self.fused_gather = fused_gather
        # plan with the library's static scratch (moe_plan_noalloc) instead of the workspace
        self.plan_noalloc = plan_noalloc
        self.s, self.rank, self.dtype, self.device = s, rank, dtype, device
        self.activation = activation
        # gated: the up projection has 2H' columns, (gate, up) pairs interleaved
        self.up_cols = 2 * s.Hp if activation == "swiglu" else s.Hp
        self.d = _mk_dims(s.R, s.S, s.K, s.E, s.B)
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        act = dict(dtype=dtype, device=device)
        self.topk_idx = torch.zeros((s.R, s.S, s.K), **i32)
        self.topk_w = torch.zeros((s.R, s.S, s.K), **f32)
        self.counts = torch.zeros((s.R, s.E), **i32)
        self.plan = torch.zeros(plan_words(self.d), **i32)
        self.status = torch.zeros(1, **i32)
        ws = max(plan_workspace_bytes(self.d), dispatch_layout_workspace_bytes(self.d))
        self.ws = torch.zeros(ws, dtype=torch.uint8, device=device)
        # the FWD and DGRAD GEMMs' scratch (split of their last round of tiles); the calls
        # run one after another on one stream, so they share it.  (The 8-bit ones take none.)
        self.gemm_ws = torch.empty(group_gemm_workspace_bytes(GEMM_FWD), dtype=torch.uint8,
                                   device=device) if dtype == torch.bfloat16 and not self.scaled else None
        self.cu = torch.zeros(s.G + 1, **i32)
        self.dest = torch.zeros(s.R * s.SK, **i32)
        self.src = torch.zeros(s.SK, **i32)
        self.x_all = torch.zeros((s.R * s.S, s.H), **act)
        self.w_up = torch.zeros((s.G, s.H, self.up_cols), **act)
        self.w_down = torch.zeros((s.G, s.Hp, s.H), **act)
        # the permuted token rows (not needed when the up projection gathers them itself)
        self.xp = None if fused_gather else torch.zeros((s.SK, s.H), **act)
        self.z = torch.zeros((s.SK, s.Hp), **act)
        # gated: the pre-activation, kept for the backward
        self.hpre = torch.zeros((s.SK, self.up_cols), **act) if activation == "swiglu" else None
        self.y_all = torch.zeros((s.R * s.SK, s.H), **act)
        self.out = torch.zeros((s.S, s.H), **act)
        if self.scaled:
            self.q_up, self.q_down = (QuantWeights(w, dgrad=backward) for w in (self.w_up, self.w_down))
            self.quantised_from = None   # what quantise_weights() read (_weights)
            e4 = torch.float8_e4m3fn
            self.xq, self.zq = QuantRows(s.SK, s.H, e4, device), QuantRows(s.SK, s.Hp, e4, device)
        self.backward_enabled = backward
        # the backward's side stream (default priority) and its fork/join events; by default
        # only where the GEMMs are long enough for the kernels beside them to gain more than
        # the cross-stream waits cost (~tens of microseconds on short steps)
        if overlap is None:
            overlap = s.S * s.K * s.H * s.Hp >= kOverlapMinWork
        self.overlap = bool(overlap)
        self.side = torch.cuda.Stream(device=device)
        self.ev_fork, self.ev_wgrad, self.ev_join = (torch.cuda.Event() for _ in range(3))
        if backward:
            self.dout_all = torch.zeros((s.R * s.S, s.H), **act)
            self.dy = torch.zeros((s.SK, s.H), **act)
            self.dz = torch.zeros((s.SK, s.Hp), **act)
            self.dh = torch.zeros((s.SK, self.up_cols), **act) if activation == "swiglu" else None
            # every rank's input-gradient rows in the layout's order; this rank's DGRAD writes
            # its slice, the other slices stand in for the peers' (the un-permute reduce reads
            # a token's K copies wherever they were processed)
            self.dxp_all = torch.zeros((s.R * s.SK, s.H), **act)
            self.dx = torch.zeros((s.S, s.H), **act)
            self.dtopk_w = torch.zeros(s.SK, **f32)
            self.dw_up = torch.zeros((s.G, s.H, self.up_cols), **f32)
            self.dw_down = torch.zeros((s.G, s.Hp, s.H), **f32)
            if self.scaled:
                self.dyq = QuantRows(s.SK, s.H, grad_format, device)
                self.dzq = QuantRows(s.SK, s.Hp, grad_format, device)
            # clip_gradients(): the sum of squares, the norm, scratch
            self.sumsq = torch.zeros(1, dtype=torch.float64, device=device)
            self.grad_norm = torch.zeros(1, **f32)
            self.clip_ws = torch.empty(grad_sumsq_workspace_bytes(), dtype=torch.uint8, device=device)

    @property
    def dxp(self):
        """This rank's slice of the input-gradient buffer (the up projection's DGRAD writes here)."""
        r, SK = self.rank, self.s.SK
        return self.dxp_all[r * SK:(r + 1) * SK]

    @property
    def y(self):
        """This rank's slice of the expert-output buffer (the down GEMM writes here)."""
        r, SK = self.rank, self.s.SK
        return self.y_all[r * SK:(r + 1) * SK]

    def _weights(self):
        """The weights and how often torch has changed them in place."""
        return [(w, None if w.is_inference() else w._version) for w in (self.w_up, self.w_down)]

    @property
    def weights_quantised(self):
        """Whether the 8-bit weights are the present ones', as far as torch counts the changes: not those by
        kernels of other libraries, fused optimizers or .data.  To be set by a caller that writes the 8-bit
        weights itself."""
        was = self.quantised_from
        return was is not None and all(w is v and n == k for (w, n), (v, k) in zip(self._weights(), was))

    @weights_quantised.setter
    def weights_quantised(self, done):
        self.quantised_from = self._weights() if done else None

    def quantise_weights(self):
        """The home experts' weights into 8 bits (gemm="scaled"): after every change of w_up or w_down.
        The slots' rows follow by the step's prefetch."""
        if not self.scaled:
            raise ValueError("quantise_weights: the layer's GEMMs are not in 8 bits")
        E = self.s.E
        for w, qw in ((self.w_up, self.q_up), (self.w_down, self.q_down)):
            moe_quant_weight(w[:E], *(None if t is None else t[:E] for t in qw.tensors()))
        self.weights_quantised = True

    def _check_logits(self, logits):
        if tuple(logits.shape) != (self.s.S, self.s.E):
            raise MoeError(f"logits of shape {tuple(logits.shape)}, expected (S, E) = ({self.s.S}, {self.s.E})")

    def route(self, logits, score="softmax_topk", bias=None, factor=1.0):
        """This rank's expert ids and router weights (its rows of topk_idx and topk_w) from its gate's
        logits [S, E]."""
        self._check_logits(logits)
        moe_router_topk(logits, self.topk_idx[self.rank], self.topk_w[self.rank], score, bias, factor)

    def route_backward(self, logits, dlogits, score="softmax_topk", factor=1.0):
        """dlogits [S, E] from the router-weight gradient of the last backward."""
        self._check_logits(logits)
        moe_router_backward(logits, self.topk_idx[self.rank],
                            self.dtopk_w.view(self.s.S, self.s.K), dlogits, score, factor)

    def clip_gradients(self, max_norm, others=()):
        """Scales the experts' weight gradients of this rank, and the gradients in `others`, in place to a
        norm over all of them of at most max_norm; returns the norm before (a one-element tensor).
        After backward(), whose fold leaves the slots' rows zero.  The norm is this rank's: an expert
        with replicas has a part of its gradient on every rank that held one.  Once those are added up,
        each gradient whole on one rank, moe_grad_sumsq, an all-reduce of its sum and moe_grad_clip give
        the norm over ranks."""
        E = self.s.E
        grads = [self.dw_up[:E], self.dw_down[:E], *others]
        moe_grad_sumsq(grads, self.sumsq, self.clip_ws)
        moe_grad_clip(grads, self.sumsq, max_norm, self.grad_norm)
        return self.grad_norm.clone()  # the buffer itself is the next call's too

    @staticmethod
    def _call(timer, name, fn, *args):
        if timer is None:
            fn(*args)
        else:
            timer(name, fn, *args)

    def forward(self, timer=None):
        s, r, c = self.s, self.rank, self._call
        if self.scaled and not self.weights_quantised:
            raise ValueError("forward: quantise_weights() has not put these weights into 8 bits, or not since they changed")
        if self.plan_noalloc:
            c(timer, "plan", moe_plan_noalloc, self.d, self.topk_idx, self.counts, self.plan,
              self.status)
        else:
            c(timer, "plan", moe_plan, self.d, self.topk_idx, self.counts, self.plan,
              self.status, self.ws)
        c(timer, "dispatch_layout", moe_dispatch_layout, self.d, r, self.topk_idx, self.plan,
          self.cu, self.dest, self.src, self.ws)
        if self.scaled:
            for qw in (self.q_up, self.q_down):
                for t in qw.tensors() if self.backward_enabled else (qw.qt, qw.qt_scale):
                    c(timer, "prefetch", moe_prefetch, self.d, r, self.plan, t)
            c(timer, "permute_quant", self._quant_rows, self.x_all, self.xq, self.xp, None)
            c(timer, "gemm_fwd_scaled", moe_group_gemm_scaled, GEMM_FWD, self.xq.q, self.xq.scale,
              self.q_up.qt, self.q_up.qt_scale, self.cu, self.z, s.H, s.Hp)
            c(timer, "quant", moe_quant_rows, self.z, self.zq.q, self.zq.scale)
            c(timer, "gemm_fwd_scaled", moe_group_gemm_scaled, GEMM_FWD, self.zq.q, self.zq.scale,
              self.q_down.qt, self.q_down.qt_scale, self.cu, self.y, s.Hp, s.H)
            c(timer, "combine", moe_combine, self.d, r, self.y_all, self.dest,
              self.topk_w.view(-1), self.out)
            return
        c(timer, "prefetch", moe_prefetch, self.d, r, self.plan, self.w_up)
        c(timer, "prefetch", moe_prefetch, self.d, r, self.plan, self.w_down)
        if self.fused_gather:   # up projection reading the token rows through src_flat
            c(timer, "gemm_fwd_gather", moe_group_gemm_gather, GEMM_FWD, self.x_all, self.src,
              s.K, self.w_up, self.cu, self.z, s.H, s.Hp, self.gemm_ws)
        else:
            c(timer, "permute", moe_permute, self.d, self.x_all, self.src, self.xp)
            if self.activation == "swiglu":
                c(timer, "gemm_fwd_swiglu", moe_group_gemm_swiglu, self.xp, self.w_up, self.cu,
                  self.z, self.hpre, s.H, self.up_cols, self.gemm_ws)
            else:
                c(timer, "gemm_fwd", moe_group_gemm, GEMM_FWD, self.xp, self.w_up, self.cu, self.z,
                  s.H, s.Hp, self.gemm_ws)
        c(timer, "gemm_fwd", moe_group_gemm, GEMM_FWD, self.z, self.w_down, self.cu, self.y, s.Hp,
          s.H, self.gemm_ws)
        c(timer, "combine", moe_combine, self.d, r, self.y_all, self.dest,
          self.topk_w.view(-1), self.out)

    def _quant_rows(self, x, to, copy, row_scale):
        """Token rows in expert order, in 8 bits and (copy) in 16."""
        moe_quant_rows(x, to.q, to.scale, gather=self.src, gather_div=self.s.K, row_scale=row_scale,
                       copy=copy)

    def _down_dgrad(self, timer):
        s = self.s
        if self.scaled:
            return (timer, "gemm_dgrad_scaled", moe_group_gemm_scaled, GEMM_DGRAD, self.dyq.q,
                    self.dyq.scale, self.q_down.q, self.q_down.q_scale, self.cu, self.dz, s.Hp, s.H)
        return (timer, "gemm_dgrad", moe_group_gemm, GEMM_DGRAD, self.dy, self.w_down, self.cu, self.dz,
                s.Hp, s.H, self.gemm_ws)

    def _up_dgrad(self, timer, dup):
        s = self.s
        if self.scaled:
            return (timer, "gemm_dgrad_scaled", moe_group_gemm_scaled, GEMM_DGRAD, self.dzq.q,
                    self.dzq.scale, self.q_up.q, self.q_up.q_scale, self.cu, self.dxp, s.H, s.Hp)
        return (timer, "gemm_dgrad", moe_group_gemm, GEMM_DGRAD, dup, self.w_up, self.cu, self.dxp,
                s.H, self.up_cols, self.gemm_ws)

    def backward(self, timer=None):
        s, r, c = self.s, self.rank, self._call
        if self.scaled:
            c(timer, "permute_weighted_quant", self._quant_rows, self.dout_all, self.dyq, self.dy,
              self.topk_w.view(-1))
        else:
            c(timer, "permute_weighted", moe_permute, self.d, self.dout_all, self.src, self.dy,
              self.topk_w.view(-1))
        cwgrad = (timer, "combine_wgrad", moe_combine_weight_grad, self.d, r, self.y_all,
                  self.dest, self.dout_all[r * s.S:(r + 1) * s.S], self.dtopk_w)
        if self.overlap:
            main = torch.cuda.current_stream()
            self.ev_fork.record(main)
        else:
            c(*cwgrad)
        c(*self._down_dgrad(timer))
        if self.overlap:  # beside the down DGRAD: it reads only forward results and dout
            self.side.wait_event(self.ev_fork)
            with torch.cuda.stream(self.side):
                c(*cwgrad)
        c(timer, "gemm_wgrad", moe_group_gemm, GEMM_WGRAD, self.z, self.dy, self.cu, self.dw_down,
          s.Hp, s.H)
        dup = self.dz
        if self.activation == "swiglu":
            c(timer, "swiglu_bwd", moe_swiglu_backward, self.hpre, self.dz, self.dh)
            dup = self.dh
        if self.scaled:
            c(timer, "quant", moe_quant_rows, self.dz, self.dzq.q, self.dzq.scale)
        up_dgrad = self._up_dgrad(timer, dup)
        if not self.overlap:
            c(*up_dgrad)
        if self.fused_gather:
            c(timer, "gemm_wgrad_gather", moe_group_gemm_gather, GEMM_WGRAD, self.x_all, self.src,
              s.K, dup, self.cu, self.dw_up, s.H, self.up_cols)
        else:
            c(timer, "gemm_wgrad", moe_group_gemm, GEMM_WGRAD, self.xp, dup, self.cu, self.dw_up,
              s.H, self.up_cols)
        folds = ((timer, "fold", moe_replica_grad_fold, self.d, r, self.plan, self.dw_up),
                 (timer, "fold", moe_replica_grad_fold, self.d, r, self.plan, self.dw_down))
        if self.overlap:  # both folds beside the up DGRAD, after both WGRADs
            self.ev_wgrad.record(main)
            c(*up_dgrad)
            self.side.wait_event(self.ev_wgrad)
            with torch.cuda.stream(self.side):
                for f in folds:
                    c(*f)
            self.ev_join.record(self.side)
        c(timer, "unpermute_reduce", moe_unpermute_reduce, self.d, r, self.dxp_all, self.dest,
          self.dx)
        if self.overlap:
            main.wait_event(self.ev_join)
        else:
            for f in folds:
                c(*f)

    def step(self, timer=None):
        self.forward(timer)
        if self.backward_enabled:
            self.backward(timer)
