"""One MoE layer's forward and backward as a sequence of C-ABI calls.

Buffers for every intermediate are allocated once (torch device memory) and
reused by each call, so a step enqueues kernels only.  The sequence is:

  forward:  moe_route -> moe_permute -> moe_grouped_swiglu_fwd -> moe_combine
  backward: moe_combine_bwd -> moe_grouped_swiglu_bwd -> moe_route_bwd

(moe_route_bwd also unpermutes and sums the expert input gradients).  With
gather=True the permutation is a plan only and the expert GEMMs read their
input rows from X through src_token (moe_grouped_swiglu_fwd_gather /
bwd_gather), so x_perm is never materialised; the results are identical.

Definitional variants: capacity_factor enables per-block expert capacity
(moe_capacity between the router and the permutation: dropped assignments get
no row), and aux_coef / z_coef add the balancing and z-loss gradients.  Either
switches the router backward to moe_route_bwd_dense; z_coef also computes the
per-block z-loss values (moe_router_zloss) in the forward.

fold_gate=True (bf16, gathered input, dims that moe_gate_folded_supported
accepts) moves the combine's gate onto the expert rows: the forward stores
h = g silu(a) b (moe_permute_gates, moe_expert_up_folded, moe_expert_down,
moe_combine without gates) and the backward reads dY through src_token
(moe_expert_dgrad_down_folded, moe_expert_dgrad_up, moe_expert_wgrad_folded,
moe_route_bwd_folded, which also sums the dgate parts; with the dense router
backward, or more than two parts per row, moe_dgate_from_parts sums them
first), so neither moe_combine_bwd nor dy_perm exists.
The results equal the unfolded layer's up to rounding.

Backward options of the expert call: wgrad_dtype=torch.float32 on a bf16 layer
keeps dW1, dW3, dW2 as the fp32 sums (not rounded to bf16), and
recompute=True hands the backward no saved a, b, h, so that it recomputes
them with the forward kernel (the forward still stores them here; the results
are the same bits).  Neither combines with fold_gate.

pre_norm=True puts the root-mean-square norm and the residual's addition in
front (moe_rmsnorm, moe_rmsnorm_bwd): the layer reads norm(x + residual), and
`stream` holds the sum that the block's output is added to, usually by the next
block's norm.

MoEServeLayer is the forward alone with the expert weights in 4 bits: norm,
router, and then moe_token_swiglu for a few tokens or moe_permute ->
moe_expert_up_mx -> moe_expert_down_mx -> moe_combine for more.
"""
from __future__ import annotations

import torch

from . import _lib as L


def _shared(a, b):
    """whether two tensors have memory in common"""
    at, to = a.data_ptr(), b.data_ptr()
    return a.numel() > 0 and b.numel() > 0 and at < to + b.nbytes and to < at + a.nbytes


def _readable(t, outs):
    """An input of the norm, or a copy of it.  The norm may write a row where it read it,
    but rows of its outputs at other places (the sequences behind one that has ended)
    may be overwritten before they are read."""
    if t is not None and any(t.data_ptr() != o.data_ptr() and _shared(t, o) for o in outs):
        return t.clone()
    return t


class MoELayer:
    def __init__(self, T: int, d: int, E: int, f: int, k: int, act: torch.dtype,
                 n_groups: int = 1, near_tie_eps: float = 1e-3, device="cuda",
                 gather: bool = False, capacity_factor=None, aux_coef: float = 0.0,
                 z_coef: float = 0.0, fold_gate: bool = False, wgrad_dtype=None,
                 recompute: bool = False, pre_norm: bool = False, norm_eps: float = 1e-6):
        self.dims = L.make_dims(T, d, E, f, k, act)
        self.wgrad_dtype = act if wgrad_dtype is None else wgrad_dtype
        self.recompute = bool(recompute)
        if fold_gate and (self.wgrad_dtype != act or self.recompute):
            raise ValueError("fold_gate takes neither another wgrad_dtype nor recompute")
        if fold_gate and not (gather and L.moe_gate_folded_supported(self.dims)):
            raise ValueError("fold_gate needs gather=True and dims that "
                             "moe_gate_folded_supported accepts (bf16, one-pass weight gradients)")
        self.fold_gate = fold_gate
        self.act = act
        self.gather = gather
        self.capacity = (None if capacity_factor is None else
                         L.moe_expert_capacity(T, k, E, n_groups, capacity_factor))
        self.aux_coef = float(aux_coef)
        self.z_coef = float(z_coef)
        self.dense_bwd = self.capacity is not None or self.aux_coef != 0.0 or self.z_coef != 0.0
        self.n_groups = n_groups
        self.eps = near_tie_eps
        R = T * k
        dev = torch.device(device)
        e32 = dict(dtype=torch.float32, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        ea = dict(dtype=act, device=dev)

        def empty(*shape, **kw):
            # never a NULL pointer, even for an empty batch (T = 0)
            t = torch.empty(max(shape[0], 1), *shape[1:], **kw)
            return t[:shape[0]]

        self.logits = empty(T, E, **e32)
        self.topk_idx = empty(T, k, **i32)
        self.topk_gate = empty(T, k, **e32)
        self.margin = empty(T, **e32)
        self.near_tie_count = empty(1, **i32)
        self.group_count = empty(n_groups, E, **i32)
        self.group_mean_prob = empty(n_groups, E, **e32)
        self.group_aux = empty(n_groups, **e32)
        self.expert_counts = empty(E, **i32)
        self.expert_offsets = empty(E + 1, **i32)
        self.pos = empty(T, k, **i32)
        self.src_token = empty(R, **i32)
        self.x_perm = empty(0 if gather else R, d, **ea)
        self.a = empty(R, f, **ea)
        self.b = empty(R, f, **ea)
        self.h = empty(R, f, **ea)
        self.y_perm = empty(R, d, **ea)
        self.y = empty(T, d, **ea)
        self.dy_perm = empty(0 if fold_gate else R, d, **ea)
        self.gate_perm = empty(R, **e32) if fold_gate else None
        self.dgate_part = (empty(R, L.moe_dgate_parts(self.dims), **e32) if fold_gate
                           else None)
        self.da = empty(R, f, **ea) if fold_gate else None
        self.db = empty(R, f, **ea) if fold_gate else None
        self.dgate = empty(T, k, **e32)
        self.dx_perm = empty(R, d, **ea)
        ew = dict(dtype=self.wgrad_dtype, device=dev)
        self.dw1 = empty(E, f, d, **ew)
        self.dw3 = empty(E, f, d, **ew)
        self.dw2 = empty(E, d, f, **ew)
        self.dx = empty(T, d, **ea)
        self.dwr = empty(E, d, **e32)
        self.kept_idx = empty(T, k, **i32) if self.capacity is not None else None
        self.group_dropped = empty(n_groups, **i32) if self.capacity is not None else None
        self.group_z = empty(n_groups, **e32) if self.z_coef != 0.0 else None
        self.dlogits = empty(T, E, **e32) if self.dense_bwd else None
        self.workspace = L.alloc_workspace(self.dims, n_groups, dev)
        if self.recompute:
            need = L.moe_grouped_swiglu_bwd_workspace_bytes(self.dims, True)
            if need > self.workspace.numel():
                self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        self.pre_norm = bool(pre_norm)
        self.norm_eps = float(norm_eps)
        self.stream = None   # what was normed: the sum, or x
        self.norm_sum = empty(T, d, **ea) if self.pre_norm else None
        self.xn = empty(T, d, **ea) if self.pre_norm else None
        self.rstd = empty(T, **e32) if self.pre_norm else None
        self.dstream = empty(T, d, **ea) if self.pre_norm else None
        self.dnorm = empty(d, **e32) if self.pre_norm else None

    # ------------------------------------------------------------------ forward
    def route(self, x, wr):
        L.moe_route(self.dims, x, wr, self.logits, self.topk_idx, self.topk_gate, self.margin,
                    self.eps, self.near_tie_count, self.n_groups, self.group_count,
                    self.group_mean_prob, self.group_aux, self.workspace)

    def forward_experts(self, x, w1, w3, w2):
        table = self.topk_idx
        if self.capacity is not None:
            L.moe_capacity(self.dims, self.n_groups, self.capacity, self.topk_idx, self.kept_idx,
                           self.group_dropped, self.workspace)
            table = self.kept_idx
        if self.z_coef != 0.0:
            L.moe_router_zloss(self.dims, self.logits, self.n_groups, self.group_z,
                               self.workspace)
        if self.fold_gate:
            L.moe_permute_gates(self.dims, table, self.topk_gate, self.expert_counts,
                                self.expert_offsets, self.pos, self.src_token, self.gate_perm,
                                self.workspace)
            L.moe_expert_up_folded(self.dims, x, self.src_token, self.expert_offsets,
                                   self.gate_perm, w1, w3, self.a, self.b, self.h)
            L.moe_expert_down(self.dims, self.h, self.expert_offsets, w2, self.y_perm)
            L.moe_combine(self.dims, self.y_perm, self.pos, None, self.y)
            return
        if self.gather:
            L.moe_permute(self.dims, table, self.expert_counts, self.expert_offsets,
                          self.pos, self.src_token, None, None, self.workspace)
            L.moe_grouped_swiglu_fwd_gather(self.dims, x, self.src_token, self.expert_offsets,
                                            w1, w3, w2, self.a, self.b, self.h, self.y_perm)
        else:
            L.moe_permute(self.dims, table, self.expert_counts, self.expert_offsets,
                          self.pos, self.src_token, x, self.x_perm, self.workspace)
            L.moe_grouped_swiglu_fwd(self.dims, self.x_perm, self.expert_offsets, w1, w3, w2,
                                     self.a, self.b, self.h, self.y_perm)
        L.moe_combine(self.dims, self.y_perm, self.pos, self.topk_gate, self.y)

    def norm(self, x, norm_weight, residual=None):
        """The pre-norm alone: the layer's input, from x and the residual."""
        if not self.pre_norm:
            raise ValueError("the layer was made without pre_norm")
        # x itself, unless the step writes there before the backward pass reads it
        total = (self.norm_sum if residual is not None
                 or any(_shared(x, t) for t in (self.xn, self.y, self.dx)) else None)
        self.stream = x if total is None else total
        L.moe_rmsnorm(self.dims, x, residual, norm_weight, self.norm_eps, total, self.xn, None,
                      None, self.rstd)
        return self.xn

    def forward(self, x, wr, w1, w3, w2, routing=None, norm_weight=None, residual=None):
        """routing: optional (topk_idx, topk_gate) device tensors that replace the
        router's decision after it has run (used to compare the downstream
        steps on a routing fixed from outside).
        norm_weight [d] fp32 and residual [T,d] or None: with pre_norm only."""
        if self.pre_norm != (norm_weight is not None) or (residual is not None
                                                          and not self.pre_norm):
            raise ValueError("norm_weight goes with pre_norm=True, and so does residual")
        with torch.cuda.device_of(x):
            return self._forward(x, wr, w1, w3, w2, routing, norm_weight, residual)

    def _forward(self, x, wr, w1, w3, w2, routing, norm_weight, residual):
        if self.pre_norm:
            x = self.norm(x, norm_weight, residual)
        self.route(x, wr)
        if routing is not None:
            self.topk_idx.copy_(routing[0])
            self.topk_gate.copy_(routing[1])
        self.forward_experts(x, w1, w3, w2)
        return self.y

    # ------------------------------------------------------------------ backward
    def backward(self, dy, x, wr, w1, w3, w2, norm_weight=None, dsum=None):
        """The gradient of the forward's x.  With pre_norm that is dstream, the
        gradient of x and of the residual alike (dx is the norm output's, dnorm
        the norm weight's); dsum [T,d] or None is added to it: the gradient that
        reaches `stream` from elsewhere."""
        if self.pre_norm != (norm_weight is not None) or (dsum is not None and not self.pre_norm):
            raise ValueError("norm_weight goes with pre_norm=True, and so does dsum")
        if self.pre_norm and self.stream is None:
            raise ValueError("backward before forward")
        with torch.cuda.device_of(dy):
            if not self.pre_norm:
                return self._layer_bwd(dy, x, wr, w1, w3, w2)
            self._layer_bwd(dy, self.xn, wr, w1, w3, w2)
            L.moe_rmsnorm_bwd(self.dims, self.dx, self.stream, norm_weight, self.rstd, dsum,
                              self.dstream, self.dnorm, self.workspace)
        return self.dstream

    def _layer_bwd(self, dy, x, wr, w1, w3, w2):
        if self.fold_gate:
            L.moe_expert_dgrad_down_folded(self.dims, dy, self.src_token, self.expert_offsets,
                                           self.gate_perm, w2, self.a, self.b, self.da, self.db,
                                           self.dgate_part)
            # with more than two parts per row the router backward's dX threads
            # would each reload them all: sum them once instead
            parts_first = self.dense_bwd or L.moe_dgate_parts(self.dims) > 2
            if parts_first:
                L.moe_dgate_from_parts(self.dims, self.dgate_part, self.pos, self.dgate)
            L.moe_expert_dgrad_up(self.dims, self.da, self.db, self.expert_offsets, w1, w3,
                                  self.dx_perm)
            L.moe_expert_wgrad_folded(self.dims, x, dy, self.src_token, self.expert_offsets,
                                      self.h, self.da, self.db, self.dw1, self.dw3, self.dw2)
            if not parts_first:   # the router backward sums the parts into dgate itself
                L.moe_route_bwd_folded(self.dims, x, wr, self.topk_idx, self.topk_gate,
                                       self.dgate_part, self.expert_offsets, self.pos,
                                       self.src_token, self.dx_perm, self.dgate, self.dx,
                                       self.dwr, self.workspace)
                return self.dx
        else:
            self._experts_bwd(dy, x, w1, w3, w2)
        self._router_bwd(x, wr)
        return self.dx

    def _experts_bwd(self, dy, x, w1, w3, w2):
        L.moe_combine_bwd(self.dims, dy, self.y_perm, self.pos, self.topk_gate, self.dy_perm,
                          self.dgate)
        saved = (None, None, None) if self.recompute else (self.a, self.b, self.h)
        if self.gather:
            L.moe_grouped_swiglu_bwd_gather(self.dims, x, self.src_token, self.expert_offsets,
                                            w1, w3, w2, *saved, self.dy_perm, self.dx_perm,
                                            self.dw1, self.dw3, self.dw2, self.workspace,
                                            wgrad_dtype=self.wgrad_dtype)
        else:
            L.moe_grouped_swiglu_bwd(self.dims, self.x_perm, self.expert_offsets, w1, w3, w2,
                                     *saved, self.dy_perm, self.dx_perm, self.dw1, self.dw3,
                                     self.dw2, self.workspace, wgrad_dtype=self.wgrad_dtype)

    def _router_bwd(self, x, wr):
        if self.dense_bwd:
            L.moe_route_bwd_dense(self.dims, x, wr, self.logits, self.topk_idx, self.topk_gate,
                                  self.dgate, self.pos, self.dx_perm, self.n_groups,
                                  self.group_count, self.aux_coef, self.z_coef, self.dx,
                                  self.dwr, self.dlogits, self.workspace)
        else:
            L.moe_route_bwd(self.dims, x, wr, self.topk_idx, self.topk_gate, self.dgate,
                            self.expert_offsets, self.pos, self.src_token, self.dx_perm, self.dx,
                            self.dwr, self.workspace)
        return self.dx

    def step(self, x, wr, w1, w3, w2, dy, norm_weight=None, residual=None, dsum=None):
        self.forward(x, wr, w1, w3, w2, norm_weight=norm_weight, residual=residual)
        self.backward(dy, x, wr, w1, w3, w2, norm_weight=norm_weight, dsum=dsum)


class MoEServeLayer:
    """The layer's forward with 4-bit expert weights, for up to max_tokens tokens.

    A few token-expert pairs go through moe_token_swiglu (activations in `act`,
    nothing sorted), more through the grouped products on 8-bit rows.  few_slots is
    how many; without it the layer takes what is faster, as measured.
    The outputs are buffers that the next forward overwrites: one forward at a time,
    on one stream or with its own ordering between them.  They, and slices of them,
    may be its inputs.
    """

    def __init__(self, max_tokens: int, d: int, E: int, f: int, k: int, act: torch.dtype,
                 norm_eps: float = 1e-6, few_slots=None, device="cuda"):
        self.T, self.d, self.E, self.f, self.k, self.act = max_tokens, d, E, f, k, act
        self.norm_eps = float(norm_eps)
        self.by_expert = few_slots is None
        self.few_slots = min(128 if self.by_expert else int(few_slots), L.MOE_TOKEN_MAX_SLOTS)
        dev = torch.device(device)
        T, R = max(max_tokens, 1), max(max_tokens * k, 1)

        def empty(*shape, dtype):
            return torch.empty(*shape, dtype=dtype, device=dev)

        f32, i32, u8 = torch.float32, torch.int32, torch.uint8
        ld, lf = L.moe_mx_scale_cols(d), L.moe_mx_scale_cols(f)
        self.w1, self.w1_scale = empty(E, f, d // 2, dtype=u8), empty(E, f, ld, dtype=u8)
        self.w3, self.w3_scale = empty(E, f, d // 2, dtype=u8), empty(E, f, ld, dtype=u8)
        self.w2, self.w2_scale = empty(E, d, f // 2, dtype=u8), empty(E, d, lf, dtype=u8)
        for scale in (self.w1_scale, self.w3_scale, self.w2_scale):
            scale.fill_(255)   # NaN, until there are weights
        if self.w1_scale.is_cuda and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.w1_scale.device).synchronize()   # load may run on any
        self.norm_sum, self.xn, self.y = (empty(T, d, dtype=act) for _ in range(3))
        self.xq, self.x_scale = empty(T, d, dtype=u8), empty(T, ld, dtype=u8)
        self.hq, self.h_scale = empty(R, f, dtype=u8), empty(R, lf, dtype=u8)
        self.y_perm = empty(R, d, dtype=act)
        self.logits, self.margin = empty(T, E, dtype=f32), empty(T, dtype=f32)
        self.topk_idx, self.topk_gate = empty(T, k, dtype=i32), empty(T, k, dtype=f32)
        self.near_tie_count = empty(1, dtype=i32)
        self.counts, self.offsets = empty(E, dtype=i32), empty(E + 1, dtype=i32)
        self.pos, self.src_token = empty(T, k, dtype=i32), empty(R, dtype=i32)
        few = self._dims(min(max_tokens, self.few_slots // k))
        need = max(L.moe_serve_workspace_bytes(self._dims(max_tokens)),
                   L.moe_token_swiglu_workspace_bytes(few), 256)
        self.workspace = empty(need, dtype=u8)

    def _dims(self, T):
        return L.make_dims(T, self.d, self.E, self.f, self.k, self.act)

    def _few(self, T):
        """Whether T tokens go through moe_token_swiglu.

        It reads an expert's weights once for every 16 of its pairs, of which there are
        at most T, and T k / E on average.  us of a forward, grouped products /
        moe_token_swiglu, bf16: d = 2048, 64 experts of 1024, k = 6: 24 pairs 68 / 54,
        126 pairs 88 / 86, 192 pairs 88 / 90; 8 experts of 2048, k = 2: 64 pairs 59 /
        54, 96 pairs 61 / 71; 4 experts of 1024, k = 4: 64 pairs 52 / 49, 96 pairs 53 /
        62; k = 1: 32 pairs 51 / 46, 64 pairs 52 / 60; d = 256, 16 experts of 256, k =
        4: 128 pairs 32 / 25, 384 pairs 33 / 36; d = 1024, 16 experts of 512, k = 16:
        128 pairs 53 / 40.  An fp32 layer crosses earlier (d = 2048, 64 experts of 1024,
        k = 6: 48 pairs 187 / 176, 96 pairs 200 / 206) but keeps fp32 rows for it."""
        R = T * self.k
        return R <= self.few_slots and (not self.by_expert or T <= 16 or R <= 8 * self.E)

    def load(self, w1, w3, w2):
        """Quantises the expert weights, [E,f,d], [E,f,d] and [E,d,f] in fp32 or bf16
        (until then every y is NaN)."""
        weights = {"w1": w1, "w3": w3, "w2": w2}
        for name, w in weights.items():
            shape = (self.E, self.d, self.f) if name == "w2" else (self.E, self.f, self.d)
            if tuple(w.shape) != shape:
                raise ValueError(f"{name} must be {shape}, is {tuple(w.shape)}")
        for name, w in weights.items():
            L.moe_mx_quantize(w, "e2m1", getattr(self, name), getattr(self, name + "_scale"))

    def forward(self, x, norm_weight, wr, residual=None):
        """x [T,d], T <= max_tokens: (y, stream), the experts' sum for norm(x +
        residual) and x + residual (without one x itself, or a copy of it where x is
        one of the layer's own outputs)."""
        T = x.shape[0]
        if x.dim() != 2 or x.shape[1] != self.d or T > self.T:
            raise ValueError(f"x must be [T, {self.d}] with T <= {self.T}, is {tuple(x.shape)}")
        if tuple(wr.shape) != (self.E, self.d):
            raise ValueError(f"wr must be [{self.E}, {self.d}], is {tuple(wr.shape)}")
        if wr.device != x.device:
            raise ValueError(f"wr must be on {x.device}, is on {wr.device}")
        with torch.cuda.device_of(x):
            return self._forward(x, norm_weight, wr, residual, T)

    def _forward(self, x, norm_weight, wr, residual, T):
        R = T * self.k
        dims, few = self._dims(T), self._few(T)
        xn, y, idx, gate = self.xn[:T], self.y[:T], self.topk_idx[:T], self.topk_gate[:T]
        xq, xs = (None, None) if few else (self.xq[:T], self.x_scale[:T])
        # the stream is x itself without a residual, unless this forward writes there
        total = (self.norm_sum[:T] if residual is not None or _shared(x, xn) or _shared(x, y)
                 else None)
        stream = x if total is None else total
        outs = (xn,) if total is None else (xn, total)
        x, residual = _readable(x, outs), _readable(residual, outs)
        L.moe_rmsnorm(dims, x, residual, norm_weight, self.norm_eps, total, xn, xq, xs, None)
        L.moe_route(dims, xn, wr, self.logits[:T], idx, gate, self.margin[:T], 0.0,
                    self.near_tie_count, 1, None, None, None, self.workspace)
        if few:
            L.moe_token_swiglu(dims, xn, idx, gate, self.w1, self.w1_scale, self.w3,
                               self.w3_scale, self.w2, self.w2_scale, y, self.workspace)
            return y, stream
        L.moe_permute(dims, idx, self.counts, self.offsets, self.pos[:T], self.src_token[:R], None,
                      None, self.workspace)
        hq, hs, y_perm = self.hq[:R], self.h_scale[:R], self.y_perm[:R]
        L.moe_expert_up_mx(dims, xq, xs, self.src_token[:R], self.offsets, self.w1, self.w1_scale,
                           self.w3, self.w3_scale, hq, hs)
        L.moe_expert_down_mx(dims, hq, hs, self.offsets, self.w2, self.w2_scale, y_perm)
        L.moe_combine(dims, y_perm, self.pos[:T], gate, y)
        return y, stream
