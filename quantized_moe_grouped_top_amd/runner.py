"""Device buffers and call sequence of one quantized MoE layer.

Allocates the routing, quantization and output buffers with torch (device
memory only) and runs the hot path as a sequence of library calls on the
current stream:

    routed formats : moe_align_block_size -> [moe_quantize_act] ->
                     moe_grouped_gemm_{fp8w8a8,int8w8a8,int8w8a16,fp8w8a16,int4w4a16} ->
                     moe_combine
    MXFP8          : moe_quantize_act(MXFP8) -> moe_grouped_gemm_mxfp8
    MXFP8 backward : input gradient = the MXFP8 call with the output gradient
                     and MOE_Q_MXFP8_COLWISE weights; weight gradient =
                     moe_quantize_act_colwise (dy, x) -> moe_grouped_gemm_mxfp8_wgrad
    activation     : moe_act_quantize (SwiGLU / SReLU + MXFP8 or fp8)
    general router : moe_route_topk -> moe_align_topk_ids in place of
                     moe_align_block_size; its gradient moe_route_topk_backward
    dense int8     : moe_quantize_act (int8 per token) -> moe_gemm_int8w8a8, e.g.
                     a shared expert added to the routed experts' sum

Every step runs in the library's HIP kernels; nothing here computes.
"""

import torch

from . import (MOE_ACT_SRELU, MOE_ACT_SWIGLU, MOE_BF16, MOE_F16, MOE_F32, MOE_GROUP_MAX,
               MOE_GROUP_TOP2, MOE_Q_FP8_PER_CHANNEL, MOE_Q_FP8_PER_TENSOR,
               MOE_Q_INT4_PER_CHANNEL, MOE_Q_INT8_PER_CHANNEL, MOE_Q_MXFP8, MOE_Q_MXFP8_COLWISE,
               MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MOE_W_FRAG,
               MOE_W_ROWMAJOR,
               MOE_W_TILED, moe_act_quantize, moe_align_block_size, moe_align_max_padded,
               moe_align_topk_ids, moe_align_workspace_bytes, moe_combine, moe_gemm_int8w8a8,
               moe_gemm_int8w8a8_workspace_bytes,
               moe_grouped_gemm_fp8w8a8, moe_grouped_gemm_fp8w8a16, moe_grouped_gemm_int4w4a16,
               moe_grouped_gemm_int8w8a8,
               moe_grouped_gemm_int8w8a16,
               moe_grouped_gemm_mxfp8, moe_grouped_gemm_mxfp8_wgrad, moe_quantize_act_colwise,
               moe_mx_scale_rows, moe_pack_weights, moe_packed_weight_bytes, moe_quantize_act,
               moe_quantize_weights, moe_quantize_workspace_bytes, moe_recommended_block_m,
               moe_route_topk, moe_route_topk_backward)

_DTYPES = {"f32": (MOE_F32, torch.float32), "bf16": (MOE_BF16, torch.bfloat16),
           "f16": (MOE_F16, torch.float16)}


def _empty(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def quantize_weights(w, fmt):
    """Offline weight quantization of float32 w [E, N, K] on its device.
    Returns (w_q, w_scale) for fp8/int8/fp8wo or (w_q, w_sf) for MXFP8."""
    E, N, K = w.shape
    dev = w.device
    if fmt == "fp8":
        q = _empty((E, N, K), torch.uint8, dev)
        s = _empty((E,), torch.float32, dev)
        ws = _empty((moe_quantize_workspace_bytes(MOE_Q_FP8_PER_TENSOR, E),), torch.uint8, dev)
        moe_quantize_weights(w, E, N, K, MOE_Q_FP8_PER_TENSOR, q, s, None, ws)
        return q, s
    if fmt == "int4wo":                  # packed codes [E, N, K/2]
        q = _empty((E, N, K // 2), torch.uint8, dev)
        s = _empty((E, N), torch.float32, dev)
        moe_quantize_weights(w, E, N, K, MOE_Q_INT4_PER_CHANNEL, q, s, None, None)
        return q, s
    if fmt == "fp8wo":
        q = _empty((E, N, K), torch.uint8, dev)
        s = _empty((E, N), torch.float32, dev)
        moe_quantize_weights(w, E, N, K, MOE_Q_FP8_PER_CHANNEL, q, s, None, None)
        return q, s
    if fmt in ("int8", "int8dq"):
        q = _empty((E, N, K), torch.int8, dev)
        s = _empty((E, N), torch.float32, dev)
        moe_quantize_weights(w, E, N, K, MOE_Q_INT8_PER_CHANNEL, q, s, None, None)
        return q, s
    if fmt == "mxfp8":
        q = _empty((E, N, K), torch.uint8, dev)
        sf = _empty((E, N, K // 32), torch.uint8, dev)
        moe_quantize_weights(w, E, N, K, MOE_Q_MXFP8, q, None, sf, None)
        return q, sf
    if fmt == "mxfp8_colwise":           # along N, transposed: [E, K, N]
        q = _empty((E, K, N), torch.uint8, dev)
        sf = _empty((E, K, N // 32), torch.uint8, dev)
        moe_quantize_weights(w, E, N, K, MOE_Q_MXFP8_COLWISE, q, None, sf, None)
        return q, sf
    raise ValueError(fmt)


def pack_weights(w_q, layout=MOE_W_TILED):
    """Packed copy (MOE_W_TILED or MOE_W_FRAG) of one-byte weights [E, N, K]
    on their device."""
    E, N, K = w_q.shape
    out = _empty((moe_packed_weight_bytes(E, N, K, layout),), torch.uint8, w_q.device)
    moe_pack_weights(w_q, E, N, K, layout, out)
    return out


def _rows_of(t, dtype, shape):
    """t holds `shape` values of `dtype` without gaps."""
    return t.dtype == dtype and tuple(t.shape) == shape and t.is_contiguous()


class TopKRouter:
    """General router of fixed (M, E, top_k): softmax or sigmoid scores, an
    optional balance bias, groups, renormalised weights.  `route` fills
    topk_ids / topk_weights; `align` groups the slots of the local experts
    [expert_first, expert_first + n_local) for the grouped GEMMs and leaves
    their loads in expert_counts; `backward` gives the logits' gradient."""

    def __init__(self, M, E, top_k, dtype="f32", score="softmax", n_group=1, topk_group=1,
                 group_rule="max", renormalize=True, scale=1.0, expert_first=0, n_local=None,
                 device="cuda"):
        self.M, self.E, self.top_k = M, E, top_k
        self.dtype, self.torch_dtype = _DTYPES[dtype]
        self.score = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}[score]
        self.n_group, self.topk_group = n_group, topk_group
        self.group_rule = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}[group_rule]
        self.renormalize, self.scale = renormalize, scale
        self.expert_first, self.n_local = expert_first, E if n_local is None else n_local
        self.holds_all = expert_first <= 0 and expert_first + self.n_local >= E
        self.topk_ids = _empty((M, top_k), torch.int32, device)
        self.topk_weights = _empty((M, top_k), torch.float32, device)
        self.expert_counts = _empty((self.n_local,), torch.int32, device)
        self.d_logits = _empty((M, E), self.torch_dtype, device)
        self.ws = _empty((moe_align_workspace_bytes(M, self.n_local, top_k),), torch.uint8, device)

    def route(self, logits, bias=None):
        assert logits.dtype == self.torch_dtype and logits.shape == (self.M, self.E)
        assert logits.stride(1) == 1
        assert bias is None or _rows_of(bias, torch.float32, (self.E,))
        moe_route_topk(logits, self.dtype, logits.stride(0), bias, self.M, self.E, self.top_k,
                       self.score, self.n_group, self.topk_group, self.group_rule,
                       self.renormalize, self.scale, self.topk_ids, self.topk_weights)

    def align(self, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded):
        n = moe_align_max_padded(self.M, self.n_local, self.top_k, block_m)
        for t, least in ((sorted_token_ids, n), (expert_ids, n // block_m),
                         (num_tokens_post_padded, 1)):
            assert t.dtype == torch.int32 and t.is_contiguous() and t.numel() >= least
        moe_align_topk_ids(self.topk_ids, self.M, self.n_local, self.top_k, block_m,
                           self.expert_first, sorted_token_ids, expert_ids,
                           num_tokens_post_padded, self.expert_counts, self.ws)

    def backward(self, d_weights, logits):
        """d_logits [M, E] for d_weights [M, top_k], the choice held fixed."""
        assert logits.dtype == self.torch_dtype and logits.shape == (self.M, self.E)
        assert logits.stride(1) == 1
        assert _rows_of(d_weights, torch.float32, (self.M, self.top_k))
        moe_route_topk_backward(d_weights, self.topk_ids, logits, self.dtype, logits.stride(0),
                                self.M, self.E, self.top_k, self.score, self.renormalize,
                                self.scale, self.d_logits, self.E)
        return self.d_logits


class Int8Linear:
    """Dense int8 W8A8 linear of fixed (M, K, N): bf16 rows quantized per token,
    int8 weights [N, K] with a scale per channel, an optional float32 bias and
    an optional addend of the output's type (which may be the output)."""

    def __init__(self, M, K, N, out="bf16", device="cuda"):
        self.M, self.K, self.N = M, K, N
        self.dtype, self.torch_dtype = _DTYPES[out]
        self.a_q = _empty((M, K), torch.int8, device)
        self.a_scale = _empty((max(M, 1),), torch.float32, device)
        self.ws = _empty((moe_gemm_int8w8a8_workspace_bytes(M, K, N),), torch.uint8, device)
        self.out = _empty((M, N), self.torch_dtype, device)

    def quantize(self, x):
        # M rows of bf16 values, or of their bits as 16-bit integers, without gaps
        assert x.dtype in (torch.bfloat16, torch.int16, torch.uint16)
        assert x.shape[-1] == self.K and x.numel() == self.M * self.K and x.is_contiguous()
        assert x.device == self.a_q.device
        moe_quantize_act(x, self.M, self.K, MOE_Q_INT8_PER_CHANNEL, None, 1, self.a_q,
                         self.a_scale, None, None)

    def gemm(self, w_q, w_scale, bias=None, addend=None, out=None):
        out = self.out if out is None else out
        assert w_q.dtype == torch.int8 and w_q.shape == (self.N, self.K) and w_q.stride(1) == 1
        assert w_scale.dtype == torch.float32 and w_scale.numel() == self.N and w_scale.is_contiguous()
        assert bias is None or _rows_of(bias, torch.float32, (self.N,))
        # the bits of 16-bit values may come as int16
        for t in (out, addend):
            assert t is None or (tuple(t.shape) == (self.M, self.N) and t.is_contiguous() and
                                 (t.dtype == self.torch_dtype or
                                  (t.dtype == torch.int16 and self.dtype == MOE_BF16)))
        moe_gemm_int8w8a8(self.a_q, self.K, self.a_scale, w_q, w_q.stride(0), w_scale, bias, addend,
                          self.M, self.K, self.N, self.dtype, out, self.N, self.ws)
        return out

    def forward(self, x, w_q, w_scale, bias=None, addend=None, out=None):
        self.quantize(x)
        return self.gemm(w_q, w_scale, bias, addend, out)


class RoutedMoE:
    """fp8 W8A8, int8 W8A16 ("int8"), int8 W8A8 with per-token activation
    scales ("int8dq"), bf16 x fp8 weight-only ("fp8wo") or bf16 x int4
    weight-only ("int4wo", block_m 16) MoE layer of fixed (M, K, N, E, top_k).
    Tokens are routed by the fused softmax routing, or by `router` (a
    TopKRouter of the same M and top_k whose local experts are the E here)."""

    def __init__(self, fmt, M, K, N, E, top_k, device="cuda", block_m=None,
                 w_layout=MOE_W_ROWMAJOR, router=None):
        assert fmt in ("fp8", "int8", "int8dq", "fp8wo", "int4wo")
        self.w_layout = w_layout
        self.fmt, self.M, self.K, self.N, self.E, self.top_k = fmt, M, K, N, E, top_k
        self.block_m = block_m or moe_recommended_block_m(M, E, top_k)
        self.max_padded = moe_align_max_padded(M, E, top_k, self.block_m)
        dev = device
        S = M * top_k
        self.router = router
        if router is not None:
            assert (router.M, router.n_local, router.top_k) == (M, E, top_k)
            self.topk_ids, self.topk_weights = router.topk_ids, router.topk_weights
        else:
            self.topk_ids = _empty((M, top_k), torch.int32, dev)
            self.topk_weights = _empty((M, top_k), torch.float32, dev)
        self.sorted_token_ids = _empty((self.max_padded,), torch.int32, dev)
        self.expert_ids = _empty((self.max_padded // self.block_m,), torch.int32, dev)
        self.num_tokens_post_padded = _empty((1,), torch.int32, dev)
        if fmt == "fp8":
            self.a_q = _empty((M, K), torch.uint8, dev)
            self.a_scale = _empty((1,), torch.float32, dev)
            self.ws = _empty((moe_quantize_workspace_bytes(MOE_Q_FP8_PER_TENSOR, 1),),
                             torch.uint8, dev)
        if fmt == "int8dq":
            self.a_q = _empty((M, K), torch.int8, dev)
            self.a_scale = _empty((max(M, 1),), torch.float32, dev)
        self.y = _empty((S, N), torch.int16, dev)      # bf16 bits, one row per slot
        self.out = _empty((M, N), torch.int16, dev)     # bf16 bits

    def route(self, logits, bias=None):
        if self.router is not None:
            self.router.route(logits, bias)
            self.router.align(self.block_m, self.sorted_token_ids, self.expert_ids,
                              self.num_tokens_post_padded)
            if not self.router.holds_all:                # slots of experts elsewhere add nothing
                self.y.zero_()
            return
        assert bias is None, "a balance bias needs a TopKRouter"
        moe_align_block_size(logits, self.M, self.E, self.top_k, self.block_m, self.topk_ids,
                             self.topk_weights, self.sorted_token_ids, self.expert_ids,
                             self.num_tokens_post_padded)

    def quantize(self, x):
        if self.fmt == "fp8":
            moe_quantize_act(x, self.M, self.K, MOE_Q_FP8_PER_TENSOR, None, 1, self.a_q,
                             self.a_scale, None, self.ws)
        elif self.fmt == "int8dq":
            moe_quantize_act(x, self.M, self.K, MOE_Q_INT8_PER_CHANNEL, None, 1, self.a_q,
                             self.a_scale, None, None)

    def gemm(self, x, w_q, w_scale):
        if self.fmt == "fp8":
            moe_grouped_gemm_fp8w8a8(self.a_q, self.a_scale, w_q, w_scale, self.w_layout,
                                     self.sorted_token_ids,
                                     self.expert_ids, self.num_tokens_post_padded,
                                     self.topk_weights, self.M, self.K, self.N, self.E,
                                     self.top_k, self.block_m, self.y)
        elif self.fmt == "int8dq":
            moe_grouped_gemm_int8w8a8(self.a_q, self.a_scale, w_q, w_scale, self.w_layout,
                                      self.sorted_token_ids, self.expert_ids,
                                      self.num_tokens_post_padded, self.topk_weights, self.M,
                                      self.K, self.N, self.E, self.top_k, self.block_m, self.y)
        elif self.fmt == "int4wo":
            moe_grouped_gemm_int4w4a16(x, w_q, w_scale, self.w_layout, self.sorted_token_ids,
                                       self.expert_ids, self.num_tokens_post_padded,
                                       self.topk_weights, self.M, self.K, self.N, self.E,
                                       self.top_k, self.block_m, self.y)
        elif self.fmt == "fp8wo":
            moe_grouped_gemm_fp8w8a16(x, w_q, w_scale, self.w_layout, self.sorted_token_ids,
                                      self.expert_ids, self.num_tokens_post_padded,
                                      self.topk_weights, self.M, self.K, self.N, self.E,
                                      self.top_k, self.block_m, self.y)
        else:
            moe_grouped_gemm_int8w8a16(x, w_q, w_scale, self.w_layout, self.sorted_token_ids,
                                       self.expert_ids,
                                       self.num_tokens_post_padded, self.topk_weights, self.M,
                                       self.K, self.N, self.E, self.top_k, self.block_m, self.y)

    def combine(self):
        moe_combine(self.y, self.M, self.N, self.top_k, self.out)

    def forward(self, x, logits, w_q, w_scale, bias=None, shared=None):
        """One pass of the hot path; returns the bf16 output bits [M, N] (int16).
        `bias`: the router's balance bias; `shared` = (Int8Linear, w_q, w_scale):
        a shared expert of the layer's M, K and N whose product is added to the
        routed experts' sum."""
        if shared is not None:
            linear = shared[0]
            assert (linear.M, linear.K, linear.N) == (self.M, self.K, self.N)
            assert linear.dtype == MOE_BF16
        self.route(logits, bias)
        self.quantize(x)
        self.gemm(x, w_q, w_scale)
        self.combine()
        if shared is not None:
            linear, sh_q, sh_scale = shared
            linear.forward(x, sh_q, sh_scale, addend=self.out, out=self.out)
        return self.out


class MxMoE:
    """MXFP8 grouped linear over expert-concatenated rows."""

    def __init__(self, rows, K, N, E, device="cuda"):
        self.rows, self.K, self.N, self.E = rows, K, N, E
        self.a_q = _empty((rows, K), torch.uint8, device)
        self.a_sf = _empty((moe_mx_scale_rows(rows, E), K // 32), torch.uint8, device)
        self.out = _empty((rows, N), torch.int16, device)

    def quantize(self, x, m_offsets):
        moe_quantize_act(x, self.rows, self.K, MOE_Q_MXFP8, m_offsets, self.E, self.a_q, None,
                         self.a_sf, None)

    def gemm(self, w_q, w_sf, m_offsets):
        moe_grouped_gemm_mxfp8(self.a_q, self.a_sf, w_q, w_sf, m_offsets, self.rows, self.K,
                               self.N, self.E, self.out)

    def forward(self, x, m_offsets, w_q, w_sf):
        self.quantize(x, m_offsets)
        self.gemm(w_q, w_sf, m_offsets)
        return self.out


class MxWgrad:
    """Weight gradient of the MXFP8 grouped linear: columnwise quantization
    of the output gradient dy [rows, N] and the input x [rows, K], then one
    grouped-GEMM launch over every expert into dw [E, N, K] (bf16 bits)."""

    def __init__(self, rows, K, N, E, m_splits, device="cuda"):
        self.rows, self.K, self.N, self.E = rows, K, N, E
        self.m_splits = [int(v) for v in m_splits]
        P = moe_mx_scale_rows(rows, E)
        self.dyT_q = _empty((N * P,), torch.uint8, device)
        self.dyT_sf = _empty((N * P // 32 + 1,), torch.uint8, device)
        self.xT_q = _empty((K * P,), torch.uint8, device)
        self.xT_sf = _empty((K * P // 32 + 1,), torch.uint8, device)
        self.dw = _empty((E, N, K), torch.int16, device)

    def quantize(self, dy, x, m_offsets):
        moe_quantize_act_colwise(dy, self.rows, self.N, m_offsets, self.E, self.dyT_q, self.dyT_sf)
        moe_quantize_act_colwise(x, self.rows, self.K, m_offsets, self.E, self.xT_q, self.xT_sf)

    def gemm(self):
        moe_grouped_gemm_mxfp8_wgrad(self.dyT_q, self.dyT_sf, self.xT_q, self.xT_sf, self.m_splits,
                                     self.E, self.N, self.K, self.dw)


class ActQuant:
    """Fused activation + quantization of expert-concatenated rows: x bf16
    [rows, 2H] (SwiGLU) or [rows, H] (SReLU) -> q [rows, H] e4m3 with MXFP8
    scale bytes (per-expert padded blocks) or one fp8 tensor scale."""

    def __init__(self, rows, H, E, act="swiglu", mode="mxfp8", device="cuda"):
        self.rows, self.H, self.E = rows, H, E
        self.act = {"swiglu": MOE_ACT_SWIGLU, "srelu": MOE_ACT_SRELU}[act]
        self.mode = {"mxfp8": MOE_Q_MXFP8, "fp8": MOE_Q_FP8_PER_TENSOR}[mode]
        self.q = _empty((rows, H), torch.uint8, device)
        self.scale = _empty((1,), torch.float32, device)
        self.sf = self.ws = None
        if self.mode == MOE_Q_MXFP8:
            self.sf = _empty((moe_mx_scale_rows(rows, E), H // 32), torch.uint8, device)
        else:
            self.ws = _empty((moe_quantize_workspace_bytes(MOE_Q_FP8_PER_TENSOR, 1),), torch.uint8,
                             device)

    def __call__(self, x, m_offsets=None):
        moe_act_quantize(x, self.rows, self.H, self.act, self.mode, m_offsets, self.E, self.q,
                         self.scale, self.sf, self.ws)
        return self.q
