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
                     a shared expert added to the routed experts' sum; moe_lora_add
                     adds the adapters of many requests
    16-bit experts : moe_gated_up -> moe_grouped_linear; backward
                     moe_gated_down_backward -> moe_grouped_linear_dgrad and
                     two moe_grouped_linear_wgrad
    block's norms  : moe_norm_residual in place of moe_combine; backward
                     moe_norm_residual_backward

Every step runs in the library's HIP kernels; nothing here computes.
"""

import torch

from . import (MOE_ACT_SRELU, MOE_ACT_SWIGLU, MOE_BF16, MOE_F16, MOE_F32, MOE_GATED_GELU,
               MOE_GATED_SILU, MOE_GATE_CHANNEL, MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GROUP_MAX,
               MOE_GROUP_TOP2, MOE_Q_FP8_PER_CHANNEL, MOE_Q_FP8_PER_TENSOR,
               MOE_Q_INT4_PER_CHANNEL, MOE_Q_INT8_PER_CHANNEL, MOE_Q_MXFP8, MOE_Q_MXFP8_COLWISE,
               MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MOE_W_FRAG,
               MOE_W_ROWMAJOR,
               MOE_W_TILED, moe_act_quantize, moe_align_block_size, moe_align_max_padded,
               moe_align_topk_ids, moe_align_workspace_bytes, moe_combine, moe_gated_down_backward,
               moe_gated_up, moe_gemm_int8w8a8,
               moe_gemm_int8w8a8_workspace_bytes,
               moe_grouped_gemm_fp8w8a8, moe_grouped_gemm_fp8w8a16, moe_grouped_gemm_int4w4a16,
               moe_grouped_gemm_int8w8a8,
               moe_grouped_gemm_int8w8a16,
               moe_grouped_gemm_mxfp8, moe_grouped_gemm_mxfp8_wgrad, moe_grouped_linear,
               moe_grouped_linear_dgrad, moe_grouped_linear_wgrad, moe_lora_add,
               moe_lora_workspace_bytes, moe_norm_backward_workspace_bytes, moe_norm_residual,
               moe_norm_residual_backward, moe_quantize_act_colwise,
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


def _row_distance(t):
    """Elements from a row of t to the next; of a single row its length, whatever
    stride it has."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


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

    def forward(self, x, w_q, w_scale, bias=None, addend=None, out=None, lora=None):
        """`lora` = (LoraAdapters, a, b, scales, ranks): the adapters' contribution,
        taken of the unquantized x, is added to the product."""
        if lora is not None:
            adapters, a, b, scales, ranks = lora
            assert adapters.T == self.M and adapters.dtype == MOE_BF16
            adapters.check(x, a, b, self.out if out is None else out, scales, ranks)
        self.quantize(x)
        out = self.gemm(w_q, w_scale, bias, addend, out)
        if lora is not None:
            adapters.add(x, a, b, out, out, scales, ranks)
        return out


class LoraAdapters:
    """Low-rank adapters of many requests beside shared projections: T tokens, L
    adapters of rank R at most, inputs of K features at most.  `plan` groups the
    tokens by adapter, once for all projections of a step; `add` adds
    scales[a] b[a] (a[a] x_t) to a projection's output (int16: the bits of bf16
    values)."""

    _OUT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16,
            torch.int16: MOE_BF16}

    def __init__(self, T, K, R, L, dtype="bf16", block_m=None, device="cuda"):
        self.T, self.K, self.R, self.L = T, K, R, L
        self.dtype, self.torch_dtype = _DTYPES[dtype]
        # Smaller blocks leave less of them empty, larger ones read an adapter's matrices less
        # often.  us with 16 / 32 / 64 / 128, 12 requests on 8 adapters of rank 64 and 4096 ->
        # 14336, and 64 on 32: 64 tokens 10.7 / 11.5 / 12.3 / 14.3 and 15.2 / 15.7 / 18.3 / 24.4;
        # 256 tokens 19.2 / 16.7 / 16.6 / 18.8 and 22.6 / 22.5 / 25.6 / 32.3; 1280 tokens 46.1 /
        # 34.9 / 33.1 / 33.6 and 53.9 / 40.1 / 43.3 / 49.5; 1700 tokens 53.9 / 40.6 / 37.7 / 37.8
        # and 61.7 / 50.8 / 46.7 / 54.2; 16384 tokens 460 / 320 / 278 / 276 and 471 / 336 / 291 / 283.
        self.block_m = block_m or (16 if T < 256 else 32 if T < 1536 else 64)
        n = moe_align_max_padded(T, L, 1, self.block_m)
        self.adapter_ids = _empty((T, 1), torch.int32, device)
        self.sorted_token_ids = _empty((n,), torch.int32, device)
        self.expert_ids = _empty((n // self.block_m,), torch.int32, device)
        self.num_tokens_post_padded = _empty((1,), torch.int32, device)
        self.align_ws = _empty((moe_align_workspace_bytes(T, L, 1),), torch.uint8, device)
        self.ws = _empty((moe_lora_workspace_bytes(T, K, R, L, self.block_m),), torch.uint8, device)

    def plan(self, adapter_ids):
        """adapter_ids [T] int32, outside [0, L) for a token without an adapter."""
        assert adapter_ids.dtype == torch.int32 and adapter_ids.numel() == self.T
        self.adapter_ids.copy_(adapter_ids.view(self.T, 1))
        moe_align_topk_ids(self.adapter_ids, self.T, self.L, 1, self.block_m, 0,
                           self.sorted_token_ids, self.expert_ids, self.num_tokens_post_padded,
                           None, self.align_ws)

    def check(self, x, a, b, out, scales=None, ranks=None):
        K, N = a.shape[2], b.shape[1]
        # the bits of bf16 values may come as 16-bit integers
        assert x.dtype == self.torch_dtype or (self.dtype == MOE_BF16 and
                                               x.dtype in (torch.int16, torch.uint16))
        assert tuple(x.shape) == (self.T, K) and K <= self.K and x.stride(1) == 1
        assert _rows_of(a, self.torch_dtype, (self.L, self.R, K))
        assert _rows_of(b, self.torch_dtype, (self.L, N, self.R))
        assert tuple(out.shape) == (self.T, N) and out.stride(1) == 1 and out.dtype in self._OUT
        assert scales is None or _rows_of(scales, torch.float32, (self.L,))
        assert ranks is None or _rows_of(ranks, torch.int32, (self.L,))

    def add(self, x, a, b, out, addend=None, scales=None, ranks=None):
        """out = addend + the adapters' part; `addend` may be out (or None: 0)."""
        self.check(x, a, b, out, scales, ranks)
        assert addend is None or (addend.dtype == out.dtype and addend.shape == out.shape and
                                  addend.stride(1) == 1 and
                                  _row_distance(addend) == _row_distance(out))
        # a workspace for K features holds that of fewer
        K, N = a.shape[2], b.shape[1]
        moe_lora_add(x, _row_distance(x), a, b, ranks, scales, self.dtype, self.adapter_ids,
                     self.sorted_token_ids, self.expert_ids, self.num_tokens_post_padded, self.T, K,
                     N, self.R, self.L, self.block_m, addend, self._OUT[out.dtype], out,
                     _row_distance(out), self.ws)
        return out


class GatedFFN:
    """Gated feed-forward of E experts in 16 bits over expert-concatenated rows:
    x [rows, K] -> y [rows, K] through w_up [E, 2H, K] (gate, then up) and w_down
    [E, K, H].  With `train` the forward pass keeps what `backward` reads."""

    def __init__(self, rows, K, H, E, dtype="bf16", act="silu", train=False, dw="same",
                 device="cuda"):
        self.rows, self.K, self.H, self.E = rows, K, H, E
        self.dtype, self.torch_dtype = _DTYPES[dtype]
        assert self.dtype != MOE_F32
        self.act = {"silu": MOE_GATED_SILU, "gelu": MOE_GATED_GELU}[act]
        t = self.torch_dtype
        self.h = _empty((rows, H), t, device)
        self.y = _empty((rows, K), t, device)
        self.gu = None
        if train:
            self.dw_dtype, dw_t = (MOE_F32, torch.float32) if dw == "f32" else (self.dtype, t)
            self.gu = _empty((rows, 2 * H), t, device)
            self.dgu = _empty((rows, 2 * H), t, device)
            self.dx = _empty((rows, K), t, device)
            self.dw_up = _empty((E, 2 * H, K), dw_t, device)
            self.dw_down = _empty((E, K, H), dw_t, device)

    def _check(self, x, w_up, w_down, m_offsets):
        t = self.torch_dtype
        assert x.dtype == t and tuple(x.shape) == (self.rows, self.K) and x.stride(1) == 1
        assert _rows_of(w_up, t, (self.E, 2 * self.H, self.K))
        assert _rows_of(w_down, t, (self.E, self.K, self.H))
        assert m_offsets is None or _rows_of(m_offsets, torch.int32, (self.E + 1,))

    def forward(self, x, w_up, w_down, m_offsets=None):
        self._check(x, w_up, w_down, m_offsets)
        moe_gated_up(x, _row_distance(x), w_up, self.dtype, m_offsets, self.rows, self.K, self.H, self.E,
                     self.act, self.gu, self.h)
        moe_grouped_linear(self.h, self.H, w_down, self.dtype, m_offsets, self.rows, self.H, self.K,
                           self.E, self.y, self.K)
        return self.y

    def backward(self, dy, x, w_up, w_down, m_offsets=None):
        """(dx, dw_up, dw_down) of the forward pass before."""
        self._check(x, w_up, w_down, m_offsets)
        assert self.gu is not None, "GatedFFN(train=True) keeps what the gradient needs"
        assert dy.dtype == self.torch_dtype and tuple(dy.shape) == (self.rows, self.K)
        assert dy.stride(1) == 1
        rows, K, H, E, t = self.rows, self.K, self.H, self.E, self.dtype
        # h is there from the forward pass
        moe_gated_down_backward(dy, _row_distance(dy), w_down, self.gu, t, m_offsets, rows, K, H, E,
                                self.act, self.dgu, None)
        moe_grouped_linear_dgrad(self.dgu, 2 * H, w_up, t, m_offsets, rows, K, 2 * H, E, self.dx, K)
        moe_grouped_linear_wgrad(self.dgu, 2 * H, x, _row_distance(x), t, m_offsets, rows, K, 2 * H, E,
                                 self.dw_dtype, self.dw_up)
        moe_grouped_linear_wgrad(dy, _row_distance(dy), self.h, H, t, m_offsets, rows, H, K, E,
                                 self.dw_dtype, self.dw_down)
        return self.dx, self.dw_up, self.dw_down


class BlockNorm:
    """What follows a block and precedes the next, for M tokens of N features:
    combine of the top_k slots, norm after the block, gate, residual, next norm."""

    def __init__(self, M, N, top_k=1, dtype="bf16", r_dtype=None, gate="none", alpha=1.0, beta=1.0,
                 eps=1e-6, train=False, device="cuda"):
        self.M, self.N, self.top_k = M, N, top_k
        self.dtype, self.torch_dtype = _DTYPES[dtype]
        self.r_dtype, self.r_torch_dtype = _DTYPES[r_dtype or dtype]
        self.gate_kind = {"none": MOE_GATE_NONE, "channel": MOE_GATE_CHANNEL,
                          "token": MOE_GATE_TOKEN}[gate]
        self.gate_size = {"none": None, "channel": (N,), "token": (M,)}[gate]
        self.alpha, self.beta, self.eps = alpha, beta, eps
        self.r = _empty((M, N), self.r_torch_dtype, device)
        self.h = _empty((M, N), self.torch_dtype, device)
        self.rstd_post = self.rstd_pre = None
        if train:
            self.rstd_post = _empty((M,), torch.float32, device)
            self.rstd_pre = _empty((M,), torch.float32, device)
            self.d_residual = _empty((M, N), self.r_torch_dtype, device)
            self.d_y = _empty((M, N), self.torch_dtype, device)
            self.d_w_post = _empty((N,), torch.float32, device)
            self.d_w_pre = _empty((N,), torch.float32, device)
            self.d_gate = _empty(self.gate_size or (0,), torch.float32, device)
            self.ws = _empty((moe_norm_backward_workspace_bytes(M, N),), torch.uint8, device)

    def check(self, y, residual, w_pre, w_post, gate):
        M, N = self.M, self.N
        # the grouped GEMMs leave the bits of bf16 values as int16
        assert y is None or _rows_of(y, self.torch_dtype, (M * self.top_k, N)) or (
            self.dtype == MOE_BF16 and _rows_of(y, torch.int16, (M * self.top_k, N)))
        assert residual is None or _rows_of(residual, self.r_torch_dtype, (M, N))
        for w in (w_pre, w_post):
            assert w is None or _rows_of(w, torch.float32, (N,))
        assert (gate is None) == (self.gate_size is None)
        assert gate is None or _rows_of(gate, torch.float32, self.gate_size)

    def forward(self, y, residual, w_pre=None, w_post=None, gate=None):
        """(r, h): the new residual and, with w_pre, the next block's input."""
        self.check(y, residual, w_pre, w_post, gate)
        h = None if w_pre is None else self.h
        moe_norm_residual(y, self.dtype, self.top_k, residual, self.r_dtype, w_post, gate,
                          self.gate_kind, self.alpha, self.beta, w_pre, self.eps, self.M, self.N,
                          self.r, h, None if w_post is None else self.rstd_post,
                          None if w_pre is None else self.rstd_pre)
        return self.r, h

    def backward(self, d_r, d_h, y, w_pre=None, w_post=None, gate=None):
        """(d_residual, d_y, d_w_pre, d_w_post, d_gate) of the forward pass before,
        None for what it did not have; d_y [M, N] is the gradient of each slot."""
        self.check(y, None, w_pre, w_post, gate)
        assert self.rstd_pre is not None, "BlockNorm(train=True) keeps what the gradient needs"
        assert d_r is None or _rows_of(d_r, self.r_torch_dtype, (self.M, self.N))
        assert d_h is None or _rows_of(d_h, self.torch_dtype, (self.M, self.N))
        d_y = None if y is None else self.d_y
        d_w_pre = None if w_pre is None else self.d_w_pre
        d_w_post = None if w_post is None else self.d_w_post
        d_gate = None if gate is None else self.d_gate
        moe_norm_residual_backward(d_r, d_h, y, self.dtype, self.top_k, self.r, self.r_dtype, w_post,
                                   gate, self.gate_kind, self.alpha, self.beta, w_pre,
                                   self.rstd_post, self.rstd_pre, self.M, self.N, self.d_residual,
                                   d_y, d_w_post, d_gate, d_w_pre, self.ws)
        return self.d_residual, d_y, d_w_pre, d_w_post, d_gate


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

    def forward(self, x, logits, w_q, w_scale, bias=None, shared=None, norm=None):
        """One pass of the hot path; returns the bf16 output bits [M, N] (int16).
        `bias`: the router's balance bias; `shared` = (Int8Linear, w_q, w_scale):
        a shared expert of the layer's M, K and N whose product is added to the
        routed experts' sum.  `norm` = (BlockNorm, residual, w_pre, w_post, gate):
        the norm after the layer, gate, residual and next norm, and their (r, h) is
        returned; without a shared expert (top_k of the BlockNorm that of the layer)
        it takes the place of the combine, with one (top_k 1) it follows the sum.
        A layer that holds part of the experts takes no norm: it needs the sum of all."""
        if norm is not None:
            assert self.router is None or self.router.holds_all
            block, norm_args = norm[0], norm[1:]
            assert (block.M, block.N, block.dtype) == (self.M, self.N, MOE_BF16)
            assert block.top_k == (1 if shared is not None else self.top_k)
            block.check(self.out if shared is not None else self.y, *norm_args)
        if shared is not None:
            linear = shared[0]
            assert (linear.M, linear.K, linear.N) == (self.M, self.K, self.N)
            assert linear.dtype == MOE_BF16
        self.route(logits, bias)
        self.quantize(x)
        self.gemm(x, w_q, w_scale)
        if norm is not None and shared is None:
            return block.forward(self.y, *norm_args)
        self.combine()
        if shared is not None:
            linear, sh_q, sh_scale = shared
            linear.forward(x, sh_q, sh_scale, addend=self.out, out=self.out)
        return self.out if norm is None else block.forward(self.out, *norm_args)


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
