/*
 * moe_block.h - the block around a Mixture-of-Experts layer (included by moe.h):
 * the experts' gated feed-forward in 16 bits with its gradients, low-rank
 * adapters of many requests beside a shared projection, and the norms before and
 * after the block fused with the combine of the routed slots, the block's gate
 * and the residual.  The conventions of moe.h hold: device pointers owned by the
 * caller, work only enqueued on `stream`, nothing allocated, arguments checked on
 * the host before anything is enqueued, the same status codes and messages.
 * Element types are MOE_F32, MOE_BF16 and MOE_F16 of moe_layer.h.
 */
#ifndef QMOE_MOE_BLOCK_H
#define QMOE_MOE_BLOCK_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- activations of the gate projection -------------------------------------- */
#define MOE_GATED_SILU 0  /* act(g) = g / (1 + exp(-g)) */
#define MOE_GATED_GELU 1  /* act(g) = g (1 + tanh(c (g + 0.044715 g^3))) / 2, c = sqrt(2/pi) */

/* ---- the block's gate (moe_norm_residual) --------------------------------------- */
#define MOE_GATE_NONE    0
#define MOE_GATE_CHANNEL 1  /* gate [N] */
#define MOE_GATE_TOKEN   2  /* gate [M] */

/* ---- limits --------------------------------------------------------------------- */
#define MOE_MAX_BLOCK_ROWS   (1 << 24) /* rows of the grouped products */
#define MOE_MAX_BLOCK_WIDTH  (1 << 20) /* K, N, 2H and row distances of them */
#define MOE_MAX_LORA_RANK    128       /* R */
#define MOE_MAX_NORM_COLUMNS 16384     /* N of the norms */
#define MOE_MAX_NORM_ROWS    (1 << 24) /* M * top_k of the norms */
#define MOE_MAX_NORM_VALUES  (1ll << 35) /* M * N of the norms */

/* ======================================================================== *
 * Gated feed-forward of the experts, 16 bits
 * ======================================================================== */

/* Shared by the five functions below.  dtype is MOE_BF16 or MOE_F16, of every
 * 16-bit array.  m_offsets [E + 1] (device, int32, non-decreasing) gives expert e
 * the rows m_offsets[e] .. m_offsets[e + 1] - 1 of the expert-concatenated arrays;
 * NULL stands for one expert (E = 1) with all rows.  Offsets are read on the
 * device; values outside [0, rows] count as the nearer end.  Rows that belong to
 * no expert are neither read nor written.  Sums are float32, on the matrix cores;
 * every output is rounded once, to nearest even.  The order of a sum hangs on the
 * call's sizes and the expert's place: the same call repeats bit by bit, a row in
 * another call agrees within the error of its float32 sum.
 *
 * Limits: 0 <= rows <= MOE_MAX_BLOCK_ROWS, 1 <= E <= MOE_MAX_EXPERTS; K, N and H
 * multiples of 8, at most MOE_MAX_BLOCK_WIDTH (2 H too); row distances (elements,
 * >= the row) multiples of 8, at most MOE_MAX_BLOCK_WIDTH; pointers 16-byte
 * aligned. */

/* Both projections, the activation and the product:
 *     g = x w[e, :H]^T,  u = x w[e, H:]^T,  h = act(g) * u
 *   x  [rows, K], rows ldx apart     w  [E, 2H, K], the gate's rows first
 *   gu [rows, 2H] = [g | u], what moe_gated_down_backward reads; or NULL
 *   h  [rows, H], of the unrounded g and u */
int moe_gated_up(const void *x, long long ldx, const void *w, int dtype, const int *m_offsets,
                 int rows, int K, int H, int E, int act, void *gu, void *h, hipStream_t stream);

/* y = x w[e]^T (the projection back down, or any linear of the experts).
 *   x [rows, K], rows ldx apart;  w [E, N, K];  y [rows, N], rows ldy apart */
int moe_grouped_linear(const void *x, long long ldx, const void *w, int dtype,
                       const int *m_offsets, int rows, int K, int N, int E, void *y,
                       long long ldy, hipStream_t stream);

/* Gradient of y = h w[e]^T, h = act(g) * u, with respect to g and u:
 *     dh = dy w[e],  dg = dh u act'(g),  du = dh act(g)
 * dh stays unrounded and is not stored.  For an infinite g (one that left the
 * type's range in moe_gated_up) act and act' are their limits: 0 and 0 at -inf, inf
 * and 1 at inf.
 *   dy [rows, N], rows lddy apart;  w [E, N, H];  gu [rows, 2H]
 *   dgu [rows, 2H] = [dg | du]; may be gu itself
 *   h [rows, H], act(g) * u once more for w's gradient; or NULL */
int moe_gated_down_backward(const void *dy, long long lddy, const void *w, const void *gu,
                            int dtype, const int *m_offsets, int rows, int N, int H, int E,
                            int act, void *dgu, void *h, hipStream_t stream);

/* Input gradient of moe_grouped_linear: dx = dy w[e].
 *   dy [rows, N], rows lddy apart;  w [E, N, K];  dx [rows, K], rows lddx apart */
int moe_grouped_linear_dgrad(const void *dy, long long lddy, const void *w, int dtype,
                             const int *m_offsets, int rows, int K, int N, int E, void *dx,
                             long long lddx, hipStream_t stream);

/* Weight gradient of moe_grouped_linear: dw[e] = dy_e^T x_e, 0 for an expert
 * without rows.
 *   dy [rows, N], rows lddy apart;  x [rows, K], rows ldx apart
 *   dw [E, N, K] of type dw_dtype: dtype or MOE_F32 */
int moe_grouped_linear_wgrad(const void *dy, long long lddy, const void *x, long long ldx,
                             int dtype, const int *m_offsets, int rows, int K, int N, int E,
                             int dw_dtype, void *dw, hipStream_t stream);

/* ======================================================================== *
 * Low-rank adapters of many requests
 * ======================================================================== */

/* Bytes of device workspace moe_lora_add needs; 0 for invalid sizes. */
size_t moe_lora_workspace_bytes(int T, int K, int R, int L, int block_m);

/* The contribution of every token's adapter, added to a shared projection's
 * output (of moe_gemm_int8w8a8, of a grouped product, ...):
 *     out_t = addend_t + scales[a] * b[a, :, :r] (a[a, :r] x_t),
 *     a = adapter_ids[t], r = ranks[a]
 * and out_t = addend_t for a token without an adapter (an id outside [0, L)).
 * The tokens grouped by adapter come from moe_align_topk_ids(adapter_ids, T, L,
 * 1, block_m, 0, ...), once for all the projections of a step.  Rows of a and
 * columns of b from r on are not used, whatever they hold.  The inner vector
 * a x_t is float32 and enters the second product in two 16-bit parts (2^-16 of
 * its value is left out at most; three parts where out is float32, 2^-24).  In
 * fp16 up to 2^-39 of the token's largest inner value is left out of each besides,
 * which is less down to values of 2^-23 (float32: 2^-15) of the largest.
 * Infinities of x, a and b count as in the definition (an inner value that is left
 * out whole as a 0).  The result is rounded once.
 *
 *   x       [T, K] of type dtype (MOE_BF16, MOE_F16), rows ldx elements apart
 *   a       [L, R, K], b [L, N, R] of type dtype
 *   ranks   [L] int32 (below 0 counts as 0, above R as R), or NULL: all R
 *   scales  [L] float32, or NULL: 1
 *   adapter_ids [T] int32; read for the tokens without an adapter only, and not
 *           at all where addend is out
 *   sorted_token_ids, expert_ids, num_tokens_post_padded: the alignment
 *   addend  [T, N] of type out_dtype (MOE_F32, MOE_BF16, MOE_F16), rows ldo
 *           apart like out's; may be out itself; NULL: 0
 *   out     [T, N] of type out_dtype
 *   workspace moe_lora_workspace_bytes(T, K, R, L, block_m) bytes, 16-byte
 *           aligned, contents on entry ignored, one for each call that may run at
 *           the same time
 * Limits: 0 <= T <= MOE_MAX_SLOTS, 1 <= L <= MOE_MAX_EXPERTS, K, N and R multiples
 * of 8, K and N at most MOE_MAX_BLOCK_WIDTH, R <= MOE_MAX_LORA_RANK, row
 * distances multiples of 8, at most MOE_MAX_BLOCK_WIDTH; x, a, b, addend and out
 * 16-byte aligned; block_m as for moe_align_topk_ids. */
int moe_lora_add(const void *x, long long ldx, const void *a, const void *b, const int *ranks,
                 const float *scales, int dtype, const int *adapter_ids,
                 const int *sorted_token_ids, const int *expert_ids,
                 const int *num_tokens_post_padded, int T, int K, int N, int R, int L,
                 int block_m, const void *addend, int out_dtype, void *out, long long ldo,
                 void *workspace, hipStream_t stream);

/* ======================================================================== *
 * The norms before and after a block, its gate and the residual
 * ======================================================================== */

/* What follows a block and precedes the next, in one pass over the rows:
 *     s = sum_j y[t * top_k + j]                    (the combine of the slots)
 *     p = w_post * s / sqrt(mean(s^2) + eps)        (without w_post: s)
 *     r = alpha * residual + beta * gate * p
 *     h = w_pre * r / sqrt(mean(r^2) + eps)
 * All of it is float32; r and h are rounded once, h is taken of the unrounded r.
 *
 *   y        [M * top_k, N] of type dtype (MOE_BF16, MOE_F16): per-slot results of
 *            the grouped GEMMs, or a block's output (top_k = 1); NULL: no block
 *            before this norm (r = alpha * residual)
 *   residual [M, N] of type r_dtype (dtype or MOE_F32), or NULL: 0
 *   w_post   [N] float32, or NULL
 *   gate     float32 as gate_kind says, NULL for MOE_GATE_NONE
 *   w_pre    [N] float32, or NULL: h is not computed
 *   r        [M, N] of type r_dtype, written; may be residual itself
 *   h        [M, N] of type dtype, written (with w_pre); may be y if top_k = 1
 *   rstd_post, rstd_pre  [M] float32: 1 / sqrt(mean + eps) of both norms, written
 *            for the backward pass; NULL where not wanted
 * Limits: N a multiple of 8, at most MOE_MAX_NORM_COLUMNS; 0 <= M, 1 <= top_k <=
 * MOE_MAX_TOPK, M * top_k <= MOE_MAX_NORM_ROWS, M * N <= MOE_MAX_NORM_VALUES; eps
 * >= 0; all arrays of M x N values, both weights and a channel gate 16-byte
 * aligned.  With M = 0 nothing is done, whichever pointers are NULL. */
int moe_norm_residual(const void *y, int dtype, int top_k, const void *residual, int r_dtype,
                      const float *w_post, const float *gate, int gate_kind, float alpha,
                      float beta, const float *w_pre, float eps, int M, int N, void *r, void *h,
                      float *rstd_post, float *rstd_pre, hipStream_t stream);

/* Bytes of device workspace moe_norm_residual_backward needs (partial sums of the
 * weights' gradients); 0 for invalid sizes. */
size_t moe_norm_backward_workspace_bytes(int M, int N);

/* Gradients of moe_norm_residual from those of r (d_r) and h (d_h), with the r
 * and the factors that it wrote:
 *     n = r rstd_pre,  d = d_h * w_pre
 *     dr = d_r + rstd_pre (d - n mean(d n)),          d_w_pre = sum_t d_h n
 *     d_residual = alpha dr,  dp = beta gate dr,      d_gate = sum beta dr p
 *     m = s rstd_post,  d = dp * w_post:
 *     d_y = rstd_post (d - m mean(d m)),              d_w_post = sum_t dp m
 * (d_y = dp without w_post; dr = d_r without w_pre).  Sums over tokens are float32
 * in an order fixed by M and N: results repeat bit by bit.
 *
 *   d_r  [M, N] of type r_dtype, or NULL: 0;  d_h [M, N] of type dtype, NULL
 *        without w_pre
 *   y, top_k, w_post, gate, gate_kind, alpha, beta, w_pre, r as in the forward
 *        call (y NULL: no block, nothing of it is computed)
 *   d_residual [M, N] of type r_dtype, written, or NULL; may be d_r
 *   d_y  [M, N] of type dtype, written (with y): the gradient of each of a
 *        token's top_k slots
 *   d_w_post [N], d_gate ([N] or [M]), d_w_pre [N] float32, written, each NULL
 *        where not wanted
 *   workspace moe_norm_backward_workspace_bytes(M, N) bytes, 16-byte aligned,
 *        contents on entry ignored, one for each call that may run at the same time
 * Limits as for moe_norm_residual.  With M = 0 the gradients of the weights and of a
 * channel gate become 0, whichever other pointers are NULL. */
int moe_norm_residual_backward(const void *d_r, const void *d_h, const void *y, int dtype,
                               int top_k, const void *r, int r_dtype, const float *w_post,
                               const float *gate, int gate_kind, float alpha, float beta,
                               const float *w_pre, const float *rstd_post,
                               const float *rstd_pre, int M, int N, void *d_residual,
                               void *d_y, float *d_w_post, float *d_gate, float *d_w_pre,
                               void *workspace, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QMOE_MOE_BLOCK_H */
