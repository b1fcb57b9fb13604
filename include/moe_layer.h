/*
 * moe_layer.h - the parts of a Mixture-of-Experts layer around the grouped
 * GEMMs of moe.h (which includes this file): the general router with its
 * gradient, the block alignment of choices made elsewhere, and the dense int8
 * product of the layers beside the experts (a shared expert, a dense
 * projection).  The conventions of moe.h hold: device pointers owned by the
 * caller, work only enqueued on `stream`, nothing allocated, arguments checked
 * on the host before anything is enqueued, the same status codes and error
 * messages.
 */
#ifndef QMOE_MOE_LAYER_H
#define QMOE_MOE_LAYER_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types of logits, gradients and int8 product outputs ---------- */
#define MOE_F32  0
#define MOE_BF16 1
#define MOE_F16  2

/* ---- router scores and group scores ---------------------------------------- */
#define MOE_SCORE_SOFTMAX 0  /* s_e = exp(x_e) / sum over all E of exp(x) */
#define MOE_SCORE_SIGMOID 1  /* s_e = 1 / (1 + exp(-x_e)) */
#define MOE_GROUP_MAX  0     /* a group counts as much as its best expert */
#define MOE_GROUP_TOP2 1     /* ... as its two best experts together */

/* ---- limits ------------------------------------------------------------------ */
#define MOE_MAX_ROUTE_EXPERTS 512     /* E of the router (one call of the grouped GEMMs
                                         takes MOE_MAX_EXPERTS of them: see expert_first
                                         of moe_align_topk_ids) */
#define MOE_MAX_ROUTE_GROUPS  64      /* n_group */
#define MOE_MAX_ROUTE_TOKENS  (1 << 25)  /* M of the router lies below (one launch) */
#define MOE_MAX_INT8_K        131071  /* K of the int8 product: |sum| <= 128*128*K < 2^31 */
#define MOE_MAX_INT8_ROWS     (1 << 27)  /* M of the int8 product lies below, M * N below
                                         2^36 (one launch) */

/* ======================================================================== *
 * Routing: scores, balance bias, groups, top-k, renormalised weights
 * ======================================================================== */

/* Chooses top_k of E experts for every token.  For token t, in order:
 *   scores   s_e from the logits x_e (MOE_SCORE_*)
 *   keys     k_e = s_e + bias[e], -inf where the logit is -inf; without a bias
 *            the logits themselves (the same order, without its rounding)
 *   groups   the E experts are n_group groups of E / n_group neighbours; a
 *            group counts as its largest key (MOE_GROUP_MAX) or as the sum of
 *            its two largest keys, without a bias its two largest scores
 *            (MOE_GROUP_TOP2; a masked expert counts -inf beside a bias, its
 *            score 0 without one); the topk_group best groups stay (on equal
 *            counts the lower group), experts of the others are never chosen.
 *            n_group = topk_group = 1: no groups
 *   choice   the top_k largest keys of those experts, largest first (on equal
 *            keys the lower expert)
 *   weights  w_j = s of the j-th choice (the bias only steers the choice); if
 *            renormalize, divided by their sum (a token whose chosen scores
 *            are all 0 gets weights 0); times scale
 *
 * Keys that rest on scores are computed in float64 and hold about 2^-40: of
 * two keys nearer than that either may come first (equal logits with equal
 * biases are exactly equal); what groups count is rounded to 38 bits.  Weights
 * are computed in float64 and rounded once to float32.
 * A logit or bias of -inf masks an expert: it is chosen only where fewer than
 * top_k others are left in the groups that stay, and a -inf logit, which masks
 * whatever the expert's bias, has score 0 (in a token without any other logit
 * every softmax score is 0).  A NaN key precedes every number, +inf the finite
 * keys; a NaN or +inf logit makes the softmax scores of its token, and so its
 * weights, NaN.  ids are distinct and inside [0, E) whatever the logits hold.
 *
 *   logits       [M, E] of type dtype (MOE_F32, MOE_BF16, MOE_F16), rows ld
 *                elements apart (ld >= E), aligned to their type
 *   bias         [E] float32, or NULL
 *   topk_ids     [M, top_k] int32, written
 *   topk_weights [M, top_k] float32, written
 *
 * Limits: 1 <= E <= MOE_MAX_ROUTE_EXPERTS, 1 <= top_k <= min(E, MOE_MAX_TOPK),
 * n_group <= MOE_MAX_ROUTE_GROUPS divides E, 1 <= topk_group <= n_group,
 * topk_group * (E / n_group) >= top_k, MOE_GROUP_TOP2 with n_group > 1 needs
 * two experts in a group, 0 <= M < MOE_MAX_ROUTE_TOKENS. */
int moe_route_topk(const void *logits, int dtype, long long ld, const float *bias, int M, int E,
                   int top_k, int score, int n_group, int topk_group, int group_rule,
                   int renormalize, float scale, int *topk_ids, float *topk_weights,
                   hipStream_t stream);

/* Gradient of the weights of moe_route_topk with respect to the logits, the
 * choice held fixed (the bias, which only steers the choice, has none).  With
 * g_j = d_weights[t, j], chosen scores s_j and S their sum:
 *   renormalised sigmoid   c = scale / S, u = sum_j g_j s_j / S:
 *                          dx_j = c (g_j - u) s_j (1 - s_j)
 *   plain sigmoid          dx_j = scale g_j s_j (1 - s_j)
 *   renormalised softmax   q = softmax over the chosen logits:
 *                          dx_j = scale q_j (g_j - sum_i g_i q_i)
 *   plain softmax          dx_e = scale p_e (g_e [e chosen] - sum_i g_i p_i)
 * and 0 for every other expert: d_logits is written in full, in the type of
 * the logits.  The scores are computed again from the logits: in float64 where
 * only the chosen ones count, in float32 for the plain softmax; where one score
 * is nearly all of the sum its difference to the weighted mean is taken over the
 * others alone, so that it holds relative to what is left.
 * Ids outside [0, E) are no choice: they take no part.  An id that stands
 * twice in a token counts twice, in the sums and in its gradient.  A token
 * whose chosen scores are all 0 gets gradient 0.
 *
 *   d_weights [M, top_k] float32; topk_ids [M, top_k] int32
 *   logits    [M, E] of type dtype, rows ld elements apart
 *   d_logits  [M, E] of type dtype, rows ldd elements apart (ldd >= E);
 *             elements between the rows are not touched; may be logits itself
 *             (with ldd = ld), but not overlap it otherwise
 * E, top_k and M as for moe_route_topk. */
int moe_route_topk_backward(const float *d_weights, const int *topk_ids, const void *logits,
                            int dtype, long long ld, int M, int E, int top_k, int score,
                            int renormalize, float scale, void *d_logits, long long ldd,
                            hipStream_t stream);

/* ======================================================================== *
 * Block alignment of given ids
 * ======================================================================== */

/* Bytes of device workspace moe_align_topk_ids needs:
 * ceil(M * top_k / 1024) * E * 4.  0 for invalid sizes. */
size_t moe_align_workspace_bytes(int M, int E, int top_k);

/* The alignment of moe_align_block_size for choices made elsewhere
 * (moe_route_topk, another device's router): slot i = t * top_k + j belongs to
 * local expert topk_ids[i] - expert_first if that lies in [0, E), and is left
 * out otherwise (an expert of another device, a dropped token).  The E local
 * experts are those the following grouped GEMMs hold.  sorted_token_ids,
 * expert_ids (local numbers) and num_tokens_post_padded are written as by
 * moe_align_block_size; a grouped GEMM then leaves the rows of y that belong
 * to left-out slots as they are.
 *
 *   topk_ids      [M, top_k] int32, read
 *   expert_counts [E] int32, written: slots of every local expert (the loads a
 *                 balance bias is adjusted by); or NULL
 *   workspace     moe_align_workspace_bytes(M, E, top_k) bytes, 4-byte aligned,
 *                 contents on entry ignored; calls that may run at the same
 *                 time need one each
 * Limits as for moe_align_block_size (E <= MOE_MAX_EXPERTS, M*top_k <=
 * MOE_MAX_SLOTS); expert_first is any int. */
int moe_align_topk_ids(const int *topk_ids, int M, int E, int top_k, int block_m,
                       int expert_first, int *sorted_token_ids, int *expert_ids,
                       int *num_tokens_post_padded, int *expert_counts, void *workspace,
                       hipStream_t stream);

/* ======================================================================== *
 * Dense int8 product
 * ======================================================================== */

/* Bytes of device workspace moe_gemm_int8w8a8 can use for this shape (at most
 * 16 MiB; 0 where it needs none or the sizes are invalid).  It splits the
 * contraction over more workgroups where the output alone has too few. */
size_t moe_gemm_int8w8a8_workspace_bytes(int M, int K, int N);

/* Product of int8 activations (moe_quantize_act with MOE_Q_INT8_PER_CHANNEL)
 * and int8 weights (moe_quantize_weights with the same mode, E = 1), with a
 * scale per token and per output channel:
 *     out[m, n] = round( (sum_k a[m,k] * w[n,k]) * a_scale[m] * w_scale[n]
 *                        + bias[n] + addend[m, n] )
 * The sums are exact (int32); they are converted to float32 once, the rest is
 * float32 and rounded once to the output type (nearest even).  With the
 * combined output of the routed experts as addend the product is the shared
 * expert's contribution to the layer.
 *
 *   a_q     [M, K] int8, rows lda bytes apart (lda >= K); a_scale [M] float32
 *   w_q     [N, K] int8, rows ldw bytes apart (ldw >= K); w_scale [N] float32
 *   bias    [N] float32, or NULL
 *   addend  [M, N] of out's type and row distance, or NULL; may be out itself
 *   out     [M, N] of type out_dtype (MOE_F32, MOE_BF16, MOE_F16), rows ldo
 *           elements apart (ldo >= N); elements between the rows stay as they are
 *   workspace moe_gemm_int8w8a8_workspace_bytes(M, K, N) bytes, 16-byte
 *           aligned, contents on entry ignored, one for each call that may run
 *           at the same time; or NULL (the same results, small shapes slower)
 * Limits: 1 <= K <= MOE_MAX_INT8_K, 0 <= M < MOE_MAX_INT8_ROWS, N >= 1, rows less
 * than 2^22 apart (so N < 2^22), M * N < 2^36; no alignment is required beyond
 * the types' own.  Fastest where a_q, w_q, lda and ldw are multiples of 16 (K
 * need not be). */
int moe_gemm_int8w8a8(const int8_t *a_q, long long lda, const float *a_scale, const int8_t *w_q,
                      long long ldw, const float *w_scale, const float *bias, const void *addend,
                      int M, int K, int N, int out_dtype, void *out, long long ldo,
                      void *workspace, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* QMOE_MOE_LAYER_H */
