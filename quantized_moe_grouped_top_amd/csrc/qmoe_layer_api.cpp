// C ABI of the operators around the grouped GEMMs (declared in moe_layer.h):
// argument validation on the host, then the launches on the caller's stream.
#include "qmoe_layer.h"
#include "qmoe_status.h"

using namespace qmoe;

namespace {

bool valid_dtype(int t) { return t == MOE_F32 || t == MOE_BF16 || t == MOE_F16; }
bool aligned_to(const void *p, int dtype) {
  return ((uintptr_t)p & (dtype == MOE_F32 ? 3u : 1u)) == 0;
}
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
// a launch holds fewer than 2^32 threads, up to 512 for 128 x 128 outputs
bool int8_rows_fit(int M, int N) {
  return M < MOE_MAX_INT8_ROWS && N < (1 << 22) && (long long)M * N < (1ll << 36);
}

// sizes shared by the router and its gradient
int check_route(int dtype, long long ld, int M, int E, int top_k, int score, const char *fn) {
  REQUIRE(valid_dtype(dtype), MOE_EINVAL, "%s: unknown element type %d", fn, dtype);
  REQUIRE(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_EINVAL,
          "%s: unknown score %d", fn, score);
  REQUIRE(M >= 0 && E >= 1, MOE_EINVAL, "%s: M=%d E=%d", fn, M, E);
  REQUIRE(M < MOE_MAX_ROUTE_TOKENS, MOE_EUNSUPPORTED, "%s: M=%d above %d", fn, M,
          MOE_MAX_ROUTE_TOKENS - 1);
  REQUIRE(E <= MOE_MAX_ROUTE_EXPERTS, MOE_EUNSUPPORTED, "%s: E=%d above %d", fn, E,
          MOE_MAX_ROUTE_EXPERTS);
  REQUIRE(top_k >= 1 && top_k <= E, MOE_EINVAL, "%s: top_k=%d outside [1, E=%d]", fn, top_k, E);
  REQUIRE(top_k <= MOE_MAX_TOPK, MOE_EUNSUPPORTED, "%s: top_k=%d above %d", fn, top_k,
          MOE_MAX_TOPK);
  REQUIRE(ld >= E, MOE_EINVAL, "%s: rows %lld apart hold no %d experts", fn, ld, E);
  REQUIRE(ld < (1ll << 31), MOE_EUNSUPPORTED, "%s: rows %lld apart", fn, ld);
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route_topk(const void *logits, int dtype, long long ld, const float *bias, int M, int E,
                   int top_k, int score, int n_group, int topk_group, int group_rule,
                   int renormalize, float scale, int *topk_ids, float *topk_weights,
                   hipStream_t stream) {
  const char *fn = "moe_route_topk";
  int rc = check_route(dtype, ld, M, E, top_k, score, fn);
  if (rc) return rc;
  REQUIRE(group_rule == MOE_GROUP_MAX || group_rule == MOE_GROUP_TOP2, MOE_EINVAL,
          "%s: unknown group rule %d", fn, group_rule);
  REQUIRE(n_group >= 1 && n_group <= E && E % n_group == 0, MOE_EINVAL,
          "%s: E=%d experts in n_group=%d groups", fn, E, n_group);
  REQUIRE(n_group <= MOE_MAX_ROUTE_GROUPS, MOE_EUNSUPPORTED, "%s: n_group=%d above %d", fn,
          n_group, MOE_MAX_ROUTE_GROUPS);
  REQUIRE(topk_group >= 1 && topk_group <= n_group, MOE_EINVAL,
          "%s: topk_group=%d outside [1, n_group=%d]", fn, topk_group, n_group);
  REQUIRE(topk_group * (E / n_group) >= top_k, MOE_EINVAL,
          "%s: %d groups of %d experts hold fewer than top_k=%d", fn, topk_group, E / n_group,
          top_k);
  REQUIRE(n_group == 1 || group_rule != MOE_GROUP_TOP2 || E / n_group >= 2, MOE_EINVAL,
          "%s: MOE_GROUP_TOP2 needs two experts in a group", fn);
  if (M == 0) return ok();
  REQUIRE(logits && topk_ids && topk_weights, MOE_EINVAL, "%s: null pointer argument", fn);
  REQUIRE(aligned_to(logits, dtype) && aligned4(bias) && aligned4(topk_ids) &&
              aligned4(topk_weights),
          MOE_EINVAL, "%s: a pointer is not aligned to its type", fn);
  const RouteArgs a{logits, ld, bias, M, E, top_k, score, n_group,
                    topk_group, group_rule, renormalize != 0, scale, topk_ids, topk_weights};
  return hip_status(launch_route_topk(a, dtype, stream), fn);
}

int moe_route_topk_backward(const float *d_weights, const int *topk_ids, const void *logits,
                            int dtype, long long ld, int M, int E, int top_k, int score,
                            int renormalize, float scale, void *d_logits, long long ldd,
                            hipStream_t stream) {
  const char *fn = "moe_route_topk_backward";
  int rc = check_route(dtype, ld, M, E, top_k, score, fn);
  if (rc) return rc;
  REQUIRE(ldd >= E, MOE_EINVAL, "%s: rows %lld apart hold no %d experts", fn, ldd, E);
  REQUIRE(ldd < (1ll << 31), MOE_EUNSUPPORTED, "%s: rows %lld apart", fn, ldd);
  if (M == 0) return ok();
  REQUIRE(d_weights && topk_ids && logits && d_logits, MOE_EINVAL, "%s: null pointer argument",
          fn);
  REQUIRE(aligned_to(logits, dtype) && aligned_to(d_logits, dtype) && aligned4(topk_ids) &&
              aligned4(d_weights),
          MOE_EINVAL, "%s: a pointer is not aligned to its type", fn);
  const RouteBwdArgs a{d_weights, topk_ids, logits, ld,       M,   E, top_k, score,
                       renormalize != 0, scale, d_logits, ldd};
  return hip_status(launch_route_backward(a, dtype, stream), fn);
}

size_t moe_align_workspace_bytes(int M, int E, int top_k) {
  if (M < 0 || E < 1 || E > MOE_MAX_EXPERTS || top_k < 1 || top_k > E || top_k > MOE_MAX_TOPK ||
      (long long)M * top_k > MOE_MAX_SLOTS)
    return 0;
  return ((size_t)M * top_k + 1023) / 1024 * E * sizeof(int);
}

int moe_align_topk_ids(const int *topk_ids, int M, int E, int top_k, int block_m,
                       int expert_first, int *sorted_token_ids, int *expert_ids,
                       int *num_tokens_post_padded, int *expert_counts, void *workspace,
                       hipStream_t stream) {
  const char *fn = "moe_align_topk_ids";
  int rc = check_routing_sizes(M, E, top_k, fn);
  if (rc) return rc;
  REQUIRE(valid_block_m(block_m), MOE_EUNSUPPORTED, "%s: block_m=%d", fn, block_m);
  REQUIRE(sorted_token_ids && expert_ids && num_tokens_post_padded, MOE_EINVAL,
          "%s: null output pointer", fn);
  REQUIRE(M == 0 || (topk_ids && workspace), MOE_EINVAL, "%s: null pointer", fn);
  REQUIRE(aligned4(topk_ids) && aligned4(workspace) && aligned4(sorted_token_ids) &&
              aligned4(expert_ids) && aligned4(num_tokens_post_padded) && aligned4(expert_counts),
          MOE_EINVAL, "%s: pointers must be 4-byte aligned", fn);
  const AlignArgs a{topk_ids, M * top_k, E, block_m, expert_first,
                    (int)max_padded_ll(M, E, top_k, block_m), sorted_token_ids, expert_ids,
                    num_tokens_post_padded, expert_counts, (int *)workspace};
  return hip_status(launch_align_ids(a, stream), fn);
}

size_t moe_gemm_int8w8a8_workspace_bytes(int M, int K, int N) {
  if (M < 1 || N < 1 || K < 1 || K > MOE_MAX_INT8_K || !int8_rows_fit(M, N)) return 0;
  return int8_workspace_bytes(M, K, N);
}

int moe_gemm_int8w8a8(const int8_t *a_q, long long lda, const float *a_scale, const int8_t *w_q,
                      long long ldw, const float *w_scale, const float *bias, const void *addend,
                      int M, int K, int N, int out_dtype, void *out, long long ldo,
                      void *workspace, hipStream_t stream) {
  const char *fn = "moe_gemm_int8w8a8";
  REQUIRE(valid_dtype(out_dtype), MOE_EINVAL, "%s: unknown element type %d", fn, out_dtype);
  REQUIRE(M >= 0 && K >= 1 && N >= 1, MOE_EINVAL, "%s: M=%d K=%d N=%d", fn, M, K, N);
  REQUIRE(K <= MOE_MAX_INT8_K, MOE_EUNSUPPORTED, "%s: K=%d above %d (int32 sums)", fn, K,
          MOE_MAX_INT8_K);
  REQUIRE(int8_rows_fit(M, N), MOE_EUNSUPPORTED, "%s: M=%d N=%d above %d, %d or 2^36 outputs", fn,
          M, N, MOE_MAX_INT8_ROWS - 1, (1 << 22) - 1);
  REQUIRE(lda >= K && ldw >= K && ldo >= N, MOE_EINVAL,
          "%s: row distances %lld, %lld, %lld below K=%d, K, N=%d", fn, lda, ldw, ldo, K, N);
  // byte offsets inside a tile of 256 rows are 32-bit
  REQUIRE(lda < (1 << 22) && ldw < (1 << 22) && ldo < (1 << 22), MOE_EUNSUPPORTED,
          "%s: rows must lie less than %d apart", fn, 1 << 22);
  if (M == 0) return ok();
  REQUIRE(a_q && a_scale && w_q && w_scale && out, MOE_EINVAL, "%s: null pointer argument", fn);
  REQUIRE(aligned4(a_scale) && aligned4(w_scale) && aligned4(bias) &&
              aligned_to(out, out_dtype) && aligned_to(addend, out_dtype),
          MOE_EINVAL, "%s: a pointer is not aligned to its type", fn);
  REQUIRE(aligned16(workspace), MOE_EINVAL, "%s: workspace must be 16-byte aligned", fn);
  const Int8Args a{a_q, lda, a_scale, w_q, ldw, w_scale, bias, addend, out, ldo, M, K, N,
                   (int *)workspace};
  return hip_status(launch_int8_gemm(a, out_dtype, stream), fn);
}

}  // extern "C"
