// C ABI of the operators of the block around the experts (declared in
// moe_block.h): argument validation on the host, then the launches on the
// caller's stream.
#include "qmoe_block.h"
#include "qmoe_status.h"

using namespace qmoe;

namespace {

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
bool type16(int t) { return t == MOE_BF16 || t == MOE_F16; }
bool type_of(int t) { return t == MOE_F32 || type16(t); }

// a width or row distance of the grouped products and adapters
int check_width(long long v, const char *what, const char *fn) {
  REQUIRE(v >= 1, MOE_EINVAL, "%s: %s=%lld", fn, what, v);
  REQUIRE(v % 8 == 0 && v <= MOE_MAX_BLOCK_WIDTH, MOE_EUNSUPPORTED,
          "%s: %s=%lld is no multiple of 8 up to %d", fn, what, v, MOE_MAX_BLOCK_WIDTH);
  return MOE_OK;
}
int check_rows(long long ld, long long row, const char *what, const char *fn) {
  int rc = check_width(ld, what, fn);
  if (rc) return rc;
  REQUIRE(ld >= row, MOE_EINVAL, "%s: %s=%lld below the row's %lld", fn, what, ld, row);
  return MOE_OK;
}
// what the five grouped products have in common
int check_grouped(int dtype, const int *m_offsets, int rows, int E, const char *fn) {
  REQUIRE(type16(dtype), MOE_EINVAL, "%s: element type %d is no 16-bit type", fn, dtype);
  REQUIRE(rows >= 0 && E >= 1, MOE_EINVAL, "%s: rows=%d E=%d", fn, rows, E);
  REQUIRE(rows <= MOE_MAX_BLOCK_ROWS, MOE_EUNSUPPORTED, "%s: rows=%d above %d", fn, rows,
          MOE_MAX_BLOCK_ROWS);
  REQUIRE(E <= MOE_MAX_EXPERTS, MOE_EUNSUPPORTED, "%s: E=%d above %d", fn, E, MOE_MAX_EXPERTS);
  REQUIRE(m_offsets || E == 1, MOE_EINVAL, "%s: E=%d experts without m_offsets", fn, E);
  REQUIRE(aligned4(m_offsets), MOE_EINVAL, "%s: m_offsets must be 4-byte aligned", fn);
  return MOE_OK;
}

#define CHECK(call)            \
  do {                         \
    const int rc_ = (call);    \
    if (rc_) return rc_;       \
  } while (0)
#define ALIGNED16(p) REQUIRE(aligned16(p), MOE_EINVAL, "%s: " #p " must be 16-byte aligned", fn)

int check_norm(int dtype, int r_dtype, int top_k, const void *y, int gate_kind, const float *gate,
               int M, int N, const char *fn) {
  REQUIRE(type16(dtype), MOE_EINVAL, "%s: element type %d is no 16-bit type", fn, dtype);
  REQUIRE(r_dtype == dtype || r_dtype == MOE_F32, MOE_EINVAL,
          "%s: the residual's type %d is neither %d nor MOE_F32", fn, r_dtype, dtype);
  REQUIRE(M >= 0 && N >= 1, MOE_EINVAL, "%s: M=%d N=%d", fn, M, N);
  REQUIRE(N % 8 == 0 && N <= MOE_MAX_NORM_COLUMNS, MOE_EUNSUPPORTED,
          "%s: N=%d is no multiple of 8 up to %d", fn, N, MOE_MAX_NORM_COLUMNS);
  REQUIRE(top_k >= 1, MOE_EINVAL, "%s: top_k=%d", fn, top_k);
  REQUIRE(top_k <= MOE_MAX_TOPK, MOE_EUNSUPPORTED, "%s: top_k=%d above %d", fn, top_k, MOE_MAX_TOPK);
  REQUIRE((long long)M * top_k <= MOE_MAX_NORM_ROWS, MOE_EUNSUPPORTED, "%s: M=%d top_k=%d above %d rows",
          fn, M, top_k, MOE_MAX_NORM_ROWS);
  REQUIRE((long long)M * N <= MOE_MAX_NORM_VALUES, MOE_EUNSUPPORTED, "%s: M=%d N=%d above %lld values", fn,
          M, N, MOE_MAX_NORM_VALUES);
  REQUIRE(gate_kind >= MOE_GATE_NONE && gate_kind <= MOE_GATE_TOKEN, MOE_EINVAL,
          "%s: unknown gate %d", fn, gate_kind);
  // arrays without elements have no address, so that without tokens nothing says which are there
  REQUIRE((gate_kind == MOE_GATE_NONE) == (gate == nullptr) || M == 0, MOE_EINVAL,
          "%s: gate kind %d and the gate's pointer disagree", fn, gate_kind);
  REQUIRE(y || gate_kind == MOE_GATE_NONE || M == 0, MOE_EINVAL, "%s: a gate without a block", fn);
  ALIGNED16(y);
  REQUIRE(gate_kind == MOE_GATE_CHANNEL ? aligned16(gate) : aligned4(gate), MOE_EINVAL,
          "%s: gate is not aligned", fn);
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_gated_up(const void *x, long long ldx, const void *w, int dtype, const int *m_offsets,
                 int rows, int K, int H, int E, int act, void *gu, void *h, hipStream_t stream) {
  const char *fn = "moe_gated_up";
  CHECK(check_grouped(dtype, m_offsets, rows, E, fn));
  REQUIRE(act == MOE_GATED_SILU || act == MOE_GATED_GELU, MOE_EINVAL, "%s: unknown activation %d", fn,
          act);
  CHECK(check_width(K, "K", fn));
  CHECK(check_width(H, "H", fn));
  CHECK(check_width(2ll * H, "2H", fn));
  CHECK(check_rows(ldx, K, "ldx", fn));
  if (rows == 0) return ok();
  REQUIRE(x && w && h, MOE_EINVAL, "%s: null pointer argument", fn);
  ALIGNED16(x);
  ALIGNED16(w);
  ALIGNED16(gu);
  ALIGNED16(h);
  GroupedArgs a{};
  a.r = (const uint16_t *)x;
  a.ldr = ldx;
  a.c = (const uint16_t *)w;
  a.ldc = K;
  a.c_expert = 2ll * H * K;
  a.off = m_offsets;
  a.rows = rows;
  a.E = E;
  a.ncol = H;
  a.depth = K;
  a.out = h;
  a.ldo = H;
  a.side = (uint16_t *)gu;
  a.H = H;
  a.act = act;
  return hip_status(launch_grouped(kLinear, kGatedUp, dtype, a, stream), fn);
}

int moe_grouped_linear(const void *x, long long ldx, const void *w, int dtype,
                       const int *m_offsets, int rows, int K, int N, int E, void *y,
                       long long ldy, hipStream_t stream) {
  const char *fn = "moe_grouped_linear";
  CHECK(check_grouped(dtype, m_offsets, rows, E, fn));
  CHECK(check_width(K, "K", fn));
  CHECK(check_width(N, "N", fn));
  CHECK(check_rows(ldx, K, "ldx", fn));
  CHECK(check_rows(ldy, N, "ldy", fn));
  if (rows == 0) return ok();
  REQUIRE(x && w && y, MOE_EINVAL, "%s: null pointer argument", fn);
  ALIGNED16(x);
  ALIGNED16(w);
  ALIGNED16(y);
  GroupedArgs a{};
  a.r = (const uint16_t *)x;
  a.ldr = ldx;
  a.c = (const uint16_t *)w;
  a.ldc = K;
  a.c_expert = (long long)N * K;
  a.off = m_offsets;
  a.rows = rows;
  a.E = E;
  a.ncol = N;
  a.depth = K;
  a.out = y;
  a.ldo = ldy;
  return hip_status(launch_grouped(kLinear, kStore, dtype, a, stream), fn);
}

int moe_gated_down_backward(const void *dy, long long lddy, const void *w, const void *gu,
                            int dtype, const int *m_offsets, int rows, int N, int H, int E,
                            int act, void *dgu, void *h, hipStream_t stream) {
  const char *fn = "moe_gated_down_backward";
  CHECK(check_grouped(dtype, m_offsets, rows, E, fn));
  REQUIRE(act == MOE_GATED_SILU || act == MOE_GATED_GELU, MOE_EINVAL, "%s: unknown activation %d", fn,
          act);
  CHECK(check_width(N, "N", fn));
  CHECK(check_width(H, "H", fn));
  CHECK(check_width(2ll * H, "2H", fn));
  CHECK(check_rows(lddy, N, "lddy", fn));
  if (rows == 0) return ok();
  REQUIRE(dy && w && gu && dgu, MOE_EINVAL, "%s: null pointer argument", fn);
  ALIGNED16(dy);
  ALIGNED16(w);
  ALIGNED16(gu);
  ALIGNED16(dgu);
  ALIGNED16(h);
  GroupedArgs a{};
  a.r = (const uint16_t *)dy;
  a.ldr = lddy;
  a.c = (const uint16_t *)w;
  a.ldc = H;
  a.c_expert = (long long)N * H;
  a.off = m_offsets;
  a.rows = rows;
  a.E = E;
  a.ncol = H;
  a.depth = N;
  a.out = dgu;
  a.ldo = 2ll * H;
  a.gu_in = (const uint16_t *)gu;
  a.side = (uint16_t *)h;
  a.H = H;
  a.act = act;
  return hip_status(launch_grouped(kDgrad, kGatedBackward, dtype, a, stream), fn);
}

int moe_grouped_linear_dgrad(const void *dy, long long lddy, const void *w, int dtype,
                             const int *m_offsets, int rows, int K, int N, int E, void *dx,
                             long long lddx, hipStream_t stream) {
  const char *fn = "moe_grouped_linear_dgrad";
  CHECK(check_grouped(dtype, m_offsets, rows, E, fn));
  CHECK(check_width(K, "K", fn));
  CHECK(check_width(N, "N", fn));
  CHECK(check_rows(lddy, N, "lddy", fn));
  CHECK(check_rows(lddx, K, "lddx", fn));
  if (rows == 0) return ok();
  REQUIRE(dy && w && dx, MOE_EINVAL, "%s: null pointer argument", fn);
  ALIGNED16(dy);
  ALIGNED16(w);
  ALIGNED16(dx);
  GroupedArgs a{};
  a.r = (const uint16_t *)dy;
  a.ldr = lddy;
  a.c = (const uint16_t *)w;
  a.ldc = K;
  a.c_expert = (long long)N * K;
  a.off = m_offsets;
  a.rows = rows;
  a.E = E;
  a.ncol = K;
  a.depth = N;
  a.out = dx;
  a.ldo = lddx;
  return hip_status(launch_grouped(kDgrad, kStore, dtype, a, stream), fn);
}

int moe_grouped_linear_wgrad(const void *dy, long long lddy, const void *x, long long ldx,
                             int dtype, const int *m_offsets, int rows, int K, int N, int E,
                             int dw_dtype, void *dw, hipStream_t stream) {
  const char *fn = "moe_grouped_linear_wgrad";
  CHECK(check_grouped(dtype, m_offsets, rows, E, fn));
  REQUIRE(dw_dtype == dtype || dw_dtype == MOE_F32, MOE_EINVAL,
          "%s: the gradient's type %d is neither %d nor MOE_F32", fn, dw_dtype, dtype);
  CHECK(check_width(K, "K", fn));
  CHECK(check_width(N, "N", fn));
  CHECK(check_rows(lddy, N, "lddy", fn));
  CHECK(check_rows(ldx, K, "ldx", fn));
  REQUIRE(dw && (rows == 0 || (dy && x)), MOE_EINVAL, "%s: null pointer argument", fn);
  ALIGNED16(dy);
  ALIGNED16(x);
  ALIGNED16(dw);
  GroupedArgs a{};
  a.r = (const uint16_t *)dy;
  a.ldr = lddy;
  a.c = (const uint16_t *)x;
  a.ldc = ldx;
  a.off = m_offsets;
  a.rows = rows;
  a.E = E;
  a.nrow = N;
  a.ncol = K;
  a.out = dw;
  a.ldo = K;
  a.out_expert = (long long)N * K;
  return hip_status(
      launch_grouped(kWgrad, dw_dtype == MOE_F32 ? kStoreF32 : kStore, dtype, a, stream), fn);
}

size_t moe_lora_workspace_bytes(int T, int K, int R, int L, int block_m) {
  if (T < 1 || T > MOE_MAX_SLOTS || L < 1 || L > MOE_MAX_EXPERTS || R < 8 || R % 8 ||
      R > MOE_MAX_LORA_RANK || K < 8 || K % 8 || K > MOE_MAX_BLOCK_WIDTH || !valid_block_m(block_m))
    return 0;
  return lora_workspace_bytes(T, K, R, L, block_m);
}

int moe_lora_add(const void *x, long long ldx, const void *a, const void *b, const int *ranks,
                 const float *scales, int dtype, const int *adapter_ids,
                 const int *sorted_token_ids, const int *expert_ids,
                 const int *num_tokens_post_padded, int T, int K, int N, int R, int L,
                 int block_m, const void *addend, int out_dtype, void *out, long long ldo,
                 void *workspace, hipStream_t stream) {
  const char *fn = "moe_lora_add";
  REQUIRE(type16(dtype), MOE_EINVAL, "%s: element type %d is no 16-bit type", fn, dtype);
  REQUIRE(type_of(out_dtype), MOE_EINVAL, "%s: unknown element type %d", fn, out_dtype);
  REQUIRE(T >= 0 && L >= 1, MOE_EINVAL, "%s: T=%d L=%d", fn, T, L);
  REQUIRE(T <= MOE_MAX_SLOTS, MOE_EUNSUPPORTED, "%s: T=%d above %d", fn, T, MOE_MAX_SLOTS);
  REQUIRE(L <= MOE_MAX_EXPERTS, MOE_EUNSUPPORTED, "%s: L=%d above %d", fn, L, MOE_MAX_EXPERTS);
  REQUIRE(valid_block_m(block_m), MOE_EUNSUPPORTED, "%s: block_m=%d", fn, block_m);
  REQUIRE(R >= 1, MOE_EINVAL, "%s: R=%d", fn, R);
  REQUIRE(R % 8 == 0 && R <= MOE_MAX_LORA_RANK, MOE_EUNSUPPORTED,
          "%s: R=%d is no multiple of 8 up to %d", fn, R, MOE_MAX_LORA_RANK);
  CHECK(check_width(K, "K", fn));
  CHECK(check_width(N, "N", fn));
  CHECK(check_rows(ldx, K, "ldx", fn));
  CHECK(check_rows(ldo, N, "ldo", fn));
  if (T == 0) return ok();
  REQUIRE(x && a && b && sorted_token_ids && expert_ids && num_tokens_post_padded && out && workspace,
          MOE_EINVAL, "%s: null pointer argument", fn);
  REQUIRE(adapter_ids || addend == out, MOE_EINVAL, "%s: null adapter_ids, and addend is not out", fn);
  ALIGNED16(x);
  ALIGNED16(a);
  ALIGNED16(b);
  ALIGNED16(addend);
  ALIGNED16(out);
  ALIGNED16(workspace);
  REQUIRE(aligned4(ranks) && aligned4(scales) && aligned4(adapter_ids) && aligned4(sorted_token_ids) &&
              aligned4(expert_ids) && aligned4(num_tokens_post_padded),
          MOE_EINVAL, "%s: a pointer is not aligned to its type", fn);
  const LoraArgs args{(const uint16_t *)x, ldx, (const uint16_t *)a, (const uint16_t *)b, ranks, scales,
                      addend == out ? nullptr : adapter_ids, sorted_token_ids, expert_ids,
                      num_tokens_post_padded, T, K, N, R, L, block_m,
                      (int)max_padded_ll(T, L, 1, block_m), addend, out, ldo, (float *)workspace};
  return hip_status(launch_lora(args, dtype, out_dtype, stream), fn);
}

int moe_norm_residual(const void *y, int dtype, int top_k, const void *residual, int r_dtype,
                      const float *w_post, const float *gate, int gate_kind, float alpha,
                      float beta, const float *w_pre, float eps, int M, int N, void *r, void *h,
                      float *rstd_post, float *rstd_pre, hipStream_t stream) {
  const char *fn = "moe_norm_residual";
  CHECK(check_norm(dtype, r_dtype, top_k, y, gate_kind, gate, M, N, fn));
  REQUIRE(eps >= 0.0f, MOE_EINVAL, "%s: eps=%g", fn, (double)eps);
  if (M == 0) return ok();
  REQUIRE(y || residual, MOE_EINVAL, "%s: neither a block nor a residual", fn);
  REQUIRE(y || !(w_post || rstd_post), MOE_EINVAL, "%s: a norm after no block", fn);
  REQUIRE((w_pre == nullptr) == (h == nullptr), MOE_EINVAL, "%s: w_pre and h go together", fn);
  REQUIRE((w_post || !rstd_post) && (w_pre || !rstd_pre), MOE_EINVAL,
          "%s: the factor of a norm that is not taken", fn);
  REQUIRE(r, MOE_EINVAL, "%s: null pointer argument", fn);
  ALIGNED16(residual);
  ALIGNED16(w_post);
  ALIGNED16(w_pre);
  ALIGNED16(r);
  ALIGNED16(h);
  REQUIRE(aligned4(rstd_post) && aligned4(rstd_pre), MOE_EINVAL, "%s: rstd must be 4-byte aligned", fn);
  const NormArgs a{(const uint16_t *)y, top_k, residual, w_post, gate, gate_kind, alpha, beta, w_pre,
                   eps, M, N, r, (uint16_t *)h, rstd_post, rstd_pre};
  return hip_status(launch_norm(a, dtype, r_dtype, stream), fn);
}

size_t moe_norm_backward_workspace_bytes(int M, int N) {
  if (M < 1 || M > MOE_MAX_NORM_ROWS || N < 8 || N % 8 || N > MOE_MAX_NORM_COLUMNS ||
      (long long)M * N > MOE_MAX_NORM_VALUES)
    return 0;
  return norm_backward_workspace_bytes(M, N);
}

int moe_norm_residual_backward(const void *d_r, const void *d_h, const void *y, int dtype,
                               int top_k, const void *r, int r_dtype, const float *w_post,
                               const float *gate, int gate_kind, float alpha, float beta,
                               const float *w_pre, const float *rstd_post,
                               const float *rstd_pre, int M, int N, void *d_residual,
                               void *d_y, float *d_w_post, float *d_gate, float *d_w_pre,
                               void *workspace, hipStream_t stream) {
  const char *fn = "moe_norm_residual_backward";
  CHECK(check_norm(dtype, r_dtype, top_k, y, gate_kind, gate, M, N, fn));
  REQUIRE((w_pre == nullptr) == (d_h == nullptr) || M == 0, MOE_EINVAL, "%s: w_pre and d_h go together", fn);
  REQUIRE(d_h || d_r || M == 0, MOE_EINVAL, "%s: no gradient comes in", fn);
  REQUIRE((y == nullptr) == (d_y == nullptr) || M == 0, MOE_EINVAL, "%s: y and d_y go together", fn);
  REQUIRE(y || !w_post || M == 0, MOE_EINVAL, "%s: a norm after no block", fn);
  REQUIRE((w_post || !d_w_post) && (w_pre || !d_w_pre) && (gate || !d_gate), MOE_EINVAL,
          "%s: the gradient of a weight or gate that is not there", fn);
  REQUIRE(!w_post || rstd_post || M == 0, MOE_EINVAL, "%s: null rstd_post", fn);
  REQUIRE(!w_pre || (rstd_pre && r) || M == 0, MOE_EINVAL, "%s: null rstd_pre or r", fn);
  REQUIRE(workspace || M == 0, MOE_EINVAL, "%s: null workspace", fn);
  ALIGNED16(d_r);
  ALIGNED16(d_h);
  ALIGNED16(r);
  ALIGNED16(w_post);
  ALIGNED16(w_pre);
  ALIGNED16(d_residual);
  ALIGNED16(d_y);
  ALIGNED16(workspace);
  REQUIRE(aligned4(rstd_post) && aligned4(rstd_pre) && aligned4(d_w_post) && aligned4(d_gate) &&
              aligned4(d_w_pre),
          MOE_EINVAL, "%s: a pointer is not aligned to its type", fn);
  const NormBwdArgs a{d_r, (const uint16_t *)d_h, (const uint16_t *)y, top_k, r, w_post, gate, gate_kind,
                      alpha, beta, w_pre, rstd_post, rstd_pre, M, N, d_residual, (uint16_t *)d_y,
                      d_w_post, d_gate, d_w_pre, (float *)workspace};
  return hip_status(launch_norm_backward(a, dtype, r_dtype, stream), fn);
}

}  // extern "C"
