// Launchers of the operators of the block around the experts (moe_block.h): the
// grouped 16-bit products of the gated feed-forward, low-rank adapters and the
// block's norms.  qmoe_block_api.cpp calls them with validated arguments.
#pragma once

#include "qmoe_layer.h"

namespace qmoe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// v_mfma_f32_16x16x32 on eight values a lane of the 16-bit type Ty.
template <typename Ty>
__device__ __forceinline__ f32x4 mfma16(const i32x4 &a, const i32x4 &b, const f32x4 &c);
template <>
__device__ __forceinline__ f32x4 mfma16<TypeBf16>(const i32x4 &a, const i32x4 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma16<TypeF16>(const i32x4 &a, const i32x4 &b, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The grouped products.  An expert's output block is rows x columns, contracted
// over `depth`; which operand is which:
//   kLinear  rows: the segment's rows of r [*, depth]; columns: c [E, cols, depth]
//   kDgrad   rows: the segment's rows of r [*, depth]; columns: c [E, depth, cols]
//   kWgrad   rows: columns of r [*, rows]; columns: columns of c [*, cols];
//            depth: the segment's rows of both
enum { kLinear = 0, kDgrad = 1, kWgrad = 2 };
// what becomes of the sums
enum { kStore = 0, kGatedUp = 1, kGatedBackward = 2, kStoreF32 = 3 };

struct GroupedArgs {
  const uint16_t *r, *c;
  long long ldr, ldc;                // elements between rows
  long long c_expert;                // ... between experts of c (kLinear, kDgrad)
  const int *off;                    // m_offsets, or null
  int rows, E;
  int nrow, ncol, depth;             // kWgrad: nrow; others: depth
  void *out;                         // kGatedUp: h, kGatedBackward: dgu
  long long ldo, out_expert;
  const uint16_t *gu_in;             // kGatedBackward
  uint16_t *side;                    // kGatedUp: gu or null; kGatedBackward: h or null
  int H, act;                        // kGated*: ncol = H; kGatedUp: c holds 2 H columns
};
hipError_t launch_grouped(int layout, int epilogue, int dtype, const GroupedArgs &a, hipStream_t s);

struct LoraArgs {
  const uint16_t *x;
  long long ldx;
  const uint16_t *a, *b;
  const int *ranks;                  // or null
  const float *scales;               // or null
  const int *ids;                    // or null: tokens without an adapter stay as they are
  const int *sorted, *labels, *num_post;
  int T, K, N, R, L, block_m, max_padded;
  const void *addend;                // or null
  void *out;
  long long ldo;
  float *ws;
};
size_t lora_workspace_bytes(int T, int K, int R, int L, int block_m);
hipError_t launch_lora(const LoraArgs &a, int dtype, int out_dtype, hipStream_t s);

struct NormArgs {
  const uint16_t *y;                 // or null
  int top_k;
  const void *residual;              // or null
  const float *w_post, *gate;        // or null
  int gate_kind;
  float alpha, beta;
  const float *w_pre;                // or null
  float eps;
  int M, N;
  void *r;
  uint16_t *h;
  float *rstd_post, *rstd_pre;       // or null
};
hipError_t launch_norm(const NormArgs &a, int dtype, int r_dtype, hipStream_t s);

struct NormBwdArgs {
  const void *d_r;                   // or null
  const uint16_t *d_h, *y;           // or null
  int top_k;
  const void *r;
  const float *w_post, *gate;
  int gate_kind;
  float alpha, beta;
  const float *w_pre, *rstd_post, *rstd_pre;
  int M, N;
  void *d_residual;                  // or null
  uint16_t *d_y;
  float *d_w_post, *d_gate, *d_w_pre;   // or null
  float *ws;
};
size_t norm_backward_workspace_bytes(int M, int N);
hipError_t launch_norm_backward(const NormBwdArgs &a, int dtype, int r_dtype, hipStream_t s);

}  // namespace qmoe
