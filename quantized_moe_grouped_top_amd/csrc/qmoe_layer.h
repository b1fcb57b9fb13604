// Launchers of the operators around the grouped GEMMs (moe_layer.h): the
// general router, its gradient, the alignment of given ids and the dense int8
// product.  qmoe_layer_api.cpp calls them with validated arguments.
#pragma once

#include <hip/hip_fp16.h>

#include "qmoe_internal.h"

namespace qmoe {

// Element types of logits, gradients and outputs: one struct per MOE_* type
// code, with the conversions from and to float32.
struct TypeF32 {
  typedef float T;
  static __device__ __forceinline__ float load(T v) { return v; }
  static __device__ __forceinline__ T store(float v) { return v; }
};
struct TypeBf16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float load(T v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ T store(float v) { return (T)f32x2_to_bf16x2(v, v); }
  static __device__ __forceinline__ int pack(float a, float b) { return (int)f32x2_to_bf16x2(a, b); }
};
struct TypeF16 {
  typedef uint16_t T;
  static __device__ __forceinline__ float load(T v) {
    return __half2float(__builtin_bit_cast(__half, v));
  }
  static __device__ __forceinline__ T store(float v) {
    return __builtin_bit_cast(uint16_t, __float2half_rn(v));
  }
  static __device__ __forceinline__ int pack(float a, float b) {
    return (int)((uint32_t)store(a) | ((uint32_t)store(b) << 16));
  }
};

struct RouteArgs {
  const void *logits;
  long long ld;
  const float *bias;                 // or null
  int M, E, top_k;
  int score, n_group, topk_group, group_rule, renormalize;
  float scale;
  int *ids;
  float *weights;
};
hipError_t launch_route_topk(const RouteArgs &a, int dtype, hipStream_t s);

struct RouteBwdArgs {
  const float *dw;
  const int *ids;
  const void *logits;
  long long ld;
  int M, E, top_k, score, renormalize;
  float scale;
  void *dx;
  long long ldd;
};
hipError_t launch_route_backward(const RouteBwdArgs &a, int dtype, hipStream_t s);

struct AlignArgs {
  const int *ids;
  int S, E, block_m, expert_first, max_padded;
  int *sorted_ids, *expert_ids, *num_post;
  int *counts;                       // or null
  int *ws;
};
hipError_t launch_align_ids(const AlignArgs &a, hipStream_t s);

struct Int8Args {
  const int8_t *a;
  long long lda;
  const float *a_scale;
  const int8_t *w;
  long long ldw;
  const float *w_scale;
  const float *bias;                 // or null
  const void *addend;                // or null
  void *out;
  long long ldo;
  int M, K, N;
  int *ws;                           // or null
};
size_t int8_workspace_bytes(int M, int K, int N);
hipError_t launch_int8_gemm(const Int8Args &a, int out_dtype, hipStream_t s);

}  // namespace qmoe
