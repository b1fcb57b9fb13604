// Dense int8 product with a scale per token and per output channel:
//   out[m, n] = round((sum_k a[m,k] w[n,k]) * a_scale[m] * w_scale[n] + bias[n] + addend[m, n])
// The sums are exact: int8 products added in int32 on the int8 MFMA.
#include "qmoe_layer.h"

namespace qmoe {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

// One output value from its exact sum.
template <typename Ty>
__device__ __forceinline__ void store_one(const Int8Args &p, int m, int n, int sum) {
  float v = (float)sum * p.a_scale[m] * p.w_scale[n];
  if (p.bias) v += p.bias[n];
  const long long i = (long long)m * p.ldo + n;
  if (p.addend) v += Ty::load(((const typename Ty::T *)p.addend)[i]);
  ((typename Ty::T *)p.out)[i] = Ty::store(v);
}

// 16 bytes of a row from byte k on: zero past K, any alignment.
__device__ __forceinline__ i32x4 load16(const int8_t *row, int k, int K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
    uint8_t b[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = k + i < K ? (uint8_t)row[k + i] : 0;
    __builtin_memcpy(&v, b, 16);
  }
  return v;
}

// 64 x 64 tile, four wavefronts of 32 x 32 (v_mfma_i32_32x32x32_i8, weights as
// the first operand), 64 k a stage through LDS rows of 80 bytes.
constexpr int kRow = 80;
template <typename Ty>
__global__ __launch_bounds__(256) void int8_any_kernel(const Int8Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t s_a[64 * kRow], s_w[64 * kRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int r = tid >> 2, c = (tid & 3) * 16;        // this thread's row and chunk of a stage
  const bool am = m0 + r < p.M, wn = n0 + r < p.N;
  const int8_t *ar = p.a + (long long)(am ? m0 + r : 0) * p.lda;
  const int8_t *wr = p.w + (long long)(wn ? n0 + r : 0) * p.ldw;
  i32x16 acc;
#pragma unroll
  for (int v = 0; v < 16; ++v) acc[v] = 0;
  const int g = lane >> 5, q = lane & 31;
  const int mw = (wave & 1) * 32, nw = (wave >> 1) * 32;
  for (int k = 0; k < p.K; k += 64) {
    const i32x4 z = {0, 0, 0, 0};
    const i32x4 av = am ? load16(ar, k + c, p.K) : z;
    const i32x4 wv = wn ? load16(wr, k + c, p.K) : z;
    __syncthreads();
    *reinterpret_cast<i32x4 *>(s_a + r * kRow + c) = av;
    *reinterpret_cast<i32x4 *>(s_w + r * kRow + c) = wv;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const i32x4 fa = *reinterpret_cast<const i32x4 *>(s_a + (mw + q) * kRow + 32 * h + 16 * g);
      const i32x4 fw = *reinterpret_cast<const i32x4 *>(s_w + (nw + q) * kRow + 32 * h + 16 * g);
      acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw, fa, acc, 0, 0, 0);
    }
  }
  const int m = m0 + mw + q;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int n = n0 + nw + 8 * (v >> 2) + 4 * g + (v & 3);
    if (m < p.M && n < p.N) store_one<Ty>(p, m, n, acc[v]);
  }
}

}  // namespace

size_t int8_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_int8_gemm(const Int8Args &a, int out_dtype, hipStream_t s) {
  const dim3 g((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64)), b(256);
  if (out_dtype == MOE_F32) hipLaunchKernelGGL(int8_any_kernel<TypeF32>, g, b, 0, s, a);
  else if (out_dtype == MOE_BF16) hipLaunchKernelGGL(int8_any_kernel<TypeBf16>, g, b, 0, s, a);
  else hipLaunchKernelGGL(int8_any_kernel<TypeF16>, g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe
