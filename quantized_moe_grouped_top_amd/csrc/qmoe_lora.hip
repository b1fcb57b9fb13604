// Low-rank adapters of many requests: out = addend + scale * B (A x), tokens
// grouped by adapter in blocks of 16 at least.
//
// Two launches.  shrink: one workgroup per 16 sorted tokens (and share of K) leaves
// v = A x as float32 in the workspace; expand: one workgroup per block of tokens and
// columns adds scale * B v.  Both are bound by the bytes they read and write (x, A,
// B, addend, out); the products are v_mfma_f32_16x16x32.
#include "qmoe_block.h"
#include "qmoe_device.h"

namespace qmoe {

namespace {

constexpr int kWaves = 4;
constexpr int kMaxRank16 = MOE_MAX_LORA_RANK / 16;

// Shares of K in the first product: enough that a few tokens read their adapters
// with more than a handful of CUs, 512 k each at least.
int shares(int T, int K, int L, int block_m) {
  const long long groups = T < 16 * L ? T : T / 16 + L;
  int n = (int)((256 + groups - 1) / groups);
  n = n < K / 512 ? n : K / 512;
  n = n < 8 ? n : 8;
  return n < 1 ? 1 : n;
}

__device__ __forceinline__ int rank_of(const LoraArgs &p, int a) {
  return p.ranks ? min(max(p.ranks[a], 0), p.R) : p.R;
}

// v[share][sorted slot][R] = the share's part of A x
template <typename Ty>
__global__ __launch_bounds__(64 * kWaves) void shrink_kernel(const LoraArgs p, int splits) {
  __shared__ f32x4 s_part[kWaves][kMaxRank16][64];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot0 = blockIdx.x * 16;
  if (slot0 >= min(p.num_post[0], p.max_padded)) return;
  const int a = p.labels[slot0 / p.block_m];
  if (a < 0 || a >= p.L) return;
  const int rank = rank_of(p, a), frags = (rank + 15) / 16;
  const int tok = p.sorted[slot0 + r16];
  const bool live = tok >= 0 && tok < p.T;
  if (__ballot(live) == 0) return;
  const uint16_t *x = p.x + (long long)(live ? tok : 0) * p.ldx;
  const uint16_t *A = p.a + (long long)a * p.R * p.K;
  f32x4 acc[kMaxRank16] = {};
  // 32 k a step, steps dealt to the wavefronts of all shares in turn
  const int steps = (p.K + 31) / 32;
  for (int st = blockIdx.y * kWaves + wave; st < steps; st += splits * kWaves) {
    const int k = 32 * st + 8 * g;
    const bool in = k < p.K;
    i32x4 xv = {0, 0, 0, 0};
    if (live && in) xv = *reinterpret_cast<const i32x4 *>(x + k);
#pragma unroll
    for (int f = 0; f < kMaxRank16; ++f) {
      if (f >= frags) break;
      i32x4 av = {0, 0, 0, 0};
      if (in && 16 * f + r16 < rank)
        av = *reinterpret_cast<const i32x4 *>(A + (long long)(16 * f + r16) * p.K + k);
      acc[f] = mfma16<Ty>(av, xv, acc[f]);
    }
  }
#pragma unroll
  for (int f = 0; f < kMaxRank16; ++f) {
    if (f >= frags) break;
    s_part[wave][f][lane] = acc[f];
  }
  __syncthreads();
  // lane: ranks 16 f + 4 g .., token r16
  float *v = p.ws + ((long long)blockIdx.y * p.max_padded + slot0 + r16) * p.R;
  for (int f = wave; f < frags; f += kWaves) {
    f32x4 sum = s_part[0][f][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += s_part[w][f][lane];
    if (16 * f + 4 * g < p.R) *reinterpret_cast<f32x4 *>(v + 16 * f + 4 * g) = sum;
  }
}

template <typename Out>
__device__ __forceinline__ void store4(typename Out::T *at, const f32x4 &v) {
  if constexpr (sizeof(typename Out::T) == 4) {
    *reinterpret_cast<f32x4 *>(at) = v;
  } else {
    *reinterpret_cast<i32x2 *>(at) = i32x2{Out::pack(v[0], v[1]), Out::pack(v[2], v[3])};
  }
}
template <typename Out>
__device__ __forceinline__ f32x4 load4(const typename Out::T *at) {
  if constexpr (sizeof(typename Out::T) == 4) {
    return *reinterpret_cast<const f32x4 *>(at);
  } else {
    const i32x2 q = *reinterpret_cast<const i32x2 *>(at);
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = Out::load((uint16_t)(q[c >> 1] >> (16 * (c & 1))));
    return v;
  }
}

// The columns that a wavefront of the second product owns.
constexpr int kCols = 64;

template <typename Ty, typename Out>
__global__ __launch_bounds__(64 * kWaves) void expand_kernel(const LoraArgs p, int splits, int blocks) {
  typedef typename Out::T T;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = (blockIdx.y * kWaves + wave) * kCols;
  const T *addend = (const T *)p.addend;
  T *out = (T *)p.out;
  if ((int)blockIdx.x >= blocks) {                    // tokens without an adapter
    const int t = blockIdx.x - blocks;
    if (p.ids[t] >= 0 && p.ids[t] < p.L) return;
    const int n = n0 + 4 * (lane & 15);
    if (lane < 16 && n < p.N) {
      const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
      store4<Out>(out + t * p.ldo + n, addend ? load4<Out>(addend + t * p.ldo + n) : zero);
    }
    return;
  }
  const int first = blockIdx.x * p.block_m;
  if (first >= min(p.num_post[0], p.max_padded) || n0 >= p.N) return;
  const int a = p.labels[blockIdx.x];
  if (a < 0 || a >= p.L) return;
  const int rank = rank_of(p, a), steps = (rank + 31) / 32;
  const float scale = p.scales ? p.scales[a] : 1.0f;
  const uint16_t *B = p.b + (long long)a * p.N * p.R;
  constexpr int kSteps = MOE_MAX_LORA_RANK / 32;
  // columns of B past the rank count as 0, whatever they hold
  i32x4 bv[4][kSteps];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      bv[j][s] = i32x4{0, 0, 0, 0};
      const int n = n0 + 16 * j + r16, k = 32 * s + 8 * g;
      if (s < steps && n < p.N && k < rank) {
        bv[j][s] = *reinterpret_cast<const i32x4 *>(B + (long long)n * p.R + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int left = rank - k - 2 * q;          // of this pair
          bv[j][s][q] &= left >= 2 ? -1 : left == 1 ? 0xFFFF : 0;
        }
      }
    }
  for (int m = 0; m < p.block_m; m += 16) {
    const int tok = p.sorted[first + m + r16];
    const bool live = tok >= 0 && tok < p.T;
    if (__ballot(live) == 0) break;                   // the rest of the block is padding
    // v of token r16, ranks 32 s + 8 g ..: the shares' sums, in float32
    float v[kSteps][8];
    float top = 0.0f;
    const float *ws = p.ws + (long long)(first + m + r16) * p.R;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[s][q] = 0.0f;
      const int k = 32 * s + 8 * g;
      if (live && s < steps && k < rank) {
        for (int y = 0; y < splits; ++y) {
          const f32x4 *part = reinterpret_cast<const f32x4 *>(ws + (long long)y * p.max_padded * p.R + k);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[s][q] += part[q >> 2][q & 3];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[s][q] = k + q < rank ? v[s][q] * scale : 0.0f;
          top = fmaxf(top, fabsf(v[s][q]));
        }
      }
    }
    // a power of two that brings a token's largest value near 1, so that both
    // 16-bit parts of every value lie in fp16's range
    float down = 1.0f, up = 1.0f;
    if constexpr (__is_same(Ty, TypeF16)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (top > 0.0f && top < __builtin_inff()) {
        const int e = min(max(ilogbf(top), -100), 100);
        down = ldexpf(1.0f, -e);
        up = ldexpf(1.0f, e);
      }
    }
    f32x4 acc[4] = {};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s >= steps) break;
      i32x4 hi, lo;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float a0 = v[s][2 * q] * down, a1 = v[s][2 * q + 1] * down;
        hi[q] = Ty::pack(a0, a1);
        const float h0 = Ty::load((uint16_t)hi[q]), h1 = Ty::load((uint16_t)((uint32_t)hi[q] >> 16));
        lo[q] = Ty::pack(__builtin_isfinite(h0) ? a0 - h0 : 0.0f, __builtin_isfinite(h1) ? a1 - h1 : 0.0f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j] = mfma16<Ty>(bv[j][s], lo, acc[j]);
        acc[j] = mfma16<Ty>(bv[j][s], hi, acc[j]);
      }
    }
    if (live) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + 16 * j + 4 * g;
        if (n >= p.N) continue;
        f32x4 o = acc[j];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] *= up;
        const long long at = tok * p.ldo + n;
        if (addend) o += load4<Out>(addend + at);
        store4<Out>(out + at, o);
      }
    }
  }
}

template <typename Ty, typename Out>
hipError_t run(const LoraArgs &a, hipStream_t s) {
  const int splits = shares(a.T, a.K, a.L, a.block_m);
  const int groups = a.max_padded / 16, blocks = a.max_padded / a.block_m;
  hipLaunchKernelGGL(shrink_kernel<Ty>, dim3(groups, splits), dim3(64 * kWaves), 0, s, a, splits);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int columns = (a.N + kCols * kWaves - 1) / (kCols * kWaves);
  hipLaunchKernelGGL((expand_kernel<Ty, Out>), dim3(blocks + (a.ids ? a.T : 0), columns), dim3(64 * kWaves), 0,
                     s, a, splits, blocks);
  return hipGetLastError();
}
template <typename Ty>
hipError_t run_out(const LoraArgs &a, int out_dtype, hipStream_t s) {
  if (out_dtype == MOE_F32) return run<Ty, TypeF32>(a, s);
  return out_dtype == MOE_BF16 ? run<Ty, TypeBf16>(a, s) : run<Ty, TypeF16>(a, s);
}

}  // namespace

size_t lora_workspace_bytes(int T, int K, int R, int L, int block_m) {
  const long long n = ((long long)T + (long long)L * (block_m - 1) + block_m - 1) / block_m * block_m;
  return (size_t)n * R * sizeof(float) * shares(T, K, L, block_m);
}

hipError_t launch_lora(const LoraArgs &a, int dtype, int out_dtype, hipStream_t s) {
  return dtype == MOE_BF16 ? run_out<TypeBf16>(a, out_dtype, s) : run_out<TypeF16>(a, out_dtype, s);
}

}  // namespace qmoe
