// The grouped 16-bit products of the experts' gated feed-forward: forward (both
// projections with the activation and the product in the epilogue), the linear
// back down, the input gradients (one with the activation's gradient in the
// epilogue) and the weight gradients.
//
// One workgroup per 64 x 64 outputs of an expert, v_mfma_f32_16x16x32 on four
// wavefronts of 32 x 32, operands through registers into LDS.
#include "qmoe_block.h"
#include "qmoe_device.h"

namespace qmoe {

namespace {

// act(g) and act'(g).  Both activations are g sigmoid(z): z = g (silu), z = 2 c (g +
// 0.044715 g^3) (gelu, since (1 + tanh(z / 2)) / 2 = sigmoid(z)).  gelu's z is that of
// g within +-1e4: act' is 0 or 1 long before, and z and dz stay finite.
__device__ __forceinline__ float act_value(float g, int act) {
  float z = g;
  if (act != MOE_GATED_SILU) {
    const float gc = __builtin_amdgcn_fmed3f(g, -1e4f, 1e4f);
    z = 1.5957691216057308f * gc * (1.0f + 0.044715f * gc * gc);
  }
  return g / (1.0f + __expf(-z));
}
__device__ __forceinline__ void act_both(float g, int act, float &a, float &da) {
  float z = g, dz = 1.0f;
  if (act != MOE_GATED_SILU) {
    const float gc = __builtin_amdgcn_fmed3f(g, -1e4f, 1e4f);
    z = 1.5957691216057308f * gc * (1.0f + 0.044715f * gc * gc);
    dz = 1.5957691216057308f * (1.0f + 3.0f * 0.044715f * gc * gc);
  }
  const float s = 1.0f / (1.0f + __expf(-z));
  a = g * s;
  da = s + a * (1.0f - s) * dz;
}

constexpr int kT = 64, kK = 32, kLd = kK + 8;

template <typename Ty, int kLayout, int kEpi>
__global__ __launch_bounds__(256) void grouped_kernel(const GroupedArgs p) {
  constexpr bool kRT = kLayout == kWgrad, kCT = kLayout != kLinear;
  constexpr int kSets = kEpi == kGatedUp ? 2 : 1;
  __shared__ uint16_t s_r[kT][kLd], s_c[kSets][kT][kLd];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, r16 = lane & 15, wm = wave & 1, wn = wave >> 1;
  // this workgroup's expert, rows and columns
  int e = 0, lo = 0, hi = 0, m0 = 0;
  const int n0 = blockIdx.y * kT;
  auto segment = [&](int i) {
    lo = p.off ? min(max(p.off[i], 0), p.rows) : 0;
    hi = p.off ? min(max(p.off[i + 1], lo), p.rows) : p.rows;
  };
  if constexpr (kLayout == kWgrad) {
    const int tiles = (p.nrow + kT - 1) / kT;
    e = blockIdx.x / tiles;
    m0 = (blockIdx.x - e * tiles) * kT;
    segment(e);
  } else {
    int t = blockIdx.x;
    for (;; ++e) {
      if (e == p.E) return;
      segment(e);
      const int n = (hi - lo + kT - 1) / kT;
      if (t < n) break;
      t -= n;
    }
    m0 = t * kT;
  }
  const int nrow = kLayout == kWgrad ? p.nrow : hi - lo;
  const int depth = kLayout == kWgrad ? hi - lo : p.depth;
  const uint16_t *r = p.r + lo * p.ldr;
  const uint16_t *c = kLayout == kWgrad ? p.c + lo * p.ldc : p.c + e * p.c_expert;

  f32x4 acc[kSets][2][2] = {};
  auto load = [&](uint16_t (*dst)[kLd], const uint16_t *src, long long ld, bool transposed, int at,
                  int count, int k0) {
    if (!transposed) {
      const int row = tid >> 2, ch = (tid & 3) * 8;
      i32x4 v = {0, 0, 0, 0};
      if (at + row < count && k0 + ch < depth)
        v = *reinterpret_cast<const i32x4 *>(src + (at + row) * ld + k0 + ch);
      *reinterpret_cast<i32x4 *>(&dst[row][ch]) = v;
    } else {
      const int k = tid >> 3, ch = (tid & 7) * 8;
      i32x4 v = {0, 0, 0, 0};
      if (k0 + k < depth && at + ch < count)
        v = *reinterpret_cast<const i32x4 *>(src + (long long)(k0 + k) * ld + at + ch);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[ch + i][k] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
  };
  for (int k0 = 0; k0 < depth; k0 += kK) {
    load(s_r, r, p.ldr, kRT, m0, nrow, k0);
#pragma unroll
    for (int s = 0; s < kSets; ++s) load(s_c[s], c + s * (long long)p.H * p.ldc, p.ldc, kCT, n0, p.ncol, k0);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[s][i][j] = mfma16<Ty>(*reinterpret_cast<const i32x4 *>(&s_c[s][32 * wn + 16 * j + r16][8 * g]),
                                    *reinterpret_cast<const i32x4 *>(&s_r[32 * wm + 16 * i + r16][8 * g]),
                                    acc[s][i][j]);
    __syncthreads();
  }
  // lane: row 16 i + r16, columns 16 j + 4 g ..
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = m0 + 32 * wm + 16 * i + r16;
    if (m >= nrow) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + 32 * wn + 16 * j + 4 * g + q;
        if (n >= p.ncol) continue;
        const float v = acc[0][i][j][q];
        const long long row = kLayout == kWgrad ? m : lo + m;
        if constexpr (kEpi == kStoreF32) {
          ((float *)p.out)[e * p.out_expert + row * p.ldo + n] = v;
        } else if constexpr (kEpi == kStore) {
          ((uint16_t *)p.out)[e * p.out_expert + row * p.ldo + n] = Ty::store(v);
        } else if constexpr (kEpi == kGatedUp) {
          const float u = acc[kSets - 1][i][j][q];
          if (p.side) {
            p.side[row * 2 * p.H + n] = Ty::store(v);
            p.side[row * 2 * p.H + p.H + n] = Ty::store(u);
          }
          ((uint16_t *)p.out)[row * p.ldo + n] = Ty::store(act_value(v, p.act) * u);
        } else {
          const long long at = row * 2 * p.H + n;
          const float gv = Ty::load(p.gu_in[at]), uv = Ty::load(p.gu_in[at + p.H]);
          float a, da;
          act_both(gv, p.act, a, da);
          ((uint16_t *)p.out)[at] = Ty::store(v * uv * da);
          ((uint16_t *)p.out)[at + p.H] = Ty::store(v * a);
          if (p.side) p.side[row * p.H + n] = Ty::store(a * uv);
        }
      }
    }
  }
}

template <typename Ty, int kLayout, int kEpi>
hipError_t launch(const GroupedArgs &a, hipStream_t s) {
  const int tiles = kLayout == kWgrad ? a.E * ((a.nrow + kT - 1) / kT) : (a.rows + kT - 1) / kT + a.E;
  hipLaunchKernelGGL((grouped_kernel<Ty, kLayout, kEpi>), dim3(tiles, (a.ncol + kT - 1) / kT), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}
template <typename Ty>
hipError_t launch_typed(int layout, int epi, const GroupedArgs &a, hipStream_t s) {
  if (layout == kLinear)
    return epi == kGatedUp ? launch<Ty, kLinear, kGatedUp>(a, s) : launch<Ty, kLinear, kStore>(a, s);
  if (layout == kDgrad)
    return epi == kGatedBackward ? launch<Ty, kDgrad, kGatedBackward>(a, s)
                                 : launch<Ty, kDgrad, kStore>(a, s);
  return epi == kStoreF32 ? launch<Ty, kWgrad, kStoreF32>(a, s) : launch<Ty, kWgrad, kStore>(a, s);
}

}  // namespace

hipError_t launch_grouped(int layout, int epilogue, int dtype, const GroupedArgs &a, hipStream_t s) {
  return dtype == MOE_BF16 ? launch_typed<TypeBf16>(layout, epilogue, a, s)
                           : launch_typed<TypeF16>(layout, epilogue, a, s);
}

}  // namespace qmoe
