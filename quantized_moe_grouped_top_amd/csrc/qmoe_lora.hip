// Low-rank adapters of many requests: out = addend + scale * B (A x), tokens
// grouped by adapter in blocks of 16 at least.
//
// Two launches.  shrink: v = A x, float32 sums left in the workspace, one workgroup per
// 16 or 32 sorted tokens, 64 ranks and share of K; expand: one workgroup per block of
// tokens and 512 columns adds scale * B v.  Both are bound by the bytes they read and
// write (x and A; B, addend and out) and, for a few tokens, by the loads that wait for
// one another: block -> adapter -> its rank, scale and matrices.  Whatever does not hang
// on the adapter is loaded beside it.  The products are v_mfma_f32_16x16x32.
#include "qmoe_block.h"
#include "qmoe_device.h"
#include <type_traits>

namespace qmoe {

namespace {

#define QMOE_INLINE __attribute__((always_inline))

constexpr int kWaves = 4;
constexpr int kMaxShares = 4;

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)p;
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
template <int n>
__device__ __forceinline__ void wait_dma() {         // all but the last n have landed
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}
// global_load_lds_dwordx4: each lane copies 16 bytes from its own address to LDS byte
// address m0 + 16 * lane.
__device__ __forceinline__ void dma16_from(const uint16_t *from, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(from), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}

// Slots of a shrink workgroup and shares of K: enough workgroups for the card where
// there are few tokens, 512 k a share at least.
int shrink_rows(int block_m) { return block_m >= 32 ? 32 : 16; }
int shares(int T, int K, int R, int L, int block_m) {
  const int per = shrink_rows(block_m);
  const long long groups = ((T < L ? T : T / per + L) + 0ll) * ((R + 63) / 64);
  int n = (int)((256 + groups - 1) / groups);
  n = n < K / 512 ? n : K / 512;
  n = n < kMaxShares ? n : kMaxShares;
  return n < 1 ? 1 : n;
}

__device__ __forceinline__ int clamp_rank(int r, int R) { return min(max(r, 0), R); }

// v[share][sorted slot][R] = the share's part of A x.  The wavefronts share out the
// share's K, 64 of it each in turn, through LDS rings of their own (whole 128-byte lines
// of x and A, D steps ahead), and add their sums at the end.
template <typename Ty, int MB, int C, int D>
__global__ __launch_bounds__(64 * kWaves) void shrink_kernel(const LoraArgs p, int splits) {
  constexpr int kSlot = 16 * (MB + C) * 128, kRingB = kWaves * D * kSlot, kPartB = kWaves * MB * C * 1024;
  constexpr int kPieces = 2 * (MB + C);
  static_assert((D - 1) * kPieces < 64, "the copies in flight are counted in 6 bits");
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kRingB > kPartB ? kRingB : kPartB];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot0 = blockIdx.x * 16 * MB, r0 = blockIdx.z * 16 * C;
  const int used = p.num_post[0], a = p.labels[slot0 / p.block_m];
  int tok[2 * MB];
#pragma unroll
  for (int u = 0; u < 2 * MB; ++u) tok[u] = p.sorted[slot0 + 8 * u + (lane >> 3)];
  if (slot0 >= min(used, p.max_padded) || a < 0 || a >= p.L) return;
  const int rank = __builtin_amdgcn_readfirstlane(p.ranks ? clamp_rank(p.ranks[a], p.R) : p.R);
  if (r0 >= rank) return;
  // chunk c of LDS row r lies at c ^ ((r >> 1) & 7); slots without a token repeat token 0
  const int ch = (lane & 7) ^ (lane >> 4);            // of the even copies; the odd ones': ^ 4
  const uint16_t *x[2 * MB];
#pragma unroll
  for (int u = 0; u < 2 * MB; ++u) x[u] = p.x + (tok[u] >= 0 && tok[u] < p.T ? tok[u] : 0) * p.ldx;
  const uint16_t *A = p.a + ((long long)a * p.R + r0) * p.K;
  uint32_t a_off[2 * C];
#pragma unroll
  for (int u = 0; u < 2 * C; ++u) {
    const int r = 8 * u + (lane >> 3);                // rows past the rank repeat its first
    a_off[u] = (uint32_t)(r0 + r < rank ? r : 0) * (uint32_t)p.K;
  }
  const uint32_t mine = lds_addr(s_ring) + (uint32_t)(wave * D * kSlot);
  const int steps = (p.K + 63) >> 6, turn = (int)blockIdx.y * kWaves + wave, turns = splits * kWaves;
  const int n = (steps - turn + turns - 1) / turns;
  auto copy = [&](int slot, int i) QMOE_INLINE {
    const int k0 = 64 * (i * turns + turn);
    const uint32_t to = mine + (uint32_t)(slot * kSlot);
    // chunks past K repeat the last one; they are masked below
    const int e = min(k0 + 8 * ch, p.K - 8), o = min(k0 + 8 * (ch ^ 4), p.K - 8);
#pragma unroll
    for (int u = 0; u < 2 * MB; ++u) dma16_from(x[u] + (u & 1 ? o : e), to + u * 1024);
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) dma16_from(A + a_off[u] + (u & 1 ? o : e), to + (2 * MB + u) * 1024);
  };
  f32x4 acc[MB][C];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < C; ++j) acc[b][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) copy(d, d);
  typedef __attribute__((address_space(3))) i32x4 *LdsV;
  int slot = 0;
  for (int i = 0; i < n; ++i) {
    if (i + D <= n) wait_dma<(D - 1) * kPieces>();
    else wait_dma_all();
    const uint32_t from = mine + (uint32_t)(slot * kSlot + r16 * 128);
    const int left = p.K - 64 * (i * turns + turn);
    i32x4 fx[MB][2], fa[C][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = from + (uint32_t)(((4 * h + g) ^ ((r16 >> 1) & 7)) << 4);
#pragma unroll
      for (int b = 0; b < MB; ++b) fx[b][h] = *(LdsV)(uintptr_t)(at + b * 2048);
#pragma unroll
      for (int j = 0; j < C; ++j) fa[j][h] = *(LdsV)(uintptr_t)(at + (MB + j) * 2048);
    }
    wait_lds();                                       // the slot has been read
    if (i + D < n) copy(slot, i + D);
    if (left < 64) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (32 * h + 8 * g >= left) {
#pragma unroll
          for (int b = 0; b < MB; ++b) fx[b][h] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < C; ++j) fa[j][h] = i32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[b][j] = mfma16<Ty>(fa[j][h], fx[b][h], acc[b][j]);
    slot = slot + 1 < D ? slot + 1 : 0;
  }
  __syncthreads();                                    // every wavefront is done with its ring
  f32x4 *part = reinterpret_cast<f32x4 *>(s_ring);
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < C; ++j) part[(wave * MB * C + b * C + j) * 64 + lane] = acc[b][j];
  __syncthreads();
  // lane: ranks 16 j + 4 g .., token r16 (sums past the rank are not used)
  for (int f = wave; f < MB * C; f += kWaves) {
    const int b = f / C, r = r0 + 16 * (f - b * C) + 4 * g;
    f32x4 sum = part[f * 64 + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += part[(w * MB * C + f) * 64 + lane];
    if (r < p.R)
      *reinterpret_cast<f32x4 *>(p.ws + ((long long)blockIdx.y * p.max_padded + slot0 + 16 * b + r16) * p.R + r) = sum;
  }
}

// Eight neighbouring values in float32, from and to the type Out.
template <typename Out>
struct Eight {
  i32x4 q[sizeof(typename Out::T) == 4 ? 2 : 1];
};
template <typename Out>
__device__ __forceinline__ Eight<Out> load8(const typename Out::T *at) {
  Eight<Out> v;
  v.q[0] = *reinterpret_cast<const i32x4 *>(at);
  if constexpr (sizeof(typename Out::T) == 4) v.q[1] = *reinterpret_cast<const i32x4 *>(at + 4);
  return v;
}
template <typename Out>
__device__ __forceinline__ float value(const Eight<Out> &v, int i) {
  if constexpr (sizeof(typename Out::T) == 4) return __int_as_float(v.q[i >> 2][i & 3]);
  else return Out::load((uint16_t)((uint32_t)v.q[0][i >> 1] >> (16 * (i & 1))));
}
template <typename Out>
__device__ __forceinline__ void store8(typename Out::T *at, const float (&f)[8]) {
  if constexpr (sizeof(typename Out::T) == 4) {
    *reinterpret_cast<f32x4 *>(at) = f32x4{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f32x4 *>(at + 4) = f32x4{f[4], f[5], f[6], f[7]};
  } else {
    *reinterpret_cast<i32x4 *>(at) = i32x4{Out::pack(f[0], f[1]), Out::pack(f[2], f[3]), Out::pack(f[4], f[5]),
                                           Out::pack(f[6], f[7])};
  }
}

// The 16-bit pairs of v with infinities and NaN as 0.
template <typename Ty>
__device__ __forceinline__ i32x4 finite_only(const i32x4 &v) {
  constexpr int kExp = std::is_same<Ty, TypeBf16>::value ? 0x7F80 : 0x7C00;     // all ones in those
  i32x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = v[q] & ((v[q] & kExp) == kExp ? ~0xFFFF : -1) & ((v[q] >> 16 & kExp) == kExp ? 0xFFFF : -1);
  return o;
}

// One workgroup per block of tokens and 512 columns, 64 a wavefront, neighbouring workgroups
// neighbouring columns: 1 KB of a token's row together (4096 tokens, 28672 columns, rank 64:
// 127 us, with 256 columns 139, neighbours in tokens 160; sums split by every wavefront for
// itself 289).  The columns' part of B stays in registers; the block's sums, 64 tokens at a time, are added over the shares of K and split
// into 16-bit parts once for the workgroup, in LDS, from where every wavefront multiplies
// 16 tokens at a time.  S: steps of 32 ranks.
constexpr int kColumns = 64, kTokens = 64, kExpandWaves = 8;

template <typename Ty, typename Out, int S>
__global__ __launch_bounds__(64 * kExpandWaves, S == 4 ? 2 : 4) void expand_kernel(const LoraArgs p, int splits, int blocks) {
  typedef typename Out::T T;
  constexpr int kRow = 32 * S + 8;                    // 16-bit values of an LDS row: off the banks
  // two parts leave out 2^-16 of v (bf16; fp16 2^-22), three 2^-24, float32's own rounding
  constexpr int kParts = sizeof(T) == 4 ? 3 : 2;
  __shared__ __attribute__((aligned(16))) uint16_t s_v[kParts][kTokens][kRow];
  __shared__ float s_up[kTokens];
  __shared__ int s_tok[kTokens];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = (blockIdx.x * kExpandWaves + wave) * kColumns;
  const T *addend = (const T *)p.addend;
  T *out = (T *)p.out;
  if ((int)blockIdx.y >= blocks) {                    // 64 tokens: those without an adapter
    const int t0 = 64 * (blockIdx.y - blocks), id = p.ids[min(t0 + lane, p.T - 1)];
    uint64_t bare = __ballot((id < 0 || id >= p.L) && t0 + lane < p.T);
    const int n = blockIdx.x * kColumns * kExpandWaves + 8 * lane;
    static_assert(kColumns * kExpandWaves == 512, "a wavefront copies all the columns of a token");
    for (int turn = 0; bare; bare &= bare - 1, ++turn) {
      const int t = t0 + __builtin_ctzll(bare);
      if ((turn & (kExpandWaves - 1)) != wave || n >= p.N) continue;
      float f[8] = {};
      if (addend) {
        const Eight<Out> v = load8<Out>(addend + t * p.ldo + n);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = value<Out>(v, i);
      }
      store8<Out>(out + t * p.ldo + n, f);
    }
    return;
  }
  const int first = blockIdx.y * p.block_m;
  const int used = p.num_post[0], a = p.labels[blockIdx.y];
  const int tokens = min(p.block_m, kTokens);         // of a pass
  const int each = 64 * kExpandWaves / tokens;              // threads of a token: 8, 16 or 32
  const int mine = tid / each, part = tid & (each - 1);
  constexpr int kQuads = S;                           // of four ranks, a thread's at most
  f32x4 v[kQuads];
  // the shares' sums of this thread's ranks: 4 (part + i each) ..
  auto fetch = [&](int m) QMOE_INLINE {
    const float *from = p.ws + (long long)(first + m + mine) * p.R;
    f32x4 w[kMaxShares][kQuads];                      // all under way at once
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int r = 4 * (part + i * each);
#pragma unroll
      for (int y = 0; y < kMaxShares; ++y) w[y][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (r < p.R) {
#pragma unroll
        for (int y = 0; y < kMaxShares; ++y)
          if (y < splits)
            w[y][i] = *reinterpret_cast<const f32x4 *>(from + (long long)y * p.max_padded * p.R + r);
      }
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      v[i] = w[0][i];
#pragma unroll
      for (int y = 1; y < kMaxShares; ++y) v[i] += w[y][i];
    }
  };
  fetch(0);                                           // beside the block's adapter
  if (first >= min(used, p.max_padded) || a < 0 || a >= p.L) return;
  const int rank = p.ranks ? clamp_rank(p.ranks[a], p.R) : p.R;
  const float scale = p.scales ? p.scales[a] : 1.0f;
  const uint16_t *B = p.b + (long long)a * p.N * p.R;
  i32x4 bv[4][S];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int n = n0 + 16 * j + r16, k = 32 * s + 8 * g;
      bv[j][s] = i32x4{0, 0, 0, 0};
      if (n < p.N && k < rank) bv[j][s] = *reinterpret_cast<const i32x4 *>(B + (long long)n * p.R + k);
    }
  // columns of B past the rank count as 0, whatever they hold
  if (rank & 7) {
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int left = rank - (32 * s + 8 * g + 2 * q);         // of this pair
        const int keep = left >= 2 ? -1 : left == 1 ? 0xFFFF : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) bv[j][s][q] &= keep;
      }
  }
  for (int m0 = 0; m0 < p.block_m; m0 += tokens) {
    // v in 16-bit parts; for fp16 through a power of two that brings a token's largest value to
    // 2^14 .. 2^15.  Below that fp16 ends at steps of 2^-24, so that beside the parts' own
    // 2^-39 of the largest value is left out at most: parts around 1 would leave out 2^-25 of
    // it, which is all of a value that far below, and more than 2^-16 of any below 2^-9.  An
    // infinity stays one in any case: the largest finite value counts.
    float top = 0.0f, down = scale, up = 1.0f;
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * (part + i * each) + q >= rank) v[i][q] = 0.0f;
        top = fmaxf(top, __builtin_isfinite(v[i][q]) ? fabsf(v[i][q]) : 0.0f);
      }
    if constexpr (std::is_same<Ty, TypeF16>::value) {
      for (int d = 1; d < each; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
      down = 1.0f;
      up = scale;
      if (top > 0.0f) {
        const int e = min(max(ilogbf(top), -100), 100);
        down = ldexpf(1.0f, 14 - e);
        up = ldexpf(scale, e - 14);
      }
    }
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int r = 4 * (part + i * each);
      if (r < 32 * S) {
        float rest[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) rest[q] = v[i][q] * down;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const i32x2 w = {Ty::pack(rest[0], rest[1]), Ty::pack(rest[2], rest[3])};
          *reinterpret_cast<i32x2 *>(&s_v[k][mine][r]) = w;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float h = Ty::load((uint16_t)((uint32_t)w[q >> 1] >> (16 * (q & 1))));
            rest[q] = __builtin_isfinite(h) ? rest[q] - h : 0.0f;    // nothing is left of an infinity
          }
        }
      }
    }
    if (part == 0) {
      s_up[mine] = up;
      const int tok = p.sorted[first + m0 + mine];
      s_tok[mine] = tok >= 0 && tok < p.T ? tok : -1;
    }
    __syncthreads();
    if (m0 + tokens < p.block_m) fetch(m0 + tokens);
    // a lane's token of 16 and its addends, loaded while the 16 before are multiplied
    const int pair = 16 * (g & 1) + 8 * (g >> 1);
    int tok, next_tok = s_tok[r16];
    Eight<Out> add[2], next_add[2];
    auto fetch_add = [&]() QMOE_INLINE {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = n0 + 32 * j + pair;
        if (addend && next_tok >= 0 && n < p.N) next_add[j] = load8<Out>(addend + next_tok * p.ldo + n);
      }
    };
    fetch_add();
    for (int m = 0; m < tokens; m += 16) {
      tok = next_tok;
      add[0] = next_add[0];
      add[1] = next_add[1];
      const bool live = tok >= 0;
      if (__ballot(live) == 0) break;                 // the rest of the block is padding
      if (m + 16 < tokens) {
        next_tok = s_tok[m + 16 + r16];
        fetch_add();
      }
      f32x4 acc[4];
      auto products = [&](auto clean) QMOE_INLINE {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          if (32 * s >= rank) break;
#pragma unroll
          for (int k = kParts - 1; k >= 0; --k) {     // the smallest first
            const i32x4 w = *reinterpret_cast<const i32x4 *>(&s_v[k][m + r16][32 * s + 8 * g]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              i32x4 b = bv[j][s];
              if constexpr (decltype(clean)::value)
                if (k > 0) {
                  asm volatile("" : "+v"(b));         // cleaned here each time, not held beside B
                  b = finite_only<Ty>(b);
                }
              acc[j] = mfma16<Ty>(b, w, acc[j]);
            }
          }
        }
      };
      products(std::false_type{});
      // An infinity of B belongs to the first part of v alone: the others may be 0 or of the
      // other sign, and with theirs its sum has become NaN.
      bool nan = false;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        nan |= __builtin_isunordered(acc[j][0], acc[j][1]) | __builtin_isunordered(acc[j][2], acc[j][3]);
      if (__ballot(nan) != 0) products(std::true_type{});
      const float by = s_up[m + r16];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float f[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const auto w = __builtin_amdgcn_permlane16_swap(__float_as_int(acc[2 * j][q]),
                                                          __float_as_int(acc[2 * j + 1][q]), false, false);
          f[q] = __int_as_float((int)w[0]) * by;
          f[4 + q] = __int_as_float((int)w[1]) * by;
        }
        const int n = n0 + 32 * j + pair;
        if (live && n < p.N) {
          if (addend) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += value<Out>(add[j], i);
          }
          store8<Out>(out + tok * p.ldo + n, f);
        }
      }
    }
    __syncthreads();                                  // the parts are read
  }
}

template <typename Ty, int MB, int C, int D>
void shrink(const LoraArgs &a, int splits, hipStream_t s) {
  hipLaunchKernelGGL((shrink_kernel<Ty, MB, C, D>), dim3(a.max_padded / (16 * MB), splits, (a.R + 16 * C - 1) / (16 * C)),
                     dim3(64 * kWaves), 0, s, a, splits);
}
template <typename Ty, typename Out, int S>
void expand(const LoraArgs &a, int splits, hipStream_t s) {
  const int blocks = a.max_padded / a.block_m, columns = (a.N + kColumns * kExpandWaves - 1) / (kColumns * kExpandWaves);
  hipLaunchKernelGGL((expand_kernel<Ty, Out, S>), dim3(columns, blocks + (a.ids ? (a.T + 63) / 64 : 0)), dim3(64 * kExpandWaves), 0,
                     s, a, splits, blocks);
}
template <typename Ty, typename Out>
hipError_t run(const LoraArgs &a, hipStream_t s) {
  const int splits = shares(a.T, a.K, a.R, a.L, a.block_m);
  if (shrink_rows(a.block_m) == 16) {
    if (a.R <= 16) shrink<Ty, 1, 1, 4>(a, splits, s);
    else if (a.R <= 32) shrink<Ty, 1, 2, 4>(a, splits, s);
    else shrink<Ty, 1, 4, 3>(a, splits, s);
  } else {
    if (a.R <= 16) shrink<Ty, 2, 1, 4>(a, splits, s);
    else if (a.R <= 32) shrink<Ty, 2, 2, 3>(a, splits, s);
    else shrink<Ty, 2, 4, 2>(a, splits, s);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.R <= 32) expand<Ty, Out, 1>(a, splits, s);
  else if (a.R <= 64) expand<Ty, Out, 2>(a, splits, s);
  else expand<Ty, Out, 4>(a, splits, s);
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
  return (size_t)n * R * sizeof(float) * shares(T, K, R, L, block_m);
}

hipError_t launch_lora(const LoraArgs &a, int dtype, int out_dtype, hipStream_t s) {
  return dtype == MOE_BF16 ? run_out<TypeBf16>(a, out_dtype, s) : run_out<TypeF16>(a, out_dtype, s);
}

}  // namespace qmoe
