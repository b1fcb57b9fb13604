// Dense int8 product with a scale per token and per output channel:
//   out[m, n] = round((sum_k a[m,k] w[n,k]) * a_scale[m] * w_scale[n] + bias[n] + addend[m, n])
// The sums are exact: int8 products added in int32 on the int8 MFMA.
#include "qmoe_device.h"
#include "qmoe_layer.h"

namespace qmoe {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

// One output value from its exact sum.  Here and in the other epilogues every
// step is rounded by itself (no multiply-add joins the second scale and the
// bias), so that all kernels give the same bits.
template <typename Ty>
__device__ __forceinline__ void store_one(const Int8Args &p, int m, int n, int sum) {
#pragma clang fp contract(off)
  float v = (float)sum * p.a_scale[m] * p.w_scale[n];
  if (p.bias) v += p.bias[n];
  const long long i = (long long)m * p.ldo + n;
  if (p.addend) v += Ty::load(((const typename Ty::T *)p.addend)[i]);
  ((typename Ty::T *)p.out)[i] = Ty::store(v);
}

// A row of K < 16 bytes, any alignment, with zeros behind it.
__device__ __forceinline__ i32x4 load_short(const int8_t *row, int K) {
  uint8_t b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = i < K ? (uint8_t)row[i] : 0;
  i32x4 v;
  __builtin_memcpy(&v, b, 16);
  return v;
}

// 16 bytes of a row of at least 16 from byte k on, zero past K: the row's last 16
// bytes moved down.
__device__ __forceinline__ i32x4 fetch_end(const int8_t *row, int k, int K) {   // as they lie
  i32x4 v;
  __builtin_memcpy(&v, row + min(k, K - 16), 16);
  return v;
}
__device__ __forceinline__ i32x4 shift_end(const i32x4 &x, int k, int K) {
  const int drop = 8 * (k - min(k, K - 16));          // bits
  const uint64_t a = (uint32_t)x[0] | ((uint64_t)(uint32_t)x[1] << 32);
  const uint64_t b = (uint32_t)x[2] | ((uint64_t)(uint32_t)x[3] << 32);
  const uint64_t lo = drop < 64 ? (a >> drop) | (b << 1 << (63 - drop)) : b >> (drop & 63);
  const uint64_t hi = drop < 64 ? b >> drop : 0;
  if (k >= K) return i32x4{0, 0, 0, 0};
  return i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
}
__device__ __forceinline__ i32x4 load_end(const int8_t *row, int k, int K) {
  return shift_end(fetch_end(row, k, K), k, K);
}

// K below 16 (the kernels below move 16 bytes of a row at a time): 64 x 64 tiles,
// four wavefronts of 32 x 32, rows byte by byte into LDS, 48 bytes apart, and one
// product of 32 k (v_mfma_i32_32x32x32_i8), the second sixteen zeros.  The weights
// are the second operand here: neighbouring lanes then hold, and store one by one,
// neighbouring columns (4096 x 8 x 28672 bf16 91 us, the other way round 284; bound
// by those stores).
constexpr int kShortRow = 48;
constexpr long long kShortGrid = 1 << 20;
template <typename Ty>
__global__ __launch_bounds__(256) void int8_short_kernel(const Int8Args p) {
  __shared__ __attribute__((aligned(16))) uint8_t s_rows[128 * kShortRow];   // activations, weights
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = (tid >> 1) & 63, c = tid & 1;        // this thread's row and half of it
  const bool of_w = tid >= 128;
  const int g = lane >> 5, q = lane & 31;
  const int mw = (wave & 1) * 32, nw = (wave >> 1) * 32;
  const long long ntn = (p.N + 63) / 64, tiles = (p.M + 63ll) / 64 * ntn;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int m0 = (int)(t / ntn) * 64, n0 = (int)(t % ntn) * 64;
    i32x4 v = {0, 0, 0, 0};
    if (c == 0) {
      if (!of_w && r < p.M - m0) v = load_short(p.a + (long long)(m0 + r) * p.lda, p.K);
      if (of_w && r < p.N - n0) v = load_short(p.w + (long long)(n0 + r) * p.ldw, p.K);
    }
    __syncthreads();                                 // the tile before has been read
    *reinterpret_cast<i32x4 *>(s_rows + (tid >> 1) * kShortRow + 16 * c) = v;
    __syncthreads();
    const i32x4 fa = *reinterpret_cast<const i32x4 *>(s_rows + (mw + q) * kShortRow + 16 * g);
    const i32x4 fw = *reinterpret_cast<const i32x4 *>(s_rows + (64 + nw + q) * kShortRow + 16 * g);
    i32x16 acc;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0;
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa, fw, acc, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int ml = mw + 8 * (e >> 2) + 4 * g + (e & 3), nl = nw + q;
      if (ml < p.M - m0 && nl < p.N - n0) store_one<Ty>(p, m0 + ml, n0 + nl, acc[e]);
    }
  }
}

// 32 columns of one row, held in the lanes l, l + 16, l + 32, l + 48 (g = 0 .. 3):
// four sums of columns 4 g .. 4 g + 3 of the first sixteen (lo) and of the second
// (hi).  Scales, bias and addend in float32; then for float32 one 16-byte store
// of each, for the 16-bit types one of eight neighbouring columns, after one swap
// of odd and even groups of 16 lanes a register pair.  `col` is the run's first
// column in the tile that starts at column n0.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef int i32x2u __attribute__((ext_vector_type(2), aligned(2)));
template <typename Ty>
__device__ __forceinline__ void store_run(const Int8Args &p, int m, int n0, int col, int g, float sa,
                                          const float *s_sw, const float *s_bias, const i32x4 &lo,
                                          const i32x4 &hi) {
#pragma clang fp contract(off)
  typedef typename Ty::T T;
  constexpr bool kWide = sizeof(T) == 4;
  const bool row_ok = m < p.M;
  const long long row = (long long)m * p.ldo;
  const bool whole = n0 + col + 32 <= p.N;             // the same in every lane
  float f[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = col + 16 * h + 4 * g;
    const f32x4 sw = *reinterpret_cast<const f32x4 *>(s_sw + at);
#pragma unroll
    for (int c = 0; c < 4; ++c) f[4 * h + c] = (float)(h ? hi[c] : lo[c]) * sa * sw[c];
    if (p.bias) {
      const f32x4 b = *reinterpret_cast<const f32x4 *>(s_bias + at);
#pragma unroll
      for (int c = 0; c < 4; ++c) f[4 * h + c] += b[c];
    }
    if (p.addend && row_ok) {
      const T *add = (const T *)p.addend + row + n0 + at;
      if (whole) {
        T v[4];
        if constexpr (kWide) {
          const f32x4u q = *reinterpret_cast<const f32x4u *>(add);
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = q[c];
        } else {
          const i32x2u q = *reinterpret_cast<const i32x2u *>(add);
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = (T)(q[c >> 1] >> (16 * (c & 1)));
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) f[4 * h + c] += Ty::load(v[c]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n0 + at + c < p.N) f[4 * h + c] += Ty::load(add[c]);
      }
    }
  }
  T *out = (T *)p.out + row + n0;
  if constexpr (kWide) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = col + 16 * h + 4 * g;
      if (!row_ok) continue;
      if (whole) {
        *reinterpret_cast<f32x4u *>(out + at) = f32x4{f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (n0 + at + c < p.N) out[at + c] = f[4 * h + c];
      }
    }
  } else {
    int x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = Ty::pack(f[2 * q], f[2 * q + 1]);
    if (whole) {
      // groups 0, 2: eight columns of the first sixteen; 1, 3: of the second
      const auto s0 = __builtin_amdgcn_permlane16_swap(x[0], x[2], false, false);
      const auto s1 = __builtin_amdgcn_permlane16_swap(x[1], x[3], false, false);
      if (row_ok)
        *reinterpret_cast<i32x4u *>(out + col + 16 * (g & 1) + 8 * (g >> 1)) =
            i32x4{(int)s0[0], (int)s1[0], (int)s0[1], (int)s1[1]};
    } else if (row_ok) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int at = col + 16 * (c >> 2) + 4 * g + (c & 3);
        if (n0 + at < p.N) out[at] = (T)(x[c >> 1] >> (16 * (c & 1)));
      }
    }
  }
}

// ---- many rows: 256 x 256 tiles ---------------------------------------------------
// One workgroup of eight wavefronts per CU, two on each SIMD; wavefront (half,
// wn) owns 128 rows x 64 columns in 128 accumulation registers.  A stage is 64 k
// of the tile's 512 rows (32 KB), copied by direct-to-LDS DMA into one of four
// slots.  The products are v_mfma_i32_16x16x64_i8: with 64 k in one instruction
// it moves half the accumulator values a product that 32x32x32 does, and where
// power sets the clock that counts (registers only, normally distributed codes:
// 4030 TOP/s at 1.98 GHz against 3350 at 1.60 GHz).
//
// The wavefronts of the upper and the lower half of the rows work in opposite
// phase: while one half reads a stage's fragments from LDS, the other multiplies
// the stage that it read in the phase before, so that one of the two wavefronts
// of every SIMD has products to do at any time.  A barrier ends each phase.  The
// DMA of the stage three ahead goes out right behind a stage's reads, where the
// wavefront would wait anyway: its copies queue up for the CU's one address path,
// and between products they held those up (770-810 cycles for 512 cycles of
// products; all copies of a 128-k stage at once in two slots: 1900).
constexpr int kBM = 256, kBN = 256, kBK = 64;
constexpr int kBigThreads = 512;
constexpr int kRing = 4;
constexpr int kBigA = kBM * kBK;                     // bytes of activations in a slot
constexpr int kBigSlot = (kBM + kBN) * kBK;
constexpr int kBigPieces = 4;                        // copies of a wavefront and stage

// 16-byte chunk c of a 64-byte LDS row r lies at c ^ swz(r): the lanes that a
// fragment read serves at a time lie on distinct banks (counted: no conflicts)
__device__ __forceinline__ int swz(int r) { return -(r >> 2) & 3; }
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)p;
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
template <int n>
__device__ __forceinline__ void wait_dma() {         // all but the last n have landed
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}
__device__ __forceinline__ void phase_end() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Tile t of an XCD-aware order: the tiles are cut into eight contiguous runs,
// one for each XCD; inside, four row tiles go together, rows fastest, so the
// 32 tiles that an XCD works on at a time are 4 x 8.
struct TileOrder {
  int ntm, ntn;
  __device__ __forceinline__ void at(int t, int &tm, int &tn) const {
    constexpr int kRows = 4;
    const int per = kRows * ntn, g = t / per, rem = t - g * per;
    const int rows = min(kRows, ntm - g * kRows);
    tn = rem / rows;
    tm = g * kRows + rem - tn * rows;
  }
};

#define QMOE_INLINE __attribute__((always_inline))

template <typename Ty>
__global__ __launch_bounds__(kBigThreads, 2) void int8_big_kernel(const Int8Args p, TileOrder order) {
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kRing * kBigSlot];
  __shared__ float s_sa[kBM], s_sw[kBN], s_bias[kBN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = wave >> 2, wn = wave & 3;          // rows 128 half .., columns 64 wn ..
  const int g = lane >> 4, r16 = lane & 15;
  const int full = p.K / kBK;                         // whole stages
  const int tail = p.K - full * kBK;

  // this workgroup's tiles: those of its XCD's run, round robin
  const int total = order.ntm * order.ntn;
  const int G = gridDim.x, b = blockIdx.x;
  const int xcd = b & (kXcds - 1), wl = b / kXcds;
  const int gx = (G - xcd + kXcds - 1) / kXcds;
  const int run = (total + kXcds - 1) / kXcds;
  const int t_end = min((xcd + 1) * run, total);
  int t = xcd * run + wl;
  if (t >= t_end) return;

  const uint32_t ring = lds_addr(s_ring);
  // this lane's 16 bytes of the first fragment of either operand
  const uint32_t ch = (uint32_t)((g ^ swz(r16)) << 4);
  const uint32_t a_rd = (uint32_t)((half * 128 + r16) * kBK) + ch;
  const uint32_t w_rd = (uint32_t)(kBigA + (wn * 64 + r16) * kBK) + ch;

  // ---- the copy cursor: stage cur_s of tile cur_t is the next to be copied.  When
  // every stage is, the last is copied again into slots nobody reads, so that
  // the counts of copies in flight stay the same.
  int cur_t = t, cur_s = 0, cur_slot = 0;
  const int8_t *a_src = nullptr, *w_src = nullptr;
  uint32_t a_off[2], w_off[2];
  auto enter = [&](int tt) QMOE_INLINE {
    int tm, tn;
    order.at(tt, tm, tn);
    const int m0 = tm * kBM, n0 = tn * kBN;
    a_src = p.a + (long long)m0 * p.lda;
    w_src = p.w + (long long)n0 * p.ldw;
    // wavefront w copies rows 32 w .. 32 w + 31 of both operands, 16 an instruction
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 32 * wave + 16 * u + (lane >> 2);
      const uint32_t ch = 16u * (uint32_t)((lane & 3) ^ swz(r));
      a_off[u] = (uint32_t)min(r, p.M - 1 - m0) * (uint32_t)p.lda + ch;
      w_off[u] = (uint32_t)min(r, p.N - 1 - n0) * (uint32_t)p.ldw + ch;
    }
  };
  auto dma_piece = [&](int u) QMOE_INLINE {
    const uint32_t at = ring + (uint32_t)(cur_slot * kBigSlot + wave * 2048 + (u & 1) * 1024);
    if (u < 2) dma16(a_src + cur_s * kBK, a_off[u], at);
    else dma16(w_src + cur_s * kBK, w_off[u - 2], at + kBigA);
  };
  auto dma_next = [&]() QMOE_INLINE {                 // the cursor's stage is on its way
    cur_slot = (cur_slot + 1) & (kRing - 1);
    if (cur_s + 1 < full) {
      ++cur_s;
    } else if (cur_t + gx < t_end) {
      cur_t += gx;
      cur_s = 0;
      enter(cur_t);
    }
  };

  i32x4 acc[8][4];
  i32x4 fa[8], fw[4];
  auto read_stage = [&](int slot) QMOE_INLINE {
    const uint8_t *base = s_ring + slot * kBigSlot;
#pragma unroll
    for (int j = 0; j < 4; ++j) fw[j] = *reinterpret_cast<const i32x4 *>(base + w_rd + j * 16 * kBK);
#pragma unroll
    for (int i = 0; i < 8; ++i) fa[i] = *reinterpret_cast<const i32x4 *>(base + a_rd + i * 16 * kBK);
  };
  auto multiply = [&]() QMOE_INLINE {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fa[i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  };
  // the cursor's copies, behind a stage's reads
  auto copy_stage = [&]() QMOE_INLINE {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kBigPieces; ++u) dma_piece(u);
    dma_next();
    __builtin_amdgcn_sched_barrier(0);
  };

  if (full > 0) {
    enter(t);
#pragma unroll
    for (int d = 0; d < kRing - 1; ++d) copy_stage();
    wait_dma<2 * kBigPieces>();                       // stage 0 has landed here ...
  }
  phase_end();                                        // ... and everywhere
  int slot = 0;                                       // of the stage being computed
  for (;;) {
    int tm, tn;
    order.at(t, tm, tn);
    const int m0 = tm * kBM, n0 = tn * kBN;
    // scales and bias of this tile, on their way while it is computed
    float side = 0.0f, side2 = 0.0f;
    if (tid < kBN) {
      side = p.w_scale[min(n0 + tid, p.N - 1)];
      if (p.bias) side2 = p.bias[min(n0 + tid, p.N - 1)];
    } else {
      side = p.a_scale[min(m0 + tid - kBN, p.M - 1)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    // Phase 2 s: the upper half reads stage s; phase 2 s + 1: the lower half
    // does.  Stage s + 1 has to be there after phase 2 s + 1, when the upper half
    // as the lower has issued the copies up to stage s + 3.
    if (full > 0) {
      if (half == 0) {
        for (int s = 0; s < full; ++s) {
          read_stage(slot);
          copy_stage();
          wait_lds();
          phase_end();
          multiply();
          wait_dma<2 * kBigPieces>();
          phase_end();
          slot = (slot + 1) & (kRing - 1);
        }
        phase_end();
      } else {
        phase_end();
        for (int s = 0; s < full; ++s) {
          read_stage(slot);
          copy_stage();
          wait_lds();
          wait_dma<2 * kBigPieces>();
          phase_end();
          multiply();
          phase_end();
          slot = (slot + 1) & (kRing - 1);
        }
      }
    }
    if (tail > 0) {
      // the rest of k, zero past K: 512 rows of 4 chunks, through registers into
      // the slot of the last stage (the next three are being filled)
      const int k0 = full * kBK, ts = (slot + kRing - 1) & (kRing - 1);
      const int8_t *ar = p.a + (long long)m0 * p.lda, *wr = p.w + (long long)n0 * p.ldw;
#pragma unroll 1
      for (int q = tid; q < (kBM + kBN) * 4; q += kBigThreads) {
        const int r = (q >> 2) & (kBM - 1), c = q & 3;
        const bool is_a = q < kBM * 4;
        const int8_t *row = is_a ? ar + (long long)min(r, p.M - 1 - m0) * p.lda
                                 : wr + (long long)min(r, p.N - 1 - n0) * p.ldw;
        *reinterpret_cast<i32x4 *>(s_ring + ts * kBigSlot + (is_a ? 0 : kBigA) + r * kBK +
                                   ((c ^ swz(r)) << 4)) = load_end(row, k0 + 16 * c, p.K);
      }
      wait_lds();
      phase_end();
      read_stage(ts);
      multiply();
      wait_lds();
      phase_end();
    }

    if (tid < kBN) {
      s_sw[tid] = side;
      s_bias[tid] = side2;
    } else {
      s_sa[tid - kBN] = side;
    }
    wait_lds();
    phase_end();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ml = half * 128 + 16 * i + r16;
      const float sa = s_sa[ml];
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        store_run<Ty>(p, m0 + ml, n0, wn * 64 + 16 * j, g, sa, s_sw, s_bias, acc[i][j], acc[i][j + 1]);
    }
    t += gx;
    if (t >= t_end) break;
  }
  wait_dma_all();                                     // no copy into LDS outlives the workgroup
}

// ---- few rows: weights through each wavefront's own LDS ----------------------------
// Four output columns of a row from their exact sums.
template <typename Ty>
__device__ __forceinline__ void store_four(const Int8Args &p, int m, int n, float sa, const float *sw,
                                           const float *bias, const i32x4 &sum) {
#pragma clang fp contract(off)
  typedef typename Ty::T T;
  if (m >= p.M) return;
  const long long at = (long long)m * p.ldo + n;
  const T *add = (const T *)p.addend + at;
  T *out = (T *)p.out + at;
  float f[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    f[c] = (float)sum[c] * sa * sw[c];
    if (p.bias) f[c] += bias[c];
  }
  if (n + 4 <= p.N) {
    if constexpr (sizeof(T) == 4) {
      if (p.addend) {
        const f32x4u q = *reinterpret_cast<const f32x4u *>(add);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] += q[c];
      }
      *reinterpret_cast<f32x4u *>(out) = f32x4{f[0], f[1], f[2], f[3]};
    } else {
      if (p.addend) {
        const i32x2u q = *reinterpret_cast<const i32x2u *>(add);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] += Ty::load((T)(q[c >> 1] >> (16 * (c & 1))));
      }
      *reinterpret_cast<i32x2u *>(out) = i32x2{Ty::pack(f[0], f[1]), Ty::pack(f[2], f[3])};
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (n + c < p.N) out[c] = Ty::store(p.addend ? f[c] + Ty::load(add[c]) : f[c]);
  }
}

// One workgroup of kW wavefronts per 16 MB rows x 16 C columns.  The wavefronts
// share out the contraction, 128 k each in turn, and add their exact partial sums
// through LDS at the end; until then each waits for nothing but its own loads, so
// those are always under way: what a weight-bound product needs.
//
// A step's rows come as whole 128-byte lines, neighbouring lanes neighbouring
// chunks, into the wavefront's own part of LDS, from where the fragments are read.
// (Loaded straight into fragments, neighbouring lanes are in different rows: 64
// line look-ups for 1 KB, and the cache's look-ups bound the kernel; 64 x 4096 x
// 14336: 18.6 us, 12.9 this way.)  With kDma the copies go to LDS directly, kD
// steps ahead, which needs rows on 16 bytes; without, they pass through registers,
// two steps ahead, and rows may begin at any byte.
// AI: copies of activation rows a step, 8 rows each.
// With `splits` > 1, workgroup (tile, y) contracts the y-th share of k and leaves
// its sums in p.ws for int8_join_kernel.
__device__ __forceinline__ int padded_cols(int N) { return (N + 3) & ~3; }

template <typename Ty, int MB, int C, int kW, int kD, int AI, bool kDma>
__global__ __launch_bounds__(64 * kW) void int8_staged_kernel(const Int8Args p, int col_tiles,
                                                              int splits) {
  constexpr int kStep = 128, kRows = 16 * (MB + C), kSlot = kRows * kStep;
  constexpr int kPieces = AI + 2 * C;
  constexpr int kSlots = kDma ? kD : 1;
  constexpr int kRingBytes = kW * kSlots * kSlot, kPartBytes = kW * MB * C * 1024;
  static_assert(!kDma || (kD - 1) * kPieces < 64, "the copies in flight are counted in 6 bits");
  __shared__ __attribute__((aligned(1024))) uint8_t
      s_ring[kRingBytes > kPartBytes ? kRingBytes : kPartBytes];   // the partial sums reuse it
  __shared__ __attribute__((aligned(1024))) uint8_t s_end[kDma ? kSlot : 16];  // a last, shorter step
  __shared__ float s_sa[16 * MB], s_sw[16 * C], s_bias[16 * C];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int m0 = (blockIdx.x / col_tiles) * (16 * MB), n0 = (blockIdx.x % col_tiles) * (16 * C);
  const int8_t *a0 = p.a + (long long)m0 * p.lda, *w0 = p.w + (long long)n0 * p.ldw;

  // 16-byte chunk c of LDS row r lies at c ^ ((r >> 1) & 7)
  uint32_t a_off[AI], w_off[2 * C];
#pragma unroll
  for (int u = 0; u < AI; ++u) {
    const int r = 8 * u + (lane >> 3);
    a_off[u] = (uint32_t)min(r, p.M - 1 - m0) * (uint32_t)p.lda +
               16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  }
#pragma unroll
  for (int u = 0; u < 2 * C; ++u) {
    const int r = 8 * u + (lane >> 3);
    w_off[u] = (uint32_t)min(r, p.N - 1 - n0) * (uint32_t)p.ldw +
               16u * (uint32_t)((lane & 7) ^ ((r >> 1) & 7));
  }
  uint8_t *mine = s_ring + wave * kSlots * kSlot;
  const uint32_t ring = lds_addr(mine);
  auto copy = [&](int slot, int k0) QMOE_INLINE {
    const uint32_t at = ring + (uint32_t)(slot * kSlot);
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) dma16(w0 + k0, w_off[u], at + (uint32_t)(16 * MB * kStep + u * 1024));
#pragma unroll
    for (int u = 0; u < AI; ++u) dma16(a0 + k0, a_off[u], at + (uint32_t)(u * 1024));
  };

  i32x4 acc[MB][C];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  // this wavefront's whole steps turn, turn + turns, ..; every workgroup begins at
  // another (a few percent where they all run through the same lines of k)
  const int turn = (int)blockIdx.y * kW + wave, turns = splits * kW;
  const int whole = p.K / kStep;
  const int steps = kDma ? whole : (p.K + kStep - 1) / kStep;        // with registers the last too
  const int n = (steps - turn + turns - 1) / turns;
  int at = n > 0 ? (int)(blockIdx.x / kXcds) % n : 0;
  auto next = [&]() QMOE_INLINE -> int {
    const int k = (at * turns + turn) * kStep;
    at = at + 1 < n ? at + 1 : 0;
    return k;
  };
  // The 16-byte chunks behind the whole steps are a step of the wavefront whose
  // turn it is, copied first (chunks past the last repeat it: activations are
  // masked below).
  const int end = whole * kStep, chunks = (p.K - end) / 16, rest = (p.K - end) & 15;
  const bool ends = whole % turns == turn;
  if (kDma && ends && chunks > 0) {
    const uint32_t at_end = lds_addr(s_end);
#pragma unroll
    for (int u = 0; u < 2 * C; ++u) {
      const int r = 8 * u + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      dma16(w0 + end, w_off[u] - 16u * (uint32_t)max(0, c - (chunks - 1)),
            at_end + (uint32_t)(16 * MB * kStep + u * 1024));
    }
#pragma unroll
    for (int u = 0; u < AI; ++u) {
      const int r = 8 * u + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      dma16(a0 + end, a_off[u] - 16u * (uint32_t)max(0, c - (chunks - 1)), at_end + (uint32_t)(u * 1024));
    }
  }
  // without kDma: a step's rows on their way to LDS
  struct Rows {
    i32x4 a[AI], w[2 * C];
  };
  auto fetch = [&](Rows &x, int k0) QMOE_INLINE {
    if (k0 + kStep <= p.K) {
#pragma unroll
      for (int u = 0; u < 2 * C; ++u) __builtin_memcpy(&x.w[u], w0 + k0 + w_off[u], 16);
#pragma unroll
      for (int u = 0; u < AI; ++u) __builtin_memcpy(&x.a[u], a0 + k0 + a_off[u], 16);
    } else {                                          // zero past K
#pragma unroll
      for (int u = 0; u < 2 * C; ++u) {
        const int c = 16 * ((lane & 7) ^ (((8 * u + (lane >> 3)) >> 1) & 7));
        x.w[u] = load_end(w0 + w_off[u] - c, k0 + c, p.K);
      }
#pragma unroll
      for (int u = 0; u < AI; ++u) {
        const int c = 16 * ((lane & 7) ^ (((8 * u + (lane >> 3)) >> 1) & 7));
        x.a[u] = load_end(a0 + a_off[u] - c, k0 + c, p.K);
      }
    }
  };
  auto put = [&](const Rows &x) QMOE_INLINE {
#pragma unroll
    for (int u = 0; u < 2 * C; ++u)
      *reinterpret_cast<i32x4 *>(mine + 16 * MB * kStep + u * 1024 + lane * 16) = x.w[u];
#pragma unroll
    for (int u = 0; u < AI; ++u) *reinterpret_cast<i32x4 *>(mine + u * 1024 + lane * 16) = x.a[u];
  };
  Rows x0, x1;
  if constexpr (kDma) {
#pragma unroll
    for (int d = 0; d < kD; ++d)
      if (d < n) copy(d, next());
  } else {
    if (n > 0) fetch(x0, next());
    if (n > 1) fetch(x1, next());
  }
  // scales and bias, behind the first copies
  float side = 0.0f, side2 = 0.0f;
  const int q = tid - 16 * C;
  if (tid < 16 * C) {
    side = p.w_scale[min(n0 + tid, p.N - 1)];
    if (p.bias) side2 = p.bias[min(n0 + tid, p.N - 1)];
  } else if (q < 16 * MB) {
    side = p.a_scale[min(m0 + q, p.M - 1)];
  }
  static_assert(16 * (MB + C) <= 64 * kW, "a thread for every scale");
  const uint32_t sw = (uint32_t)((r16 >> 1) & 7);
  i32x4 fa[MB][2], fw[C][2];
  auto read = [&](const uint8_t *from) QMOE_INLINE {
    const uint8_t *base = from + r16 * kStep;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t ch = (((uint32_t)(4 * c + g)) ^ sw) << 4;
#pragma unroll
      for (int j = 0; j < C; ++j)
        fw[j][c] = *reinterpret_cast<const i32x4 *>(base + ch + 16 * (MB + j) * kStep);
#pragma unroll
      for (int i = 0; i < MB; ++i)
        fa[i][c] = *reinterpret_cast<const i32x4 *>(base + ch + 16 * i * kStep);
    }
  };
  auto multiply = [&](int c) QMOE_INLINE {
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int i = 0; i < MB; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j][c], fa[i][c], acc[i][j], 0, 0, 0);
  };
  if constexpr (kDma) {
    int slot = 0;
    for (int i = 0; i < n; ++i) {
      if (i + kD <= n) wait_dma<(kD - 1) * kPieces>();
      else wait_dma_all();
      read(mine + slot * kSlot);
      wait_lds();                                     // the slot has been read
      if (i + kD < n) copy(slot, next());
      multiply(0);
      multiply(1);
      slot = slot + 1 < kD ? slot + 1 : 0;
    }
    if (ends && chunks > 0) {
      wait_dma_all();
      read(s_end);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
          if (4 * c + g >= chunks) fa[i][c] = i32x4{0, 0, 0, 0};
        multiply(c);
      }
    }
    if (ends && rest > 0) {                           // the last bytes, straight from memory
      const int k = p.K - rest;
#pragma unroll
      for (int j = 0; j < C; ++j)
        fw[j][0] = load_end(w0 + (long long)min(16 * j + r16, p.N - 1 - n0) * p.ldw, k, p.K);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        fa[i][0] = load_end(a0 + (long long)min(16 * i + r16, p.M - 1 - m0) * p.lda, k, p.K);
        if (g > 0) fa[i][0] = i32x4{0, 0, 0, 0};
      }
      multiply(0);
    }
  } else {
    // a wavefront's LDS accesses are carried out in order: no barrier between its
    // writes and reads
    auto step = [&](Rows &x, int i) QMOE_INLINE {
      put(x);
      if (i + 2 < n) fetch(x, next());
      wait_lds();
      read(mine);
      wait_lds();
      multiply(0);
      multiply(1);
    };
    for (int i = 0; i < n; i += 2) {
      step(x0, i);
      if (i + 1 < n) step(x1, i + 1);
    }
  }

  if (tid < 16 * C) {
    s_sw[tid] = side;
    s_bias[tid] = side2;
  } else if (q < 16 * MB) {
    s_sa[q] = side;
  }
  __syncthreads();                                    // every wavefront is done with its ring
  i32x4 *part = reinterpret_cast<i32x4 *>(s_ring);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < C; ++j) part[(wave * MB * C + i * C + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int f = wave; f < MB * C; f += kW) {
    i32x4 sum = part[f * 64 + lane];
#pragma unroll
    for (int w = 1; w < kW; ++w) sum += part[(w * MB * C + f) * 64 + lane];
    const int i = f / C, col = 16 * (f - i * C) + 4 * g, m = m0 + 16 * i + r16, nn = n0 + col;
    if (splits == 1) {
      store_four<Ty>(p, m, nn, s_sa[16 * i + r16], s_sw + col, s_bias + col, sum);
    } else if (m < p.M && nn < p.N) {
      const long long np = padded_cols(p.N);
      *reinterpret_cast<i32x4 *>(p.ws + ((long long)blockIdx.y * p.M + m) * np + nn) = sum;
    }
  }
}

// The shares' exact sums added, four columns a thread, and the epilogue.
template <typename Ty>
__global__ __launch_bounds__(256) void int8_join_kernel(const Int8Args p, int splits) {
  const int np = padded_cols(p.N), quads = np / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)p.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i - (long long)m * quads) * 4;
  i32x4 sum = {0, 0, 0, 0};
  for (int y = 0; y < splits; ++y)
    sum += *reinterpret_cast<const i32x4 *>(p.ws + ((long long)y * p.M + m) * np + n);
  float sw[4], bias[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    sw[c] = p.w_scale[min(n + c, p.N - 1)];
    bias[c] = p.bias ? p.bias[min(n + c, p.N - 1)] : 0.0f;
  }
  store_four<Ty>(p, m, n, p.a_scale[m], sw, bias, sum);
}

// ---- a few hundred rows: 128 x 128 tiles, the contraction in two halves -----------------
// Eight wavefronts in two groups of four; each group contracts one half of k over
// the whole tile (wavefront: 64 x 64 outputs), with its own ring of four 64-k
// stages, so every SIMD has two wavefronts even where the output has no more
// tiles than the card CUs.  A stage's fragments are read while the one before is
// multiplied; one barrier a stage.  The groups' exact sums meet in LDS.  Without
// kDma (rows that begin at any byte) a stage passes through registers: fetched
// two steps before it is written to LDS, which is one before it is read.
// With more than one share of k, workgroup (tile, y) contracts the y-th and leaves
// its sums in p.ws for int8_join_kernel.
struct Shares {
  int n, each, more;                                  // `each` stages, one more in the first `more`
};
constexpr int kMM = 128, kMN = 128;
constexpr int kMidSlot = (kMM + kMN) * kBK;          // 16 KB
constexpr int kMidPieces = 4;

template <typename Ty, bool kDma>
__global__ __launch_bounds__(512, 2) void int8_mid_kernel(const Int8Args p, TileOrder order,
                                                           Shares shares) {
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[2 * kRing * kMidSlot];
  __shared__ float s_sa[kMM], s_sw[kMN], s_bias[kMN];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2, wm = wave & 1, wn = (wave >> 1) & 1;
  const int g = lane >> 4, r16 = lane & 15;
  const int total = order.ntm * order.ntn, run = (total + kXcds - 1) / kXcds;
  const int t = (int)(blockIdx.x & (kXcds - 1)) * run + (int)blockIdx.x / kXcds;
  if ((int)blockIdx.x / kXcds >= run || t >= total) return;
  int tm, tn;
  order.at(t, tm, tn);
  const int m0 = tm * kMM, n0 = tn * kMN;
  const int8_t *a0 = p.a + (long long)m0 * p.lda, *w0 = p.w + (long long)n0 * p.ldw;

  // this share's whole stages: group 0 the first half
  const int all = p.K / kBK, y = blockIdx.y;
  const int from = y * shares.each + min(y, shares.more), whole = shares.each + (y < shares.more);
  const int first = from + (grp ? (whole + 1) / 2 : 0);
  const int mine = grp ? whole / 2 : (whole + 1) / 2, steps = (whole + 1) / 2;

  // this wavefront's copies: rows 32 w .. of both operands, w its number in the group
  const int w4 = wave & 3;
  uint32_t a_off[2], w_off[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = 32 * w4 + 16 * u + (lane >> 2);
    const uint32_t ch = 16u * (uint32_t)((lane & 3) ^ swz(r));
    a_off[u] = (uint32_t)min(r, p.M - 1 - m0) * (uint32_t)p.lda + ch;
    w_off[u] = (uint32_t)min(r, p.N - 1 - n0) * (uint32_t)p.ldw + ch;
  }
  uint8_t *base = s_ring + grp * kRing * kMidSlot;
  const uint32_t ring = lds_addr(base);
  // past the last stage it is copied again, into a slot that is not read any more
  auto copy = [&](int s) QMOE_INLINE {
    const int k0 = (first + min(s, mine - 1)) * kBK;
    const uint32_t at = ring + (uint32_t)((s & (kRing - 1)) * kMidSlot + w4 * 2048);
#pragma unroll
    for (int u = 0; u < 2; ++u) dma16(a0 + k0, a_off[u], at + (uint32_t)(u * 1024));
#pragma unroll
    for (int u = 0; u < 2; ++u) dma16(w0 + k0, w_off[u], at + (uint32_t)(kMM * kBK + u * 1024));
  };
  const uint32_t ch = (uint32_t)((g ^ swz(r16)) << 4);
  const uint32_t a_rd = (uint32_t)((wm * 64 + r16) * kBK) + ch;
  const uint32_t w_rd = (uint32_t)((kMM + wn * 64 + r16) * kBK) + ch;
  struct Frags {
    i32x4 a[4], w[4];
  };
  auto read = [&](Frags &f, int s) QMOE_INLINE {
    const uint8_t *q = base + (s & (kRing - 1)) * kMidSlot;
#pragma unroll
    for (int j = 0; j < 4; ++j) f.w[j] = *reinterpret_cast<const i32x4 *>(q + w_rd + j * 16 * kBK);
#pragma unroll
    for (int i = 0; i < 4; ++i) f.a[i] = *reinterpret_cast<const i32x4 *>(q + a_rd + i * 16 * kBK);
  };
  i32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto multiply = [&](const Frags &f) QMOE_INLINE {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[j], f.a[i], acc[i][j], 0, 0, 0);
  };

  struct Rows {
    i32x4 v[kMidPieces];
  };
  auto fetch = [&](Rows &x, int s) QMOE_INLINE {
    const int k0 = (first + min(s, mine - 1)) * kBK;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      __builtin_memcpy(&x.v[u], a0 + k0 + a_off[u], 16);
      __builtin_memcpy(&x.v[u + 2], w0 + k0 + w_off[u], 16);
    }
  };
  auto put = [&](const Rows &x, int s) QMOE_INLINE {
    uint8_t *at = base + (s & (kRing - 1)) * kMidSlot + w4 * 2048 + lane * 16;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      *reinterpret_cast<i32x4 *>(at + u * 1024) = x.v[u];
      *reinterpret_cast<i32x4 *>(at + kMM * kBK + u * 1024) = x.v[u + 2];
    }
  };
  float side = 0.0f, side2 = 0.0f;
  Frags f0, f1;
  Rows x0, x1;
  if (mine > 0) {
    if constexpr (kDma) {
#pragma unroll
      for (int s = 0; s < kRing; ++s) copy(s);
    } else {
      Rows y0, y1;
      fetch(y0, 0);
      fetch(y1, 1);
      fetch(x0, 2);
      fetch(x1, 3);
      put(y0, 0);
      put(y1, 1);
    }
  }
  if (tid < kMN) {
    side = p.w_scale[min(n0 + tid, p.N - 1)];
    if (p.bias) side2 = p.bias[min(n0 + tid, p.N - 1)];
  } else if (tid < kMN + kMM) {
    side = p.a_scale[min(m0 + tid - kMN, p.M - 1)];
  }
  if (tid < kMN) {
    s_sw[tid] = side;
    s_bias[tid] = side2;
  } else if (tid < kMN + kMM) {
    s_sa[tid - kMN] = side;
  }
  // the last bytes of the rows, straight from memory: fetched here, used at the end
  Frags fe;
  const bool ends = grp == 1 && y == shares.n - 1 && p.K > all * kBK;
  const int ke = all * kBK + 16 * g;
  if (ends) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      fe.w[j] = fetch_end(w0 + (long long)min(wn * 64 + 16 * j + r16, p.N - 1 - n0) * p.ldw, ke, p.K);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      fe.a[i] = fetch_end(a0 + (long long)min(wm * 64 + 16 * i + r16, p.M - 1 - m0) * p.lda, ke, p.K);
  }
  // Stage s + 1 has landed everywhere, and everybody has read stage s, after the
  // barrier of step s; the copies of the two stages behind it may be under way.
  if constexpr (kDma) wait_dma<3 * kMidPieces>();
  wait_lds();
  phase_end();
  if (mine > 0) read(f0, 0);
  wait_lds();
  // a step's reads and copies go between its products, where they do not hold them up
  auto step = [&](Frags &now, Frags &then, Rows &x, int s) QMOE_INLINE {
    if constexpr (kDma) wait_dma<2 * kMidPieces>();
    phase_end();
    const uint8_t *q = base + ((s + 1) & (kRing - 1)) * kMidSlot;
    const int k0 = (first + min(s + kRing, mine - 1)) * kBK;
    const uint32_t at = ring + (uint32_t)((s & (kRing - 1)) * kMidSlot + w4 * 2048);
    if (s < mine) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int j = e >> 2, i = e & 3;
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(now.w[j], now.a[i], acc[i][j], 0, 0, 0);
        if ((e & 1) == 0) {
          const int r = e >> 1;
          if (r < 4) then.w[r] = *reinterpret_cast<const i32x4 *>(q + w_rd + r * 16 * kBK);
          else then.a[r - 4] = *reinterpret_cast<const i32x4 *>(q + a_rd + (r - 4) * 16 * kBK);
        } else if (!kDma) {
          if (e == 1) put(x, s + 2);
          if (e == 9) fetch(x, s + 4);
        } else if ((e & 3) == 3) {
          const int u = e >> 2;
          if (u < 2) dma16(a0 + k0, a_off[u], at + (uint32_t)(u * 1024));
          else dma16(w0 + k0, w_off[u - 2], at + (uint32_t)(kMM * kBK + (u - 2) * 1024));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_lds();
  };
  for (int s = 0; s < steps; s += 2) {
    step(f0, f1, x0, s);
    if (s + 1 < steps) step(f1, f0, x1, s + 1);
  }
  if (ends) {
#pragma unroll
    for (int j = 0; j < 4; ++j) fe.w[j] = shift_end(fe.w[j], ke, p.K);
#pragma unroll
    for (int i = 0; i < 4; ++i) fe.a[i] = shift_end(fe.a[i], ke, p.K);
    multiply(fe);
  }

  wait_dma_all();                                     // no copy lands in what follows
  phase_end();
  // group 0 finishes the rows i = 0, 1 of its wavefronts, group 1 the rows i = 2, 3
  i32x4 *part = reinterpret_cast<i32x4 *>(s_ring);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      part[((wave * 2 + i) * 4 + j) * 64 + lane] = grp ? acc[i][j] : acc[i + 2][j];
  wait_lds();
  phase_end();
  const int other = wave ^ 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int ml = wm * 64 + 16 * (2 * grp + i) + r16;
    const float sa = s_sa[ml];
    i32x4 sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sum[j] = (grp ? acc[i + 2][j] : acc[i][j]) + part[((other * 2 + i) * 4 + j) * 64 + lane];
    if (shares.n > 1) {
      const int m = m0 + ml, np = padded_cols(p.N);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + wn * 64 + 16 * j + 4 * g;
        if (m < p.M && n < np)
          *reinterpret_cast<i32x4 *>(p.ws + ((long long)y * p.M + m) * np + n) = sum[j];
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      store_run<Ty>(p, m0 + ml, n0, wn * 64 + 16 * j, g, sa, s_sw, s_bias, sum[j], sum[j + 1]);
  }
}

}  // namespace

namespace {

int compute_units() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  return n;
}

long long tiles_of(int M, int N, int tm, int tn) {
  return (long long)((M + tm - 1) / tm) * ((N + tn - 1) / tn);
}

// The kernels and their tiles, by the time they take: rounds of one workgroup a CU
// (of two for up to 16 rows), each a fixed part and one that grows with K, in us
// for K = 4096, fitted to measured calls.  The least by that count wins.
//   int8_staged_kernel, 64 rows: 16, 32, 64 columns 1.5 + 2.5, 2 + 3, 3.2 + 5.6
//     (64 x 4096 x 4096: 6.4, 7.3, 9.7 with the launch; 64 x 4096 x 14336: 20.5,
//     14.5, 12.9); up to 16 rows: 16, 32 columns 0.6 + 0.5, 0.9 + 0.9 (1 x 4096 x
//     14336: 11.0, 10.3)
//   int8_mid_kernel 2.7 + 18, int8_big_kernel 5.5 + 33
// On both sides of the borders (us, staged / mid / big, M x K x N): 512 x 2048 x
// 4096 14.0 / 13.1 / 23.3, 512 x 4096 x 4096 19.9 / 20.4 / 38.1, 200 x 512 x 16384
// 16.2 / 8.2 / 11.9, 1024 x 64 x 8192 30.4 / 10.1 / 9.9, 1024 x 2048 x 8192 52.1 /
// 29.5 / 25.0, 732 x 7872 x 7168 104.8 / 81.5 / 79.1.
constexpr int kCus = 256;
struct Cost {
  double fixed, at_4096;
  double of(long long tiles, int at_once, int K) const {
    return (double)((tiles + at_once - 1) / at_once) * (fixed + at_4096 * K / 4096.0);
  }
};
struct StagedShape {
  int mb, c, splits;                                  // 16 mb rows, 16 c columns, shares of k
  double us;
};
StagedShape staged_shape(int M, int K, int N) {
  constexpr Cost kFew[2] = {{0.6, 0.5}, {0.9, 0.9}}, kMore[3] = {{1.5, 2.5}, {2.0, 3.0}, {3.2, 5.6}};
  const int mb = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  StagedShape best{mb, 1, 1, 1e300};
  for (int i = 0; i < (mb == 1 ? 2 : 3); ++i) {
    const long long tiles = tiles_of(M, N, 16 * mb, 16 << i);
    double us = mb == 1 ? kFew[i].of(tiles, 2 * kCus, K) : kMore[i].of(tiles, kCus, K);
    // every tile reads its rows of both operands, at 14 TB/s together (by that count
    // 128 x 128 tiles in shares: 512 x 14336 x 4096 76.0 -> 47.7 us, 256 x 14336 x
    // 4096 39.6 -> 30.8; nearest border 256 x 14336 x 2048 21.9, in shares 24.2)
    const double read = (double)tiles * (16 * mb + (16 << i)) * K / 14e6;
    if (mb > 1 && us < read) us = read;
    if (us < best.us) best = {mb, 1 << i, 1, us};
  }
  // Shares of k where the tiles leave three quarters of the CUs idle and each
  // has a long way to go: 512 k of every wavefront (a second launch costs 4 us;
  // 64 x 14336 x 1024 in shares: 10.4 us, whole: 13.9)
  const long long tiles = tiles_of(M, N, 16 * mb, 16 * best.c);
  if (tiles <= kCus / 4) {
    const long long room = kCus / tiles, work = K / 2048;
    best.splits = (int)(room < work ? room : work);
    if (best.splits < 3) best.splits = 1;
  }
  return best;
}

// 128 x 128 tiles, in shares of k where the tiles are few and the sums' way through
// the workspace costs less than it saves: 4.5 us for the second launch and 4 TB/s
// for the sums (whole, in shares: 512 x 14336 x 4096 60.3, 47.1 us, 384 x 14336 x
// 4096 58.8, 42.0, 768 x 8192 x 2048 34.3, 29.5).  All shares run at once: each XCD
// has 32 CUs for its run of the tiles (84 tiles in three shares, 33 a XCD: 35.2 us,
// in two 25.3).
struct MidShape {
  int splits;
  double us;
};
MidShape mid_shape(int M, int K, int N) {
  constexpr Cost kMidCost{2.7, 18.0};
  const long long tiles = tiles_of(M, N, kMM, kMN), run = (tiles + kXcds - 1) / kXcds;
  MidShape best{1, kMidCost.of(tiles, kCus, K)};
  for (int s = 2; s <= 16 && run * s <= kCus / kXcds && K / kBK >= 8 * s; ++s) {
    const double us = 2.7 + 18.0 * K / 4096.0 / s + 4.5 + 8.0 * s * M * (double)N / 4e6;
    if (us < best.us) best = {s, us};
  }
  return best;
}

enum Kind { kStaged, kMid, kBig };
Kind kind_of(int M, int K, int N) {
  constexpr Cost kBigCost{5.5, 33.0};
  const double staged = staged_shape(M, K, N).us;
  const double mid = mid_shape(M, K, N).us;
  const double big = kBigCost.of(tiles_of(M, N, kBM, kBN), kCus, K);
  if (staged <= mid && staged <= big) return kStaged;
  return mid < big ? kMid : kBig;
}

size_t sums_bytes(int splits, int M, int N) {
  return splits == 1 ? 0 : (size_t)splits * M * ((N + 3) / 4 * 4) * sizeof(int);
}

template <typename Ty>
hipError_t launch_join(const Int8Args &a, int splits, hipStream_t s) {
  const long long quads = (long long)a.M * ((a.N + 3) / 4);
  hipLaunchKernelGGL(int8_join_kernel<Ty>, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s, a,
                     splits);
  return hipGetLastError();
}

template <typename Ty, int MB, int C, int kD, int AI, bool kDma>
hipError_t launch_staged(const Int8Args &a, int splits, hipStream_t s) {
  constexpr int kW = 4;
  const int cols = (a.N + 16 * C - 1) / (16 * C), rows = (a.M + 16 * MB - 1) / (16 * MB);
  hipLaunchKernelGGL((int8_staged_kernel<Ty, MB, C, kW, kD, AI, kDma>),
                     dim3((unsigned)(cols * rows), (unsigned)splits), dim3(64 * kW), 0, s, a, cols,
                     splits);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || splits == 1 ? e : launch_join<Ty>(a, splits, s);
}

template <typename Ty, bool kDma>
hipError_t launch_staged_shape(const Int8Args &a, StagedShape t, hipStream_t s) {
  if (!a.ws) t.splits = 1;
  if (t.mb == 1 && t.c == 1)
    return a.M <= 8 ? launch_staged<Ty, 1, 1, 4, 1, kDma>(a, t.splits, s)
                    : launch_staged<Ty, 1, 1, 4, 2, kDma>(a, t.splits, s);
  if (t.mb == 1)
    return a.M <= 8 ? launch_staged<Ty, 1, 2, 3, 1, kDma>(a, t.splits, s)
                    : launch_staged<Ty, 1, 2, 3, 2, kDma>(a, t.splits, s);
  if (t.mb == 2)
    return t.c == 1   ? launch_staged<Ty, 2, 1, 4, 4, kDma>(a, t.splits, s)
           : t.c == 2 ? launch_staged<Ty, 2, 2, 4, 4, kDma>(a, t.splits, s)
                      : launch_staged<Ty, 2, 4, 3, 4, kDma>(a, t.splits, s);
  return t.c == 1   ? launch_staged<Ty, 4, 1, 2, 8, kDma>(a, t.splits, s)
         : t.c == 2 ? launch_staged<Ty, 4, 2, 2, 8, kDma>(a, t.splits, s)
                    : launch_staged<Ty, 4, 4, 2, 8, kDma>(a, t.splits, s);
}

template <typename Ty>
hipError_t launch(const Int8Args &a, hipStream_t s) {
  if (a.K < 16) {
    const long long tiles = tiles_of(a.M, a.N, 64, 64);
    hipLaunchKernelGGL(int8_short_kernel<Ty>, dim3((unsigned)(tiles < kShortGrid ? tiles : kShortGrid)),
                       dim3(256), 0, s, a);
    return hipGetLastError();
  }
  // rows that direct-to-LDS copies can take
  const bool aligned = ((uintptr_t)a.a & 15) == 0 && ((uintptr_t)a.w & 15) == 0 && a.lda % 16 == 0 &&
                       a.ldw % 16 == 0;
  const Kind kind = kind_of(a.M, a.K, a.N);
  if (!aligned && kind == kStaged)
    return launch_staged_shape<Ty, false>(a, staged_shape(a.M, a.K, a.N), s);
  if (kind == kStaged) return launch_staged_shape<Ty, true>(a, staged_shape(a.M, a.K, a.N), s);
  if (kind == kMid || !aligned) {
    const TileOrder order{(a.M + kMM - 1) / kMM, (a.N + kMN - 1) / kMN};
    const long long tiles = (long long)order.ntm * order.ntn;
    const int splits = kind == kMid && a.ws ? mid_shape(a.M, a.K, a.N).splits : 1;
    const dim3 grid((unsigned)((tiles + kXcds - 1) / kXcds * kXcds), (unsigned)splits);
    const Shares shares{splits, a.K / kBK / splits, a.K / kBK % splits};
    if (aligned) hipLaunchKernelGGL((int8_mid_kernel<Ty, true>), grid, dim3(512), 0, s, a, order, shares);
    else hipLaunchKernelGGL((int8_mid_kernel<Ty, false>), grid, dim3(512), 0, s, a, order, shares);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || splits == 1 ? e : launch_join<Ty>(a, splits, s);
  }
  const TileOrder order{(a.M + kBM - 1) / kBM, (a.N + kBN - 1) / kBN};
  const long long tiles = (long long)order.ntm * order.ntn;
  // a workgroup for every tile of every XCD's run, as far as there are CUs
  const long long all = (tiles + kXcds - 1) / kXcds * kXcds, cus = compute_units();
  hipLaunchKernelGGL(int8_big_kernel<Ty>, dim3((unsigned)(all < cus ? all : cus)), dim3(kBigThreads), 0,
                     s, a, order);
  return hipGetLastError();
}

}  // namespace

size_t int8_workspace_bytes(int M, int K, int N) {
  if (K < 16) return 0;
  switch (kind_of(M, K, N)) {
    case kStaged: return sums_bytes(staged_shape(M, K, N).splits, M, N);
    case kMid: return sums_bytes(mid_shape(M, K, N).splits, M, N);
    default: return 0;
  }
}

hipError_t launch_int8_gemm(const Int8Args &a, int out_dtype, hipStream_t s) {
  if (out_dtype == MOE_F32) return launch<TypeF32>(a, s);
  if (out_dtype == MOE_BF16) return launch<TypeBf16>(a, s);
  return launch<TypeF16>(a, s);
}

}  // namespace qmoe
