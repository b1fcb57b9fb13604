// Dense int8 product with a scale per token and per output channel:
//   out[m, n] = round((sum_k a[m,k] w[n,k]) * a_scale[m] * w_scale[n] + bias[n] + addend[m, n])
// The sums are exact: int8 products added in int32 on the int8 MFMA.
#include "qmoe_device.h"
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
                                   ((c ^ swz(r)) << 4)) = load16(row, k0 + 16 * c, p.K);
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

}  // namespace

size_t int8_workspace_bytes(int, int, int) { return 0; }

namespace {

int compute_units() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  return n;
}

template <typename Ty>
hipError_t launch(const Int8Args &a, hipStream_t s) {
  // rows that direct-to-LDS copies can take
  const bool aligned = ((uintptr_t)a.a & 15) == 0 && ((uintptr_t)a.w & 15) == 0 && a.lda % 16 == 0 &&
                       a.ldw % 16 == 0;
  if (aligned && a.M > 256) {
    const TileOrder order{(a.M + kBM - 1) / kBM, (a.N + kBN - 1) / kBN};
    const long long tiles = (long long)order.ntm * order.ntn;
    const int cus = compute_units();
    hipLaunchKernelGGL(int8_big_kernel<Ty>, dim3((unsigned)(tiles < cus ? tiles : cus)),
                       dim3(kBigThreads), 0, s, a, order);
    return hipGetLastError();
  }
  const dim3 g((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64)), b(256);
  hipLaunchKernelGGL(int8_any_kernel<Ty>, g, b, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_gemm(const Int8Args &a, int out_dtype, hipStream_t s) {
  if (out_dtype == MOE_F32) return launch<TypeF32>(a, s);
  if (out_dtype == MOE_BF16) return launch<TypeBf16>(a, s);
  return launch<TypeF16>(a, s);
}

}  // namespace qmoe
