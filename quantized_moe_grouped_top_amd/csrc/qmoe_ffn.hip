// The grouped 16-bit products of the experts' gated feed-forward: forward (both
// projections with the activation and the product in the epilogue), the linear
// back down, the input gradients (one with the activation's gradient in the
// epilogue) and the weight gradients.
//
// All five are one kernel over three operand layouts.  An operand whose rows run
// along the contraction is copied to LDS row by row and its fragments are read as
// they lie; one whose rows run across it (the weights of an input gradient, both
// operands of a weight gradient) is copied row by row as well and its fragments are
// read by ds_read_b64_tr_b16, which transposes 16-bit values on the way: no operand
// is ever laid out again in memory.
//
// Between two products h and [dg | du] are rounded to the caller's 16-bit type: the matrix
// instructions take no wider one, and a second part of them would double the products
// behind and the bytes in between.  A whole pass is off by 1.41 times what the last
// rounding alone costs (bf16 0.0024 of its rms against 0.0017, fp16 0.00029 and 0.00021).
#include "qmoe_block.h"
#include "qmoe_device.h"
#include <type_traits>

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
// The gradient's g is the stored one, infinite where it left its type's range on the way
// forward: there act and act' are their limits, 0 and 0, an infinity and 1.
__device__ __forceinline__ void act_both(float g, int act, float &a, float &da) {
  float z = g, dz = 1.0f;
  if (act != MOE_GATED_SILU) {
    const float gc = __builtin_amdgcn_fmed3f(g, -1e4f, 1e4f);
    z = 1.5957691216057308f * gc * (1.0f + 0.044715f * gc * gc);
    dz = 1.5957691216057308f * (1.0f + 3.0f * 0.044715f * gc * gc);
  }
  const float s = 1.0f / (1.0f + __expf(-z));
  a = __builtin_elementwise_maximum(g, -__FLT_MAX__) * s;             // (these keep a NaN)
  da = s + __builtin_elementwise_minimum(a, __FLT_MAX__) * (1.0f - s) * dz;
}

#define QMOE_INLINE __attribute__((always_inline))

typedef short s16x4 __attribute__((ext_vector_type(4)));

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

// buffer_load_dwordx4 to LDS: lane l copies 16 bytes from base + voff to LDS byte
// address m0 + 16 l, zeros where voff is kOut.  (The wait states are those between
// a vector instruction that writes a scalar register and a memory one reading it.)
constexpr uint32_t kOut = 0x80000000u;
__device__ __forceinline__ void dma16z(const uint16_t *base, uint32_t voff, uint32_t lds) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  i32x4 rsrc;
  rsrc[0] = __builtin_amdgcn_readfirstlane((int)b);
  rsrc[1] = __builtin_amdgcn_readfirstlane((int)(b >> 32) & 0xFFFF);
  rsrc[2] = (int)kOut;                                // bytes from base that are memory
  rsrc[3] = 0x00020000;
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory", "m0");
}

// Where the experts' rows lie and how their tiles are counted.
struct Segments {
  int lo[kMaxExperts], hi[kMaxExperts];
  int first[kMaxExperts + 2];                         // first tile of every expert; then the total
  float cost[kMaxExperts + 2];                        // the cost of all tiles before its first
};
// All threads (two wavefronts at least) take part; `tiles` gives an expert's tiles
// by its rows, `cost` what one of them takes.
template <typename F, typename C>
__device__ __forceinline__ void find_segments(Segments &s, const int *off, int rows, int E, F tiles, C cost) {
  const int tid = threadIdx.x;
  if (tid < kMaxExperts) {
    int lo = 0, hi = 0;
    if (tid < E) {
      lo = off ? min(max(off[tid], 0), rows) : 0;
      hi = off ? min(max(off[tid + 1], lo), rows) : rows;
    }
    s.lo[tid] = lo;
    s.hi[tid] = hi;
  }
  __syncthreads();
  if (tid < 64) {                                     // two experts a lane
    const int e = 2 * tid;
    const int na = s.hi[e] - s.lo[e], nb = s.hi[e + 1] - s.lo[e + 1];
    const int a = e < E ? tiles(na) : 0, b = e + 1 < E ? tiles(nb) : 0;
    const float ca = a ? (float)a * cost(na) : 0.0f, cb = b ? (float)b * cost(nb) : 0.0f;
    int sum = a + b;
    float all = ca + cb;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d);
      const float c = __shfl_up(all, d);
      if (tid >= d) {
        sum += v;
        all += c;
      }
    }
    s.first[e] = sum - a - b;
    s.first[e + 1] = sum - b;
    s.cost[e] = all - ca - cb;
    s.cost[e + 1] = all - cb;
    if (tid == 63) {
      s.first[kMaxExperts] = sum;
      s.cost[kMaxExperts] = all;
    }
  }
  __syncthreads();
}
// First tile of the x-th of eight contiguous runs of equal cost.
__device__ __forceinline__ int run_start(const Segments &s, int E, int x) {
  const int total = __builtin_amdgcn_readfirstlane(s.first[kMaxExperts]);
  if (x == 0) return 0;
  if (x >= kXcds) return total;
  const float at = s.cost[kMaxExperts] * ((float)x / (float)kXcds);
  int e = 0;                                          // the last expert that begins at or before it
  while (e + 1 < E && s.cost[e + 1] <= at) ++e;
  const int n = s.first[e + 1] - s.first[e];
  const float each = n > 0 ? (s.cost[e + 1] - s.cost[e]) / (float)n : 1.0f;
  const int t = s.first[e] + min(n, (int)((at - s.cost[e]) / each));
  return __builtin_amdgcn_readfirstlane(min(t, total));
}

// Eight neighbouring columns a lane from two fragments of four each: groups 0 and 2
// get the first fragment's, 1 and 3 the second's, columns 8 (g >> 1) .. of it.
__device__ __forceinline__ i32x4 join8(int a0, int a1, int b0, int b1) {
  const auto s0 = __builtin_amdgcn_permlane16_swap(a0, b0, false, false);
  const auto s1 = __builtin_amdgcn_permlane16_swap(a1, b1, false, false);
  return i32x4{(int)s0[0], (int)s1[0], (int)s0[1], (int)s1[1]};
}
template <typename Ty>
__device__ __forceinline__ i32x4 join8(const f32x4 &a, const f32x4 &b) {
  return join8(Ty::pack(a[0], a[1]), Ty::pack(a[2], a[3]), Ty::pack(b[0], b[1]), Ty::pack(b[2], b[3]));
}

// A wavefront's sums to memory: 16 FI rows from m0 on of expert e (nrow in all, the
// first one row lo of the arrays) and the columns from col0 on.  Fragment (i, j) of a
// lane: row 16 i + r16, columns 16 j + 4 g ..; with both projections in one tile
// fragment 2 j is the gate's, 2 j + 1 the other projection's of the same columns.
template <typename Ty, int kLayout, int kEpi, int FI, int FJ>
__device__ __forceinline__ void store_tile(const GroupedArgs &p, int e, int lo, int m0, int nrow, int col0,
                                           const f32x4 (&acc)[FI][FJ]) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r16 = lane & 15;
  // groups 0 and 2 of a joined pair of fragments hold the first one's columns
  const int pair = 16 * (g & 1) + 8 * (g >> 1);
#pragma unroll
  for (int i = 0; i < FI; ++i) {
    const bool ok = m0 + 16 * i + r16 < nrow;
    const long long row = lo + m0 + 16 * i + r16;
    if constexpr (kEpi == kStoreF32) {
      float *out = (float *)p.out + e * p.out_expert + row * p.ldo;
#pragma unroll
      for (int j = 0; j < FJ; ++j) {
        const int n0 = col0 + 16 * j + 4 * g;
        if (ok && n0 < p.ncol) *reinterpret_cast<f32x4 *>(out + n0) = acc[i][j];
      }
    } else if constexpr (kEpi == kStore) {
      uint16_t *out = (uint16_t *)p.out + e * p.out_expert + row * p.ldo;
      if constexpr (FJ == 1) {
        const int n0 = col0 + 4 * g;
        const f32x4 &v = acc[i][0];
        if (ok && n0 < p.ncol)
          *reinterpret_cast<i32x2 *>(out + n0) = i32x2{Ty::pack(v[0], v[1]), Ty::pack(v[2], v[3])};
      } else {
#pragma unroll
        for (int j = 0; j < FJ; j += 2) {
          const int n0 = col0 + 16 * j + pair;
          const i32x4 v = join8<Ty>(acc[i][j], acc[i][j + 1]);
          if (ok && n0 < p.ncol) *reinterpret_cast<i32x4 *>(out + n0) = v;
        }
      }
    } else if constexpr (kEpi == kGatedUp && FJ % 4 == 0) {
#pragma unroll
      for (int j = 0; j < FJ; j += 4) {
        const int n0 = col0 + 8 * j + pair;
        const bool in = ok && n0 < p.ncol;
        if (p.side) {
          const i32x4 gv = join8<Ty>(acc[i][j], acc[i][j + 2]), uv = join8<Ty>(acc[i][j + 1], acc[i][j + 3]);
          uint16_t *gu = p.side + row * 2 * p.H + n0;
          if (in) {
            *reinterpret_cast<i32x4 *>(gu) = gv;
            *reinterpret_cast<i32x4 *>(gu + p.H) = uv;
          }
        }
        f32x4 h0, h1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h0[q] = act_value(acc[i][j][q], p.act) * acc[i][j + 1][q];
          h1[q] = act_value(acc[i][j + 2][q], p.act) * acc[i][j + 3][q];
        }
        const i32x4 hv = join8<Ty>(h0, h1);
        if (in) *reinterpret_cast<i32x4 *>((uint16_t *)p.out + row * p.ldo + n0) = hv;
      }
    } else if constexpr (kEpi == kGatedUp) {          // one pair: four columns a lane
      static_assert(kEpi != kGatedUp || FJ % 4 == 0 || FJ == 2, "pairs of fragments");
      const int n0 = col0 + 4 * g;
      f32x4 h0;
#pragma unroll
      for (int q = 0; q < 4; ++q) h0[q] = act_value(acc[i][0][q], p.act) * acc[i][1][q];
      if (ok && n0 < p.ncol) {
        auto put = [&](uint16_t *at, const f32x4 &v) QMOE_INLINE {
          *reinterpret_cast<i32x2 *>(at) = i32x2{Ty::pack(v[0], v[1]), Ty::pack(v[2], v[3])};
        };
        if (p.side) {
          put(p.side + row * 2 * p.H + n0, acc[i][0]);
          put(p.side + row * 2 * p.H + p.H + n0, acc[i][1]);
        }
        put((uint16_t *)p.out + row * p.ldo + n0, h0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < FJ; j += 2) {
        const int n0 = col0 + 16 * j + pair;
        float d[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const auto s = __builtin_amdgcn_permlane16_swap(__float_as_int(acc[i][j][q]),
                                                          __float_as_int(acc[i][j + 1][q]), false, false);
          d[q] = __int_as_float((int)s[0]);
          d[4 + q] = __int_as_float((int)s[1]);
        }
        if (ok && n0 < p.ncol) {
          const long long at = row * 2 * p.H + n0;
          const i32x4 gv = *reinterpret_cast<const i32x4 *>(p.gu_in + at);
          const i32x4 uv = *reinterpret_cast<const i32x4 *>(p.gu_in + at + p.H);
          i32x4 dg, du, hv;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float vg[2], vu[2], vh[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float gf = Ty::load((uint16_t)((uint32_t)gv[q] >> (16 * b)));
              const float uf = Ty::load((uint16_t)((uint32_t)uv[q] >> (16 * b)));
              float a, da;
              act_both(gf, p.act, a, da);
              vg[b] = d[2 * q + b] * uf * da;
              vu[b] = d[2 * q + b] * a;
              vh[b] = a * uf;
            }
            dg[q] = Ty::pack(vg[0], vg[1]);
            du[q] = Ty::pack(vu[0], vu[1]);
            hv[q] = Ty::pack(vh[0], vh[1]);
          }
          *reinterpret_cast<i32x4 *>((uint16_t *)p.out + at) = dg;
          *reinterpret_cast<i32x4 *>((uint16_t *)p.out + at + p.H) = du;
          if (p.side) *reinterpret_cast<i32x4 *>(p.side + row * p.H + n0) = hv;
        }
      }
    }
  }
}

// c += a b, v_mfma_f32_16x16x32 with the sum in accumulation registers (as an
// instruction of its own: left to the compiler the sums move between both halves of
// the register file).  Whoever reads c afterwards waits for the product to end.
template <typename Ty>
__device__ __forceinline__ void mfma_into(f32x4 &c, const i32x4 &a, const i32x4 &b) {
  if constexpr (std::is_same<Ty, TypeBf16>::value)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// The same with a copy behind it: 16 bytes a lane from src + voff to LDS byte address
// lds + offset + 16 l (zeros where voff is kOut).  The product stands between the write
// of m0 and its use, which need a wait state between them.
template <typename Ty>
__device__ __forceinline__ void mfma_copy(f32x4 &c, const i32x4 &a, const i32x4 &b, const i32x4 &src,
                                          uint32_t voff, uint32_t lds, int offset) {
  if constexpr (std::is_same<Ty, TypeBf16>::value)
    asm volatile("s_add_u32 m0, %5, %6\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\t"
                 "buffer_load_dwordx4 %3, %4, 0 offen lds"
                 : "+a"(c) : "v"(a), "v"(b), "v"(voff), "s"(src), "s"(lds), "i"(offset)
                 : "memory", "m0", "scc");
  else
    asm volatile("s_add_u32 m0, %5, %6\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0\n\t"
                 "buffer_load_dwordx4 %3, %4, 0 offen lds"
                 : "+a"(c) : "v"(a), "v"(b), "v"(voff), "s"(src), "s"(lds), "i"(offset)
                 : "memory", "m0", "scc");
}
// ... and without a product
__device__ __forceinline__ void dma16s(const i32x4 &src, uint32_t voff, uint32_t lds, int offset) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(src), "s"(lds), "i"(offset)
               : "memory", "m0", "scc");
}

// ---- many rows: 256 x 256 tiles on four wavefronts --------------------------------
// One workgroup per CU, one wavefront per SIMD with 128 x 128 outputs in 256
// accumulation registers (eight wavefronts of 128 x 64 in opposite phases read a half
// more from LDS for the same products: 8192 x 4096 x 28672 1681 us, this 1306).
//
// The contraction comes in stages that direct-to-LDS DMA copies into a ring of slots, 128
// KB in all, across tiles.  A stage of 64 is 128 bytes of a row, whole lines: halves of
// them, which stages of 32 ask for, are twice the requests to the L2 (1463 us).  Where
// both operands run across the contraction a line is whole anyway, and stages of 32,
// copied three ahead instead of one, take 1307 us instead of 1358.  Copies past an
// operand's rows, columns or depth bring zeros, so ragged segments and ends need no code
// of their own.
//
// While the 64 products of 32 of the contraction run, the fragments of the next 32 are read
// between them, and the copies of a later stage go out, evenly spread: a wavefront issues
// in order, and more than three instructions between two products, or copies faster than
// the address path takes them (16 cycles each), hold up the next (all copies in the
// second half of a stage 1527 us, spread but with their bookkeeping between 1450).  One
// barrier for each stage of copies; behind it the slot read last is free.  The products
// stand in inline assembly so that the sums stay in their half of the register file.
//
// Persistent: the tiles are ordered expert by expert, inside in groups of four row
// tiles, rows fastest; the 32 tiles that an XCD works on at a time are 4 x 8 neighbours
// that share rows and columns in its L2.
//
// Power sets the clock (1.5 to 1.9 GHz); the matrix units are busy about 80% of the time.
// What is left: the epilogue, during which no products run, tiles that the experts' rows
// fill in part, and the last round of tiles.
template <typename Ty, int kLayout, int kEpi, int TM>
__global__ __launch_bounds__(256, 1) void wide_kernel(const GroupedArgs p) {
  constexpr int T = 256;                              // columns of a tile
  constexpr int FI = TM / 32;                         // row fragments of a wavefront
  constexpr bool kRT = kLayout == kWgrad, kCT = kLayout != kLinear;
  constexpr bool kFine = kRT && kCT;                  // stages of 32, four slots
  constexpr int kStage = kFine ? 32 : 64, kSlots = kFine ? 4 : 2;
  constexpr int kPart = TM * 2 * kStage, kSlot = kPart + T * 2 * kStage, kRowB = 2 * T;
  static_assert(TM == T || !kRT, "rows across come in rows of 256");
  // copies of a wavefront and stage: of the rows, of the columns
  constexpr int PR = kFine ? 4 : TM / 32, P = kFine ? 4 : 8;
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kSlots * kSlot];
  __shared__ Segments s_seg;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int g = lane >> 4, r16 = lane & 15;
  constexpr int kTN = kEpi == kGatedUp ? T / 2 : T;
  const int ntn = (p.ncol + kTN - 1) / kTN;
  const int ntr = (p.nrow + TM - 1) / TM;             // kWgrad
  // twice 32 of the contraction that a tile takes; without any (an expert without rows)
  // zeros are contracted
  auto pairs = [](int depth) QMOE_INLINE { return max(1, (depth + 63) >> 6); };
  // tiles of an expert with n rows, and what one takes: its pairs, the epilogue as four
  find_segments(s_seg, p.off, p.rows, p.E,
                [&](int n) { return (kLayout == kWgrad ? ntr : (n + TM - 1) / TM) * ntn; },
                [&](int n) { return kLayout == kWgrad ? (float)(pairs(n) + 4) : 1.0f; });

  // This workgroup's tiles.  The tiles are cut into eight contiguous runs of equal cost, one
  // for each XCD; its workgroups take the run's tiles round robin.
  const int G = gridDim.x, wg = blockIdx.x;
  const int xcd = wg & (kXcds - 1), wl = wg / kXcds;
  const int gx = (G - xcd + kXcds - 1) / kXcds;
  const int t_end = run_start(s_seg, p.E, xcd + 1);
  int t = run_start(s_seg, p.E, xcd) + wl;
  if (t >= t_end) return;

  struct Tile {
    int e, lo, nrow, depth, m0, n0;
    int rows;                                         // of the tile: TM at most
  };
  // tile tt (its expert is e or a later one)
  auto decode = [&](int tt, int e) QMOE_INLINE -> Tile {
    while (__builtin_amdgcn_readfirstlane(s_seg.first[e + 1]) <= tt) ++e;
    Tile w;
    w.e = e;
    w.lo = __builtin_amdgcn_readfirstlane(s_seg.lo[e]);
    const int n = __builtin_amdgcn_readfirstlane(s_seg.hi[e]) - w.lo;
    w.nrow = kLayout == kWgrad ? p.nrow : n;
    w.depth = kLayout == kWgrad ? n : p.depth;
    const int local = tt - __builtin_amdgcn_readfirstlane(s_seg.first[e]);
    constexpr int kRows = 4;
    const int ntm = kLayout == kWgrad ? ntr : (n + TM - 1) / TM;
    const int per = kRows * ntn, grp = local / per, rem = local - grp * per;
    const int rows = min(kRows, ntm - grp * kRows);
    const int tn = rem / rows;
    w.m0 = (grp * kRows + rem - tn * rows) * TM;
    w.n0 = tn * kTN;
    w.rows = min(TM, w.nrow - w.m0);
    return w;
  };

  // ---- copies.  LDS rows of an operand along the contraction: 128 bytes, 16-byte chunk c
  // of row r at c ^ swz(r); across it: kRowB bytes, 32-byte granule q of row k at q ^
  // swt(k).  Either way the lanes that a fragment read serves at a time lie on distinct
  // banks.
  auto swz = [](int r) QMOE_INLINE { return (r >> 1) & 7; };
  auto swt = [](int k) QMOE_INLINE { return (k & 3) | ((k >> 1) & 4); };
  const uint32_t ring = lds_addr(s_ring);
  const uint32_t my_ring = __builtin_amdgcn_readfirstlane(ring + (uint32_t)(PR * wave * 1024));
  const uint32_t my_cols = kPart + (P - PR) * wave * 1024;            // from there to the columns' part
  // the copies' cursor: stages of tile cur_t that are left, what of its contraction is
  int cur_t = t, cur_left = 0, cur_valid = 0, cur_e = 0;
  uint32_t cur_slot = my_ring, cur_cols = my_ring + my_cols;          // this wavefront's parts of the slot
  // resources of the cursor's stage: base address (advanced stage by stage), bytes that
  // are memory, format
  i32x4 r_src = {0, 0, (int)kOut, 0x00020000}, c_src = r_src, c_src2 = r_src;
  const long long r_step = 2 * kStage * (kRT ? p.ldr : 1), c_step = 2 * kStage * (kCT ? p.ldc : 1);   // bytes
  auto set_base = [](i32x4 &s, const uint16_t *at) QMOE_INLINE {
    const uint64_t b = (uint64_t)(uintptr_t)at;
    s[0] = __builtin_amdgcn_readfirstlane((int)b);
    s[1] = __builtin_amdgcn_readfirstlane((int)(b >> 32) & 0xFFFF);
  };
  auto advance = [](i32x4 &s, long long by) QMOE_INLINE {
    const uint64_t b = ((uint64_t)(uint32_t)s[1] << 32 | (uint32_t)s[0]) + (uint64_t)by;
    s[0] = (int)b;
    s[1] = (int)(b >> 32);
  };
  // Copy u of an operand that runs along the contraction: LDS rows 8 (copies wave + u) .. + 7,
  // of one that runs across it: LDS rows 2 (copies wave + u), + 1.  A lane's place there:
  auto row_of = [&](int u, int copies) QMOE_INLINE { return 8 * (copies * wave + u) + (lane >> 3); };
  auto along_k = [&](int u) QMOE_INLINE { return 8 * ((lane & 7) ^ swz(8 * u + (lane >> 3))); };
  auto across_k = [&](int u) QMOE_INLINE { return 2 * P * wave + 2 * u + (lane >> 5); };
  auto across_at = [&](int u) QMOE_INLINE {
    const int q = lane & 31;
    return 8 * (((q >> 1 ^ swt(across_k(u))) << 1) | (q & 1));
  };
  uint32_t r_off[PR], c_off[P];                       // bytes from the stage's base, or kOut
  auto enter = [&]() QMOE_INLINE {
    const Tile w = decode(cur_t, cur_e);
    cur_e = w.e;
    cur_left = __builtin_amdgcn_readfirstlane(pairs(w.depth) * (64 / kStage));
    cur_valid = __builtin_amdgcn_readfirstlane(w.depth);
    set_base(r_src, kRT ? p.r + w.lo * p.ldr + w.m0 : p.r + (w.lo + w.m0) * p.ldr);
    const uint16_t *c = kLayout == kWgrad ? p.c + w.lo * p.ldc + w.n0
                        : kCT             ? p.c + w.e * p.c_expert + w.n0
                                          : p.c + w.e * p.c_expert + w.n0 * p.ldc;
    set_base(c_src, c);
    if constexpr (kEpi == kGatedUp) set_base(c_src2, c + (long long)p.H * p.ldc);
    // wait states between a vector instruction that writes a scalar register and a memory
    // instruction that reads it
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 4");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < PR; ++u) {
      const int row = row_of(u, PR);
      if (kRT)
        r_off[u] = across_at(u) < w.rows
                       ? 2u * ((uint32_t)across_k(u) * (uint32_t)p.ldr + (uint32_t)across_at(u)) : kOut;
      else
        r_off[u] = row < w.rows ? 2u * ((uint32_t)row * (uint32_t)p.ldr + (uint32_t)along_k(u)) : kOut;
    }
#pragma unroll
    for (int u = 0; u < P; ++u) {
      if (kCT) {
        c_off[u] = w.n0 + across_at(u) < p.ncol
                       ? 2u * ((uint32_t)across_k(u) * (uint32_t)p.ldc + (uint32_t)across_at(u)) : kOut;
      } else {
        // of both projections: sixteen columns of the gate's, the same of the other's, ..
        const int row = row_of(u, P), at = kEpi == kGatedUp ? (row >> 5) * 16 + (row & 15) : row;
        c_off[u] = w.n0 + at < p.ncol ? 2u * ((uint32_t)at * (uint32_t)p.ldc + (uint32_t)along_k(u)) : kOut;
      }
    }
  };
  // the copies of a stage that is not all of it contraction: zeros behind
  auto cut = [&]() QMOE_INLINE {
    if (cur_valid < kStage) {
#pragma unroll
      for (int u = 0; u < PR; ++u) r_off[u] = (kRT ? across_k(u) : along_k(u)) < cur_valid ? r_off[u] : kOut;
#pragma unroll
      for (int u = 0; u < P; ++u) c_off[u] = (kCT ? across_k(u) : along_k(u)) < cur_valid ? c_off[u] : kOut;
    }
  };
  // The cursor's copies are under way: on to the next stage.  The plain steps first, ..
  auto next_stage = [&]() QMOE_INLINE {
    cur_slot = cur_slot - my_ring == (kSlots - 1) * kSlot ? my_ring : cur_slot + kSlot;
    cur_cols = cur_slot + my_cols;
    --cur_left;
    cur_valid -= kStage;
    advance(r_src, r_step);
    advance(c_src, c_step);
    if constexpr (kEpi == kGatedUp) advance(c_src2, c_step);
  };
  // .. then what a tile's last stage and a next tile need
  auto next_tile = [&]() QMOE_INLINE {
    if (cur_valid < kStage) {
      if (cur_left == 0) {
        if (cur_t + gx < t_end) {
          cur_t += gx;
          enter();
        } else {
          cur_left = 1 << 30;                         // zeros from here on
        }
      }
      cut();
    }
  };
  // copy q of the cursor's stage: resource, offset, place in the ring
  auto piece_src = [&](int q) QMOE_INLINE -> const i32x4 & {
    return q < PR ? r_src : kEpi == kGatedUp && ((q - PR) >> 1 & 1) ? c_src2 : c_src;
  };
  auto piece_off = [&](int q) QMOE_INLINE { return q < PR ? r_off[q] : c_off[q - PR]; };
  auto piece_to = [&](int q) QMOE_INLINE { return q < PR ? cur_slot : cur_cols; };
  auto piece_at = [](int q) QMOE_INLINE { return (q < PR ? q : q - PR) * 1024; };

  // ---- fragments.  A stage of 64 is read in halves of 32.
  const uint32_t ch = (uint32_t)((g ^ swz(r16)) << 4);
  const uint32_t tr = (uint32_t)((8 * g + (r16 >> 2)) * kRowB + 8 * (r16 & 3));
  const uint32_t tf = (uint32_t)((r16 >> 2) | ((g & 1) << 2));        // swt of the lane's rows
  const uint32_t c_rd = (uint32_t)kPart + (kCT ? tr + (((uint32_t)(wn * 8) ^ tf) << 5)
                                               : (uint32_t)((wn * 128 + r16) * 128) + ch);
  const uint32_t r_rd = kRT ? tr + (((uint32_t)(wm * 8) ^ tf) << 5) : (uint32_t)((wm * (TM / 2) + r16) * 128) + ch;
  typedef __attribute__((address_space(3))) s16x4 *LdsT;
  typedef __attribute__((address_space(3))) i32x4 *LdsV;
  auto read_across = [&](uint32_t at) QMOE_INLINE -> i32x4 {
    const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(uintptr_t)at);
    const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(uintptr_t)(at + 4 * kRowB));
    const i32x2 x = __builtin_bit_cast(i32x2, a), y = __builtin_bit_cast(i32x2, b);
    return i32x4{x[0], x[1], y[0], y[1]};
  };
  struct Frags {
    i32x4 r[FI], c[8];
  };
  // ra, ca: addresses of the wavefront's first fragments; fragment k: 0 .. 7 of the
  // columns, then of the rows
  auto read_frag = [&](Frags &f, uint32_t ra, uint32_t ca, int k) QMOE_INLINE {
    if (k >= 8) f.r[k - 8] = kRT ? read_across(ra ^ (uint32_t)((k - 8) << 5)) : *(LdsV)(uintptr_t)(ra + (k - 8) * 2048);
    else f.c[k] = kCT ? read_across(ca ^ (uint32_t)(k << 5)) : *(LdsV)(uintptr_t)(ca + k * 2048);
  };
  auto half_at = [](uint32_t rd, bool is_across, uint32_t base, bool second) QMOE_INLINE -> uint32_t {
    return is_across ? base + rd + (second ? 32 * kRowB : 0) : (base + rd) ^ (second ? 64u : 0u);
  };
  f32x4 acc[FI][8];
  // The products of `f`, the first or second half of the stage in hand; the fragments of
  // the half that follows (in slot `base`) come into `nf` on the way, with a second half
  // also the copies of the stage two ahead.  A product takes 16 cycles, another instruction
  // 4 of them: what stands between two products are three at most.
  auto step = [&](const Frags &f, Frags &nf, uint32_t base, auto second_) QMOE_INLINE {
    constexpr bool second = kFine || decltype(second_)::value;
    if constexpr (second) {
      wait_dma<kFine ? 2 * (PR + P) : 0>();              // the next stage has landed here,
      wait_lds();                                     // the one in hand is read ...
      phase_end();                                    // ... here and everywhere
    }
    // between how many products a copy goes out
    constexpr int kEvery = kFine ? 8 : FI == 8 ? 4 : 3;
    uint32_t ra = 0, ca = 0;
    int read = 0, copy = 0;
#pragma unroll
    for (int q = 0; q < 8 * FI; ++q) {
      const int j = q / FI, i = q % FI;
      if (second && q % kEvery == kEvery / 2 && copy < PR + P) {
        mfma_copy<Ty>(acc[i][j], f.c[j], f.r[i], piece_src(copy), piece_off(copy), piece_to(copy), piece_at(copy));
        ++copy;
      } else {
        mfma_into<Ty>(acc[i][j], f.c[j], f.r[i]);
      }
      if (q == 0) {
        ra = half_at(r_rd, kRT, base, !second);
        ca = half_at(c_rd, kCT, base, !second);
        asm volatile("" : "+v"(ra), "+v"(ca));        // 2048 k is added in the instruction
      }
      if (read < FI + 8 && (kFine ? q % 3 == 2 : second ? q % kEvery == kEvery - 1 : q % 2 == 0 && q > 0)) {
        read_frag(nf, ra, ca, read);
        ++read;
      }
      if (second && q == 8 * FI - 1) next_stage();
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (second) next_tile();
  };

  enter();
  cut();
#pragma unroll
  for (int d = 0; d < kSlots; ++d) {
#pragma unroll
    for (int q = 0; q < PR + P; ++q) dma16s(piece_src(q), piece_off(q), piece_to(q), piece_at(q));
    next_stage();
    next_tile();
  }
  wait_dma<(kSlots - 1) * (PR + P)>();                  // stage 0 has landed here ...
  phase_end();                                        // ... and everywhere
  uint32_t base = ring;                               // slot of the stage in hand
  auto next_base = [&]() QMOE_INLINE { base = base - ring == (kSlots - 1) * kSlot ? ring : base + kSlot; };
  Tile w = decode(t, 0);
  Frags fa, fb;
#pragma unroll
  for (int k = 0; k < FI + 8; ++k) read_frag(fa, base + r_rd, base + c_rd, k);
  for (;;) {
    const int n = pairs(w.depth);
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        asm volatile("" : "+a"(acc[i][j]));
      }
    // wait states between a write of a register and the product that adds to it
    asm volatile("s_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    for (int s = 0; s < n; ++s) {
      if (kFine) next_base();
      step(fa, fb, base, std::false_type{});
      next_base();
      step(fb, fa, base, std::true_type{});
    }
    // the last products are written before anything else reads their registers
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
    store_tile<Ty, kLayout, kEpi, FI, 8>(p, w.e, kLayout == kWgrad ? 0 : w.lo, w.m0 + wm * (TM / 2), w.m0 + w.rows,
                                        w.n0 + wn * (kTN / 2), acc);
    t += gx;
    if (t >= t_end) break;
    w = decode(t, w.e);
  }
  wait_dma_all();                                     // no copy into LDS outlives the workgroup
}

// ---- few tiles: T x T outputs -----------------------------------------------------
// One workgroup of four wavefronts per tile, T / 2 x T / 2 outputs each, for products
// whose 256 x 256 tiles are fewer than the card has CUs.  Stages of 64 of the
// contraction, copied kSlots - 1 ahead; one barrier a stage, behind which the slot read
// last is free.  Many tiles of 64 x 64 are bound by what the L2 gives (224 of them, depth
// 3584: 9 TB/s), those of 128 by the LDS (its reads take 1.5 times as long as the products).
// Few tiles are bound by the time of a stage, 0.3 us from a barrier to the next, whatever
// the copies' lead (seven stages instead of three: 10 to 20% slower): there two groups of
// four wavefronts take every other stage each and add their sums through LDS (130 rows, 8192
// -> 512 back 40.5 us with one group, 29.9 with two; 128 rows, 4096 -> 2 x 512 19.2,
// 15.6; but 256 tiles, 256 x 2048 -> 4096 back, 14.1, 14.8).
template <typename Ty, int kLayout, int kEpi, int T, int kGroups = 1>
__global__ __launch_bounds__(256 * kGroups, 2) void square_kernel(const GroupedArgs p) {
  constexpr bool kRT = kLayout == kWgrad, kCT = kLayout != kLinear;
  constexpr int kSlots = T == 64 ? 4 : 2;
  constexpr int kPart = T * 128, kSlot = 2 * kPart, kRowB = 2 * T;
  constexpr int P = T / 32;                           // copies of a wavefront, stage and operand
  constexpr int F = T / 32;                           // fragments of a wavefront either way
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kGroups * kSlots * kSlot];
  __shared__ f32x4 s_part[kGroups == 1 ? 1 : F * F * 256];
  __shared__ Segments s_seg;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3, group = __builtin_amdgcn_readfirstlane(tid >> 8);
  const int wm = wave >> 1, wn = wave & 1;
  const int g = lane >> 4, r16 = lane & 15;
  constexpr int kTN = kEpi == kGatedUp ? T / 2 : T;
  const int ntn = (p.ncol + kTN - 1) / kTN;
  const int ntr = (p.nrow + T - 1) / T;               // kWgrad
  find_segments(s_seg, p.off, p.rows, p.E,
                [&](int n) { return (kLayout == kWgrad ? ntr : (n + T - 1) / T) * ntn; },
                [](int) { return 1.0f; });
  const int total = __builtin_amdgcn_readfirstlane(s_seg.first[kMaxExperts]);
  const uint32_t ring = lds_addr(s_ring) + (uint32_t)(group * kSlots * kSlot);
  auto swz = [](int r) QMOE_INLINE { return (r >> 1) & 7; };
  // 32-byte granules of an LDS row across: 8 of them for T = 128, 4 for T = 64, whose rows
  // of 128 bytes take two of k into each 256 bytes of banks
  auto swt = [](int k) QMOE_INLINE {
    return T == 128 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
  };
  typedef __attribute__((address_space(3))) s16x4 *LdsT;
  typedef __attribute__((address_space(3))) i32x4 *LdsV;
  auto read_across = [&](uint32_t at) QMOE_INLINE -> i32x4 {
    const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(uintptr_t)at);
    const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsT)(uintptr_t)(at + 4 * kRowB));
    const i32x2 x = __builtin_bit_cast(i32x2, a), y = __builtin_bit_cast(i32x2, b);
    return i32x4{x[0], x[1], y[0], y[1]};
  };
  const uint32_t ch = (uint32_t)((g ^ swz(r16)) << 4);
  // of the lane's rows in a read across: 8 g + (r16 >> 2) and four behind it (their swizzle
  // differs in nothing for T = 128; for T = 64 bit 2 of k takes no part)
  const int kk = 8 * g + (r16 >> 2);
  const uint32_t tr = (uint32_t)(kk * kRowB + 8 * (r16 & 3)), tf = (uint32_t)swt(kk);
  const uint32_t r_rd = kRT ? tr : (uint32_t)((wm * (T / 2) + r16) * 128) + ch;
  const uint32_t c_rd = (uint32_t)kPart + (kCT ? tr : (uint32_t)((wn * (T / 2) + r16) * 128) + ch);

  int e = 0;
  for (int tt = blockIdx.x; tt < total; tt += gridDim.x) {
    while (__builtin_amdgcn_readfirstlane(s_seg.first[e + 1]) <= tt) ++e;
    const int lo = __builtin_amdgcn_readfirstlane(s_seg.lo[e]);
    const int n = __builtin_amdgcn_readfirstlane(s_seg.hi[e]) - lo;
    const int nrow = kLayout == kWgrad ? p.nrow : n, depth = kLayout == kWgrad ? n : p.depth;
    const int local = tt - __builtin_amdgcn_readfirstlane(s_seg.first[e]);
    // rows fastest: the workgroups of a column tile share its columns
    const int ntm = kLayout == kWgrad ? ntr : (n + T - 1) / T;
    const int tn = local / ntm, m0 = (local - tn * ntm) * T, n0 = tn * kTN;
    const int stages = (depth + 64 * kGroups - 1) / (64 * kGroups);      // of a group

    const uint16_t *r_src = kRT ? p.r + lo * p.ldr + m0 : p.r + (lo + m0) * p.ldr;
    const uint16_t *c_src = kLayout == kWgrad ? p.c + lo * p.ldc + n0
                            : kCT             ? p.c + e * p.c_expert + n0
                                              : p.c + e * p.c_expert + n0 * p.ldc;
    const long long r_step = kRT ? 64 * p.ldr : 64, c_step = kCT ? 64 * p.ldc : 64;
    // copy u: 8 LDS rows along the contraction, 1 KB of rows across it
    constexpr int kAcross = 1024 / kRowB;             // rows across of a copy
    uint32_t r_off[P], c_off[P];
    int r_k[P], c_k[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int row = 8 * (P * wave + u) + (lane >> 3);
      const int along = 8 * ((lane & 7) ^ swz(row));
      const int q = lane & (kRowB / 16 - 1), k = kAcross * (P * wave + u) + lane / (kRowB / 16);
      const int at = 8 * (((q >> 1 ^ swt(k)) << 1) | (q & 1));
      r_k[u] = kRT ? k : along;
      c_k[u] = kCT ? k : along;
      if (kRT) r_off[u] = m0 + at < nrow ? 2u * ((uint32_t)k * (uint32_t)p.ldr + (uint32_t)at) : kOut;
      else r_off[u] = m0 + row < nrow ? 2u * ((uint32_t)row * (uint32_t)p.ldr + (uint32_t)along) : kOut;
      if (kCT) {
        c_off[u] = n0 + at < p.ncol ? 2u * ((uint32_t)k * (uint32_t)p.ldc + (uint32_t)at) : kOut;
      } else {
        const int col = kEpi == kGatedUp ? (row >> 5) * 16 + (row & 15) : row;
        c_off[u] = n0 + col < p.ncol ? 2u * ((uint32_t)col * (uint32_t)p.ldc + (uint32_t)along) : kOut;
      }
    }
    // behind the last stage zeros go into slots that nobody reads, so that the counts of
    // copies in flight stay the same
    auto copy_stage = [&](int s) QMOE_INLINE {
      const uint32_t at = ring + (uint32_t)((s & (kSlots - 1)) * kSlot + P * wave * 1024);
      const int from = s * kGroups + group, left = depth - 64 * from;
#pragma unroll
      for (int u = 0; u < P; ++u)
        dma16z(r_src + from * r_step, r_k[u] < left ? r_off[u] : kOut, at + u * 1024);
#pragma unroll
      for (int u = 0; u < P; ++u) {
        const bool second = kEpi == kGatedUp && ((P * wave + u) >> 1 & 1);      // rows 16 .. 31 of 32
        dma16z(c_src + from * c_step + (second ? (long long)p.H * p.ldc : 0), c_k[u] < left ? c_off[u] : kOut,
               at + kPart + u * 1024);
      }
    };
    f32x4 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    __syncthreads();                                  // the slots of the tile before are read
#pragma unroll
    for (int s = 0; s < kSlots - 1; ++s) copy_stage(s);
    for (int s = 0; s < stages; ++s) {
      wait_dma<(kSlots - 2) * 2 * P>();               // stage s has landed here,
      wait_lds();                                     // the one before is read ...
      phase_end();                                    // ... here and everywhere
      copy_stage(s + kSlots - 1);
      const uint32_t base = ring + (uint32_t)((s & (kSlots - 1)) * kSlot);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        i32x4 fr[F], fc[F];
#pragma unroll
        for (int j = 0; j < F; ++j)
          fc[j] = kCT ? read_across(base + c_rd + h * 32 * kRowB + (((uint32_t)(wn * F + j) ^ tf) << 5))
                      : *(LdsV)(uintptr_t)(((base + c_rd) ^ (uint32_t)(64 * h)) + j * 2048);
#pragma unroll
        for (int i = 0; i < F; ++i)
          fr[i] = kRT ? read_across(base + r_rd + h * 32 * kRowB + (((uint32_t)(wm * F + i) ^ tf) << 5))
                      : *(LdsV)(uintptr_t)(((base + r_rd) ^ (uint32_t)(64 * h)) + i * 2048);
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int i = 0; i < F; ++i) acc[i][j] = mfma16<Ty>(fc[j], fr[i], acc[i][j]);
      }
    }
    if constexpr (kGroups == 2) {
      f32x4 *const part = s_part + (tid & 255);
      if (group == 1) {
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
          for (int j = 0; j < F; ++j) part[256 * (i * F + j)] = acc[i][j];
      }
      __syncthreads();
      if (group == 1) continue;
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] += part[256 * (i * F + j)];
    }
    store_tile<Ty, kLayout, kEpi, F, F>(p, e, kLayout == kWgrad ? 0 : lo, m0 + wm * (T / 2), nrow,
                                        n0 + wn * (kTN / 2), acc);
  }
  wait_dma_all();                                     // no copy into LDS outlives the workgroup
}

// ---- a few rows an expert: weights through each wavefront's own LDS -----------------
// One workgroup of four wavefronts per expert and 16 columns (of both projections, or 16 C
// of a linear); it takes 16 MB of the expert's rows at a time.  The wavefronts share out
// the contraction, 64 of it each in turn, and add their sums through LDS at the end;
// until then each waits for nothing but its own copies, D steps ahead, so that those are
// always under way: what a product bound by its weights needs.  A step's rows come as
// whole 128-byte lines.
constexpr int kStreamWaves = 4;

template <typename Ty, int kEpi, int MB, int C, int D>
__global__ __launch_bounds__(64 * kStreamWaves) void stream_kernel(const GroupedArgs p, int col_tiles) {
  constexpr int kSlot = 16 * (MB + C) * 128, kRingB = kStreamWaves * D * kSlot;
  constexpr int kPieces = 2 * (MB + C);
  constexpr int kPartB = kStreamWaves * MB * C * 1024;
  static_assert((D - 1) * kPieces < 64, "the copies in flight are counted in 6 bits");
  __shared__ __attribute__((aligned(1024))) uint8_t s_ring[kRingB > kPartB ? kRingB : kPartB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int e = blockIdx.x / col_tiles;
  constexpr int kTN = kEpi == kGatedUp ? 16 : 16 * C;
  const int n0 = (blockIdx.x - e * col_tiles) * kTN;
  const int lo = p.off ? min(max(p.off[e], 0), p.rows) : 0;
  const int hi = p.off ? min(max(p.off[e + 1], lo), p.rows) : p.rows;

  // chunk c of LDS row r lies at c ^ ((r >> 1) & 7)
  const uint16_t *w0 = p.c + e * p.c_expert + n0 * p.ldc;
  const int ch = (lane & 7) ^ (lane >> 4);            // of the even copies; the odd ones': ^ 4
  uint32_t w_off[2 * C];
#pragma unroll
  for (int u = 0; u < 2 * C; ++u) {
    const int col = kEpi == kGatedUp ? 8 * (u & 1) + (lane >> 3) : 8 * u + (lane >> 3);
    w_off[u] = n0 + col < p.ncol ? 2u * ((uint32_t)col * (uint32_t)p.ldc + 8u * (uint32_t)(ch ^ (4 * (u & 1)))) : kOut;
  }
  const uint32_t mine = lds_addr(s_ring) + (uint32_t)(wave * D * kSlot);
  const int steps = (p.depth + 63) >> 6;
  const int n = (steps - wave + kStreamWaves - 1) / kStreamWaves;    // this wavefront's
  const int turn = n > 0 ? (int)(blockIdx.x / kXcds) % n : 0;        // .. from another on in each workgroup
  typedef __attribute__((address_space(3))) i32x4 *LdsV;

  for (int m0 = lo; m0 < hi; m0 += 16 * MB) {
    const uint16_t *a0 = p.r + m0 * p.ldr;
    uint32_t a_off[2 * MB];
#pragma unroll
    for (int u = 0; u < 2 * MB; ++u) {
      const int r = 8 * u + (lane >> 3);
      a_off[u] = m0 + r < hi ? 2u * ((uint32_t)r * (uint32_t)p.ldr + 8u * (uint32_t)(ch ^ (4 * (u & 1)))) : kOut;
    }
    auto copy = [&](int slot, int i) QMOE_INLINE {
      int at = turn + i;
      at = at < n ? at : at - n;
      const int k0 = 64 * (at * kStreamWaves + wave), left = p.depth - k0;
      const uint32_t to = mine + (uint32_t)(slot * kSlot);
#pragma unroll
      for (int u = 0; u < 2 * C; ++u)
        dma16z(w0 + k0 + (kEpi == kGatedUp && u >= 2 ? (long long)p.H * p.ldc : 0),
               8 * (ch ^ (4 * (u & 1))) < left ? w_off[u] : kOut, to + 16 * MB * 128 + u * 1024);
#pragma unroll
      for (int u = 0; u < 2 * MB; ++u)
        dma16z(a0 + k0, 8 * (ch ^ (4 * (u & 1))) < left ? a_off[u] : kOut, to + u * 1024);
    };
    f32x4 acc[MB][C];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < C; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (d < n) copy(d, d);
    int slot = 0;
    for (int i = 0; i < n; ++i) {
      if (i + D <= n) wait_dma<(D - 1) * kPieces>();
      else wait_dma_all();
      const uint32_t from = mine + (uint32_t)(slot * kSlot + r16 * 128);
      i32x4 fa[MB][2], fw[C][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = from + (uint32_t)(((4 * h + g) ^ ((r16 >> 1) & 7)) << 4);
#pragma unroll
        for (int j = 0; j < C; ++j) fw[j][h] = *(LdsV)(uintptr_t)(at + (MB + j) * 2048);
#pragma unroll
        for (int b = 0; b < MB; ++b) fa[b][h] = *(LdsV)(uintptr_t)(at + b * 2048);
      }
      wait_lds();                                     // the slot has been read
      if (i + D < n) copy(slot, i + D);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int b = 0; b < MB; ++b) acc[b][j] = mfma16<Ty>(fw[j][h], fa[b][h], acc[b][j]);
      slot = slot + 1 < D ? slot + 1 : 0;
    }
    __syncthreads();                                  // every wavefront is done with its ring
    f32x4 *part = reinterpret_cast<f32x4 *>(s_ring);
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < C; ++j) part[(wave * MB * C + b * C + j) * 64 + lane] = acc[b][j];
    __syncthreads();
    for (int b = wave; b < MB; b += kStreamWaves) {
      f32x4 sum[1][C];
#pragma unroll
      for (int j = 0; j < C; ++j) {
        sum[0][j] = part[(b * C + j) * 64 + lane];
#pragma unroll
        for (int v = 1; v < kStreamWaves; ++v) sum[0][j] += part[(v * MB * C + b * C + j) * 64 + lane];
      }
      store_tile<Ty, kLinear, kEpi, 1, C>(p, e, lo, m0 - lo + 16 * b, hi - lo, n0, sum);
    }
    __syncthreads();                                  // the sums are read: the ring is free
  }
}

constexpr int kCus = 256;

template <typename Ty, int kEpi, int MB, int C, int D>
hipError_t launch_stream(const GroupedArgs &a, hipStream_t s) {
  const int tn = kEpi == kGatedUp ? 16 : 16 * C, cols = (a.ncol + tn - 1) / tn;
  hipLaunchKernelGGL((stream_kernel<Ty, kEpi, MB, C, D>), dim3((unsigned)cols * a.E), dim3(64 * kStreamWaves), 0, s,
                     a, cols);
  return hipGetLastError();
}

// Which kernel, by the experts' average rows (of one expert: its rows; of several the
// fullest is taken to have twice the average: how the rows really lie only the device
// knows) and the widths.  The kernels add in orders of their own: a row of a call of other
// rows, experts or widths, or in another expert's place, may differ in the last bits of its
// float32 sums; the same call repeats bit by bit.  Other splits of the rows cost time only:
// 2048 -> 1024, 4096 rows in 128 experts 131 us, half of them in one 205, all 308 (alone, as
// one expert, 25); 4096 -> 7168, 128 rows in 8 experts 88, half in one 93, all 40.
//   A linear of up to 64 rows of one expert, or 48 on average of several: weights streamed
//   past 16, 32 or 64 of them (up and down of one token, 4096 x 14336: 37.7 + 18.8 us, in tiles
//   43.3 + 57.1; 128 rows in 8 experts of 4096 x 7168: 156 + 95 us with 32 rows, 192 + 107 with
//   16, 186 + 92 with 64, 206 + 156 in tiles; 320 rows: 205 + 103 with 64, 218 + 159 in tiles).
//   Else 256 x 256 tiles where half of the CUs have one (E = 8, rows of 2048 x 4096 x 14336:
//   128 tiles of the linear back down 366 us, with 128 x 128 499; 777 x 1024 x 3584, 70 tiles,
//   28 us, with 128 x 128 16), 128 x 128 where these are 192 at least, 64 x 64 below (777 x
//   1792 x 1024 in 5 experts, 80 tiles of 128: 22 us, with 64 x 64 14; 2048 x 4096 x 2048 in 4,
//   256 tiles: 72, with 64 x 64 112).  Tiles of 192 rows where they need fewer rounds over the
//   card by more than their products cost (8192 rows in 8 experts, 14336 -> 4096: 3 rounds
//   either way, 968 us against 1030; 28672 -> 4096 1834 against 1960).
//   A weight gradient over few rows in few tiles is its prologues and stores, which two
//   workgroups of 128 x 128 a CU overlap (3584 x 1024 in 5 experts, 280 tiles: 777 rows 17.7
//   us against 23.8, 12800 rows the same; 2048 x 1408 in 5, 240 tiles, 2048 rows 21.4 against
//   29.3, but 1792 x 1024, 140 tiles, 3200 rows 25.8 against 24.4; 8192 x 2048 in 4, 1024
//   tiles, 2048 rows 81.7 against 74.9).
template <typename Ty, int kLayout, int kEpi>
hipError_t launch(const GroupedArgs &a, hipStream_t s) {
  auto tiles = [&](int T) {
    const long long each = ((long long)a.rows + a.E - 1) / a.E, tn = kEpi == kGatedUp ? T / 2 : T;
    const long long m = a.E * (((kLayout == kWgrad ? a.nrow : each) + T - 1) / T);
    return m * ((a.ncol + tn - 1) / tn);
  };
  // rounds of tiles of TM x 256 over the card; of several experts each leaves a tile half full
  auto rounds = [&](int TM) {
    const int tn = kEpi == kGatedUp ? 128 : 256, cols = (a.ncol + tn - 1) / tn;
    const double m = a.E == 1 ? (double)((a.rows + TM - 1) / TM) : (double)a.rows / TM + 0.5 * a.E;
    return (double)(long long)((m * cols + kCus - 1) / kCus);
  };
  const dim3 block(256);
  if constexpr (kLayout == kLinear) {
    constexpr int C = kEpi == kGatedUp ? 2 : 1;
    const int most = a.E == 1 ? a.rows : 2 * ((a.rows + a.E - 1) / a.E);
    if (most <= 16) return launch_stream<Ty, kEpi, 1, C, 5 - C>(a, s);
    if (most <= 32) return launch_stream<Ty, kEpi, 2, C, 4 - C>(a, s);
    if (most <= (a.E == 1 ? 64 : 96)) return launch_stream<Ty, kEpi, 4, 2, 3>(a, s);
  }
  const bool shallow = kLayout == kWgrad && a.rows <= 512ll * a.E && tiles(256) <= 5 * kCus / 2;
  if (tiles(256) >= kCus / 2 && !shallow) {
    if constexpr (kLayout != kWgrad) {
      if (rounds(192) * 192 * 1.06 < rounds(256) * 256) {
        hipLaunchKernelGGL((wide_kernel<Ty, kLayout, kEpi, 192>), dim3(kCus), block, 0, s, a);
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((wide_kernel<Ty, kLayout, kEpi, 256>), dim3(kCus), block, 0, s, a);
  } else if (tiles(128) >= 192) {
    hipLaunchKernelGGL((square_kernel<Ty, kLayout, kEpi, 128>), dim3(2 * kCus), block, 0, s, a);
  } else if (tiles(64) <= kCus / 2) {
    hipLaunchKernelGGL((square_kernel<Ty, kLayout, kEpi, 64, 2>), dim3(kCus), dim3(512), 0, s, a);
  } else {
    hipLaunchKernelGGL((square_kernel<Ty, kLayout, kEpi, 64>), dim3(2 * kCus), block, 0, s, a);
  }
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
