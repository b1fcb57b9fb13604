// The general router (scores, balance bias, groups, top-k, renormalised
// weights), its gradient, and the block alignment of given ids.
#include "qmoe_layer.h"

namespace qmoe {

namespace {

// ---- rows of logits spread over lanes -------------------------------------------
// G neighbouring lanes share a token; lane i of them holds the experts i*V ..
// i*V + V - 1 in registers.

// A lane's vectors of a row of whole vectors, `left` elements from its end on: all
// at once where the row has them all (a few percent faster than one by one).
template <typename T, typename Vec, int n>
__device__ __forceinline__ void load_vectors(const T *x, int left, Vec (&q)[n]) {
  constexpr int kEach = sizeof(Vec) / sizeof(T);
  if (left >= n * kEach) {
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = *reinterpret_cast<const Vec *>(x + i * kEach);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      q[i] = Vec{};
      if (left > i * kEach) q[i] = *reinterpret_cast<const Vec *>(x + i * kEach);
    }
  }
}
template <typename T, typename Vec, int n>
__device__ __forceinline__ void store_vectors(T *x, int left, const Vec (&q)[n]) {
  constexpr int kEach = sizeof(Vec) / sizeof(T);
  if (left >= n * kEach) {
#pragma unroll
    for (int i = 0; i < n; ++i) *reinterpret_cast<Vec *>(x + i * kEach) = q[i];
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (left > i * kEach) *reinterpret_cast<Vec *>(x + i * kEach) = q[i];
  }
}

// V values of a row from element e0 on as float32; elements at or past E read 0.
// `vec`: rows and base are 16-byte aligned and E is whole vectors (vector_rows), so
// a vector's values exist all or not at all.
template <int V>
__device__ __forceinline__ void load_values(const void *base, long long row_at, int dtype, bool vec,
                                            int e0, int E, float (&v)[V]) {
#pragma unroll
  for (int u = 0; u < V; ++u) v[u] = 0.0f;
  if (dtype == MOE_F32) {
    const float *x = (const float *)base + row_at + e0;
    if constexpr (V % 4 == 0) {
      if (vec) {
        f32x4 q[V / 4];
        load_vectors(x, E - e0, q);
#pragma unroll
        for (int u = 0; u < V; ++u) v[u] = q[u / 4][u % 4];
        return;
      }
    }
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (e0 + u < E) v[u] = x[u];
    return;
  }
  const uint16_t *x = (const uint16_t *)base + row_at + e0;
  const bool bf = dtype == MOE_BF16;
  if constexpr (V % 4 == 0) {
    if (vec) {
      constexpr int kW = V % 8 == 0 ? 4 : 2;               // dwords per load
      typedef uint32_t words __attribute__((ext_vector_type(kW)));
      words q[V / (2 * kW)];
      load_vectors(x, E - e0, q);
#pragma unroll
      for (int u = 0; u < V; u += 2) {
        const uint32_t two = q[u / (2 * kW)][u / 2 % kW];
        v[u] = bf ? bf16_bits_to_f32(two & 0xFFFFu) : TypeF16::load((uint16_t)two);
        v[u + 1] = bf ? bf16_bits_to_f32(two >> 16) : TypeF16::load((uint16_t)(two >> 16));
      }
      return;
    }
  }
#pragma unroll
  for (int u = 0; u < V; ++u)
    if (e0 + u < E) v[u] = bf ? bf16_bits_to_f32(x[u]) : TypeF16::load(x[u]);
}

// The value of the lane that a step of a G-lane reduction pairs this one with.
// Step 0 and 1: the neighbours in a quad; 2: the other quad of 8 lanes; 3: the
// other 8 of 16; 4 and 5: the other 16 of 32, the other 32 of 64.  After step
// s all 2^(s+1) lanes hold the same, so mirrored lanes serve as partners.
template <int kStep>
__device__ __forceinline__ int lane_partner(int x) {
  if constexpr (kStep == 0) return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);
  else if constexpr (kStep == 1) return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);
  else if constexpr (kStep == 2) return __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true);
  else if constexpr (kStep == 3) return __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true);
  else return __shfl_xor(x, 1 << kStep);
}
template <int kStep>
__device__ __forceinline__ float lane_partner(float x) {
  return __int_as_float(lane_partner<kStep>(__float_as_int(x)));
}
template <int kStep>
__device__ __forceinline__ double lane_partner(double x) {
  const int lo = lane_partner<kStep>(__double2loint(x));
  const int hi = lane_partner<kStep>(__double2hiint(x));
  return __hiloint2double(hi, lo);
}

template <int G>
struct Log2 {
  static constexpr int value = 1 + Log2<G / 2>::value;
};
template <>
struct Log2<1> {
  static constexpr int value = 0;
};
template <int kStep, int kEnd, typename T>
__device__ __forceinline__ T lanes_sum(T x) {
  if constexpr (kStep < kEnd) return lanes_sum<kStep + 1, kEnd>(x + lane_partner<kStep>(x));
  else return x;
}
template <int kStep, int kEnd>
__device__ __forceinline__ float lanes_max(float x) {      // a NaN loses
  if constexpr (kStep < kEnd) return lanes_max<kStep + 1, kEnd>(fmaxf(x, lane_partner<kStep>(x)));
  else return x;
}

// ---- router: keys ------------------------------------------------------------------
// A key is a double that carries its expert in the low 9 bits (so that its
// order is that of (value, lower expert first) and one maximum instruction
// compares both): what is below 2^-43 of a key's value is given up for it.
// NaN keys and infinities are stood for by large finite values; -inf is
// no key at all (an expert of a group that was left out, or none).
constexpr int kIdBits = 9;
constexpr int kIdMask = (1 << kIdBits) - 1;
static_assert(MOE_MAX_ROUTE_EXPERTS == 1 << kIdBits, "a key holds its expert's number");

__device__ __forceinline__ double stand_in_nan() { return __hiloint2double(0x7FEF0000, 0); }
__device__ __forceinline__ double stand_in_inf() { return __hiloint2double(0x7FDF0000, 0); }

// NaN and infinities replaced by their stand-ins
__device__ __forceinline__ double finite(double k) {
  const double c = stand_in_inf();
  return k != k ? stand_in_nan() : k > c ? c : k < -c ? -c : k;
}
// and back
__device__ __forceinline__ double unfinite(double k) {
  const double c = stand_in_inf();
  return k > c ? __builtin_nan("") : k == c ? INFINITY : k == -c ? -INFINITY : k;
}

template <int kBits>
__device__ __forceinline__ double with_id(double k, int id) {
  constexpr int kMask = (1 << kBits) - 1;
  k += 0.0;                                                // -0 is +0
  const int hi = __double2hiint(k), lo = __double2loint(k);
  // below zero a larger magnitude is a smaller value
  return __hiloint2double(hi, (lo & ~kMask) | ((id ^ ~(hi >> 31)) & kMask));
}
__device__ __forceinline__ int id_of(double k) {
  return (__double2loint(k) ^ ~(__double2hiint(k) >> 31)) & kIdMask;
}

// 2^t for t <= 1000, about 2^-45 of the value: Chebyshev interpolation of
// degree 9 on [-1/2, 1/2].
__device__ __forceinline__ double fma_const(double p, double r, double c) {
  // the constant stays in scalar registers (the compiler's choice copies it into
  // the result's vector registers first, at every use)
  double d;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(p), "v"(r), "s"(c));
  return d;
}
// The leading coefficient, kept in vector registers by the caller.
__device__ __forceinline__ double exp2_lead() {
  double c = 1.0205905373362123e-07;
  asm("" : "+v"(c));
  return c;
}
__device__ __forceinline__ double exp2_poly(double t, double lead) {
  const double n = __builtin_rint(t);
  const double r = t - n;
  double p = fma_const(lead, r, 1.3259645246593194e-06);
  p = fma_const(p, r, 1.525267292505434e-05);
  p = fma_const(p, r, 0.0001540343375123525);
  p = fma_const(p, r, 0.0013333558200794313);
  p = fma_const(p, r, 0.009618129193934349);
  p = fma_const(p, r, 0.05550410866465167);
  p = fma_const(p, r, 0.2402265069564034);
  p = fma_const(p, r, 0.6931471805599462);
  p = fma_const(p, r, 1.0000000000000135);
  return ldexp(p, (int)n);
}
constexpr double kLog2e = 1.4426950408889634;

// 1 / (1 + exp(-x)) to about 2^-42 (absolute): beyond |x| = 80 the score is 0
// or 1 within 2^-115, and 1 + exp(80) is still a float32, whose hardware
// reciprocal starts one Newton step.
__device__ __forceinline__ double sigmoid_key(float x, double lead) {
  const float c = __builtin_amdgcn_fmed3f(x, -80.0f, 80.0f);
  const double d = 1.0 + exp2_poly(-kLog2e * (double)c, lead);
  const double y = (double)__builtin_amdgcn_rcpf((float)d);
  return fma(y, fma(-d, y, 1.0), y);
}

// The score and 1 - score, by the exponential that cannot overflow.
__device__ __forceinline__ double sigmoid64(double x, double &rest) {
  const double e = exp(-__builtin_fabs(x)), d = 1.0 / (1.0 + e), small = e * d;
  rest = x < 0.0 ? d : small;
  return x < 0.0 ? small : d;
}

// ---- router: sorted lists ------------------------------------------------------------
// Larger and smaller of two keys (never NaN).  As instructions: the compiler's
// fmax and fmin first quiet every operand that it knows nothing about, here one
// in two.  It does not see either that these write registers which a lane
// exchange may not read in the two cycles after: settle() goes in between.
__device__ __forceinline__ double larger(double a, double b) {
  double d;
  asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
__device__ __forceinline__ double smaller(double a, double b) {
  double d;
  asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
  return d;
}
__device__ __forceinline__ void settle(double (&a)[8]) {
  asm volatile("s_nop 1"
               : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]), "+v"(a[4]), "+v"(a[5]), "+v"(a[6]),
                 "+v"(a[7]));
}
__device__ __forceinline__ void settle(double (&a)[2]) {
  asm volatile("s_nop 1" : "+v"(a[0]), "+v"(a[1]));
}
__device__ __forceinline__ void exchange(double &a, double &b) {   // a >= b afterwards
  const double hi = larger(a, b), lo = smaller(a, b);
  a = hi;
  b = lo;
}
// the larger KK of two descending lists, descending: the maxima of opposite
// places form a bitonic sequence
template <int KK>
__device__ __forceinline__ void merge_lists(double (&a)[KK], const double (&b)[KK]) {
#pragma unroll
  for (int i = 0; i < KK; ++i) a[i] = larger(a[i], b[KK - 1 - i]);
#pragma unroll
  for (int d = KK / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < KK; ++i)
      if ((i & d) == 0) exchange(a[i], a[i + d]);
}
template <int KK, int kStep, int kEnd>
__device__ __forceinline__ void merge_lanes(double (&a)[KK]) {
  if constexpr (kStep < kEnd) {
    double b[KK];
    settle(a);
#pragma unroll
    for (int i = 0; i < KK; ++i) b[i] = lane_partner<kStep>(a[i]);
    merge_lists<KK>(a, b);
    merge_lanes<KK, kStep + 1, kEnd>(a);
  }
}
// 8 values, descending (a network of 19 exchanges)
__device__ __forceinline__ void sort8(double (&a)[8]) {
#define QMOE_X(i, j) exchange(a[i], a[j]);
  QMOE_X(0, 2) QMOE_X(1, 3) QMOE_X(4, 6) QMOE_X(5, 7)
  QMOE_X(0, 4) QMOE_X(1, 5) QMOE_X(2, 6) QMOE_X(3, 7)
  QMOE_X(0, 1) QMOE_X(2, 3) QMOE_X(4, 5) QMOE_X(6, 7)
  QMOE_X(2, 4) QMOE_X(3, 5)
  QMOE_X(1, 4) QMOE_X(3, 6)
  QMOE_X(1, 2) QMOE_X(3, 4) QMOE_X(5, 6)
#undef QMOE_X
}
// the KK largest of a lane's V keys, descending, -inf where there are fewer
template <int V, int KK>
__device__ __forceinline__ void local_list(const double (&key)[V], double (&a)[KK]) {
  if constexpr (KK == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = i < V ? key[i < V ? i : 0] : -INFINITY;
    if constexpr (V > 1) sort8(a);
#pragma unroll
    for (int q = 8; q < V; q += 8) {
      double b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = q + i < V ? key[q + i < V ? q + i : 0] : -INFINITY;
      sort8(b);
      merge_lists<8>(a, b);
    }
  } else {
    static_assert(KK == 2, "lists of 2 or 8");
    a[0] = key[0];
    a[1] = -INFINITY;
#pragma unroll
    for (int i = 1; i < V; ++i) {
      a[1] = larger(a[1], smaller(a[0], key[i]));
      a[0] = larger(a[0], key[i]);
    }
  }
}

// the two largest of a lane's values joined over 2^n lanes
template <int kStep, int kEnd>
__device__ __forceinline__ void top2_lanes(double &m1, double &m2, int steps) {
  if constexpr (kStep < kEnd) {
    if (kStep < steps) {
      double m[2] = {m1, m2};
      settle(m);
      m1 = m[0];
      m2 = m[1];
      const double o1 = lane_partner<kStep>(m1), o2 = lane_partner<kStep>(m2);
      m2 = larger(smaller(m1, o1), larger(m2, o2));
      m1 = larger(m1, o1);
      top2_lanes<kStep + 1, kEnd>(m1, m2, steps);
    }
  }
}

// What groups are ranked by, with the group's number in the low 6 bits.  It is
// rounded to 38 bits first: sums that are equal in exact arithmetic, as
// sigmoid(x) + sigmoid(-x) = 1 for every x, then tie in spite of the last bits
// of their scores.
static_assert(MOE_MAX_ROUTE_GROUPS == 64, "a group's worth holds its number");
__device__ __forceinline__ double group_worth(double m1, double m2, bool top2, int g) {
  const double w = top2 ? finite(unfinite(m1) + unfinite(m2)) : m1;
  const long long bits = __double_as_longlong(w + 0.0);
  return with_id<6>(__longlong_as_double((bits + 0x2000) & ~0x3FFFll), g);
}

enum { kNoGroups = 0, kLaneGroups = 1, kAnyGroups = 2 };

// One token per G lanes.  The scores that keys rest on are computed in float64
// by a polynomial; every lane sorts its V keys, and log2(G) merges of sorted
// lists of KK leave the token's choice in every lane.  Groups: kLaneGroups
// where a group is 2^n whole lanes (n = lane_bits), joined by lane steps;
// kAnyGroups ranks them through LDS, 2^lane_bits lanes a group.
template <int G, int V, int KK, int kGroups>
__global__ __launch_bounds__(256) void route_topk_kernel(const RouteArgs a, int dtype, bool vec,
                                                         int lane_bits) {
  constexpr int kTokens = 256 / G, kSteps = Log2<G>::value;
  constexpr int kGroupSlots = G * V < 64 ? G * V : 64;
  __shared__ float s_x[kTokens][G * V];                    // logits, for the chosen ones' weights
  __shared__ double s_key[kGroups == kAnyGroups ? kTokens : 1][kGroups == kAnyGroups ? G * V : 1];
  __shared__ double s_worth[kGroups == kAnyGroups ? kTokens : 1]
                           [kGroups == kAnyGroups ? kGroupSlots : 1];
  __shared__ uint8_t s_keep[kGroups == kAnyGroups ? kTokens : 1]
                           [kGroups == kAnyGroups ? kGroupSlots : 1];
  const int i = threadIdx.x & (G - 1), tok = threadIdx.x / G;
  const long long t = (long long)blockIdx.x * kTokens + tok;
  const bool live = t < a.M;                               // the same for a token's lanes
  const int E = a.E, e0 = i * V;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;

  float v[V];
  load_values<V>(a.logits, (live ? t : 0) * a.ld, dtype, vec, e0, E, v);
#pragma unroll
  for (int u = 0; u < V; ++u) s_x[tok][e0 + u] = v[u];

  // ---- scores, where keys or groups rest on them
  const bool top2 = kGroups != kNoGroups && a.group_rule == MOE_GROUP_TOP2;
  const bool plain_softmax = soft && !a.renormalize;       // its weights need the whole sum
  const bool scored = a.bias != nullptr || top2;
  float m = -INFINITY;
  double z = 0.0;
  double key[V], sc[V];
  const double lead = exp2_lead();
  bool odd = false;                                        // NaN or infinities here
#pragma unroll
  for (int u = 0; u < V; ++u) odd |= !(__builtin_fabsf(v[u]) < INFINITY);
  if (soft && (scored || plain_softmax)) {
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (e0 + u < E) m = fmaxf(m, v[u]);
    m = lanes_max<0, kSteps>(m);
    if (m == -INFINITY) m = 0.0f;                          // nothing above -inf: scores 0 (or NaN)
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const double d = kLog2e * ((double)v[u] - (double)m);
      sc[u] = d < -1100.0 ? 0.0 : exp2_poly(d, lead);            // (a NaN stays one)
      if (e0 + u < E) z += sc[u];
    }
    z = lanes_sum<0, kSteps>(z);
    const double inv = z == 0.0 ? 0.0 : 1.0 / z;
#pragma unroll
    for (int u = 0; u < V; ++u) sc[u] *= inv;
  } else if (scored) {
#pragma unroll
    for (int u = 0; u < V; ++u) sc[u] = sigmoid_key(v[u], lead);
    if (__any(odd)) {
#pragma unroll
      for (int u = 0; u < V; ++u) sc[u] = v[u] != v[u] ? (double)v[u] : sc[u];
    }
  }
  if (a.bias) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const float b = e0 + u < E ? a.bias[e0 + u] : 0.0f;
      odd |= !(__builtin_fabsf(b) < INFINITY);
      sc[u] += (double)b;
      key[u] = sc[u];
    }
  } else {
#pragma unroll
    for (int u = 0; u < V; ++u) key[u] = (double)v[u];
  }
  if (__any(odd)) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      key[u] = finite(key[u]);
      if (top2) sc[u] = finite(sc[u]);
      if (a.bias && v[u] == -INFINITY) key[u] = sc[u] = -stand_in_inf();   // masked, whatever its bias
    }
  }
#pragma unroll
  for (int u = 0; u < V; ++u) key[u] = e0 + u < E ? with_id<kIdBits>(key[u], e0 + u) : -INFINITY;

  // ---- groups
  if constexpr (kGroups == kLaneGroups) {
    // lanes [g * 2^n, (g + 1) * 2^n) are group g
    double m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const double w = top2 ? sc[u] : key[u];
      if (e0 + u < E) {
        m2 = larger(m2, smaller(m1, w));
        m1 = larger(m1, w);
      }
    }
    top2_lanes<0, kSteps>(m1, m2, lane_bits);
    const int g = i >> lane_bits;
    double w = group_worth(m1, m2, top2, g);
    if (e0 >= E) w = -INFINITY;
    int before = 0;                                        // groups better than this one
    for (int o = 1; o < (G >> lane_bits); ++o) {
      const int from = (threadIdx.x & 63) ^ (o << lane_bits);
      const double other = __hiloint2double(__shfl(__double2hiint(w), from),
                                            __shfl(__double2loint(w), from));
      before += other > w;
    }
    if (before >= a.topk_group) {
#pragma unroll
      for (int u = 0; u < V; ++u) key[u] = -INFINITY;
    }
  } else if constexpr (kGroups == kAnyGroups) {
    const int gs = E / a.n_group;
#pragma unroll
    for (int u = 0; u < V; ++u) s_key[tok][e0 + u] = top2 ? sc[u] : key[u];
    __syncthreads();
    // 2^lane_bits lanes scan a group
    const int each = 1 << lane_bits, part = i & (each - 1);
    for (int g0 = 0; g0 < a.n_group; g0 += G >> lane_bits) {
      const int g = g0 + (i >> lane_bits);
      double m1 = -INFINITY, m2 = -INFINITY;
      if (g < a.n_group) {
#pragma unroll 4
        for (int q = part; q < gs; q += each) {
          const double w = s_key[tok][g * gs + q];
          m2 = larger(m2, smaller(m1, w));
          m1 = larger(m1, w);
        }
      }
      top2_lanes<0, kSteps>(m1, m2, lane_bits);
      if (g < a.n_group && part == 0) s_worth[tok][g] = group_worth(m1, m2, top2, g);
    }
    __syncthreads();
    for (int g = i; g < a.n_group; g += G) {
      const double w = s_worth[tok][g];
      int before = 0;
#pragma unroll 8
      for (int o = 0; o < a.n_group; ++o) before += s_worth[tok][o] > w;
      s_keep[tok][g] = before < a.topk_group;
    }
    __syncthreads();
    int g = e0 / gs, left = gs - (e0 - g * gs);            // experts of group g from here on
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (e0 + u < E && !s_keep[tok][g]) key[u] = -INFINITY;
      if (--left == 0) {
        ++g;
        left = gs;
      }
    }
  }

  // ---- choice: the KK largest keys, in every lane of the token
  double best[KK];
  local_list<V, KK>(key, best);
  merge_lanes<KK, 0, kSteps>(best);
  __syncthreads();

  // ---- weights: lane j the j-th choice
  double mine = best[0];
#pragma unroll
  for (int j = 1; j < KK; ++j) mine = i == j ? best[j] : mine;
  const bool chosen = i < a.top_k;
  const int id = chosen ? id_of(mine) : 0;
  const float xj = s_x[tok][id];
  double w;
  if (soft) {
    if (a.renormalize) {
      m = lanes_max<0, 3>(chosen ? xj : -INFINITY);
      if (m == -INFINITY) m = 0.0f;
      // z is only summed up where keys rest on scores: NaN then by any expert's
      // logit, chosen or not.  Elsewhere such a logit is itself chosen.
      w = z != z ? z : exp((double)xj - (double)m);
    } else {
      w = z == 0.0 ? 0.0 : exp((double)xj - (double)m) / z;
    }
  } else {
    double rest;
    w = sigmoid64((double)xj, rest);
  }
  if (a.renormalize) {
    const double sum = lanes_sum<0, 3>(chosen ? w : 0.0);
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (live && chosen) {
    a.ids[t * a.top_k + i] = id;
    a.weights[t * a.top_k + i] = (float)(w * (double)a.scale);
  }
}

// ---- gradient -----------------------------------------------------------------
// One token per G lanes.  Lane j takes the j-th choice and its share of the sums
// and puts its gradient into the token's row in LDS; then every lane stores the V
// gradients of its experts.  A token with one expert twice is gathered choice by
// choice instead, in their order; the plain softmax, which reads the whole row for
// its scores, joins such choices first.  The others read only the chosen logits.
//
// Renormalised, q_j = s_j / S: dx_j = scale q_j t_j (g_j sum_{i != j} q_i - sum_{i != j}
// g_i q_i) in float64, t_j = 1 (softmax) or 1 - s_j (sigmoid).
// Plain softmax: dx_e = scale p_e (g_e - sum_i g_i p_i) in float32, but of a chosen
// expert with a score above one half, where that would be a difference of nearly
// equal terms,
//   dx_e = scale p_e (g_e sum_{i != e} p_i - sum_{i != e} g_i p_i),
// its sums taken without e.  Only a wavefront with such a token does that (16384 x
// 256 bf16 in the caches: 6.8 us, 7.2 where every token is one).
template <int V>
__device__ __forceinline__ void store_values(void *base, long long row_at, int dtype, bool vec,
                                             int e0, int E, const float (&v)[V]) {
  if (dtype == MOE_F32) {
    float *x = (float *)base + row_at + e0;
    if constexpr (V % 4 == 0) {
      if (vec) {
        f32x4 q[V / 4];
#pragma unroll
        for (int u = 0; u < V; ++u) q[u / 4][u % 4] = v[u];
        store_vectors(x, E - e0, q);
        return;
      }
    }
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (e0 + u < E) x[u] = v[u];
    return;
  }
  uint16_t *x = (uint16_t *)base + row_at + e0;
  const bool bf = dtype == MOE_BF16;
  if constexpr (V % 4 == 0) {
    if (vec) {
      constexpr int kW = V % 8 == 0 ? 4 : 2;
      typedef uint32_t words __attribute__((ext_vector_type(kW)));
      words q[V / (2 * kW)];
#pragma unroll
      for (int u = 0; u < V; u += 2)
        q[u / (2 * kW)][u / 2 % kW] =
            bf ? f32x2_to_bf16x2(v[u], v[u + 1])
               : (uint32_t)TypeF16::store(v[u]) | ((uint32_t)TypeF16::store(v[u + 1]) << 16);
      store_vectors(x, E - e0, q);
      return;
    }
  }
#pragma unroll
  for (int u = 0; u < V; ++u)
    if (e0 + u < E) x[u] = bf ? TypeBf16::store(v[u]) : TypeF16::store(v[u]);
}

// Lanes 0 .. 7 of a token: the sum over the other seven (others), and over all
// eight (all).
template <typename T>
__device__ __forceinline__ void sums_of_eight(T x, T &others, T &all) {
  others = lane_partner<0>(x);
  all = x + others;
  T o = lane_partner<1>(all);
  others += o;
  all += o;
  o = lane_partner<2>(all);
  others += o;
  all += o;
}
// The value of the lane whose number differs in the bits of kXor (1 .. 7).
template <int kXor>
__device__ __forceinline__ int lane_xor(int x) {
  if constexpr (kXor == 1) return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);
  else if constexpr (kXor == 2) return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);
  else if constexpr (kXor == 3) return __builtin_amdgcn_mov_dpp(x, 0x1B, 0xF, 0xF, true);
  else if constexpr (kXor == 7) return __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true);
  else return lane_xor<7 - kXor>(lane_xor<7>(x));
}
// Another choice has this lane's expert.
template <int kXor>
__device__ __forceinline__ bool has_twin(int id) {
  const bool here = lane_xor<kXor>(id) == id;
  if constexpr (kXor < 7) return here | has_twin<kXor + 1>(id);
  else return here;
}
// Choices of one expert joined in the first of them: its g is their sum, the
// later ones become no choice.
template <int kXor>
__device__ __forceinline__ void join_twins(int i, int id, float g, int &first_id, float &sum) {
  const int other = lane_xor<kXor>(id);
  const float og = __int_as_float(lane_xor<kXor>(__float_as_int(g)));
  if (other == id) {
    if ((i ^ kXor) < i) first_id = -1;
    else sum += og;
  }
  if constexpr (kXor < 7) join_twins<kXor + 1>(i, id, g, first_id, sum);
}

// exp(x - m).  The difference comes first: m log2(e) alone overflows where a whole
// row holds its type's lowest value.  Off by up to about 2 + 2.5 |x - m| half steps
// (2^-24): the difference, its product and log2(e) itself are rounded to float32.
__device__ __forceinline__ float exp_less(float x, float m) {
  constexpr float kL = 1.44269504f;
  return __builtin_amdgcn_exp2f((x - m) * kL);
}

template <int G, int V, bool kDense>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteBwdArgs a, int dtype,
                                                             bool vec_in, bool vec_out) {
  constexpr int kTokens = 256 / G, kSteps = Log2<G>::value;
  __shared__ __attribute__((aligned(16))) float s_row[kTokens][G * V];
  const int i = threadIdx.x & (G - 1), tok = threadIdx.x / G;
  const long long t = (long long)blockIdx.x * kTokens + tok;
  const bool live = t < a.M;
  const int E = a.E, e0 = i * V, k = a.top_k;
  const long long row = live ? t : 0;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  float p[V];
  if constexpr (kDense) load_values<V>(a.logits, row * a.ld, dtype, vec_in, e0, E, p);
  // lane j < top_k: the j-th choice
  int id = -1;
  float g = 0.0f, x = 0.0f;
  if (i < k) {
    id = a.ids[row * k + i];
    g = a.dw[row * k + i];
  }
  if ((unsigned)id >= (unsigned)E) {                // no choice: takes no part
    id = -1;
    g = 0.0f;
  }
  if constexpr (kDense) {
    if (__any(has_twin<1>(id) && id >= 0)) {
      int first_id = id;
      float sum = g;
      join_twins<1>(i, id, g, first_id, sum);
      id = first_id;
      g = id < 0 ? 0.0f : sum;
    }
  }
  const bool valid = id >= 0;
  if (valid) {
    if (dtype == MOE_F32) x = ((const float *)a.logits)[row * a.ld + id];
    else if (dtype == MOE_BF16) x = TypeBf16::load(((const uint16_t *)a.logits)[row * a.ld + id]);
    else x = TypeF16::load(((const uint16_t *)a.logits)[row * a.ld + id]);
  }
  float d = 0.0f;                                   // the choice's gradient, less p_e where dense
  float none = 0.0f;                                // and of an expert that is not chosen
  const int first = (threadIdx.x & 63) & ~(G - 1);
  if constexpr (kDense) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (e0 + u < E) m = fmaxf(m, p[u]);
    m = lanes_max<0, kSteps>(m);
    if (m == -INFINITY) m = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      p[u] = e0 + u < E ? exp_less(p[u], m) : 0.0f;
      z += p[u];
    }
    z = lanes_sum<0, kSteps>(z);
    const float inv = z == 0.0f ? 0.0f : 1.0f / z;
    const float ej = valid ? exp_less(x, m) : 0.0f;
    const float gp = g * (ej * inv);
    none = -a.scale * lanes_sum<0, kSteps>(gp);
    d = a.scale * g + none;
    const bool steep = z < 2.0f;                    // the one exponential that is 1 takes over half
    if (__any(steep)) {
      float rest = 0.0f, others, all;
#pragma unroll
      for (int u = 0; u < V; ++u) rest += p[u] == 1.0f ? 0.0f : p[u];
      rest = lanes_sum<0, kSteps>(rest);
      sums_of_eight(gp, others, all);
      if (steep && ej == 1.0f) d = a.scale * (g * (rest * inv) - others);
    }
#pragma unroll
    for (int u = 0; u < V; ++u) p[u] *= inv;
  } else {
    double s = 0.0, tail = 1.0;
    if (soft) {
      float m = lanes_max<0, 3>(valid ? x : -INFINITY);
      if (m == -INFINITY) m = 0.0f;
      if (valid) s = exp((double)x - (double)m);
    } else if (valid) {
      s = sigmoid64((double)x, tail);
    }
    double c = (double)g;
    if (a.renormalize) {
      const double sum = lanes_sum<0, 3>(s);
      s = sum == 0.0 ? 0.0 : s / sum;
      double other_s, other_gs, all;
      sums_of_eight(s, other_s, all);
      sums_of_eight((double)g * s, other_gs, all);
      c = c * other_s - other_gs;
    }
    d = (float)((double)a.scale * s * c * tail);
  }
  float o[V];
#pragma unroll
  for (int u = 0; u < V; ++u) o[u] = 0.0f;
  bool twice = false;                               // another choice has this expert
  if constexpr (!kDense) {
#pragma unroll
    for (int j = 1; j < kMaxTopK; ++j)
      twice |= __shfl(id, first + ((i + j) & (kMaxTopK - 1))) == id && valid && i < kMaxTopK;
  }
  if (__any(twice)) {
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) {
      if (j >= k) break;
      const int at = __shfl(id, first + j) - e0;
      const float dj = __shfl(d, first + j);
#pragma unroll
      for (int u = 0; u < V; ++u) o[u] += at == u ? dj : 0.0f;
    }
  } else {
    // a wavefront's LDS accesses are carried out in order, and no other touches
    // its tokens' rows
    float *row_s = s_row[tok];
#pragma unroll
    for (int u = 0; u < V; ++u) row_s[e0 + u] = none;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (valid) row_s[id] = d;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int u = 0; u < V; ++u) o[u] = row_s[e0 + u];
  }
  if constexpr (kDense) {
#pragma unroll
    for (int u = 0; u < V; ++u) o[u] *= p[u];
  }
  if (live) store_values<V>(a.dx, row * a.ldd, dtype, vec_out, e0, E, o);
}

// ---- alignment ------------------------------------------------------------------
// A stable counting sort of the slots by local expert.  Every wavefront owns a
// run of slots; for 64 of them one ballot per bit of the expert's number gives
// each lane the lanes with the same expert, so ranks need no atomics and keep
// the slots' order.
constexpr int kAlignThreads = 1024;
constexpr int kAlignWaves = kAlignThreads / 64;
// Chunks up to which one workgroup does it all: 2048 slots 4.4 - 6.2 us by the
// number of experts, two launches 6.5; 2560 of 128 experts 7.7 against 6.5.
constexpr int kOneWorkgroupChunks = 2;
constexpr int kChunk = 1024;                     // slots of one workgroup where there are many

// local expert of a slot, or -1
__device__ __forceinline__ int local_expert(int id, int first, int E) {
  return id >= first && (unsigned)id - (unsigned)first < (unsigned)E ? (int)((unsigned)id - (unsigned)first)
                                                                     : -1;
}

__device__ __forceinline__ unsigned long long peers_of(int e, int nbits) {
  unsigned long long peers = __ballot(e >= 0);
  for (int b = 0; b < nbits; ++b) {
    const bool bit = (e >> b) & 1;
    const unsigned long long mb = __ballot(bit);
    peers &= bit ? mb : ~mb;
  }
  return peers;
}
__device__ __forceinline__ int lanes_below(unsigned long long mask) {
  return __builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0u));
}

// Exclusive scan of the padded group sizes by wavefront 0: lane l holds the
// experts l and l + 64.  Fills s_off[0 .. E].
__device__ __forceinline__ void padded_starts(const int *s_cnt, int E, int block_m, int *s_off) {
  const int lane = threadIdx.x;
  const int n0 = lane < E ? s_cnt[lane] : 0, n1 = lane + 64 < E ? s_cnt[lane + 64] : 0;
  const int c0 = (n0 + block_m - 1) & -block_m, c1 = (n1 + block_m - 1) & -block_m;  // a power of two
  int x0 = c0, x1 = c1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y0 = __shfl_up(x0, d), y1 = __shfl_up(x1, d);
    if (lane >= d) {
      x0 += y0;
      x1 += y1;
    }
  }
  const int half = __shfl(x0, 63);
  if (lane < E) s_off[lane] = x0 - c0;
  if (lane + 64 < E) s_off[lane + 64] = half + x1 - c1;
  const int total = half + __shfl(x1, 63);
  if (lane == 0) s_off[E] = total;
}

// Everything that is not a slot: block labels, padding, the tail, counts; the
// `part`-th of `parts` workgroups does its share.
__device__ __forceinline__ void align_rest(const AlignArgs &a, const int *s_off, const int *s_cnt,
                                           int part, int parts) {
  const int tid = threadIdx.x, total = s_off[a.E];
  const int step = parts * kAlignThreads, at = part * kAlignThreads + tid;
  for (int b = at; b < a.max_padded / a.block_m; b += step) {
    const int p = b * a.block_m;
    int label = -1;
    if (p < total) {
      int lo = 0, hi = a.E - 1;                  // the last expert that starts at or before p
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_off[mid] <= p) lo = mid;
        else hi = mid - 1;
      }
      label = lo;
    }
    a.expert_ids[b] = label;
  }
  for (int e = part * kAlignWaves + (tid >> 6); e < a.E; e += parts * kAlignWaves)
    for (int p = s_off[e] + s_cnt[e] + (tid & 63); p < s_off[e + 1]; p += 64) a.sorted_ids[p] = a.S;
  for (int p = total + at; p < a.max_padded; p += step) a.sorted_ids[p] = a.S;
  if (part == 0) {
    if (a.counts && tid < a.E) a.counts[tid] = s_cnt[tid];
    if (tid == 0) *a.num_post = total;
  }
}

// Slots [begin, end) of one workgroup, wavefront w its w-th run of `per` (a
// multiple of 64): the counts of every wavefront and expert ...
__device__ __forceinline__ void count_slots(const AlignArgs &a, int begin, int end, int per, int nbits,
                                            int (*s_wave)[kMaxExperts]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lo = begin + wave * per, hi = min(lo + per, end);
  for (int base = lo; base < hi; base += 64) {
    const int e = base + lane < hi ? local_expert(a.ids[base + lane], a.expert_first, a.E) : -1;
    const unsigned long long peers = peers_of(e, nbits);
    if (e >= 0 && lanes_below(peers) == 0) s_wave[wave][e] += __popcll(peers);
  }
}
// ... and their places, s_wave holding each wavefront's next place per expert.
__device__ __forceinline__ void place_slots(const AlignArgs &a, int begin, int end, int per, int nbits,
                                            int (*s_wave)[kMaxExperts]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lo = begin + wave * per, hi = min(lo + per, end);
  for (int base = lo; base < hi; base += 64) {
    const int e = base + lane < hi ? local_expert(a.ids[base + lane], a.expert_first, a.E) : -1;
    const unsigned long long peers = peers_of(e, nbits);
    if (e >= 0) {
      const int rank = lanes_below(peers), at = s_wave[wave][e];   // read by every lane first ...
      a.sorted_ids[at + rank] = base + lane;
      if (rank == 0) s_wave[wave][e] = at + __popcll(peers);       // ... then written by one
    }
  }
}

__device__ __forceinline__ int bits_for(int E) { return E > 1 ? 32 - __builtin_clz((unsigned)(E - 1)) : 0; }

// Few slots: one workgroup does it all.
__global__ __launch_bounds__(kAlignThreads) void align_one_kernel(const AlignArgs a) {
  __shared__ int s_wave[kAlignWaves][kMaxExperts];
  __shared__ int s_cnt[kMaxExperts], s_off[kMaxExperts + 1];
  const int tid = threadIdx.x, nbits = bits_for(a.E);
  const int per = ((a.S + kAlignWaves - 1) / kAlignWaves + 63) & ~63;
  for (int x = tid; x < kAlignWaves * kMaxExperts; x += kAlignThreads) (&s_wave[0][0])[x] = 0;
  __syncthreads();
  count_slots(a, 0, a.S, per, nbits, s_wave);
  __syncthreads();
  if (tid < a.E) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kAlignWaves; ++w) n += s_wave[w][tid];
    s_cnt[tid] = n;
  }
  __syncthreads();
  if (tid < 64) padded_starts(s_cnt, a.E, a.block_m, s_off);
  __syncthreads();
  if (tid < a.E) {
    int at = s_off[tid];
#pragma unroll
    for (int w = 0; w < kAlignWaves; ++w) {
      const int n = s_wave[w][tid];
      s_wave[w][tid] = at;
      at += n;
    }
  }
  __syncthreads();
  place_slots(a, 0, a.S, per, nbits, s_wave);
  align_rest(a, s_off, s_cnt, 0, 1);
}

// Many slots: workgroup b counts chunk b into ws[b], [E] each ...
__global__ __launch_bounds__(kAlignThreads) void align_count_kernel(const AlignArgs a) {
  __shared__ int s_wave[kAlignWaves][kMaxExperts];
  const int tid = threadIdx.x, begin = blockIdx.x * kChunk;
  for (int x = tid; x < kAlignWaves * kMaxExperts; x += kAlignThreads) (&s_wave[0][0])[x] = 0;
  __syncthreads();
  count_slots(a, begin, min(begin + kChunk, a.S), 64, bits_for(a.E), s_wave);
  __syncthreads();
  if (tid < a.E) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kAlignWaves; ++w) n += s_wave[w][tid];
    a.ws[blockIdx.x * a.E + tid] = n;
  }
}

// ... and, from the counts of all chunks, places its own.
__global__ __launch_bounds__(kAlignThreads) void align_place_kernel(const AlignArgs a) {
  constexpr int kParts = kAlignThreads / kMaxExperts;
  constexpr int kEach = kMaxSlots / kChunk / kParts;   // chunks of one thread at most
  __shared__ int s_wave[kAlignWaves][kMaxExperts];
  __shared__ int s_all[kParts][kMaxExperts], s_pre[kParts][kMaxExperts];
  __shared__ int s_cnt[kMaxExperts], s_off[kMaxExperts + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nbits = bits_for(a.E);
  const int i = (int)blockIdx.x * kChunk + tid;        // this thread's slot
  const int id = i < a.S ? a.ids[i] : 0;
  // slots of an expert in all chunks and in those before this one: every
  // kParts-th chunk by one group of kMaxExperts threads, all loads at once
  const int x = tid % kMaxExperts, part = tid / kMaxExperts, chunks = gridDim.x;
  int n[kEach];
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    const int c = part + q * kParts;
    n[q] = x < a.E && c < chunks ? a.ws[c * a.E + x] : 0;
  }
  for (int q = tid; q < kAlignWaves * kMaxExperts; q += kAlignThreads) (&s_wave[0][0])[q] = 0;
  const int e = i < a.S ? local_expert(id, a.expert_first, a.E) : -1;
  const unsigned long long peers = peers_of(e, nbits);
  const int rank = lanes_below(peers);
  int all = 0, pre = 0;
#pragma unroll
  for (int q = 0; q < kEach; ++q) {
    all += n[q];
    pre += part + q * kParts < (int)blockIdx.x ? n[q] : 0;
  }
  s_all[part][x] = all;
  s_pre[part][x] = pre;
  __syncthreads();
  if (e >= 0 && rank == 0) s_wave[wave][e] = __popcll(peers);
  if (tid < kMaxExperts) {
    int sum = 0;
#pragma unroll
    for (int q = 0; q < kParts; ++q) sum += s_all[q][tid];
    s_cnt[tid] = sum;
  }
  __syncthreads();
  if (tid < 64) padded_starts(s_cnt, a.E, a.block_m, s_off);
  __syncthreads();
  if (tid < a.E) {
    int at = s_off[tid];
#pragma unroll
    for (int q = 0; q < kParts; ++q) at += s_pre[q][tid];
#pragma unroll
    for (int w = 0; w < kAlignWaves; ++w) {
      const int m = s_wave[w][tid];
      s_wave[w][tid] = at;
      at += m;
    }
  }
  __syncthreads();
  if (e >= 0) a.sorted_ids[s_wave[wave][e] + rank] = i;
  align_rest(a, s_off, s_cnt, blockIdx.x, chunks);
}

}  // namespace

namespace {

// Rows and base 16-byte aligned, and whole vectors in a row: 16 bytes, of the 16-bit
// types 8 where a lane's V values are no multiple of 16 bytes.
bool vector_rows(const void *p, long long ld, int dtype, int E, int V) {
  const long long bytes = ld * (dtype == MOE_F32 ? 4 : 2);
  return ((uintptr_t)p & 15u) == 0 && bytes % 16 == 0 && E % (dtype == MOE_F32 || V % 8 ? 4 : 8) == 0;
}

// Groups of gs experts are 2^n whole lanes of V.
bool whole_lanes(int gs, int V) {
  const int lanes = gs / V;
  return gs % V == 0 && (lanes & (lanes - 1)) == 0;
}

template <int G, int V>
hipError_t route_with(const RouteArgs &a, int dtype, hipStream_t s) {
  const bool vec = vector_rows(a.logits, a.ld, dtype, a.E, V);
  const long long blocks = ((long long)a.M * G + 255) / 256;
  const dim3 grid((unsigned)blocks), block(256);
  const int gs = a.E / a.n_group, lanes = gs / V;
  const bool grouped = a.topk_group < a.n_group;
  const bool by_lanes = whole_lanes(gs, V);
  // lanes of a group: those that hold it, or as many as there are for its scan
  int bits = 0;
  while (by_lanes ? (1 << bits) < lanes : (a.n_group << (bits + 1)) <= G) ++bits;
#define QMOE_ROUTE(kk, mode) \
  hipLaunchKernelGGL((route_topk_kernel<G, V, kk, mode>), grid, block, 0, s, a, dtype, vec, bits)
#define QMOE_ROUTE_K(mode)                 \
  do {                                     \
    if (a.top_k <= 2) QMOE_ROUTE(2, mode); \
    else QMOE_ROUTE(8, mode);              \
  } while (0)
  if (!grouped) {
    QMOE_ROUTE_K(kNoGroups);
  } else if (by_lanes) {
    QMOE_ROUTE_K(kLaneGroups);
  } else if constexpr (V <= 8) {         // launch_route_topk's wider lanes take no others
    QMOE_ROUTE_K(kAnyGroups);
  } else {
    return hipErrorInvalidValue;
  }
#undef QMOE_ROUTE_K
#undef QMOE_ROUTE
  return hipGetLastError();
}

template <int G, int V>
hipError_t backward_with(const RouteBwdArgs &a, int dtype, hipStream_t s) {
  const bool vin = vector_rows(a.logits, a.ld, dtype, a.E, V);
  const bool vout = vector_rows(a.dx, a.ldd, dtype, a.E, V);
  const dim3 grid((unsigned)(((long long)a.M * G + 255) / 256)), block(256);
  if (a.score == MOE_SCORE_SOFTMAX && !a.renormalize)
    hipLaunchKernelGGL((route_backward_kernel<G, V, true>), grid, block, 0, s, a, dtype, vin, vout);
  else
    hipLaunchKernelGGL((route_backward_kernel<G, V, false>), grid, block, 0, s, a, dtype, vin, vout);
  return hipGetLastError();
}

}  // namespace

// Lanes and keys per lane.  Few tokens: four keys, the shortest way through the
// lane's sort (64 tokens of 256 experts 4.9 us, with eight keys 5.8).  From a
// wavefront on every SIMD on, eight: fewer lanes repeat the merges (16384 tokens
// of 128 experts: 5.5 us, with four 8.3).  From 8192 tokens on 16 to 24, by which
// the lanes have work best (16384 tokens with 16 keys and with the number taken:
// 160 experts 9.9, 7.5 us, 320 17.9, 12.4; of 256 in groups 14.9, with eight
// 16.7).  Groups that are no whole lanes go through LDS, which costs more
// than the wider lanes save: those stay at eight keys (16384 tokens of 200 experts
// in 8 groups 18.5 us, with sixteen 23.7; 256 in 32 groups, whole lanes of eight,
// 17.6, with sixteen 25.3; 160 in 8, whole lanes of twenty, 9.2, with sixteen 20.4).
hipError_t launch_route_topk(const RouteArgs &a, int dtype, hipStream_t s) {
  constexpr int kWaves = 1024;                       // SIMDs of the card
  if (a.E <= 8) return route_with<8, 1>(a, dtype, s);
  if (a.E <= 32) return route_with<8, 4>(a, dtype, s);
  if (a.E <= 64) return route_with<8, 8>(a, dtype, s);
  const bool few = (long long)a.M * (a.E <= 128 ? 32 : 64) <= 64 * kWaves;
  const bool grouped = a.topk_group < a.n_group;
#define QMOE_MANY(limit, G, V) \
  if (a.E <= limit && (!grouped || whole_lanes(a.E / a.n_group, V))) return route_with<G, V>(a, dtype, s);
  if (a.M >= 8192) {
    QMOE_MANY(128, 8, 16)
    QMOE_MANY(160, 8, 20)
    QMOE_MANY(192, 8, 24)
    QMOE_MANY(256, 16, 16)
    QMOE_MANY(320, 16, 20)
    QMOE_MANY(384, 16, 24)
    QMOE_MANY(512, 32, 16)
  }
#undef QMOE_MANY
  if (a.E <= 128) return few ? route_with<32, 4>(a, dtype, s) : route_with<16, 8>(a, dtype, s);
  if (a.E <= 256) return few ? route_with<64, 4>(a, dtype, s) : route_with<32, 8>(a, dtype, s);
  return route_with<64, 8>(a, dtype, s);
}

hipError_t launch_route_backward(const RouteBwdArgs &a, int dtype, hipStream_t s) {
  if (a.E <= 8) return backward_with<8, 1>(a, dtype, s);
  if (a.E <= 32) return backward_with<8, 4>(a, dtype, s);
  if (a.E <= 64) return backward_with<8, 8>(a, dtype, s);
  if (a.E <= 128) return backward_with<16, 8>(a, dtype, s);
  if (a.E <= 256) return backward_with<32, 8>(a, dtype, s);
  return backward_with<64, 8>(a, dtype, s);
}

hipError_t launch_align_ids(const AlignArgs &a, hipStream_t s) {
  const int chunks = (a.S + kChunk - 1) / kChunk;
  const dim3 b(kAlignThreads);
  if (chunks <= kOneWorkgroupChunks) {
    hipLaunchKernelGGL(align_one_kernel, dim3(1), b, 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(align_count_kernel, dim3(chunks), b, 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(align_place_kernel, dim3(chunks), b, 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe
