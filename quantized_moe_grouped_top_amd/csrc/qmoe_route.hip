// The general router (scores, balance bias, groups, top-k, renormalised
// weights), its gradient, and the block alignment of given ids.
#include "qmoe_layer.h"

namespace qmoe {

namespace {

// ---- router -------------------------------------------------------------------
// Keys as 64-bit integers in the order of the doubles: NaN above every number,
// -0 equal to +0.
__device__ __forceinline__ uint64_t ordered(double v) {
  if (v != v) return ~0ull;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | (1ull << 63));
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// One token per thread; keys are computed again wherever they are needed.
template <typename Ty>
__global__ __launch_bounds__(64) void route_topk_kernel(const RouteArgs a) {
  const int t = blockIdx.x * 64 + threadIdx.x;
  if (t >= a.M) return;
  const typename Ty::T *x = (const typename Ty::T *)a.logits + (long long)t * a.ld;
  const int E = a.E;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  double m = 0.0, z = 1.0;
  if (soft) {
    m = -INFINITY;
    for (int e = 0; e < E; ++e) m = fmax(m, (double)Ty::load(x[e]));
    if (m == -INFINITY) m = 0.0;                    // no logit above -inf: scores 0 (or NaN)
    z = 0.0;
    for (int e = 0; e < E; ++e) z += exp((double)Ty::load(x[e]) - m);
  }
  auto score = [&](int e) -> double {
    const double v = (double)Ty::load(x[e]);
    if (!soft) return sigmoid64(v);
    return z == 0.0 ? 0.0 : exp(v - m) / z;
  };
  auto biased = [&](int e) -> double {
    return a.bias ? score(e) + (double)a.bias[e] : score(e);
  };
  auto key = [&](int e) -> uint64_t {
    return ordered(a.bias ? biased(e) : (double)Ty::load(x[e]));
  };
  uint64_t groups = ~0ull;                         // groups that stay
  const int gs = E / a.n_group;
  if (a.topk_group < a.n_group) {
    groups = 0;
    for (int r = 0; r < a.topk_group; ++r) {
      int best = -1;
      uint64_t best_v = 0;
      for (int g = 0; g < a.n_group; ++g) {
        if (groups >> g & 1) continue;
        uint64_t v;
        if (a.group_rule == MOE_GROUP_MAX) {
          v = 0;
          for (int e = g * gs; e < (g + 1) * gs; ++e) v = max(v, key(e));
        } else {
          double b1 = biased(g * gs), b2 = -INFINITY;
          bool first = true;
          for (int e = g * gs; e < (g + 1) * gs; ++e) {
            const double w = biased(e);
            if (first) {
              b1 = w;
              first = false;
            } else if (ordered(w) > ordered(b1)) {
              b2 = b1;
              b1 = w;
            } else if (ordered(w) > ordered(b2)) {
              b2 = w;
            }
          }
          v = ordered(b1 + b2);
        }
        if (best < 0 || v > best_v) {
          best = g;
          best_v = v;
        }
      }
      groups |= 1ull << best;
    }
  }
  // the j-th choice is the first expert, in the order of (key descending,
  // expert ascending), after the (j-1)-th
  int ids[kMaxTopK];
  uint64_t prev = ~0ull;
  int prev_id = -1;
  for (int j = 0; j < a.top_k; ++j) {
    int best = -1;
    uint64_t best_v = 0;
    for (int e = 0; e < E; ++e) {
      if (!(groups >> (e / gs) & 1)) continue;
      const uint64_t v = key(e);
      const bool after = j == 0 || v < prev || (v == prev && e > prev_id);
      if (after && (best < 0 || v > best_v)) {
        best = e;
        best_v = v;
      }
    }
    ids[j] = best;
    prev = best_v;
    prev_id = best;
  }
  double w[kMaxTopK], sum = 0.0, mc = -INFINITY;
  for (int j = 0; j < a.top_k; ++j) mc = fmax(mc, (double)Ty::load(x[ids[j]]));
  if (mc == -INFINITY) mc = 0.0;
  for (int j = 0; j < a.top_k; ++j) {
    if (soft && a.renormalize) {
      w[j] = exp((double)Ty::load(x[ids[j]]) - mc);
    } else {
      w[j] = score(ids[j]);
    }
    sum += w[j];
  }
  for (int j = 0; j < a.top_k; ++j) {
    const double q = a.renormalize ? (sum == 0.0 ? 0.0 : w[j] / sum) : w[j];
    a.ids[(long long)t * a.top_k + j] = ids[j];
    a.weights[(long long)t * a.top_k + j] = (float)(q * (double)a.scale);
  }
}

// ---- gradient -----------------------------------------------------------------
// One token per thread.
template <typename Ty>
__global__ __launch_bounds__(64) void route_backward_kernel(const RouteBwdArgs a) {
  const int t = blockIdx.x * 64 + threadIdx.x;
  if (t >= a.M) return;
  const typename Ty::T *x = (const typename Ty::T *)a.logits + (long long)t * a.ld;
  typename Ty::T *dx = (typename Ty::T *)a.dx + (long long)t * a.ldd;
  const int *ids = a.ids + (long long)t * a.top_k;
  const float *dw = a.dw + (long long)t * a.top_k;
  const int E = a.E, k = a.top_k;
  const bool soft = a.score == MOE_SCORE_SOFTMAX;
  double d[kMaxTopK];                               // gradient of every choice's logit
  double m = -INFINITY, z = 0.0, u = 0.0;
  if (soft && !a.renormalize) {
    for (int e = 0; e < E; ++e) m = fmax(m, (double)Ty::load(x[e]));
    if (m == -INFINITY) m = 0.0;
    for (int e = 0; e < E; ++e) z += exp((double)Ty::load(x[e]) - m);
  } else if (soft) {
    for (int j = 0; j < k; ++j)
      if ((unsigned)ids[j] < (unsigned)E) m = fmax(m, (double)Ty::load(x[ids[j]]));
    if (m == -INFINITY) m = 0.0;
  }
  double sum = 0.0;
  for (int j = 0; j < k; ++j) {
    d[j] = 0.0;
    if ((unsigned)ids[j] >= (unsigned)E) continue;
    const double v = (double)Ty::load(x[ids[j]]);
    d[j] = soft ? exp(v - m) : sigmoid64(v);
    sum += d[j];
  }
  if (soft && !a.renormalize) sum = z;
  const double inv = sum != 0.0 ? 1.0 / sum : 0.0;
  const bool ratio = soft || a.renormalize;         // shares of a sum
  for (int j = 0; j < k; ++j) {
    if ((unsigned)ids[j] < (unsigned)E && ratio) u += (double)dw[j] * (d[j] * inv);
  }
  for (int j = 0; j < k; ++j) {
    if ((unsigned)ids[j] >= (unsigned)E) continue;
    const double v = (double)Ty::load(x[ids[j]]);
    const double s = ratio ? d[j] * inv : d[j];
    const double tail = soft ? 1.0 : 1.0 / (1.0 + exp(v));
    // plain softmax: the -u term of every expert is added below
    const double g = (double)dw[j] - (ratio && !(soft && !a.renormalize) ? u : 0.0);
    d[j] = (double)a.scale * s * g * tail;
  }
  for (int e = 0; e < E; ++e) {
    double g = 0.0;
    for (int j = 0; j < k; ++j)
      if (ids[j] == e) g += d[j];
    if (soft && !a.renormalize)
      g -= (double)a.scale * u * (exp((double)Ty::load(x[e]) - m) * inv);
    dx[e] = Ty::store((float)g);
  }
}

// ---- alignment ------------------------------------------------------------------
// One workgroup: thread e counts, places and labels the slots of expert e.
__global__ __launch_bounds__(kMaxExperts) void align_ids_kernel(const AlignArgs a) {
  __shared__ int s_cnt[kMaxExperts];
  __shared__ int s_off[kMaxExperts + 1];
  const int e = threadIdx.x;
  int n = 0;
  if (e < a.E) {
    for (int i = 0; i < a.S; ++i) n += (long long)a.ids[i] - a.expert_first == e;
    s_cnt[e] = n;
    if (a.counts) a.counts[e] = n;
  }
  __syncthreads();
  if (e == 0) {
    int at = 0;
    for (int q = 0; q < a.E; ++q) {
      s_off[q] = at;
      at += (s_cnt[q] + a.block_m - 1) / a.block_m * a.block_m;
    }
    s_off[a.E] = at;
    *a.num_post = at;
  }
  __syncthreads();
  if (e < a.E) {
    int p = s_off[e];
    for (int b = p; b < s_off[e + 1]; b += a.block_m) a.expert_ids[b / a.block_m] = e;
    for (int i = 0; i < a.S; ++i)
      if ((long long)a.ids[i] - a.expert_first == e) a.sorted_ids[p++] = i;
    for (; p < s_off[e + 1]; ++p) a.sorted_ids[p] = a.S;
  }
  for (int p = s_off[a.E] + e; p < a.max_padded; p += blockDim.x) a.sorted_ids[p] = a.S;
  for (int b = s_off[a.E] / a.block_m + e; b < a.max_padded / a.block_m; b += blockDim.x)
    a.expert_ids[b] = -1;
}

}  // namespace

hipError_t launch_route_topk(const RouteArgs &a, int dtype, hipStream_t s) {
  const dim3 g((unsigned)((a.M + 63) / 64)), b(64);
  if (dtype == MOE_F32) hipLaunchKernelGGL(route_topk_kernel<TypeF32>, g, b, 0, s, a);
  else if (dtype == MOE_BF16) hipLaunchKernelGGL(route_topk_kernel<TypeBf16>, g, b, 0, s, a);
  else hipLaunchKernelGGL(route_topk_kernel<TypeF16>, g, b, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBwdArgs &a, int dtype, hipStream_t s) {
  const dim3 g((unsigned)((a.M + 63) / 64)), b(64);
  if (dtype == MOE_F32) hipLaunchKernelGGL(route_backward_kernel<TypeF32>, g, b, 0, s, a);
  else if (dtype == MOE_BF16) hipLaunchKernelGGL(route_backward_kernel<TypeBf16>, g, b, 0, s, a);
  else hipLaunchKernelGGL(route_backward_kernel<TypeF16>, g, b, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_align_ids(const AlignArgs &a, hipStream_t s) {
  hipLaunchKernelGGL(align_ids_kernel, dim3(1), dim3(kMaxExperts), 0, s, a);
  return hipGetLastError();
}

}  // namespace qmoe
