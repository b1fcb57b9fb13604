// The norms before and after a block, fused with the combine of its routed slots,
// its gate and the residual, and their gradients.
//
// Memory streams: a workgroup holds a whole row in registers (eight columns a
// thread and chunk, 16-byte loads and stores), so every byte is read and written
// once; the two sums of a row go through one wavefront reduction and LDS.  4096 rows of
// 4096 with two slots, norms before and after (168 MB): 32.5 us a call among others, the
// kernel 30.5 (29.4 at least), 5.5 TB/s; the gradients of 8192 rows of 6144 (604 MB): 138
// us a call, 4.4 TB/s, 5 of them the weights' sums (traced launch by launch, which starts
// each with the card empty, 147 + 5, at least 138 + 4.7).
#include "qmoe_block.h"
#include "qmoe_device.h"

namespace qmoe {

namespace {

typedef float f32x8 __attribute__((ext_vector_type(8)));

template <typename Ty>
__device__ __forceinline__ f32x8 unpack8(const i32x4 &v) {
  f32x8 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = Ty::load((uint16_t)((uint32_t)v[i >> 1] >> (16 * (i & 1))));
  return f;
}
template <typename Ty>
__device__ __forceinline__ f32x8 load8(const void *base, long long at) {
  if constexpr (sizeof(typename Ty::T) == 4) {
    const f32x4 *p = reinterpret_cast<const f32x4 *>((const float *)base + at);
    const f32x4 a = p[0], b = p[1];
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    return unpack8<Ty>(__builtin_nontemporal_load(reinterpret_cast<const i32x4 *>((const uint16_t *)base + at)));
  }
}
template <typename Ty>
__device__ __forceinline__ void store8(void *base, long long at, const f32x8 &v) {
  if constexpr (sizeof(typename Ty::T) == 4) {
    f32x4 *p = reinterpret_cast<f32x4 *>((float *)base + at);
    p[0] = __builtin_shufflevector(v, v, 0, 1, 2, 3);
    p[1] = __builtin_shufflevector(v, v, 4, 5, 6, 7);
  } else {
    i32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = Ty::pack(v[2 * i], v[2 * i + 1]);
    __builtin_nontemporal_store(o, reinterpret_cast<i32x4 *>((uint16_t *)base + at));
  }
}
__device__ __forceinline__ f32x8 zero8() { return f32x8{0, 0, 0, 0, 0, 0, 0, 0}; }
__device__ __forceinline__ float sum8(const f32x8 &v) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// The sum of v over the workgroup, the same in every thread and in every run.
// `part` is one of two buffers used in turn, so that one barrier is enough.
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += part[w];
  return s;
}

// s of chunk c of token t: the slots added in float32 in their order
template <typename Ty>
__device__ __forceinline__ f32x8 slots8(const uint16_t *y, int top_k, long long t, int N, int c) {
  f32x8 s = load8<Ty>(y, t * top_k * N + 8 * c);
  for (int j = 1; j < top_k; ++j) s += load8<Ty>(y, (t * top_k + j) * N + 8 * c);
  return s;
}

// V: chunks a thread
template <typename Ty, typename Res, int V>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs p) {
  __shared__ float s_part[2][16];
  const int N = p.N, chunks = N / 8;
  const float inv = 1.0f / (float)N;
  const long long t = blockIdx.x;
  f32x8 r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    r[i] = p.y && c < chunks ? slots8<Ty>(p.y, p.top_k, t, N, c) : zero8();
  }
  f32x8 x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    x[i] = p.residual && c < chunks ? load8<Res>(p.residual, t * N + 8 * c) : zero8();
  }
  float f = 1.0f;
  if (p.w_post) {
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) q += sum8(r[i] * r[i]);
    f = 1.0f / sqrtf(row_sum(q, s_part[0]) * inv + p.eps);
    if (p.rstd_post && threadIdx.x == 0) p.rstd_post[t] = f;
  }
  float scale = p.beta;
  if (p.gate_kind == MOE_GATE_TOKEN) scale *= p.gate[t];
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) {
      if (p.w_post) r[i] = r[i] * f * load8<TypeF32>(p.w_post, 8 * c);
      if (p.gate_kind == MOE_GATE_CHANNEL) r[i] *= load8<TypeF32>(p.gate, 8 * c);
      r[i] = p.alpha * x[i] + scale * r[i];
      store8<Res>(p.r, t * N + 8 * c, r[i]);
      q += sum8(r[i] * r[i]);
    }
  }
  if (!p.w_pre) return;
  f = 1.0f / sqrtf(row_sum(q, s_part[1]) * inv + p.eps);
  if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[t] = f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) store8<Ty>(p.h, t * N + 8 * c, r[i] * f * load8<TypeF32>(p.w_pre, 8 * c));
  }
}

// Eight neighbouring values as they lie in memory.
template <typename Ty>
struct Packed {
  i32x4 q[sizeof(typename Ty::T) == 4 ? 2 : 1];
};
template <typename Ty>
__device__ __forceinline__ Packed<Ty> load_packed(const void *base, long long at) {
  Packed<Ty> v;
  if constexpr (sizeof(typename Ty::T) == 4) {
    const i32x4 *p = reinterpret_cast<const i32x4 *>((const float *)base + at);
    v.q[0] = p[0];
    v.q[1] = p[1];
  } else {
    v.q[0] = *reinterpret_cast<const i32x4 *>((const uint16_t *)base + at);
  }
  return v;
}
template <typename Ty>
__device__ __forceinline__ f32x8 unpack(const Packed<Ty> &v) {
  if constexpr (sizeof(typename Ty::T) == 4) {
    f32x8 f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __int_as_float(v.q[i >> 2][i & 3]);
    return f;
  } else {
    return unpack8<Ty>(v.q[0]);
  }
}

// Workgroup b takes tokens b, b + grid, ..; the weights' gradients are added up
// column by column in registers and left, one row of each workgroup, in the
// workspace: [3][grid][N] (w_pre, w_post, channel gate).  A row's two sums wait for
// its loads and for each other, so the next row's loads go out before them.
// (8192 rows of 6144: 259 us without, 165 with two chunks a thread, of whose workgroups a CU
// holds one of six wavefronts.  Rows of more than 8192 need two chunks of 1024 threads, whose
// registers do not hold the next row.)
template <typename Ty, typename Res, int V>
__global__ __launch_bounds__(1024) void norm_backward_kernel(const NormBwdArgs p) {
  constexpr bool kAhead = V == 1;
  __shared__ float s_part[4][16];
  const int N = p.N, chunks = N / 8;
  const float inv = 1.0f / (float)N;
  const bool channel = p.gate_kind == MOE_GATE_CHANNEL;
  f32x8 g_pre[V], g_post[V], g_gate[V];
#pragma unroll
  for (int i = 0; i < V; ++i) g_pre[i] = g_post[i] = g_gate[i] = zero8();
  struct Row {
    Packed<Res> dr[V], r[V];
    Packed<Ty> dh[V], y[V];                           // y: the first slot
    float f_pre, f_post, gate;
  } next;
  auto fetch = [&](long long t) __attribute__((always_inline)) {
    if (p.w_pre) next.f_pre = p.rstd_pre[t];
    if (p.w_post) next.f_post = p.rstd_post[t];
    if (p.gate_kind == MOE_GATE_TOKEN) next.gate = p.gate[t];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        const long long at = t * N + 8 * c;
        if (p.w_pre) {
          next.r[i] = load_packed<Res>(p.r, at);
          next.dh[i] = load_packed<Ty>(p.d_h, at);
        }
        if (p.d_r) next.dr[i] = load_packed<Res>(p.d_r, at);
        if (p.y) next.y[i] = load_packed<Ty>(p.y, t * p.top_k * N + 8 * c);
      }
    }
  };
  int turn = 0;
  long long t = blockIdx.x;
  if (kAhead) fetch(t);
  for (; t < p.M; t += gridDim.x, turn ^= 2) {
    if (!kAhead) fetch(t);
    const float f = next.f_pre, fp = p.w_post ? next.f_post : 1.0f;
    const float gate_t = p.gate_kind == MOE_GATE_TOKEN ? next.gate : 1.0f;
    f32x8 dr[V], s[V], n[V], d[V];
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      dr[i] = s[i] = n[i] = d[i] = zero8();
      if (c < chunks) {
        if (p.d_r) dr[i] = unpack<Res>(next.dr[i]);
        if (p.y) s[i] = unpack<Ty>(next.y[i]);
        if (p.w_pre) {
          n[i] = unpack<Res>(next.r[i]) * f;
          const f32x8 dh = unpack<Ty>(next.dh[i]);
          g_pre[i] += dh * n[i];
          d[i] = dh * load8<TypeF32>(p.w_pre, 8 * c);
          q += sum8(d[i] * n[i]);
        }
      }
    }
    if (kAhead && t + gridDim.x < p.M) fetch(t + gridDim.x);
    if (p.y && p.top_k > 1) {                         // the slots added in their order
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < chunks)
          for (int j = 1; j < p.top_k; ++j) s[i] += load8<Ty>(p.y, (t * p.top_k + j) * N + 8 * c);
      }
    }
    if (p.w_pre) {
      const float mean = row_sum(q, s_part[turn]) * inv;
#pragma unroll
      for (int i = 0; i < V; ++i) dr[i] += f * (d[i] - n[i] * mean);
    }
    if (p.d_residual) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c < chunks) store8<Res>(p.d_residual, t * N + 8 * c, p.alpha * dr[i]);
      }
    }
    if (!p.y) continue;
    // the sum of dr p (by the channel gate) is both the token gate's gradient and, times it,
    // the norm's mean
    float u = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        s[i] *= fp;                                   // m, or s
        dr[i] *= p.beta;
        const f32x8 pv = p.w_post ? s[i] * load8<TypeF32>(p.w_post, 8 * c) : s[i];
        if (channel) {
          const f32x8 gv = load8<TypeF32>(p.gate, 8 * c);
          g_gate[i] += dr[i] * pv;
          dr[i] *= gv;
        }
        u += sum8(dr[i] * pv);
      }
    }
    if (p.w_post || p.gate_kind == MOE_GATE_TOKEN) u = row_sum(u, s_part[turn + 1]);
    if (p.gate_kind == MOE_GATE_TOKEN && p.d_gate && threadIdx.x == 0) p.d_gate[t] = u;
    const float mean = gate_t * u * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < chunks) {
        f32x8 dp = dr[i] * gate_t;
        if (p.w_post) {
          g_post[i] += dp * s[i];
          dp = fp * (dp * load8<TypeF32>(p.w_post, 8 * c) - s[i] * mean);
        }
        store8<Ty>(p.d_y, t * N + 8 * c, dp);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < chunks) {
      const long long at = (long long)blockIdx.x * N + 8 * c, set = (long long)gridDim.x * N;
      if (p.d_w_pre) store8<TypeF32>(p.ws, at, g_pre[i]);
      if (p.d_w_post) store8<TypeF32>(p.ws, set + at, g_post[i]);
      if (p.d_gate && channel) store8<TypeF32>(p.ws, 2 * set + at, g_gate[i]);
    }
  }
}

// The workgroups' rows added up in a fixed order: 64 columns a workgroup, its 16
// wavefronts a sixteenth of the rows each (four of them with a quarter: 33 us for 512
// rows of 6144 where this takes 9).
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void norm_join_kernel(const NormBwdArgs p, int rows) {
  __shared__ float s_part[kJoinWaves][64];
  float *const outs[3] = {p.d_w_pre, p.d_w_post, p.gate_kind == MOE_GATE_CHANNEL ? p.d_gate : nullptr};
  float *out = outs[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 63, col = blockIdx.x * 64 + lane, part = threadIdx.x >> 6;
  float v[4] = {};
  if (col < p.N) {
    const float *ws = p.ws + (long long)blockIdx.y * rows * p.N + col;
    const int to = rows * (part + 1) / kJoinWaves;
    int r = rows * part / kJoinWaves;
    for (; r + 4 <= to; r += 4)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += ws[(long long)(r + i) * p.N];
    for (; r < to; ++r) v[0] += ws[(long long)r * p.N];
  }
  s_part[part][lane] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  if (part == 0 && col < p.N) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWaves; ++w) sum += s_part[w][lane];
    out[col] = sum;
  }
}

// threads for rows of N columns with at most `most` chunks a thread
int threads_for(int N, int most) {
  const int chunks = N / 8;
  int t = 64;
  while (t < 1024 && t * most < chunks) t += 64;
  return t;
}

// As many workgroups as the card holds at once (a CU one where rows of more than 4096 take
// nine wavefronts or more), fewer where that gives each the same number of tokens.
int backward_grid(int M, int N) {
  const int most = N > 4096 ? 256 : 512, each = (M + most - 1) / most;
  return each ? (M + each - 1) / each : 0;
}

template <typename Ty, typename Res>
hipError_t run(const NormArgs &a, hipStream_t s) {
  const int t = threads_for(a.N, 2);
  const dim3 grid(a.M), block(t);
  if (a.N / 8 <= t) hipLaunchKernelGGL((norm_kernel<Ty, Res, 1>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_kernel<Ty, Res, 2>), grid, block, 0, s, a);
  return hipGetLastError();
}
template <typename Ty, typename Res>
hipError_t run_backward(const NormBwdArgs &a, hipStream_t s) {
  const int rows = backward_grid(a.M, a.N);
  if (a.M > 0) {
    const int t = threads_for(a.N, 1);
    const dim3 grid(rows), block(t);
    if (a.N / 8 <= t) hipLaunchKernelGGL((norm_backward_kernel<Ty, Res, 1>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((norm_backward_kernel<Ty, Res, 2>), grid, block, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool sums = a.d_w_pre || a.d_w_post || (a.d_gate && a.gate_kind == MOE_GATE_CHANNEL);
  if (!sums) return hipSuccess;
  hipLaunchKernelGGL(norm_join_kernel, dim3((a.N + 63) / 64, 3), dim3(64 * kJoinWaves), 0, s, a, rows);
  return hipGetLastError();
}

}  // namespace

size_t norm_backward_workspace_bytes(int M, int N) {
  return (size_t)3 * backward_grid(M, N) * N * sizeof(float);
}

hipError_t launch_norm(const NormArgs &a, int dtype, int r_dtype, hipStream_t s) {
  if (dtype == MOE_BF16)
    return r_dtype == MOE_F32 ? run<TypeBf16, TypeF32>(a, s) : run<TypeBf16, TypeBf16>(a, s);
  return r_dtype == MOE_F32 ? run<TypeF16, TypeF32>(a, s) : run<TypeF16, TypeF16>(a, s);
}

hipError_t launch_norm_backward(const NormBwdArgs &a, int dtype, int r_dtype, hipStream_t s) {
  if (dtype == MOE_BF16)
    return r_dtype == MOE_F32 ? run_backward<TypeBf16, TypeF32>(a, s)
                              : run_backward<TypeBf16, TypeBf16>(a, s);
  return r_dtype == MOE_F32 ? run_backward<TypeF16, TypeF32>(a, s)
                            : run_backward<TypeF16, TypeF16>(a, s);
}

}  // namespace qmoe
