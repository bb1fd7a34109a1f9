// Layer norm and its gradients (sm_103a).
//
//   m = mean x (0 if not centred), r = 1 / sqrt(mean (x - m)^2 + eps), h = (x - m) r, y = h w + b
//   g = dy w,  dx = r (g - mean g (0 if not centred) - h mean(g h)) + add
//   dw (+)= sum over rows of dy h,  db (+)= sum over rows of dy
//
// Bound: HBM (about 7 operations an element forward, 14 backward).
#include <algorithm>
#include <type_traits>

#include "fsp_rows.cuh"

namespace fsp {
namespace {

constexpr int64_t kMostDim = int64_t(1) << 20;   // a thread of the widest rows adds 1024 elements
constexpr int kParts = 152;                      // most partial sums of the weight's gradient: one per SM

__device__ __forceinline__ float load_any(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : widen(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int V>
__device__ __forceinline__ void load_any(const void* p, bool f32, int64_t i, float* f) {
  if (f32)
    load_vec<float, V>(static_cast<const float*>(p) + i, f);
  else
    load_vec<__nv_bfloat16, V>(static_cast<const __nv_bfloat16*>(p) + i, f);
}
template <int V>
__device__ __forceinline__ void store_any(void* p, bool f32, int64_t i, const float* f) {
  if (f32)
    store_vec<float, V>(static_cast<float*>(p) + i, f);
  else
    store_vec<__nv_bfloat16, V>(static_cast<__nv_bfloat16*>(p) + i, f);
}

struct NormArgs {
  const void* x;
  const void* weight;   // NULL: ones
  const void* bias;     // NULL: zeros
  void* out;
  float2* stats;        // (m, r) of each row, or NULL
  int64_t rows, dim, x_stride, out_stride;
  float eps;
  bool center, param_f32, out_f32;
};

struct GradArgs {
  const void* x;
  const float2* stats;
  const void* grad;
  const void* weight;   // NULL: ones
  const void* add;      // NULL: zeros
  void* grad_x;         // NULL: not wanted
  float* parts;         // [kParts][2][dim]
  void* grad_weight;    // NULL: not wanted
  void* grad_bias;
  int64_t rows, dim, x_stride, grad_stride, add_stride, grad_x_stride;
  int n_parts;
  bool center, weight_f32, grad_param_f32, accumulate;
};

// The sums over the CTA of N values per thread, in every thread.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float (*share)[N]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < N; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
    if (lane == 0) share[warp][j] = v[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    v[j] = lane < int(blockDim.x >> 5) ? share[lane][j] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  }
  __syncthreads();
}

// ---- rows that fit in registers -------------------------------------------------------

// T threads hold a row, E elements each: accesses of V elements, T * V apart.  T < 32 divides
// a warp among rows.
template <int T>
__device__ __forceinline__ float row_sum(float v) {   // over T <= 32 lanes
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rows of T threads, R of them in flight per thread.  A warp or less per row needs no
// barrier; a longer row has a CTA of its own.
template <typename X, int V, int T, int E, int R>
__global__ void __launch_bounds__(T > 256 ? T : 256) norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kThreads = T > 256 ? T : 256, N = E / V, kRows = kThreads / T;
  static_assert(T <= 32 || R == 1);
  __shared__ float share[2][T > 32 ? kThreads / 32 : 1];
  launch_dependents();
  grid_dependency_wait();
  const int t = threadIdx.x % T;
  const int64_t row0 = (int64_t(blockIdx.x) * kRows + threadIdx.x / T) * R;
  auto sum = [&](float v, int which) {
    if constexpr (T <= 32) {
      return row_sum<T>(v);
    } else {
      constexpr int W = T / 32;
      v = row_sum<32>(v);
      float* mine = share[which] + threadIdx.x / T * W;
      if (threadIdx.x % 32 == 0) mine[t / 32] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) v += mine[k];
      return v;
    }
  };
  alignas(32) X raw[R][N][V];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * T + t) * V;
      if (row0 + i < a.rows && c < a.dim) {
        load_raw<X, V>(static_cast<const X*>(a.x) + (row0 + i) * a.x_stride + c, raw[i][n]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) raw[i][n][j] = narrow<X>(0.f);
      }
    }
  const float count = float(a.dim);
  float m[R], r[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = 0.f;
    if (a.center) {
      float v = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < V; ++j) v += widen(raw[i][n][j]);
      m[i] = sum(v, 0) / count;
    }
    float v = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if ((n * T + t) * V < a.dim) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = widen(raw[i][n][j]) - m[i];
          v = __fmaf_rn(d, d, v);
        }
      }
    r[i] = 1.f / sqrtf(sum(v, 1) / count + a.eps);
    if (a.stats && t == 0 && row0 + i < a.rows) a.stats[row0 + i] = make_float2(m[i], r[i]);
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * T + t) * V;
    if (c >= a.dim) break;
    float w[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[j] = 1.f;
      b[j] = 0.f;
    }
    if (a.weight) load_any<V>(a.weight, a.param_f32, c, w);
    if (a.bias) load_any<V>(a.bias, a.param_f32, c, b);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = __fmaf_rn((widen(raw[i][n][j]) - m[i]) * r[i], w[j], b[j]);
      if (row0 + i < a.rows) store_any<V>(a.out, a.out_f32, (row0 + i) * a.out_stride + c, f);
    }
  }
}

// All gradients in one pass over x and dy.  A thread holds the same columns of every row it
// takes part in, and adds their terms of dw and db in registers; the CTA's rows are joined
// in shared memory at the end, so that a launch leaves one pair of partial sums per CTA.
// The next row's loads are in flight while a row is reduced.
constexpr int kGradThreads = 512;

template <typename X, typename G, int V, int T, int E>
__global__ void __launch_bounds__(kGradThreads, 1) grad_kernel(const __grid_constant__ GradArgs a) {
  constexpr int N = E / V, kGroups = kGradThreads / T;
  extern __shared__ __align__(16) float joined[];   // [2][kGroups][T * E]
  __shared__ float2 share[2][kGradThreads / 32];
  launch_dependents();
  grid_dependency_wait();
  const int group = threadIdx.x / T, t = threadIdx.x % T;
  // rows of a warp's groups advance together: `first` is that of its first group
  const int64_t step = int64_t(gridDim.x) * kGroups;
  int64_t row = int64_t(blockIdx.x) * kGroups + group;
  int64_t first = int64_t(blockIdx.x) * kGroups + threadIdx.x / (T < 32 ? 32 : T) * (T < 32 ? 32 / T : 1);
  float w[E], dw[E] = {}, db[E] = {};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * T + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) w[n * V + j] = 1.f;
    if (a.weight && c < a.dim) load_any<V>(a.weight, a.weight_f32, c, &w[n * V]);
  }
  alignas(32) X xr[N][V], ar[N][V];
  alignas(32) G gr[N][V];
  float2 st;
  auto fetch = [&](auto* to, const auto* from, int64_t stride) {
    using Y = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * T + t) * V;
      if (row < a.rows && c < a.dim) {
        load_raw<Y, V>(from + row * stride + c, to[n]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) to[n][j] = narrow<Y>(0.f);
      }
    }
  };
  auto fetch_row = [&] {
    fetch(xr, static_cast<const X*>(a.x), a.x_stride);
    fetch(gr, static_cast<const G*>(a.grad), a.grad_stride);
    st = row < a.rows ? a.stats[row] : make_float2(0.f, 0.f);
  };
  fetch_row();
  if (a.add) fetch(ar, static_cast<const X*>(a.add), a.add_stride);
  const float count = float(a.dim);
  for (int which = 0; first < a.rows; which ^= 1) {
    float h[E], g[E], s0 = 0.f, s1 = 0.f;
    const float r = st.y;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = n * V + j;
        const float dy = widen(gr[n][j]);
        h[e] = (widen(xr[n][j]) - st.x) * r;
        dw[e] = __fmaf_rn(dy, h[e], dw[e]);
        db[e] += dy;
        g[e] = dy * w[e];
        s0 += g[e];
        s1 = __fmaf_rn(g[e], h[e], s1);
      }
    const int64_t now = row;
    first += step;
    row += step;
    fetch_row();
    if (a.grad_x) {
      s0 = row_sum<(T < 32 ? T : 32)>(s0);
      s1 = row_sum<(T < 32 ? T : 32)>(s1);
      if constexpr (T > 32) {
        constexpr int W = T / 32;
        float2* mine = share[which] + group * W;
        if (threadIdx.x % 32 == 0) mine[t / 32] = make_float2(s0, s1);
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
        s0 = s1 = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          s0 += mine[k].x;
          s1 += mine[k].y;
        }
      }
      const float mean_g = a.center ? s0 / count : 0.f, mean_gh = s1 / count;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = (n * T + t) * V;
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = n * V + j;
          f[j] = __fmaf_rn(r, __fmaf_rn(-h[e], mean_gh, g[e] - mean_g), a.add ? widen(ar[n][j]) : 0.f);
        }
        if (now < a.rows && c < a.dim) store_vec<X, V>(static_cast<X*>(a.grad_x) + now * a.grad_x_stride + c, f);
      }
      if (a.add) fetch(ar, static_cast<const X*>(a.add), a.add_stride);
    }
  }
  if (!a.grad_weight && !a.grad_bias) return;
  constexpr int kCols = T * E;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (n * T + t) * V + j;
      joined[group * kCols + c] = dw[n * V + j];
      joined[(kGroups + group) * kCols + c] = db[n * V + j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kCols; i += kGradThreads) {
    const int which = i / kCols, c = i % kCols;
    if (c >= a.dim || !(which ? a.grad_bias : a.grad_weight)) continue;
    float v = 0.f;
#pragma unroll 8
    for (int k = 0; k < kGroups; ++k) v += joined[(which * kGroups + k) * kCols + c];
    a.parts[(int64_t(blockIdx.x) * 2 + which) * a.dim + c] = v;
  }
}

// ---- rows through shared memory -------------------------------------------------------
//
// Many rows: each CTA stays and takes every gridDim.x-th set of 512 / T rows.  A thread
// holds the same E columns of every row it takes part in, so its parameters are read once,
// and copies those columns of the rows ahead into its own part of a ring of stages in shared
// memory (cp.async): the copies of kStages - 1 rows are in flight while a row is reduced,
// without registers for them, and what a thread copied is read by itself alone, so that the
// ring needs no barriers.

constexpr int kRingThreads = 512;
constexpr int kHold = 16;   // columns of a thread (bf16 and fp32 rows)

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {   // 16 bytes, or zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {   // until at most N groups of this thread's copies are in flight
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_at(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

// A thread's columns of one row of Y, as N accesses of V elements, T * V apart: in a stage
// [n][thread] of accesses.
template <typename Y, int V, int T, int N>
struct Columns {
  static constexpr int kBytes = int(sizeof(Y)) * V;
  static constexpr int kStage = N * kRingThreads * kBytes;
  static_assert(kBytes % 16 == 0);
  static __device__ __forceinline__ void copy(char* stage, const void* from, int64_t stride, int64_t row, int64_t rows, int64_t dim, int t) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * T + t) * V;
      const bool there = row < rows && c < dim;
      const char* src = reinterpret_cast<const char*>(static_cast<const Y*>(from) + (there ? row * stride + c : 0));
      const uint32_t dst = smem_at(stage) + (n * kRingThreads + threadIdx.x) * kBytes;
#pragma unroll
      for (int k = 0; k < kBytes; k += 16) copy_async(dst + k, src + k, there);
    }
  }
  static __device__ __forceinline__ void read(const char* stage, int n, float* f) {
    alignas(16) Y y[V];
    const uint4* from = reinterpret_cast<const uint4*>(stage + (n * kRingThreads + threadIdx.x) * kBytes);
#pragma unroll
    for (int k = 0; k < kBytes / 16; ++k) reinterpret_cast<uint4*>(y)[k] = from[k];
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = widen(y[j]);
  }
};

// Sums over the T threads of a group, of which a CTA has several.  `which` alternates from
// sum to sum: a thread is past the barrier of a sum only when all have read the one before.
template <int T, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float (*share)[kRingThreads / 32][K], int which) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = row_sum<(T < 32 ? T : 32)>(v[k]);
  if constexpr (T > 32) {
    const int group = threadIdx.x / T;
    float(*mine)[K] = share[which] + group * (T / 32);
    if (threadIdx.x % 32 == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) mine[threadIdx.x % T / 32][k] = v[k];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(T) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += mine[w][k];
  }
}

// The rows of a thread: `row` its group's, `first` that of its warp's first group (the groups
// of a warp advance together), `step` to the next.
template <int T>
struct Walk {
  int64_t row, first, step;
  int t;
  __device__ __forceinline__ Walk() {
    constexpr int kGroups = kRingThreads / T, kUnit = T < 32 ? 32 : T;
    t = threadIdx.x % T;
    step = int64_t(gridDim.x) * kGroups;
    row = int64_t(blockIdx.x) * kGroups + threadIdx.x / T;
    first = int64_t(blockIdx.x) * kGroups + threadIdx.x / kUnit * (kUnit / T);
  }
};

template <typename X, int V, int T, int kStages>
__global__ void __launch_bounds__(kRingThreads, 1) norm_ring_kernel(const __grid_constant__ NormArgs a) {
  constexpr int E = kHold, N = E / V;
  using C = Columns<X, V, T, N>;
  extern __shared__ __align__(16) char ring[];
  __shared__ float share[2][kRingThreads / 32][1];
  launch_dependents();
  grid_dependency_wait();
  Walk<T> at;
  const int t = at.t;
#pragma unroll
  for (int d = 0; d < kStages; ++d) {
    C::copy(ring + d * C::kStage, a.x, a.x_stride, at.row + d * at.step, a.rows, a.dim, t);
    copies_issued();
  }
  float w[E], b[E];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * T + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[n * V + j] = 1.f;
      b[n * V + j] = 0.f;
    }
    if (a.weight && c < a.dim) load_any<V>(a.weight, a.param_f32, c, &w[n * V]);
    if (a.bias && c < a.dim) load_any<V>(a.bias, a.param_f32, c, &b[n * V]);
  }
  const float count = float(a.dim);
  int slot = 0, which = 0;
  for (; at.first < a.rows; at.first += at.step, at.row += at.step, which ^= 1) {
    char* stage = ring + slot * C::kStage;
    slot = slot + 1 == kStages ? 0 : slot + 1;
    copies_wait<kStages - 1>();
    float f[E], m = 0.f, s[1];
#pragma unroll
    for (int n = 0; n < N; ++n) C::read(stage, n, &f[n * V]);
    if (a.center) {
      s[0] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] += f[e];
      group_sum<T>(s, share, 0);
      m = s[0] / count;
    }
    s[0] = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = n * V + j;
        f[e] -= m;
        if ((n * T + t) * V < a.dim) s[0] = __fmaf_rn(f[e], f[e], s[0]);
      }
    group_sum<T>(s, share, a.center ? 1 : which);
    C::copy(stage, a.x, a.x_stride, at.row + kStages * at.step, a.rows, a.dim, t);   // (what was read is in registers)
    copies_issued();
    const float r = 1.f / sqrtf(s[0] / count + a.eps);
    if (at.row < a.rows) {
      if (a.stats && t == 0) a.stats[at.row] = make_float2(m, r);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = (n * T + t) * V;
        float y[V];
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = __fmaf_rn(f[n * V + j] * r, w[n * V + j], b[n * V + j]);
        if (c < a.dim) store_any<V>(a.out, a.out_f32, at.row * a.out_stride + c, y);
      }
    }
  }
  copies_wait<0>();
}

// All gradients in one pass over x and dy.  A thread adds its columns' terms of dw and db in
// registers; the CTA's groups are joined in shared memory at the end, so that a launch leaves
// one pair of partial sums per CTA.
template <typename X, typename G, int V, int T, int kStages>
__global__ void __launch_bounds__(kRingThreads, 1) grad_ring_kernel(const __grid_constant__ GradArgs a) {
  constexpr int E = kHold, N = E / V, kGroups = kRingThreads / T;
  using CX = Columns<X, V, T, N>;
  using CG = Columns<G, V, T, N>;
  constexpr int kStage = 2 * CX::kStage + CG::kStage;   // dy, x, add
  extern __shared__ __align__(16) char ring[];
  __shared__ float share[2][kRingThreads / 32][2];
  launch_dependents();
  grid_dependency_wait();
  Walk<T> at;
  const int t = at.t;
  auto copy_row = [&](char* stage, int64_t row) {
    CG::copy(stage, a.grad, a.grad_stride, row, a.rows, a.dim, t);
    CX::copy(stage + CG::kStage, a.x, a.x_stride, row, a.rows, a.dim, t);
    if (a.add) CX::copy(stage + CG::kStage + CX::kStage, a.add, a.add_stride, row, a.rows, a.dim, t);
    copies_issued();
  };
#pragma unroll
  for (int d = 0; d < kStages; ++d) copy_row(ring + d * kStage, at.row + d * at.step);
  float w[E], dw[E] = {}, db[E] = {};
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * T + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) w[n * V + j] = 1.f;
    if (a.weight && c < a.dim) load_any<V>(a.weight, a.weight_f32, c, &w[n * V]);
  }
  const float count = float(a.dim);
  float2 next = at.row < a.rows ? a.stats[at.row] : make_float2(0.f, 0.f);
  int slot = 0;
  for (int which = 0; at.first < a.rows; which ^= 1) {
    char* stage = ring + slot * kStage;
    slot = slot + 1 == kStages ? 0 : slot + 1;
    const float2 st = next;
    if (at.row + at.step < a.rows) next = a.stats[at.row + at.step];
    copies_wait<kStages - 1>();
    float h[E], g[E], s[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      CG::read(stage, n, &g[n * V]);
      CX::read(stage + CG::kStage, n, &h[n * V]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int e = n * V + j;
        h[e] = (h[e] - st.x) * st.y;
        dw[e] = __fmaf_rn(g[e], h[e], dw[e]);
        db[e] += g[e];
        g[e] *= w[e];
        s[0] += g[e];
        s[1] = __fmaf_rn(g[e], h[e], s[1]);
      }
    }
    if (a.grad_x) {
      group_sum<T>(s, share, which);
      const float mean_g = a.center ? s[0] / count : 0.f, mean_gh = s[1] / count;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = (n * T + t) * V;
        float f[V] = {};
        if (a.add) CX::read(stage + CG::kStage + CX::kStage, n, f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = n * V + j;
          f[j] = __fmaf_rn(st.y, __fmaf_rn(-h[e], mean_gh, g[e] - mean_g), f[j]);
        }
        if (at.row < a.rows && c < a.dim) store_vec<X, V>(static_cast<X*>(a.grad_x) + at.row * a.grad_x_stride + c, f);
      }
    }
    copy_row(stage, at.row + kStages * at.step);
    at.first += at.step;
    at.row += at.step;
  }
  copies_wait<0>();
  if (!a.grad_weight && !a.grad_bias) return;
  __syncthreads();
  constexpr int kCols = T * E;
  float* joined = reinterpret_cast<float*>(ring);   // [2][kGroups][kCols]
  static_assert(2 * kGroups * kCols * 4 <= kStages * kStage);
  const int group = threadIdx.x / T;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (n * T + t) * V + j;
      joined[group * kCols + c] = dw[n * V + j];
      joined[(kGroups + group) * kCols + c] = db[n * V + j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kCols; i += kRingThreads) {
    const int which = i / kCols, c = i % kCols;
    if (c >= a.dim || !(which ? a.grad_bias : a.grad_weight)) continue;
    float v = 0.f;
#pragma unroll 8
    for (int k = 0; k < kGroups; ++k) v += joined[(which * kGroups + k) * kCols + c];
    a.parts[(int64_t(blockIdx.x) * 2 + which) * a.dim + c] = v;
  }
}

// ---- rows of any length: a CTA per row, which reads it again for each pass ------------

constexpr int kWideThreads = 1024;

template <typename X, int V>
__global__ void __launch_bounds__(kWideThreads) wide_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float share[32][1];
  launch_dependents();
  grid_dependency_wait();
  const int64_t row = blockIdx.x, first = int64_t(threadIdx.x) * V, step = int64_t(blockDim.x) * V;
  const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
  float f[V], m = 0.f, s[1];
  if (a.center) {
    s[0] = 0.f;
    for (int64_t c = first; c < a.dim; c += step) {
      load_vec<X, V>(x + c, f);
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) t += f[j];
      s[0] += t;
    }
    cta_sum<1>(s, share);
    m = s[0] / float(a.dim);
  }
  s[0] = 0.f;
  for (int64_t c = first; c < a.dim; c += step) {
    load_vec<X, V>(x + c, f);
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) t = __fmaf_rn(f[j] - m, f[j] - m, t);
    s[0] += t;
  }
  cta_sum<1>(s, share);
  const float r = 1.f / sqrtf(s[0] / float(a.dim) + a.eps);
  if (a.stats && threadIdx.x == 0) a.stats[row] = make_float2(m, r);
  for (int64_t c = first; c < a.dim; c += step) {
    load_vec<X, V>(x + c, f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float h = (f[j] - m) * r;
      f[j] = __fmaf_rn(h, a.weight ? load_any(a.weight, a.param_f32, c + j) : 1.f,
                       a.bias ? load_any(a.bias, a.param_f32, c + j) : 0.f);
    }
    store_any<V>(a.out, a.out_f32, row * a.out_stride + c, f);
  }
}

template <typename X, typename G, int V>
__global__ void __launch_bounds__(kWideThreads) wide_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float share[32][2];
  launch_dependents();
  grid_dependency_wait();
  const int64_t row = blockIdx.x, first = int64_t(threadIdx.x) * V, step = int64_t(blockDim.x) * V;
  const X* x = static_cast<const X*>(a.x) + row * a.x_stride;
  const G* dy = static_cast<const G*>(a.grad) + row * a.grad_stride;
  const float2 st = a.stats[row];
  float h[V], g[V], s[2] = {0.f, 0.f};
  auto load = [&](int64_t c) {
    load_vec<X, V>(x + c, h);
    load_vec<G, V>(dy + c, g);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[j] = (h[j] - st.x) * st.y;
      if (a.weight) g[j] *= load_any(a.weight, a.weight_f32, c + j);
    }
  };
  for (int64_t c = first; c < a.dim; c += step) {
    load(c);
    float t = 0.f, u = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      t += g[j];
      u = __fmaf_rn(g[j], h[j], u);
    }
    s[0] += t;
    s[1] += u;
  }
  cta_sum<2>(s, share);
  const float mean_g = a.center ? s[0] / float(a.dim) : 0.f, mean_gh = s[1] / float(a.dim);
  for (int64_t c = first; c < a.dim; c += step) {
    load(c);
    float add[V] = {};
    if (a.add) load_vec<X, V>(static_cast<const X*>(a.add) + row * a.add_stride + c, add);
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = __fmaf_rn(st.y, g[j] - mean_g - h[j] * mean_gh, add[j]);
    store_vec<X, V>(static_cast<X*>(a.grad_x) + row * a.grad_x_stride + c, g);
  }
}

// The weight's and the bias's gradient: part p of the rows, 32 x V columns a CTA.
constexpr int kColumnWarps = 8;

template <typename X, typename G, int V>
__global__ void __launch_bounds__(kColumnWarps * 32) column_sums_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float share[kColumnWarps][2][32 * V];
  launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = (int64_t(blockIdx.x) * 32 + lane) * V;
  const int64_t begin = a.rows * blockIdx.y / a.n_parts, end = a.rows * (blockIdx.y + 1) / a.n_parts;
  float dw[V] = {}, db[V] = {};
  if (col < a.dim)
    for (int64_t row = begin + warp; row < end; row += kColumnWarps) {
      float h[V], g[V];
      load_vec<X, V>(static_cast<const X*>(a.x) + row * a.x_stride + col, h);
      load_vec<G, V>(static_cast<const G*>(a.grad) + row * a.grad_stride + col, g);
      const float2 st = a.stats[row];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dw[j] = __fmaf_rn(g[j], (h[j] - st.x) * st.y, dw[j]);
        db[j] += g[j];
      }
    }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    share[warp][0][j * 32 + lane] = dw[j];
    share[warp][1][j * 32 + lane] = db[j];
  }
  __syncthreads();
  if (warp < 2 && col < a.dim) {
    float sum[V] = {};
    for (int w = 0; w < kColumnWarps; ++w)
#pragma unroll
      for (int j = 0; j < V; ++j) sum[j] += share[w][warp][j * 32 + lane];
    store_vec<float, V>(a.parts + (int64_t(blockIdx.y) * 2 + warp) * a.dim + col, sum);
  }
}

// Adds the parts, 32 columns of one of the two gradients a CTA; warp w adds parts w, w + 32, ...
constexpr int kJoinWarps = 32;

__global__ void __launch_bounds__(kJoinWarps * 32) join_columns_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float share[kJoinWarps][32];
  launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  void* out = blockIdx.y == 0 ? a.grad_weight : a.grad_bias;
  if (!out) return;
  const int64_t col = int64_t(blockIdx.x) * 32 + lane;
  float sum = 0.f;
  if (col < a.dim) {
#pragma unroll
    for (int k = 0; k < (kParts + kJoinWarps - 1) / kJoinWarps; ++k) {
      const int p = warp + k * kJoinWarps;
      if (p < a.n_parts) sum += a.parts[(int64_t(p) * 2 + blockIdx.y) * a.dim + col];
    }
  }
  share[warp][lane] = sum;
  __syncthreads();
  if (warp > 0 || col >= a.dim) return;
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) sum += share[w][lane];
  if (a.accumulate) sum += load_any(out, a.grad_param_f32, col);
  store_any<1>(out, a.grad_param_f32, col, &sum);
}

// ---- host -----------------------------------------------------------------------------

fsp_status check_sizes(int64_t rows, int64_t dim) {
  if (rows < 0 || dim < 0) return fail(FSP_EINVAL, "rows and dim must be >= 0");
  if (dim > kMostDim) return fail(FSP_EUNSUPPORTED, "dim must be at most 2^20");
  if (rows > INT32_MAX) return fail(FSP_EUNSUPPORTED, "rows must be below 2^31");
  return FSP_OK;
}

fsp_status check_vector(const void* p, int64_t dim, int32_t dtype, const char* name) {
  return p ? check_form(p, 1, dim, std::max<int64_t>(1, dim), dtype, name) : FSP_OK;
}
Operand vector_operand(const void* p, int64_t dim, int32_t dtype, const char* name) {
  return {p, p ? size_t(dim) * size_of(dtype) : 0, name};
}

fsp_status check_stats(const float* stats) {
  return reinterpret_cast<uintptr_t>(stats) % 8 ? fail(FSP_EINVAL, "stats is not 8-byte aligned") : FSP_OK;
}

template <typename X, int V, int T, int E, int R>
fsp_status launch_rows(const NormArgs& a, cudaStream_t st) {
  constexpr int kThreads = T > 256 ? T : 256, kRows = kThreads / T * R;
  return launch_next(norm_kernel<X, V, T, E, R>, dim3(unsigned((a.rows + kRows - 1) / kRows)), kThreads, 0, 1, a, st, "layer norm kernel launch");
}

template <typename X, int V, int T>
fsp_status launch_ring(const NormArgs& a, cudaStream_t st) {
  constexpr int kStages = sizeof(X) == 2 ? 6 : 4, kSmem = kStages * Columns<X, V, T, kHold / V>::kStage;
  void (*kernel)(NormArgs) = norm_ring_kernel<X, V, T, kStages>;
  const fsp_status s = allow_kernel(reinterpret_cast<const void*>(kernel), kSmem);
  if (s != FSP_OK) return s;
  const int64_t ctas = std::min<int64_t>(kParts, (a.rows + kRingThreads / T - 1) / (kRingThreads / T));
  return launch_next(kernel, dim3(unsigned(ctas)), kRingThreads, kSmem, 1, a, st, "layer norm kernel launch");
}

template <typename X>
fsp_status launch_norm_vec(const NormArgs& a, cudaStream_t st) {
  constexpr int V = 16 / int(sizeof(X));
  if (a.dim <= 8 * kHold) return launch_ring<X, V, 8>(a, st);
  if (a.dim <= 16 * kHold) return launch_ring<X, V, 16>(a, st);
  if (a.dim <= 32 * kHold) return launch_ring<X, V, 32>(a, st);
  if (a.dim <= 64 * kHold) return launch_ring<X, V, 64>(a, st);
  if (a.dim <= 128 * kHold) return launch_ring<X, V, 128>(a, st);
  if (a.dim <= 256 * kHold) return launch_ring<X, V, 256>(a, st);
  return launch_ring<X, V, 512>(a, st);
}

template <typename X, int V>
fsp_status launch_norm(const NormArgs& a, cudaStream_t st) {
  if (V > 1 && a.rows >= 1024 && a.dim <= 512 * kHold) return launch_norm_vec<X>(a, st);
  if (a.dim <= 128) return launch_rows<X, V, 16, 8, 4>(a, st);
  if (a.dim <= 256) return launch_rows<X, V, 32, 8, 4>(a, st);
  if (a.dim <= 512) return launch_rows<X, V, 32, 16, 2>(a, st);
  if (a.dim <= 1024) return launch_rows<X, V, 32, 32, 1>(a, st);
  if (a.dim <= 2048) return launch_rows<X, V, 32, 64, 1>(a, st);
  if (a.dim <= 4096) return launch_rows<X, V, 128, 32, 1>(a, st);
  if (a.dim <= 8192) return launch_rows<X, V, 256, 32, 1>(a, st);
  if (a.dim <= 16384) return launch_rows<X, V, 512, 32, 1>(a, st);
  return launch_next(wide_norm_kernel<X, V>, dim3(unsigned(a.rows)), kWideThreads, 0, 1, a, st, "layer norm kernel launch");
}

fsp_status norm(const void* x, int32_t xd, int64_t rows, int64_t dim, int64_t xs, const void* weight, const void* bias,
                int32_t pd, float eps, int32_t center, void* out, int32_t od, int64_t os, float* stats, void* stream) {
  fsp_status s = check_sizes(rows, dim);
  if (s != FSP_OK) return s;
  if (!(eps >= 0.f) || eps > 3.4e38f) return fail(FSP_EINVAL, "eps must be finite and >= 0");
  if ((weight || bias) && !known(pd)) return fail(FSP_EINVAL, "unknown dtype of the parameters");
  s = check_form(x, rows, dim, xs, xd, "x");
  if (s == FSP_OK) s = check_vector(weight, dim, pd, "weight");
  if (s == FSP_OK) s = check_vector(bias, dim, pd, "bias");
  if (s == FSP_OK) s = check_form(out, rows, dim, os, od, "out");
  if (s == FSP_OK) s = check_stats(stats);
  if (s != FSP_OK || rows == 0 || dim == 0) return s;
  const Operand outs[] = {rows_operand(out, rows, dim, os, od, "out"), {stats, stats ? size_t(rows) * 8 : 0, "stats"}};
  const Operand ins[] = {rows_operand(x, rows, dim, xs, xd, "x"), vector_operand(weight, dim, pd, "weight"),
                         vector_operand(bias, dim, pd, "bias")};
  s = check_operands(outs, 2, ins, 3);
  if (s != FSP_OK) return s;
  NormArgs a{x, weight, bias, out, reinterpret_cast<float2*>(stats), rows, dim, xs, os, eps, center != 0, pd == FSP_DTYPE_F32, od == FSP_DTYPE_F32};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = dim % 8 == 0 && rows_fit(x, xs, xd, 8) && rows_fit(out, os, od, 8) && (!weight || rows_fit(weight, 0, pd, 8)) &&
                   (!bias || rows_fit(bias, 0, pd, 8));
  using B = __nv_bfloat16;
  if (xd == FSP_DTYPE_F32) return vec ? launch_norm<float, 8>(a, st) : launch_norm<float, 1>(a, st);
  return vec ? launch_norm<B, 8>(a, st) : launch_norm<B, 1>(a, st);
}

int64_t parts_of(int64_t rows) { return std::min<int64_t>(kParts, rows); }
size_t workspace_of(int64_t rows, int64_t dim) { return size_t(parts_of(rows)) * 2 * size_t(dim) * 4 + 256; }   // (from a multiple of 256)

fsp_status launch_join(const GradArgs& a, cudaStream_t st) {
  return launch_next(join_columns_kernel, dim3(unsigned((a.dim + 31) / 32), 2), kJoinWarps * 32, 0, 1, a, st,
                     "layer norm gradient (join) kernel launch");
}

template <typename X, typename G, int V, int T, int E>
fsp_status launch_rows_grad(GradArgs a, cudaStream_t st) {
  constexpr int kGroups = kGradThreads / T, kSmem = 2 * kGroups * T * E * 4;
  void (*kernel)(GradArgs) = grad_kernel<X, G, V, T, E>;
  fsp_status s = allow_kernel(reinterpret_cast<const void*>(kernel), kSmem);
  if (s != FSP_OK) return s;
  a.n_parts = int(std::min<int64_t>(kParts, (a.rows + kGroups - 1) / kGroups));
  if (a.rows > 0) s = launch_next(kernel, dim3(unsigned(a.n_parts)), kGradThreads, kSmem, 1, a, st, "layer norm gradient kernel launch");
  return s == FSP_OK && (a.grad_weight || a.grad_bias) ? launch_join(a, st) : s;
}

template <typename X, typename G, int T>
fsp_status launch_ring_grad(GradArgs a, cudaStream_t st) {
  constexpr int V = sizeof(X) + sizeof(G) == 8 ? 4 : 8, N = kHold / V, kGroups = kRingThreads / T;
  constexpr int kStages = sizeof(X) == 4 ? 2 : sizeof(G) == 4 ? 3 : 4;
  constexpr int kSmem = kStages * (2 * Columns<X, V, T, N>::kStage + Columns<G, V, T, N>::kStage);
  void (*kernel)(GradArgs) = grad_ring_kernel<X, G, V, T, kStages>;
  fsp_status s = allow_kernel(reinterpret_cast<const void*>(kernel), kSmem);
  if (s != FSP_OK) return s;
  a.n_parts = int(std::min<int64_t>(kParts, (a.rows + kGroups - 1) / kGroups));
  if (a.rows > 0) s = launch_next(kernel, dim3(unsigned(a.n_parts)), kRingThreads, kSmem, 1, a, st, "layer norm gradient kernel launch");
  return s == FSP_OK && (a.grad_weight || a.grad_bias) ? launch_join(a, st) : s;
}

template <typename X, typename G>
fsp_status launch_grad_vec(const GradArgs& a, cudaStream_t st) {
  if (a.dim <= 8 * kHold) return launch_ring_grad<X, G, 8>(a, st);
  if (a.dim <= 16 * kHold) return launch_ring_grad<X, G, 16>(a, st);
  if (a.dim <= 32 * kHold) return launch_ring_grad<X, G, 32>(a, st);
  if (a.dim <= 64 * kHold) return launch_ring_grad<X, G, 64>(a, st);
  if (a.dim <= 128 * kHold) return launch_ring_grad<X, G, 128>(a, st);
  if (a.dim <= 256 * kHold) return launch_ring_grad<X, G, 256>(a, st);
  return launch_ring_grad<X, G, 512>(a, st);
}

template <typename X, typename G, int V>
fsp_status launch_wide_grad(const GradArgs& a, cudaStream_t st) {
  fsp_status s = FSP_OK;
  if (a.grad_weight || a.grad_bias) {   // (first: grad_x may take the place of x or grad_out)
    const dim3 grid(unsigned((a.dim + 32 * V - 1) / (32 * V)), unsigned(a.n_parts));
    if (a.rows > 0)
      s = launch_next(column_sums_kernel<X, G, V>, grid, kColumnWarps * 32, 0, 1, a, st, "layer norm gradient (columns) kernel launch");
    if (s == FSP_OK) s = launch_join(a, st);
  }
  if (s != FSP_OK || !a.grad_x || a.rows == 0) return s;
  return launch_next(wide_grad_kernel<X, G, V>, dim3(unsigned(a.rows)), kWideThreads, 0, 1, a, st, "layer norm gradient kernel launch");
}

template <typename X, typename G, int V>
fsp_status launch_grad(const GradArgs& a, cudaStream_t st) {
  if (V > 1 && a.dim <= 512 * kHold) return launch_grad_vec<X, G>(a, st);
  // sixteen elements a thread, eight where fp32 rows would not leave the registers for the row ahead
  constexpr int E = sizeof(X) + sizeof(G) > 4 ? 8 : 16;
  if (a.dim <= 8 * E) return launch_rows_grad<X, G, V, 8, E>(a, st);
  if (a.dim <= 16 * E) return launch_rows_grad<X, G, V, 16, E>(a, st);
  if (a.dim <= 32 * E) return launch_rows_grad<X, G, V, 32, E>(a, st);
  if (a.dim <= 64 * E) return launch_rows_grad<X, G, V, 64, E>(a, st);
  if (a.dim <= 128 * E) return launch_rows_grad<X, G, V, 128, E>(a, st);
  if (a.dim <= 256 * E) return launch_rows_grad<X, G, V, 256, E>(a, st);
  if (a.dim <= 512 * E) return launch_rows_grad<X, G, V, 512, E>(a, st);
  if (a.dim <= 1024 * E) return launch_rows_grad<X, G, V, 512, 2 * E>(a, st);
  return launch_wide_grad<X, G, V>(a, st);
}

template <typename X, typename G>
fsp_status launch_grad_v(const GradArgs& a, bool vec, cudaStream_t st) {
  return vec ? launch_grad<X, G, 8>(a, st) : launch_grad<X, G, 1>(a, st);
}

fsp_status backward(const void* x, int32_t xd, int64_t rows, int64_t dim, int64_t xs, const float* stats, int32_t center,
                    const void* grad, int32_t gd, int64_t gs, const void* weight, int32_t wd, const void* add, int64_t as,
                    void* grad_x, int64_t ds, void* grad_weight, void* grad_bias, int32_t pd, int32_t accumulate,
                    void* workspace, size_t workspace_bytes, void* stream) {
  fsp_status s = check_sizes(rows, dim);
  if (s != FSP_OK) return s;
  const bool columns = grad_weight || grad_bias;
  if (weight && !known(wd)) return fail(FSP_EINVAL, "unknown dtype of weight");
  if (columns && !known(pd)) return fail(FSP_EINVAL, "unknown dtype of the parameters' gradients");
  if (add && !grad_x) return fail(FSP_EINVAL, "add needs grad_x");
  s = check_form(x, rows, dim, xs, xd, "x");
  if (s == FSP_OK) s = check_form(grad, rows, dim, gs, gd, "grad_out");
  if (s == FSP_OK && rows > 0 && dim > 0 && !stats) s = fail(FSP_EINVAL, "stats is NULL");
  if (s == FSP_OK) s = check_stats(stats);
  if (s == FSP_OK) s = check_vector(weight, dim, wd, "weight");
  if (s == FSP_OK && add) s = check_form(add, rows, dim, as, xd, "add");
  if (s == FSP_OK && grad_x) s = check_form(grad_x, rows, dim, ds, xd, "grad_x");
  if (s == FSP_OK) s = check_vector(grad_weight, dim, pd, "grad_weight");
  if (s == FSP_OK) s = check_vector(grad_bias, dim, pd, "grad_bias");
  if (s != FSP_OK) return s;
  if (dim == 0 || (!grad_x && !columns) || (rows == 0 && (!columns || accumulate))) return FSP_OK;
  const size_t need = columns && rows > 0 ? workspace_of(rows, dim) : 0;
  if (need) {
    if (!workspace) return fail(FSP_EINVAL, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return fail(FSP_EINVAL, "workspace is not 16-byte aligned");
    if (workspace_bytes < need) return fail(FSP_EINVAL, "workspace is smaller than fsp_layer_norm_backward_workspace_bytes");
  }
  const Operand outs[] = {rows_operand(grad_x, rows, dim, ds, xd, "grad_x"),
                          vector_operand(grad_weight, dim, pd, "grad_weight"),
                          vector_operand(grad_bias, dim, pd, "grad_bias"), {workspace, need, "workspace"}};
  const Operand ins[] = {rows_operand(x, rows, dim, xs, xd, "x"), rows_operand(grad, rows, dim, gs, gd, "grad_out"),
                         rows_operand(add, rows, dim, as, xd, "add"), vector_operand(weight, dim, wd, "weight"),
                         {stats, size_t(rows) * 8, "stats"}};
  s = check_operands(outs, 4, ins, 5);
  if (s != FSP_OK) return s;
  GradArgs a{};
  a.x = x;
  a.stats = reinterpret_cast<const float2*>(stats);
  a.grad = grad;
  a.weight = weight;
  a.add = add;
  a.grad_x = grad_x;
  a.parts = reinterpret_cast<float*>(round256(reinterpret_cast<uintptr_t>(workspace)));
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.rows = rows;
  a.dim = dim;
  a.x_stride = xs;
  a.grad_stride = gs;
  a.add_stride = as;
  a.grad_x_stride = ds;
  a.n_parts = int(parts_of(rows));
  a.center = center != 0;
  a.weight_f32 = wd == FSP_DTYPE_F32;
  a.grad_param_f32 = pd == FSP_DTYPE_F32;
  a.accumulate = accumulate != 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool vec = dim % 8 == 0 && rows_fit(x, xs, xd, 8) && rows_fit(grad, gs, gd, 8) && (!add || rows_fit(add, as, xd, 8)) &&
                   (!grad_x || rows_fit(grad_x, ds, xd, 8)) && (!weight || rows_fit(weight, 0, wd, 8));
  using B = __nv_bfloat16;
  if (xd == FSP_DTYPE_F32)
    return gd == FSP_DTYPE_F32 ? launch_grad_v<float, float>(a, vec, st) : launch_grad_v<float, B>(a, vec, st);
  return gd == FSP_DTYPE_F32 ? launch_grad_v<B, float>(a, vec, st) : launch_grad_v<B, B>(a, vec, st);
}

}  // namespace
}  // namespace fsp

extern "C" fsp_status fsp_layer_norm(const void* x, int32_t x_dtype, int64_t rows, int64_t dim, int64_t x_stride,
                                     const void* weight, const void* bias, int32_t param_dtype, float eps, int32_t center,
                                     void* out, int32_t out_dtype, int64_t out_stride, float* stats, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::norm(x, x_dtype, rows, dim, x_stride, weight, bias, param_dtype, eps, center, out, out_dtype, out_stride,
                     stats, cuda_stream);
  });
}

extern "C" fsp_status fsp_layer_norm_backward_workspace_bytes(int64_t rows, int64_t dim, size_t* bytes) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (!bytes) return fsp::fail(FSP_EINVAL, "bytes is NULL");
    const fsp_status s = fsp::check_sizes(rows, dim);
    if (s == FSP_OK) *bytes = fsp::workspace_of(rows, dim);
    return s;
  });
}

extern "C" fsp_status fsp_layer_norm_backward(const void* x, int32_t x_dtype, int64_t rows, int64_t dim, int64_t x_stride,
                                              const float* stats, int32_t center, const void* grad_out,
                                              int32_t grad_dtype, int64_t grad_stride, const void* weight,
                                              int32_t weight_dtype, const void* add, int64_t add_stride, void* grad_x,
                                              int64_t grad_x_stride, void* grad_weight, void* grad_bias,
                                              int32_t grad_param_dtype, int32_t accumulate, void* workspace,
                                              size_t workspace_bytes, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::backward(x, x_dtype, rows, dim, x_stride, stats, center, grad_out, grad_dtype, grad_stride, weight,
                         weight_dtype, add, add_stride, grad_x, grad_x_stride, grad_weight, grad_bias, grad_param_dtype,
                         accumulate, workspace, workspace_bytes, cuda_stream);
  });
}
