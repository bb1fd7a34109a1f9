// Layer norm and its gradients (sm_103a).
//
//   m = mean x (0 if not centred), r = 1 / sqrt(mean (x - m)^2 + eps), h = (x - m) r, y = h w + b
//   g = dy w,  dx = r (g - mean g (0 if not centred) - h mean(g h)) + add
//   dw (+)= sum over rows of dy h,  db (+)= sum over rows of dy
//
// Bound: HBM (about 7 operations an element forward, 14 backward; 4 to 12 bytes forward).
//
//   few rows (below kRingElements): rows in registers, 8 elements a thread, everything asked for
//     at once (one row of 1024 1.6 us);
//   many rows of up to 16384 elements: a CTA per SM that stays, rows ahead in a ring in shared
//     memory, the gradients of all three in one pass and a join of one pair of partial sums per
//     CTA (32768 x 2048 bf16: forward 46 us, 0.87 of the measured copy, gradients with the
//     residual's 82 us, 0.97; 131072 x 128 12 and 21 us; odd rows 20000 x 1001 20 and 35 us, bound by
//     their instructions);
//   longer rows: a CTA per row, which reads it three times.
// All sums are fp32; no sum's order depends on timing.  In the ring a mean is a corrected product
// with 1 / dim and r a corrected rsqrtf (divisions and a root cost a short row a tenth of its
// instructions).
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
  float* parts;         // [n_parts][2][dim]
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

// T threads hold a row, E elements each: accesses of V elements, T * V apart.  T < 32 divides
// a warp among rows.
template <int T>
__device__ __forceinline__ float row_sum(float v) {   // over T <= 32 lanes
#pragma unroll
  for (int o = T / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- few rows: in registers -----------------------------------------------------------

// Everything that a row needs is asked for at once, and eight elements a thread keep the
// sums short: what counts is a launch's latency.
template <typename X, int V, int T, int E>
__global__ void __launch_bounds__(T > 128 ? T : 128) norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kThreads = T > 128 ? T : 128, N = E / V, kRows = kThreads / T;
  __shared__ float share[2][kThreads / 32];
  launch_dependents();
  grid_dependency_wait();
  const int t = threadIdx.x % T;
  const int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / T;
  auto sum = [&](float v, int which) {
    v = row_sum<32>(v);
    if constexpr (T > 32) {
      float* mine = share[which] + threadIdx.x / T * (T / 32);
      if (threadIdx.x % 32 == 0) mine[t / 32] = v;
      __syncthreads();
      v = threadIdx.x % 32 < T / 32 ? mine[threadIdx.x % 32] : 0.f;
      v = row_sum<32>(v);
    }
    return v;
  };
  float f[E], w[E], b[E];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * T + t) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f[n * V + j] = b[n * V + j] = 0.f;
      w[n * V + j] = 1.f;
    }
    if (c < a.dim) {
      if (row < a.rows) load_vec<X, V>(static_cast<const X*>(a.x) + row * a.x_stride + c, &f[n * V]);
      if (a.weight) load_any<V>(a.weight, a.param_f32, c, &w[n * V]);
      if (a.bias) load_any<V>(a.bias, a.param_f32, c, &b[n * V]);
    }
  }
  const float count = float(a.dim);
  float m = 0.f, v = 0.f;
  if (a.center) {
#pragma unroll
    for (int e = 0; e < E; ++e) v += f[e];
    m = sum(v, 0) / count;
    v = 0.f;
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = n * V + j;
      f[e] -= m;
      if ((n * T + t) * V < a.dim) v = __fmaf_rn(f[e], f[e], v);
    }
  const float r = 1.f / sqrtf(sum(v, 1) / count + a.eps);
  if (row >= a.rows) return;
  if (a.stats && t == 0) a.stats[row] = make_float2(m, r);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = (n * T + t) * V;
    if (c >= a.dim) break;
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = __fmaf_rn(f[n * V + j] * r, w[n * V + j], b[n * V + j]);
    store_any<V>(a.out, a.out_f32, row * a.out_stride + c, y);
  }
}

// ---- many rows: through shared memory ---------------------------------------------------
//
// Each CTA stays and takes every gridDim.x-th set of 512 / T rows.  The T threads of a group
// hold the same columns of every row that the group takes, and copy the rows ahead into the
// group's part of a ring of stages in shared memory (cp.async): the copies of kStages - 1
// rows are in flight while a row is reduced, without registers for them.
//
// Rows whose accesses of eight elements begin at multiples of their size (kWhole), and others of
// an even count of bf16 elements or of fp32 ones, in pieces of four or eight bytes (kPart): a
// thread copies what it reads itself, so that the ring needs no barriers.  Otherwise (kShift) the
// group copies the 16-byte pieces that cover the row, and a thread reads pairs of elements from
// wherever they begin; a row of results is laid down in shared memory likewise and leaves in
// 16-byte pieces.  A piece that reaches past a matrix's first or last byte is filled with the
// elements that are the matrix's.  (Measured, kPart and kShift, us: forward 20000 x 700 bf16 15.9
// and 17.9, but 4099 x 1001 fp32 to bf16 9.4 and 8.1, so the forward pass of fp32 takes kShift;
// gradients of 20000 x 700 bf16 23.8 and 33.5.)

constexpr int kRingThreads = 512;

template <int kPiece>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {   // 4, 8 or 16 bytes, or zeros
  if constexpr (kPiece == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kPiece), "r"(there ? kPiece : 0) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {   // until at most N groups of this thread's copies are in flight
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_at(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

// The barrier of the T threads that this one's group (T < 32: its warp) has.
template <int T>
__device__ __forceinline__ void group_sync() {
  if constexpr (T <= 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(int(threadIdx.x) / T + 1), "n"(T) : "memory");
}

// Sums over the threads of a group.  `which` alternates from sum to sum: a thread is past the
// barrier of one only when all have read the one before.
template <int T, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float (*share)[kRingThreads / 32][K], int which) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = row_sum<(T < 32 ? T : 32)>(v[k]);
  if constexpr (T > 32) {
    float(*mine)[K] = share[which] + threadIdx.x / T * (T / 32);
    if (threadIdx.x % 32 == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) mine[threadIdx.x % T / 32][k] = v[k];
    }
    group_sync<T>();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += mine[w][k];
  }
}

// Two elements an instruction, each rounded as its own.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float sum_of(float2 x) { return x.x + x.y; }

// s / n, share = 1 / n.  q = s share is off by up to 2^-23 of itself; what is missing, s - q n,
// is exact in a fused product, and q plus its share is s / n within 2^-24 and, where s / n is a
// float, that float.  (An infinite sum has an infinite mean: fminf takes the other for NaN.)
__device__ __forceinline__ float mean_of(float s, float n, float share) {
  const float q = s * share;
  return __fmaf_rn(fminf(__fmaf_rn(-q, n, s), 3.4e38f), share, q);
}
// 1 / sqrt(v) of v >= 0: rsqrtf, up to two steps of 2^-23 off, and a step of Newton's method on
// 1 / r^2 = v, after which the roundings are left (1.5 * 2^-24; likewise for zeros and infinities).
__device__ __forceinline__ float root_of(float v) {
  const float r = rsqrtf(v);
  return __fmaf_rn(0.5f * r, fminf(__fmaf_rn(-v * r, r, 1.f), 1.f), r);
}

// The rows of a thread: `row` its group's, `first` that of its warp's first group (the groups
// of a warp advance together), `step` to the next.  (Below 2^32, also those past the last.)
template <int T>
struct Walk {
  uint32_t row, first, step;
  __device__ __forceinline__ Walk() {
    constexpr int kGroups = kRingThreads / T, kUnit = T < 32 ? 32 : T;
    step = gridDim.x * kGroups;
    row = blockIdx.x * kGroups + threadIdx.x / T;
    first = blockIdx.x * kGroups + threadIdx.x / kUnit * (kUnit / T);
  }
  __device__ __forceinline__ void next() {
    row += step;
    first += step;
  }
};

// One of the matrices that go through the ring.
struct Stream {
  const void* p;
  int64_t stride;
};

// How the rows of a call lie: kWhole, kPart or kShift, above.
enum Rows { kWhole, kPart, kShift };

// Which columns a thread of a group of T holds, as E / 2 pairs.  kWhole: accesses n of V
// elements, from column (n T + t) V on (V = 4 or 8).  Otherwise pair i is columns 2 (i T + t)
// and the next (V = 2), or 2 i T + t and T further (V = 1, fp32 alone), so that a warp reads
// words of shared memory side by side.
template <int V, int T, int E>
struct Held {
  static constexpr bool kPairs = V < 4;
  static constexpr int N = kPairs ? E / 2 : E / V;        // accesses, or pairs
  static constexpr int W = kPairs ? 2 : V;                // elements of one
  enum { kStep = V == 1 ? T : 1 };            // between the two columns of a pair
  static __device__ __forceinline__ int thread() { return threadIdx.x % T; }
  static __device__ __forceinline__ int column(int n) { return V == 1 ? 2 * n * T + thread() : (n * T + thread()) * W; }
  // Zeros for what lies past the row's end.
  static __device__ __forceinline__ void mask(int dim, float2 (&f)[E / 2]) {
#pragma unroll
    for (int n = N - 1; n >= 0; --n) {
      if ((n + 1) * T * W <= dim) break;   // (whole from here on, for the whole group)
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const int c = column(n) + 2 * i;
        if (c >= dim) f[n * W / 2 + i].x = 0.f;
        if (c + kStep >= dim) f[n * W / 2 + i].y = 0.f;
      }
    }
  }
  // Its columns of a vector of parameters, `otherwise` where there is none.
  static __device__ __forceinline__ void load(const void* p, bool f32, int dim, float otherwise, float2 (&f)[E / 2]) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) f[i] = both(otherwise);
    if (!p) return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = column(n);
      if constexpr (kPairs) {
        if (c < dim) f[n].x = load_any(p, f32, c);
        if (c + kStep < dim) f[n].y = load_any(p, f32, c + kStep);
      } else if (c < dim) {
        float y[V];
        load_any<V>(p, f32, c, y);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) f[n * V / 2 + i] = make_float2(y[2 * i], y[2 * i + 1]);
      }
    }
  }
};

// Rows of Y in a stage of the ring.
template <typename Y, int V, int T, int E, Rows R>
struct Columns {
  using H = Held<V, T, E>;
  static constexpr int kSize = int(sizeof(Y)), kBytes = kSize * V;
  static constexpr int kGroup = T * E * kSize + (R == kShift ? 16 : 0);   // of a group; kShift: and what surrounds a row
  static constexpr int kStage = kRingThreads / T * kGroup;
  static_assert(kGroup % 16 == 0 && (R != kWhole || kBytes % 16 == 0) && (R == kWhole) == (V >= 4));

  static __device__ __forceinline__ char* group(char* stage) { return stage + threadIdx.x / T * kGroup; }
  static __device__ __forceinline__ const char* address(Stream s, uint32_t row) {
    return static_cast<const char*>(s.p) + int64_t(row) * s.stride * kSize;
  }
  // Zeros for the columns past a row's end, which no copy writes.
  static __device__ __forceinline__ void clear(char* stage, int dim) {
    const int t = H::thread();
    stage = group(stage);
    if constexpr (R == kWhole) {
#pragma unroll
      for (int n = 0; n < H::N; ++n)
        if (n * T * V >= dim - t * V) {
#pragma unroll
          for (int k = 0; k < kBytes; k += 16) *reinterpret_cast<uint4*>(stage + (n * T + t) * kBytes + k) = make_uint4(0, 0, 0, 0);
        }
    } else if constexpr (R == kPart) {
#pragma unroll
      for (int n = 0; n < H::N; ++n) {
        Y* at = reinterpret_cast<Y*>(stage) + H::column(n);
        if (H::column(n) >= dim) at[0] = narrow<Y>(0.f);
        if (H::column(n) + H::kStep >= dim) at[H::kStep] = narrow<Y>(0.f);
      }
    }
  }
  // Starts the copies of a row; past the last, zeros where other groups of the warp go on (T < 32).
  static __device__ __forceinline__ void copy(char* stage, Stream s, uint32_t row, uint32_t rows, int dim) {
    const int t = H::thread();
    stage = group(stage);
    if constexpr (R != kShift) {
      const bool there = row < rows;
      if (T >= 32 && !there) return;
      // (V = 1: two columns a pair, each a copy)
      constexpr int kCopies = R == kPart && V == 1 ? 2 * H::N : H::N, kPiece = kBytes < 16 ? kBytes : 16;
      const char* src = address(s, there ? row : 0) + t * kBytes;
      const uint32_t dst = smem_at(stage) + t * kBytes;
#pragma unroll
      for (int n = 0; n < kCopies; ++n)
        if (n * T * V < dim - t * V) {
#pragma unroll
          for (int k = 0; k < kBytes; k += kPiece) copy_async<kPiece>(dst + n * T * kBytes + k, src + n * T * kBytes + k, there);
        }
    } else if (row < rows) {
      const char* begin = address(s, row);
      const int before = int(reinterpret_cast<uintptr_t>(begin) & 15), bytes = (before + dim * kSize + 15) & ~15;
      const char* src = begin - before + t * 16;
      const uint32_t dst = smem_at(stage) + t * 16;
      if (inside(s, row, rows)) {
#pragma unroll
        for (int k = 0; k < kGroup; k += T * 16)
          if (k + t * 16 < bytes) copy_async<16>(dst + k, src + k, true);
      } else {
        const char *lowest = static_cast<const char*>(s.p), *highest = address(s, rows - 1) + dim * kSize;
        for (int k = t * 16; k < bytes; k += T * 16) {
          const char* p = begin - before + k;
          if (p >= lowest && p + 16 <= highest) {
            copy_async<16>(smem_at(stage) + k, p, true);
          } else {
            for (const char* q = p < lowest ? lowest : p; q < p + 16 && q < highest; q += kSize)
              *reinterpret_cast<Y*>(stage + k + (q - p)) = *reinterpret_cast<const Y*>(q);
          }
        }
      }
    }
  }
  // Whether the 16-byte pieces that cover a row lie within the matrix for certain.
  static __device__ __forceinline__ bool inside(Stream s, uint32_t row, uint32_t rows) {
    const uint32_t margin = s.stride * kSize >= 16 ? 1 : 16;   // rows of 16 bytes
    return row >= margin && row + margin < rows;
  }
  // Bytes of a stage before a row's first.
  static __device__ __forceinline__ int skip(Stream s, uint32_t row) {
    return R == kShift ? int((uint32_t(reinterpret_cast<uintptr_t>(s.p)) + row * uint32_t(s.stride) * kSize) & 15u) : 0;
  }
  static __device__ __forceinline__ float2 pair_of(uint32_t w) {   // bf16
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  // This thread's access n of the row, at multiples of 16 bytes.
  static __device__ __forceinline__ void read(char* stage, int n, float2* f) {
    const uint4* from = reinterpret_cast<const uint4*>(group(stage) + (n * T + H::thread()) * kBytes);
#pragma unroll
    for (int k = 0; k < kBytes / 16; ++k) {
      const uint4 q = from[k];
      if constexpr (kSize == 2) {
        f[0] = pair_of(q.x);
        f[1] = pair_of(q.y);
        f[2] = pair_of(q.z);
        f[3] = pair_of(q.w);
      } else {
        f[2 * k] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
        f[2 * k + 1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
      }
    }
  }
  // Pair n of this thread's columns (not kWhole), zeros past the row's end.
  static __device__ __forceinline__ float2 read_pair(char* stage, int skip, int dim, int n) {
    const uint32_t* from = reinterpret_cast<const uint32_t*>(group(stage) + (skip & ~3));
    float2 f;
    if constexpr (kSize == 4) {
      from += H::column(n);
      f = make_float2(__uint_as_float(from[0]), __uint_as_float(from[H::kStep]));
    } else {
      from += n * T + H::thread();
      f = skip & 2 ? make_float2(__uint_as_float(from[0] & 0xffff0000u), __uint_as_float(from[1] << 16)) : pair_of(from[0]);
    }
    if (R == kShift && (n + 1) * T * 2 > dim) {   // (not the whole group)
      if (H::column(n) >= dim) f.x = 0.f;
      if (H::column(n) + H::kStep >= dim) f.y = 0.f;
    }
    return f;
  }
  // All of this thread's columns, zeros past the row's end.
  static __device__ __forceinline__ void read_row(char* stage, int skip, int dim, float2 (&f)[E / 2]) {
    if constexpr (R == kWhole) {
#pragma unroll
      for (int n = 0; n < H::N; ++n) read(stage, n, f + n * V / 2);
    } else {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(group(stage) + (skip & ~3));
      if constexpr (kSize == 4) {
        from += H::column(0);
#pragma unroll
        for (int n = 0; n < H::N; ++n) f[n] = make_float2(__uint_as_float(from[2 * n * T]), __uint_as_float(from[2 * n * T + H::kStep]));
      } else {
        from += H::thread();
        if (R == kShift && skip & 2) {   // (the same for the whole group) pairs across two words
#pragma unroll
          for (int n = 0; n < H::N; ++n)
            f[n] = make_float2(__uint_as_float(from[n * T] & 0xffff0000u), __uint_as_float(from[n * T + 1] << 16));
        } else {
#pragma unroll
          for (int n = 0; n < H::N; ++n) f[n] = pair_of(from[n * T]);
        }
      }
      if constexpr (R == kShift) H::mask(dim, f);
    }
  }
};

// A row of results: result(n, f) gives access (or pair) n of a thread.  kShift: by way of
// `staging`, 16 bytes more than the group's E * T elements in shared memory, which the barriers
// of the sums before it have left free.  there: whether the group has a row.
template <typename O, int V, int T, int E, Rows R, typename Result>
__device__ __forceinline__ void write_row(O* out, int dim, bool there, char* staging, Result result) {
  using H = Held<V, T, E>;
  const int t = H::thread();
  if constexpr (R != kShift) {
    if (!there) return;
#pragma unroll
    for (int n = 0; n < H::N; ++n) {
      float2 f[H::W / 2];
      result(n, f);
      const int c = H::column(n);
      if constexpr (V == 1) {
        if (c < dim) store_vec<O, 1>(out + c, &f->x);
        if (c + T < dim) store_vec<O, 1>(out + c + T, &f->y);
      } else if (c < dim) {
        store_vec<O, V>(out + c, reinterpret_cast<const float*>(f));
      }
    }
  } else {
    // laid down as far from a multiple of 16 bytes as it is in memory, so that whole pieces leave
    constexpr int kSize = int(sizeof(O));
    const int ahead = int(reinterpret_cast<uintptr_t>(out) & 15), end = ahead + (there ? dim * kSize : 0);
    O* to = reinterpret_cast<O*>(staging + ahead) + H::column(0);
    constexpr int kNext = V == 1 ? 2 * T : T * 2;   // columns from pair to pair
    float2 f;
    if (kSize == 2 && V == 2 && (ahead & 2) == 0) {
#pragma unroll
      for (int n = 0; n < H::N; ++n) {
        result(n, &f);
        *reinterpret_cast<__nv_bfloat162*>(to + n * kNext) = __floats2bfloat162_rn(f.x, f.y);
      }
    } else {
#pragma unroll
      for (int n = 0; n < H::N; ++n) {
        result(n, &f);
        to[n * kNext] = narrow<O>(f.x);
        to[n * kNext + H::kStep] = narrow<O>(f.y);
      }
    }
    group_sync<T>();
    char* base = reinterpret_cast<char*>(out) - ahead;
    const int whole = ahead > 0 ? 16 : 0;   // the first whole piece
#pragma unroll
    for (int k = 0; k < T * E * kSize + 16; k += T * 16)
      if (k + t * 16 >= whole && k + t * 16 + 16 <= end)
        __stcs(reinterpret_cast<uint4*>(base + t * 16 + k), *reinterpret_cast<const uint4*>(staging + t * 16 + k));
    if (t < 16 / kSize) {   // elements before and after them
      const int head = ahead + t * kSize, tail = max(whole, end & ~15) + t * kSize;
      if (head < min(whole, end)) *reinterpret_cast<O*>(base + head) = *reinterpret_cast<const O*>(staging + head);
      if (tail < end) *reinterpret_cast<O*>(base + tail) = *reinterpret_cast<const O*>(staging + tail);
    }
  }
}

template <typename X, int V, int T, int E, int kStages, Rows R>
__global__ void __launch_bounds__(kRingThreads, 1) norm_ring_kernel(const __grid_constant__ NormArgs a) {
  using C = Columns<X, V, T, E, R>;
  using H = Held<V, T, E>;
  extern __shared__ __align__(16) char ring[];
  __shared__ float share[2][kRingThreads / 32][1];
  launch_dependents();
  grid_dependency_wait();
  Walk<T> at;
  const Stream x{a.x, a.x_stride};
  const int dim = int(a.dim);
  const uint32_t rows = uint32_t(a.rows);
#pragma unroll
  for (int d = 0; d < kStages; ++d) {
    C::clear(ring + d * C::kStage, dim);
    C::copy(ring + d * C::kStage, x, at.row + d * at.step, rows, dim);
    copies_issued();
  }
  float2 w[E / 2], b[E / 2];
  H::load(a.weight, a.param_f32, dim, 1.f, w);
  H::load(a.bias, a.param_f32, dim, 0.f, b);
  const float count = float(dim), share_of = 1.f / count;
  int slot = 0;
  for (int which = 0; at.first < rows; at.next(), which ^= 1) {
    char* stage = ring + slot * C::kStage;
    slot = slot + 1 == kStages ? 0 : slot + 1;
    copies_wait<kStages - 1>();
    if constexpr (R == kShift) group_sync<T>();
    float2 f[E / 2], part[2] = {};
    float m = 0.f, s[1];
    C::read_row(stage, C::skip(x, at.row), dim, f);
    if (a.center) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) part[i & 1] = __fadd2_rn(part[i & 1], f[i]);
      s[0] = sum_of(__fadd2_rn(part[0], part[1]));
      group_sum<T>(s, share, 0);
      m = mean_of(s[0], count, share_of);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) f[i] = __fadd2_rn(f[i], both(-m));
      H::mask(dim, f);
      part[0] = part[1] = both(0.f);
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) part[i & 1] = __ffma2_rn(f[i], f[i], part[i & 1]);
    s[0] = sum_of(__fadd2_rn(part[0], part[1]));
    group_sum<T>(s, share, a.center ? 1 : which);
    if constexpr (R == kShift && T <= 32) __syncwarp();   // (of larger groups the sum's barrier: all have read the stage)
    C::copy(stage, x, at.row + kStages * at.step, rows, dim);
    copies_issued();
    const float r = root_of(s[0] * share_of + a.eps);
    const bool there = at.row < rows;
    if (a.stats && H::thread() == 0 && there) a.stats[at.row] = make_float2(m, r);
    auto result = [&](int n, float2* y) {
#pragma unroll
      for (int i = 0; i < H::W / 2; ++i) {
        const int k = n * H::W / 2 + i;
        y[i] = __ffma2_rn(__fmul2_rn(f[k], both(r)), w[k], b[k]);
      }
    };
    auto write = [&](auto* out) {
      using O = std::remove_pointer_t<decltype(out)>;
      char* staging = ring + kStages * C::kStage + threadIdx.x / T * (T * E * int(sizeof(O)) + 16);
      write_row<O, V, T, E, R>(out + (there ? at.row : 0) * a.out_stride, dim, there, staging, result);
    };
    if (a.out_f32)
      write(static_cast<float*>(a.out));
    else
      write(static_cast<__nv_bfloat16*>(a.out));
  }
  copies_wait<0>();
}

// All gradients in one pass over x and dy.  A thread adds its columns' terms of dw and db in
// registers; the CTA's groups are joined in shared memory at the end, so that a launch leaves
// one pair of partial sums per CTA.  What is multiplied is d = x - m, and r joins dy for dw and
// the row's sum for mean(g h): past a row's end, where dy is 0 and d is -m, h = d r may be infinite
// and 0 h not a number.  kKeep: d and g stay in registers from the sums to dx
// (E = 16; kShift: dx then takes x's place in the stage); otherwise they are read again (20000
// odd bf16 rows of 1001: 35 us with 16 columns a thread, 49 with 32 that are read again).
template <typename X, typename G, int V, int T, int E, int kStages, Rows R>
__global__ void __launch_bounds__(kRingThreads, 1) grad_ring_kernel(const __grid_constant__ GradArgs a) {
  constexpr int kGroups = kRingThreads / T;
  constexpr bool kKeep = E <= 16;
  using H = Held<V, T, E>;
  using CX = Columns<X, V, T, E, R>;
  using CG = Columns<G, V, T, E, R>;
  constexpr int kStage = 2 * CX::kStage + CG::kStage;   // dy, x, add
  extern __shared__ __align__(16) char ring[];
  __shared__ float share[2][kRingThreads / 32][2];
  launch_dependents();
  grid_dependency_wait();
  Walk<T> at;
  const Stream x{a.x, a.x_stride}, dy{a.grad, a.grad_stride}, add{a.add, a.add_stride};
  const int dim = int(a.dim);
  const uint32_t rows = uint32_t(a.rows);
  auto copy_row = [&](char* stage, uint32_t row) {
    CG::copy(stage, dy, row, rows, dim);
    CX::copy(stage + CG::kStage, x, row, rows, dim);
    if (a.add) CX::copy(stage + CG::kStage + CX::kStage, add, row, rows, dim);
    copies_issued();
  };
#pragma unroll
  for (int d = 0; d < kStages; ++d) {
    CG::clear(ring + d * kStage, dim);
    CX::clear(ring + d * kStage + CG::kStage, dim);
    copy_row(ring + d * kStage, at.row + d * at.step);
  }
  float2 w[E / 2], dw[E / 2] = {}, db[E / 2] = {};
  H::load(a.weight, a.weight_f32, dim, 1.f, w);
  const float count = float(dim), share_of = 1.f / count;
  float2 next = at.row < rows ? a.stats[at.row] : make_float2(0.f, 0.f);
  int slot = 0;
  for (int which = 0; at.first < rows; at.next(), which ^= 1) {
    char* stage = ring + slot * kStage;
    slot = slot + 1 == kStages ? 0 : slot + 1;
    const bool there = at.row < rows;
    const float2 st = there ? next : make_float2(0.f, 0.f);
    if (at.row + at.step < rows) next = a.stats[at.row + at.step];
    copies_wait<kStages - 1>();
    if constexpr (R == kShift) group_sync<T>();
    const int end = there ? dim : 0;   // kShift: nothing of what an earlier row left
    const int skip_dy = CG::skip(dy, at.row), skip_x = CX::skip(x, at.row), skip_add = CX::skip(add, at.row);
    float2 d[(kKeep ? E : H::W) / 2], g[(kKeep ? E : H::W) / 2], sg = both(0.f), sgd = both(0.f);
    auto centre = [&](float2& x) { x = __fadd2_rn(x, both(-st.x)); };
    auto add_terms = [&](int e, float2& g, float2 d) {   // pair e; g becomes dy w
      dw[e] = __ffma2_rn(__fmul2_rn(g, both(st.y)), d, dw[e]);
      db[e] = __fadd2_rn(db[e], g);
      g = __fmul2_rn(g, w[e]);
      sg = __fadd2_rn(sg, g);
      sgd = __ffma2_rn(g, d, sgd);
    };
    auto read = [&](int n) {   // (not kKeep) access n of dy and d
      if constexpr (H::kPairs) {
        g[0] = CG::read_pair(stage, skip_dy, end, n);
        d[0] = CX::read_pair(stage + CG::kStage, skip_x, end, n);
      } else {
        CG::read(stage, n, g);
        CX::read(stage + CG::kStage, n, d);
      }
#pragma unroll
      for (int i = 0; i < H::W / 2; ++i) centre(d[i]);
    };
    if constexpr (kKeep) {
      CG::read_row(stage, skip_dy, end, g);
      CX::read_row(stage + CG::kStage, skip_x, end, d);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        centre(d[e]);
        add_terms(e, g[e], d[e]);
      }
    } else {
#pragma unroll
      for (int n = 0; n < H::N; ++n) {
        read(n);
#pragma unroll
        for (int i = 0; i < H::W / 2; ++i) add_terms(n * H::W / 2 + i, g[i], d[i]);
      }
    }
    if (a.grad_x) {
      float s[2] = {sum_of(sg), sum_of(sgd)};
      group_sum<T>(s, share, which);
      if constexpr (R == kShift && kKeep && T <= 32) __syncwarp();   // dx takes the place of x, which all have read
      const float2 mean_g = both(a.center ? -mean_of(s[0], count, share_of) : 0.f), r = both(st.y);
      const float2 of_d = both(-(mean_of(s[1], count, share_of) * st.y) * st.y);   // h mean(g h) = d times this
      float2 plus[H::kPairs && kKeep ? E / 2 : 1];
      if constexpr (H::kPairs && kKeep) {
        if (a.add) {
          CX::read_row(stage + CG::kStage + CX::kStage, skip_add, end, plus);
        } else {
#pragma unroll
          for (int i = 0; i < E / 2; ++i) plus[i] = both(0.f);
        }
      }
      auto result = [&](int n, float2* f) {
        if constexpr (H::kPairs && kKeep) {
          f[0] = plus[n];
        } else if constexpr (H::kPairs) {
          f[0] = a.add ? CX::read_pair(stage + CG::kStage + CX::kStage, skip_add, end, n) : both(0.f);
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) f[i] = both(0.f);
          if (a.add) CX::read(stage + CG::kStage + CX::kStage, n, f);
        }
        if constexpr (!kKeep) {
          read(n);
#pragma unroll
          for (int i = 0; i < H::W / 2; ++i) g[i] = __fmul2_rn(g[i], w[n * H::W / 2 + i]);
        }
#pragma unroll
        for (int i = 0; i < H::W / 2; ++i) {
          const int k = kKeep ? n * H::W / 2 + i : i;
          f[i] = __ffma2_rn(r, __ffma2_rn(d[k], of_d, __fadd2_rn(g[k], mean_g)), f[i]);
        }
      };
      char* staging = kKeep ? CX::group(stage + CG::kStage) : ring + kStages * kStage + threadIdx.x / T * (T * E * int(sizeof(X)) + 16);
      write_row<X, V, T, E, R>(static_cast<X*>(a.grad_x) + (there ? at.row : 0) * a.grad_x_stride, dim, there, staging, result);
    }
    if constexpr (R == kShift) group_sync<T>();   // all have read the stage
    copy_row(stage, at.row + kStages * at.step);
  }
  copies_wait<0>();
  if (!a.grad_weight && !a.grad_bias) return;
  __syncthreads();
  constexpr int kCols = T * E;
  float* joined = reinterpret_cast<float*>(ring);   // [2][kGroups][kCols], of dw and db
  static_assert(2 * kGroups * kCols * 4 <= kStages * kStage);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.grad_bias : a.grad_weight)) continue;
    const float2* y = which ? db : dw;
    float* to = joined + (which * kGroups + threadIdx.x / T) * kCols;
#pragma unroll
    for (int n = 0; n < H::N; ++n) {
      if constexpr (H::kPairs) {
        to[H::column(n)] = y[n].x;
        to[H::column(n) + H::kStep] = y[n].y;
      } else {
#pragma unroll
        for (int i = 0; i < V / 2; i += 2)
          *reinterpret_cast<float4*>(&to[H::column(n) + 2 * i]) = make_float4(y[n * V / 2 + i].x, y[n * V / 2 + i].y, y[n * V / 2 + i + 1].x, y[n * V / 2 + i + 1].y);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    void* out = which ? a.grad_bias : a.grad_weight;
    if (!out) continue;
    const float* from = joined + which * kGroups * kCols;
    float* part = a.parts + (int64_t(blockIdx.x) * 2 + which) * dim;
    for (int c = threadIdx.x; c < kCols && c < dim; c += kRingThreads) {
      float v = 0.f;
#pragma unroll 8
      for (int k = 0; k < kGroups; ++k) v += from[k * kCols + c];
      if (gridDim.x > 1) {
        part[c] = v;
      } else {   // nothing to add these to: no second launch
        if (a.accumulate) v += load_any(out, a.grad_param_f32, c);
        store_any<1>(out, a.grad_param_f32, c, &v);
      }
    }
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
#pragma unroll 4
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
#pragma unroll 2
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
constexpr int64_t kPartRows = 64;   // rows of a part, while there are few: parts are written and read again

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
  float sum = 0.f, old = 0.f;
  if (col < a.dim) {
    if (warp == 0 && a.accumulate) old = load_any(out, a.grad_param_f32, col);
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
  sum += old;
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

template <typename X, int V, int T, int E>
fsp_status launch_few(const NormArgs& a, cudaStream_t st) {
  constexpr int kThreads = T > 128 ? T : 128, kRows = kThreads / T;
  return launch_next(norm_kernel<X, V, T, E>, dim3(unsigned((a.rows + kRows - 1) / kRows)), kThreads, 0, 1, a, st, "layer norm kernel launch");
}

// Most shared memory that a ring takes.
constexpr int kRingBytes = 226 << 10;

template <typename X, Rows R, int T, int E>
fsp_status launch_ring(const NormArgs& a, cudaStream_t st) {
  constexpr int V = R == kWhole ? 16 / int(sizeof(X)) : sizeof(X) == 4 ? 1 : 2;
  using C = Columns<X, V, T, E, R>;
  constexpr int kStaging = R == kShift ? kRingThreads / T * (T * E * 4 + 16) : 0;
  constexpr int kStages = std::min((kRingBytes - kStaging) / C::kStage, C::kStage > 48 << 10 ? 3 : C::kStage > 24 << 10 ? 4 : 6);
  constexpr int kSmem = kStages * C::kStage + kStaging;
  void (*kernel)(NormArgs) = norm_ring_kernel<X, V, T, E, kStages, R>;
  const fsp_status s = allow_kernel(reinterpret_cast<const void*>(kernel), kSmem);
  if (s != FSP_OK) return s;
  const int64_t ctas = std::min<int64_t>(kParts, (a.rows + kRingThreads / T - 1) / (kRingThreads / T));
  return launch_next(kernel, dim3(unsigned(ctas)), kRingThreads, kSmem, 1, a, st, "layer norm kernel launch");
}

// From this many elements on the ring pays for its start (few rows or many, us: 256 x 1024
// 2.1 and 3.0, 1024 x 1024 3.1 and 3.1, 2048 x 1024 5.1 and 3.3; 2048 x 128 2.3 and 2.7,
// 8192 x 128 3.8 and 2.7; 64 x 8192 2.8 and 3.4, 256 x 8192 6.1 and 3.9).
constexpr int64_t kRingElements = 3 << 18;

template <typename X, Rows R>
fsp_status launch_norm(const NormArgs& a, cudaStream_t st) {
  constexpr int V = R == kWhole ? 8 : 1;
  if (a.rows * a.dim < kRingElements) {
    if (a.dim <= 256) return launch_few<X, V, 32, 8>(a, st);
    if (a.dim <= 512) return launch_few<X, V, 64, 8>(a, st);
    if (a.dim <= 1024) return launch_few<X, V, 128, 8>(a, st);
    if (a.dim <= 2048) return launch_few<X, V, 256, 8>(a, st);
    if (a.dim <= 4096) return launch_few<X, V, 512, 8>(a, st);
    if (a.dim <= 8192) return launch_few<X, V, 1024, 8>(a, st);
  } else {
    if (a.dim <= 64) return launch_ring<X, R, 8, 8>(a, st);
    if (a.dim <= 128) return launch_ring<X, R, 8, 16>(a, st);
    if (a.dim <= 256) return launch_ring<X, R, 16, 16>(a, st);
    if (a.dim <= 512) return launch_ring<X, R, 32, 16>(a, st);
    if (a.dim <= 1024) return launch_ring<X, R, 32, 32>(a, st);
    if (a.dim <= 2048) return launch_ring<X, R, 64, 32>(a, st);
    if (a.dim <= 4096) return launch_ring<X, R, 128, 32>(a, st);
    if (a.dim <= 8192) return launch_ring<X, R, 256, 32>(a, st);
  }
  if (a.dim <= 16384) return launch_ring<X, R, 512, 32>(a, st);
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
  auto fit = [&](int v) { return dim % v == 0 && rows_fit(x, xs, xd, v) && rows_fit(out, os, od, v); };
  const bool whole = fit(8) && (!weight || rows_fit(weight, 0, pd, 8)) && (!bias || rows_fit(bias, 0, pd, 8));
  using B = __nv_bfloat16;
  if (xd == FSP_DTYPE_F32) return whole ? launch_norm<float, kWhole>(a, st) : launch_norm<float, kShift>(a, st);
  return whole ? launch_norm<B, kWhole>(a, st) : fit(2) ? launch_norm<B, kPart>(a, st) : launch_norm<B, kShift>(a, st);
}

// Where the parameters' gradients are wanted, one CTA takes up to this many rows a group, which
// saves the second launch (32 x 512 and 16 x 1024 4.3 and 4.7 us, on two CTAs 4.8 and 5.1; four
// rows a group 5.7 and 6.3 for 64 and 32 rows, on several CTAs 4.8 and 5.0).  The gradient of x
// alone has no second launch to save (32 x 512 3.1 us on one CTA, 2.3 on two).
constexpr int kAlone = 2;

// Threads of a group for rows of up to 8192 elements (0: of more).
constexpr int grad_threads(int64_t dim) {
  return dim <= 128 ? 8 : dim <= 256 ? 16 : dim <= 512 ? 32 : dim <= 1024 ? 64 : dim <= 2048 ? 128 : dim <= 4096 ? 256 : dim <= 8192 ? 512 : 0;
}
bool alone(int64_t rows, int64_t dim) { return grad_threads(dim) && rows <= kAlone * (kRingThreads / grad_threads(dim)); }

size_t workspace_of(int64_t rows, int64_t dim) {   // (from a multiple of 256)
  return rows == 0 || alone(rows, dim) ? 0 : size_t(std::min<int64_t>(kParts, rows)) * 2 * size_t(dim) * 4 + 256;
}

fsp_status launch_join(const GradArgs& a, cudaStream_t st) {
  return launch_next(join_columns_kernel, dim3(unsigned((a.dim + 31) / 32), 2), kJoinWarps * 32, 0, 1, a, st,
                     "layer norm gradient (join) kernel launch");
}

template <typename X, typename G, Rows R, int T, int E>
fsp_status launch_ring_grad(GradArgs a, cudaStream_t st) {
  constexpr bool kWide = sizeof(X) + sizeof(G) == 8;
  constexpr int V = R == kWhole ? (kWide ? 4 : 8) : kWide ? 1 : 2, kGroups = kRingThreads / T;
  constexpr int kStage = 2 * Columns<X, V, T, E, R>::kStage + Columns<G, V, T, E, R>::kStage;
  constexpr int kStaging = R == kShift && E > 16 ? kGroups * (T * E * int(sizeof(X)) + 16) : 0;
  constexpr int kStages = std::min(4, (kRingBytes - kStaging) / kStage), kSmem = kStages * kStage + kStaging;
  void (*kernel)(GradArgs) = grad_ring_kernel<X, G, V, T, E, kStages, R>;
  fsp_status s = allow_kernel(reinterpret_cast<const void*>(kernel), kSmem);
  if (s != FSP_OK) return s;
  a.n_parts = int(std::min<int64_t>(kParts, (a.rows + kGroups - 1) / kGroups));
  if (a.rows > 0 && (a.grad_weight || a.grad_bias) && alone(a.rows, a.dim)) a.n_parts = 1;
  if (a.rows > 0) s = launch_next(kernel, dim3(unsigned(a.n_parts)), kRingThreads, kSmem, 1, a, st, "layer norm gradient kernel launch");
  return s == FSP_OK && (a.grad_weight || a.grad_bias) && a.n_parts != 1 ? launch_join(a, st) : s;   // (one CTA joins by itself)
}

template <typename X, typename G, int V>
fsp_status launch_wide_grad(GradArgs a, cudaStream_t st) {
  fsp_status s = FSP_OK;
  a.n_parts = int(std::min<int64_t>(kParts, (a.rows + kPartRows - 1) / kPartRows));
  if (a.grad_weight || a.grad_bias) {   // (first: grad_x may take the place of x or grad_out)
    const dim3 grid(unsigned((a.dim + 32 * V - 1) / (32 * V)), unsigned(a.n_parts));
    if (a.rows > 0)
      s = launch_next(column_sums_kernel<X, G, V>, grid, kColumnWarps * 32, 0, 1, a, st, "layer norm gradient (columns) kernel launch");
    if (s == FSP_OK) s = launch_join(a, st);
  }
  if (s != FSP_OK || !a.grad_x || a.rows == 0) return s;
  return launch_next(wide_grad_kernel<X, G, V>, dim3(unsigned(a.rows)), kWideThreads, 0, 1, a, st, "layer norm gradient kernel launch");
}

template <typename X, typename G, Rows R>
fsp_status launch_grad(const GradArgs& a, cudaStream_t st) {
  switch (grad_threads(a.dim)) {
    case 8: return a.dim <= 64 ? launch_ring_grad<X, G, R, 8, 8>(a, st) : launch_ring_grad<X, G, R, 8, 16>(a, st);
    case 16: return launch_ring_grad<X, G, R, 16, 16>(a, st);
    case 32: return launch_ring_grad<X, G, R, 32, 16>(a, st);
    case 64: return launch_ring_grad<X, G, R, 64, 16>(a, st);
    case 128: return launch_ring_grad<X, G, R, 128, 16>(a, st);
    case 256: return launch_ring_grad<X, G, R, 256, 16>(a, st);
    case 512: return launch_ring_grad<X, G, R, 512, 16>(a, st);
  }
  // (odd rows of fp32 beside bf16: 32 columns a thread leave no room for a row of results beside one of each input)
  if constexpr (R != kShift || sizeof(X) + sizeof(G) == 4)
    if (a.dim <= 16384) return launch_ring_grad<X, G, R, 512, 32>(a, st);
  return launch_wide_grad<X, G, R == kWhole ? 8 : 1>(a, st);
}

template <typename X, typename G>
fsp_status launch_grad(const GradArgs& a, Rows rows, cudaStream_t st) {
  if (rows == kWhole) return launch_grad<X, G, kWhole>(a, st);
  if constexpr (sizeof(X) + sizeof(G) == 8) return launch_grad<X, G, kPart>(a, st);   // (elements of four bytes)
  else return rows == kPart ? launch_grad<X, G, kPart>(a, st) : launch_grad<X, G, kShift>(a, st);
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
  const size_t need = columns ? workspace_of(rows, dim) : 0;
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
  a.center = center != 0;
  a.weight_f32 = wd == FSP_DTYPE_F32;
  a.grad_param_f32 = pd == FSP_DTYPE_F32;
  a.accumulate = accumulate != 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto fit = [&](int v) {
    return dim % v == 0 && rows_fit(x, xs, xd, v) && rows_fit(grad, gs, gd, v) && (!add || rows_fit(add, as, xd, v)) &&
           (!grad_x || rows_fit(grad_x, ds, xd, v));
  };
  const Rows lie = fit(8) && (!weight || rows_fit(weight, 0, wd, 8)) ? kWhole : fit(2) ? kPart : kShift;
  using B = __nv_bfloat16;
  if (xd == FSP_DTYPE_F32) return gd == FSP_DTYPE_F32 ? launch_grad<float, float>(a, lie, st) : launch_grad<float, B>(a, lie, st);
  return gd == FSP_DTYPE_F32 ? launch_grad<B, float>(a, lie, st) : launch_grad<B, B>(a, lie, st);
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
