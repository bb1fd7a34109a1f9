// Embedding lookup with scaling and its gradient by sorted tokens (sm_103a).
//
//   y_i = s W[t_i],   dW_r (+)= s sum_{i: t_i = r} dy_i
//
// Bound: HBM.  The lookup reads each named row and writes each output row once.
// The gradient reads dy once and writes the table once (or reads and writes the
// named rows, when accumulating); no atomic addition touches a value, so the
// result depends on the tokens alone.
//
// Gradient, three launches, with programmatic stream serialisation (their CTAs are
// there when the launch before them ends):
//   1. sort_tokens_kernel: one cluster sorts (token, position) pairs by token,
//      stably (radix sort), and marks the tokens that occur in a bitmap;
//   2. sum_rows_kernel: the sorted pairs in chunks of 32; a warp owns 32 x V columns
//      of a chunk and adds its rows in fp32 in sorted order.  A token whose pairs
//      lie within one chunk is finished there; the parts of one that spans chunks
//      go to the workspace, so a token that fills half of a batch is spread over as
//      many CTAs as any other half;
//   3. join_rows_kernel: adds such a token's parts, eight warps a share each.
// Zeros into the rows that no token names (not when accumulating) are written by
// other CTAs of 2 or 3.
#include <cooperative_groups.h>

#include <algorithm>

#include "fsp_rows.cuh"

namespace fsp {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kErrToken = 16u;   // a token outside [0, vocab)
__device__ unsigned int g_token_error = 0;

// From L2: written by another CTA of this grid.
__device__ __forceinline__ uint32_t load_l2(const uint32_t* p) {
  uint32_t x;
  asm volatile("ld.global.cg.b32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ uint2 load_l2(const uint2* p) {
  uint2 x;
  asm volatile("ld.global.cg.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p) : "memory");
  return x;
}

__device__ __forceinline__ int64_t token_at(const void* tokens, int index_bytes, int64_t i) {
  return index_bytes == 8 ? static_cast<const int64_t*>(tokens)[i] : int64_t(static_cast<const int32_t*>(tokens)[i]);
}

// ---- lookup ---------------------------------------------------------------------

constexpr int kLookupThreads = 256;

struct LookupArgs {
  const void* weight;
  const void* tokens;
  void* out;
  int64_t vocab, dim, weight_stride, out_stride, n_tokens;
  float scale;
  int index_bytes;
};

// A warp per token: the row in steps of 32 x V elements, four in flight.
template <typename W, typename O, int V>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(const __grid_constant__ LookupArgs a) {
  constexpr int kAhead = 4;
  launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * (kLookupThreads / 32) + (threadIdx.x >> 5);
  if (i >= a.n_tokens) return;
  const int64_t t = token_at(a.tokens, a.index_bytes, i);
  const bool ok = t >= 0 && t < a.vocab;
  if (!ok && lane == 0) atomicOr(&g_token_error, kErrToken);
  const W* row = static_cast<const W*>(a.weight) + (ok ? t : 0) * a.weight_stride;
  O* out = static_cast<O*>(a.out) + i * a.out_stride;
  for (int64_t c0 = int64_t(lane) * V; c0 < a.dim; c0 += kAhead * 32 * V) {
    alignas(32) W x[kAhead][V];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c0 + k * 32 * V < a.dim) load_raw<W, V>(row + c0 + k * 32 * V, x[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c0 + k * 32 * V < a.dim) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = ok ? widen(x[k][j]) * a.scale : 0.f;
        store_vec<O, V>(out + c0 + k * 32 * V, f);
      }
  }
}

// ---- gradient: sort ----------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortCluster = 16;            // most CTAs of a sort (65536 tokens: 23 us, in eight CTAs 36)
constexpr int kHeld = 8;                    // items of a lane that stay in registers
constexpr int kSortOne = 2048;              // tokens that one CTA sorts in its shared memory
constexpr int64_t kSortPerCta = 1024;       // tokens per CTA of a cluster from which twice as many pay (4099: 12 us, of 2048 14)
constexpr int kSortSmem = kSortWarps * kBins * 4 + kBins * 4 + kSortWarps * 4;
constexpr int kSortSmemOne = kSortSmem + 2 * kSortOne * 8;
static_assert(kSortOne <= kSortThreads * kHeld, "one CTA holds its items");
// Most tokens: the sort counts them in 32 bits, in steps of up to all of its threads
// (the last step may end that far past the last token).
constexpr int64_t kSortMost = int64_t(INT32_MAX) - kSortCluster * kSortThreads;
static_assert(32 * kHeld <= kSortCluster * kSortThreads, "a warp's rounds end within the same reach");

struct SortArgs {
  const void* tokens;
  uint2* a;             // (key, position) after an odd number of passes
  uint2* b;             // ... an even number
  uint32_t* present;    // bitmap of the tokens that occur
  uint32_t* totals;     // [kSortCluster][kBins]
  int64_t vocab;
  int64_t padding_idx;
  int n;
  int index_bytes;
  int n_words;          // of the bitmap
  int passes, bits;     // passes of `bits` bits
};

// The sort key: the token, or `vocab` (which sorts last) for one whose gradient
// is dropped.
__device__ __forceinline__ uint32_t token_key(const SortArgs& s, int i) {
  const int64_t t = token_at(s.tokens, s.index_bytes, i);
  if (t < 0 || t >= s.vocab) {
    atomicOr(&g_token_error, kErrToken);
    return uint32_t(s.vocab);
  }
  return t == s.padding_idx ? uint32_t(s.vocab) : uint32_t(t);
}

// The lanes of the warp whose digit equals this one's (kDigitBits ballots).
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool valid) {
  uint32_t mask = __ballot_sync(0xffffffffu, valid);
#pragma unroll
  for (int b = 0; b < kDigitBits; ++b) {
    const uint32_t v = __ballot_sync(0xffffffffu, (d >> b) & 1u);
    mask &= (d >> b) & 1u ? v : ~v;
  }
  return mask;
}

// Least significant digit first.  CTA c of the cluster holds a contiguous run
// of the items and each of its warps a contiguous run of that, so "earlier
// CTA, earlier warp, earlier round, lower lane" is the input's order and every
// pass is stable.  Per pass: each warp ranks its items within their digit,
// counting in shared memory; the counts become each warp's first output slot per
// digit (a scan over digits, CTAs and warps); the items are placed.  Up to
// kHeld rounds of 32 a warp keeps items and ranks in registers (131072 tokens in
// 16 CTAs); beyond, it walks them a second time.  kOne: a single CTA, whose passes
// before the last stay in shared memory.
template <bool kOne>
__global__ void __launch_bounds__(kSortThreads) sort_tokens_kernel(const __grid_constant__ SortArgs s) {
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* hist = smem;                            // [kSortWarps][kBins]
  uint32_t* total = hist + kSortWarps * kBins;      // [kBins]: first slot of this CTA's items of the digit
  uint32_t* sums = total + kBins;                   // [kSortWarps]
  uint2* local = reinterpret_cast<uint2*>(sums + kSortWarps);   // kOne: two buffers of items
  auto sync = [] {
    if constexpr (kOne)
      __syncthreads();
    else
      cg::this_cluster().sync();
  };
  auto item_at = [](const uint2* p) {   // written by any CTA of the cluster before its last sync
    if constexpr (kOne)
      return *p;
    else
      return load_l2(p);
  };
  launch_dependents();
  grid_dependency_wait();
  const int n_ctas = int(gridDim.x), cta = int(blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = cta * kSortThreads + tid; i < s.n_words; i += n_ctas * kSortThreads) s.present[i] = 0;
  const int per_warp = ((s.n + n_ctas * kSortWarps - 1) / (n_ctas * kSortWarps) + 31) / 32 * 32;
  const int64_t first = int64_t(cta * kSortWarps + warp) * per_warp;
  const int begin = int(min(first, int64_t(s.n))), end = int(min(first + per_warp, int64_t(s.n)));
  const bool held = per_warp <= 32 * kHeld;
  const uint32_t digit_mask = (1u << s.bits) - 1u;
  uint32_t* mine = hist + warp * kBins;
  uint2 item[kHeld];
  uint32_t rank[kHeld];
  uint2* dst = s.b;
  for (int pass = 0; pass < s.passes; ++pass) {
    const int shift = pass * s.bits;
    const uint2* src = kOne ? local + ((pass + 1) & 1) * kSortOne : pass & 1 ? s.a : s.b;
    dst = kOne && pass + 1 < s.passes ? local + (pass & 1) * kSortOne : pass & 1 ? s.b : s.a;
    auto load = [&](int from) {   // kHeld rounds of this warp's items
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int i = from + 32 * k + lane;
        if (i < end) item[k] = pass == 0 ? make_uint2(token_key(s, i), uint32_t(i)) : item_at(&src[i]);
      }
    };
    auto rank_round = [&](int k, int i) {   // item k's rank among this warp's items of its digit so far
      const bool valid = i < end;
      const uint32_t d = valid ? (item[k].x >> shift) & digit_mask : 0u;
      const uint32_t peers = same_digit(d, valid);
      const uint32_t at = mine[d];
      __syncwarp();
      const uint32_t before = __popc(peers & ((1u << lane) - 1u));
      if (valid && before == 0) mine[d] = at + __popc(peers);
      __syncwarp();
      return at + before;
    };
    load(begin);
    for (int i = tid; i < kSortWarps * kBins; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    for (int from = begin; from < end; from += 32 * kHeld) {
      if (from > begin) load(from);
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        if (from + 32 * k >= end) break;
        rank[k] = rank_round(k, from + 32 * k + lane);
      }
    }
    __syncthreads();
    if (tid < kBins) {   // counts -> each warp's offset within this CTA's items of the digit
      uint32_t c[kSortWarps], run = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * kBins + tid];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        hist[w * kBins + tid] = run;
        run += c[w];
      }
      total[tid] = run;
      if (!kOne) s.totals[cta * kBins + tid] = run;
    }
    if (!kOne) sync();
    // first slot of each digit (over all CTAs), then of this CTA's items of it
    uint32_t all = 0, before = 0;
    if (kOne && tid < kBins) {
      all = total[tid];
    } else if (tid < kBins) {
      uint32_t t[kSortCluster];
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) t[c] = c < n_ctas ? load_l2(&s.totals[c * kBins + tid]) : 0u;
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        if (c < cta) before += t[c];
        all += t[c];
      }
    }
    uint32_t scan = all;   // inclusive over the warp's digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    if (tid < kBins) {
      uint32_t base = 0;
      for (int w = 0; w < warp; ++w) base += sums[w];
      total[tid] = base + scan - all + before;
    }
    __syncthreads();
    if (held) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k)
        if (begin + 32 * k + lane < end) {
          const uint32_t d = (item[k].x >> shift) & digit_mask;
          dst[total[d] + mine[d] + rank[k]] = item[k];
        }
    } else {
      for (int from = begin; from < end; from += 32 * kHeld) {
        load(from);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          const int i = from + 32 * k + lane;
          if (from + 32 * k >= end) break;
          const uint32_t at = rank_round(k, i);   // (from the warp's offset on)
          if (i < end) dst[total[(item[k].x >> shift) & digit_mask] + at] = item[k];
        }
      }
    }
    sync();   // the pass's items, and totals[] before it is written again
  }
  // the first item of each token marks it
  const int step = n_ctas * kSortThreads;
  for (int i = cta * kSortThreads + tid; i < s.n; i += step) {
    const uint32_t key = item_at(&dst[i]).x;
    if (key < uint32_t(s.vocab) && (i == 0 || item_at(&dst[i - 1]).x != key)) atomicOr(&s.present[key >> 5], 1u << (key & 31));
  }
}

// ---- gradient: rows ------------------------------------------------------------------

constexpr int kRowThreads = 128;
constexpr int kChunk = 32;       // sorted pairs of one warp's walk
constexpr int kZeroRows = 32;    // rows of one CTA that writes zeros: a word of the bitmap

struct RowArgs {
  const uint2* items;        // sorted (key, position)
  const uint32_t* present;
  const void* grad;
  void* weight;
  float* parts;              // [chunk][2][dim]: of a token begun before / going on after the chunk
  int64_t vocab, dim, grad_stride, weight_stride;
  float scale;
  int n;
  int accumulate;
  int cols;                  // threads along the columns: 32, 64 or 128
  int col_ctas;              // CTAs along the columns
  int64_t sum_ctas, zero_ctas;   // of the sums' launch
  uint32_t join_zeros;            // CTAs of the join, per CTA along the columns, that write zeros
};

template <typename T, int V>
__device__ __forceinline__ void finish_row(const RowArgs& a, uint32_t row, int64_t col, const float* acc) {
  T* p = static_cast<T*>(a.weight) + int64_t(row) * a.weight_stride + col;
  float f[V], old[V];
  if (a.accumulate) {
    load_vec<T, V>(p, old);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = __fmaf_rn(acc[j], a.scale, old[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = acc[j] * a.scale;
  }
  store_vec<T, V>(p, f);
}

// A warp: 32 x V columns of one chunk.
template <typename G, typename T, int V>
__device__ __forceinline__ void sum_chunk(const RowArgs& a, int64_t chunk, int64_t col, int lane) {
  constexpr int kAhead = 8;   // rows in flight (16: 4099 tokens 33 us instead of 30, long batches the same)
  const int64_t begin = chunk * kChunk;
  if (begin >= a.n) return;
  const uint32_t none = uint32_t(a.vocab);
  const uint2 it = begin + lane < a.n ? a.items[begin + lane] : make_uint2(none, 0);
  const uint32_t prev = begin > 0 ? a.items[begin - 1].x : none;
  const uint32_t next = begin + kChunk < a.n ? a.items[begin + kChunk].x : none;
  const int count = __popc(__ballot_sync(0xffffffffu, it.x < none));   // dropped tokens sort last
  if (count == 0) return;
  const bool in = col < a.dim;
  const G* grad = static_cast<const G*>(a.grad) + col;
  uint32_t row = __shfl_sync(0xffffffffu, it.x, 0);
  bool head = prev == row;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  for (int k0 = 0; k0 < count; k0 += kAhead) {
    alignas(32) G x[kAhead][V];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t at = __shfl_sync(0xffffffffu, it.y, (k0 + k) & 31);
      if (k0 + k < count && in) load_raw<G, V>(grad + int64_t(at) * a.grad_stride, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k >= count) break;
      const uint32_t key = __shfl_sync(0xffffffffu, it.x, k0 + k);
      if (key != row) {   // the token before is complete: its end lies in this chunk
        if (in) {
          if (head)
            store_vec<float, V>(a.parts + (chunk * 2) * a.dim + col, acc);
          else
            finish_row<T, V>(a, row, col, acc);
        }
        head = false;
        row = key;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = 0.f;
      }
      if (in) {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += widen(x[k][j]);
      }
    }
  }
  if (!in) return;
  const bool tail = count == kChunk && next == row;
  if (head || tail)
    store_vec<float, V>(a.parts + (chunk * 2 + (head ? 0 : 1)) * a.dim + col, acc);
  else
    finish_row<T, V>(a, row, col, acc);
}

// Zeros into the rows of one word of the bitmap that no token of the batch has.
template <typename T, int V, int kThreads>
__device__ __forceinline__ void write_zeros(const RowArgs& a, int64_t word) {
  const int64_t row0 = word * kZeroRows;
  if (row0 >= a.vocab) return;
  const int cx = threadIdx.x & (a.cols - 1), cy = threadIdx.x / a.cols;
  const uint32_t present = a.present[word];
  const float zero[V] = {};
  const int rows = int(min(int64_t(kZeroRows), a.vocab - row0));
  for (int r = cy; r < rows; r += kThreads / a.cols) {
    if (present >> r & 1u) continue;
    T* p = static_cast<T*>(a.weight) + (row0 + r) * a.weight_stride;
    for (int64_t c = int64_t(cx) * V; c < a.dim; c += a.cols * V) store_vec<T, V>(p + c, zero);
  }
}

template <typename G, typename T, int V>
__global__ void __launch_bounds__(kRowThreads) sum_rows_kernel(const __grid_constant__ RowArgs a) {
  launch_dependents();
  grid_dependency_wait();
  // CTAs that sum and CTAs that write zeros, in proportion all along the grid:
  // reads and writes then share the launch's time
  const int64_t ctas = a.sum_ctas + a.zero_ctas, i = blockIdx.x;
  const int64_t sums = i * a.sum_ctas / ctas;
  if ((i + 1) * a.sum_ctas / ctas > sums) {
    const int cx = threadIdx.x & (a.cols - 1), cy = threadIdx.x / a.cols;
    const int64_t chunk = sums / a.col_ctas * (kRowThreads / a.cols) + cy;
    sum_chunk<G, T, V>(a, chunk, (sums % a.col_ctas * a.cols + cx) * V, threadIdx.x & 31);
  } else {
    write_zeros<T, V, kRowThreads>(a, i - sums);
  }
}

// The join's additions wait for one another and leave the memory idle, so the zeros
// of a large table are written beside them instead of beside the sums (text-like tokens,
// fp32 rows of 1024: 65536 into 151936 rows 143 us, beside the sums 154; 4096 107 and 112;
// 16384 into 32000 47 and 50).  Of a small table (4096 x 1024 into 66 MB: 30 us either
// way) or of few tokens (300 into 151936 rows: 100 and 98) the sums hide as much.
constexpr size_t kLateBytes = size_t(100) << 20;
constexpr int64_t kLateChunks = 64;

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// A CTA: the tokens that begin in one of eight chunks and go on after it, 32 x V
// columns.  A token of up to kAlone parts (its chunks') is added by the warp of its
// first chunk; of a longer one each warp adds parts w, w + 8, ..., and then the
// eight sums are added in order.  (One token after the other, by the whole CTA,
// took 40 us on 65536 text-like tokens.)
constexpr int kAlone = 16;

// VZ: elements of an access of a CTA that writes zeros.
template <typename T, int V, int VZ>
__global__ void __launch_bounds__(kJoinThreads) join_rows_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float share[kJoinWarps][32 * V];
  __shared__ int64_t count[kJoinWarps];   // parts of the token that begins in this chunk
  launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x < a.join_zeros) {
    write_zeros<T, VZ, kJoinThreads>(a, int64_t(blockIdx.y) * a.join_zeros + blockIdx.x);
    return;
  }
  const int64_t first = int64_t(blockIdx.x - a.join_zeros) * kJoinWarps;
  const int64_t col = (int64_t(blockIdx.y) * 32 + lane) * V;
  // parts begin, begin + step, ... of the token that begins in `chunk`
  float acc[V];
  auto add_parts = [&](int64_t chunk, int64_t begin, int64_t parts, int step) {
    constexpr int kAhead = 4;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int64_t p = begin; p < parts && col < a.dim; p += kAhead * step) {
      float f[kAhead][V];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t at = p + k * step;
        if (at < parts) load_vec<float, V>(a.parts + ((chunk + at) * 2 + (at == 0 ? 1 : 0)) * a.dim + col, f[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (p + k * step < parts) {
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] += f[k][j];
        }
    }
  };
  {
    const int64_t chunk = first + warp, begin = chunk * kChunk, end = begin + kChunk;
    int64_t parts = 0;
    uint32_t row = 0;
    if (end < a.n) {
      row = a.items[end - 1].x;
      const uint32_t next = a.items[end].x, head = a.items[begin].x, prev = begin > 0 ? a.items[begin - 1].x : ~0u;
      if (row < uint32_t(a.vocab) && next == row && !(head == row && prev == row)) {   // goes on, and not begun before
        // the chunks after this one that begin with it, 128 at a time
        parts = 1;
        for (bool more = true; more;) {
          bool same[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t at = (chunk + parts + 32 * k + lane) * kChunk;
            same[k] = at < a.n && a.items[at].x == row;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int got = __popc(__ballot_sync(0xffffffffu, same[k]));   // sorted: no gaps
            parts += more ? got : 0;
            more = more && got == 32;
          }
        }
      }
    }
    if (parts > 0 && parts <= kAlone) {
      add_parts(chunk, 0, parts, 1);
      if (col < a.dim) finish_row<T, V>(a, row, col, acc);
    }
    if (lane == 0) count[warp] = parts > kAlone ? parts : 0;
  }
  __syncthreads();
  for (int t = 0; t < kJoinWarps; ++t) {
    const int64_t parts = count[t];
    if (parts == 0) continue;   // the whole CTA
    add_parts(first + t, warp, parts, kJoinWarps);
#pragma unroll
    for (int j = 0; j < V; ++j) share[warp][j * 32 + lane] = acc[j];
    __syncthreads();
    if (warp == 0 && col < a.dim) {
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += share[w][j * 32 + lane];
      finish_row<T, V>(a, a.items[(first + t) * kChunk + kChunk - 1].x, col, acc);
    }
    __syncthreads();
  }
}

// ---- host ----------------------------------------------------------------------------

fsp_status check_tokens(const void* tokens, int32_t index_bytes, int64_t n) {
  if (index_bytes != 4 && index_bytes != 8) return fail(FSP_EINVAL, "index_bytes must be 4 or 8");
  if (n < 0 || n > (int64_t(1) << 58)) return fail(FSP_EINVAL, "n_tokens is out of range");
  if (n == 0) return FSP_OK;
  if (!tokens) return fail(FSP_EINVAL, "tokens is NULL");
  if (reinterpret_cast<uintptr_t>(tokens) % size_t(index_bytes)) return fail(FSP_EINVAL, "tokens is not aligned to its elements");
  return check_allocation(tokens, size_t(n) * size_t(index_bytes), "tokens");
}

template <typename W, typename O>
fsp_status launch_lookup(const LookupArgs& a, int v, cudaStream_t st) {
  const dim3 ctas(unsigned((a.n_tokens + kLookupThreads / 32 - 1) / (kLookupThreads / 32)));
  return launch_next(v == 8 ? lookup_kernel<W, O, 8> : v == 4 ? lookup_kernel<W, O, 4> : lookup_kernel<W, O, 1>, ctas, kLookupThreads, 0, 1, a, st,
                     "embedding kernel launch");
}

fsp_status lookup(const void* weight, int32_t wd, int64_t vocab, int64_t dim, int64_t ws, const void* tokens,
                  int32_t index_bytes, int64_t n, float scale, void* out, int32_t od, int64_t os, void* stream) {
  if (vocab < 0 || dim < 0) return fail(FSP_EINVAL, "vocab and dim must be >= 0");
  fsp_status s = check_tokens(tokens, index_bytes, n);
  if (s == FSP_OK) s = check_matrix(weight, vocab, dim, ws, wd, "weight");
  if (s == FSP_OK) s = check_matrix(out, n, dim, os, od, "out");
  if (s != FSP_OK) return s;
  const size_t ob = span_bytes(n, dim, os, od);
  if (overlap(out, ob, weight, span_bytes(vocab, dim, ws, wd)) || overlap(out, ob, tokens, size_t(n) * size_t(index_bytes)))
    return fail(FSP_EINVAL, "out overlaps an input");
  if (n == 0 || dim == 0) return FSP_OK;
  if (vocab == 0) return fail(FSP_EINVAL, "tokens look up an empty table");
  if (n > int64_t(INT32_MAX) * (kLookupThreads / 32)) return fail(FSP_EUNSUPPORTED, "too many tokens");
  const LookupArgs a{weight, tokens, out, vocab, dim, ws, os, n, scale, index_bytes};
  int v = 1;
  for (int k : {8, 4})
    if (v == 1 && dim % k == 0 && rows_fit(weight, ws, wd, k) && rows_fit(out, os, od, k)) v = k;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (wd == FSP_DTYPE_F32)
    return od == FSP_DTYPE_F32 ? launch_lookup<float, float>(a, v, st) : launch_lookup<float, B>(a, v, st);
  return od == FSP_DTYPE_F32 ? launch_lookup<B, float>(a, v, st) : launch_lookup<B, B>(a, v, st);
}

struct Workspace {   // byte offsets
  size_t a, b, present, totals, parts, bytes;
};
Workspace workspace_of(int64_t vocab, int64_t dim, int64_t n) {
  Workspace w{};
  const size_t items = round256(size_t(n) * sizeof(uint2));
  const size_t chunks = size_t((n + kChunk - 1) / kChunk);
  w.a = 0;
  w.b = w.a + items;
  w.present = w.b + items;
  w.totals = w.present + round256(size_t((vocab + 31) / 32) * 4);
  w.parts = w.totals + size_t(kSortCluster) * kBins * 4;
  w.bytes = w.parts + round256(chunks * 2 * size_t(dim) * 4) + 256;   // (the offsets count from a multiple of 256)
  return w;
}

fsp_status check_sizes(int64_t vocab, int64_t dim, int64_t n) {
  if (vocab < 0 || dim < 0 || n < 0) return fail(FSP_EINVAL, "vocab, dim and n_tokens must be >= 0");
  if (vocab >= INT32_MAX) return fail(FSP_EUNSUPPORTED, "vocab must be below 2^31 - 1");
  if (n > kSortMost) return fail(FSP_EUNSUPPORTED, "n_tokens must be below 2^31 - 16384");
  if (dim > (int64_t(1) << 24)) return fail(FSP_EUNSUPPORTED, "dim must be at most 2^24");
  return FSP_OK;
}

fsp_status launch_sort(const SortArgs& s, cudaStream_t st) {
  if (s.n <= kSortOne) {
    const fsp_status ok = allow_kernel(reinterpret_cast<const void*>(&sort_tokens_kernel<true>), kSortSmemOne);
    if (ok != FSP_OK) return ok;
    return launch_next(sort_tokens_kernel<true>, dim3(1), kSortThreads, kSortSmemOne, 1, s, st, "token sort kernel launch");
  }
  // (clusters of 16 are beyond the size every device has to offer)
  const fsp_status ok = allow_kernel(reinterpret_cast<const void*>(&sort_tokens_kernel<false>), kSortSmem, true);
  if (ok != FSP_OK) return ok;
  int ctas = 4;
  while (ctas < kSortCluster && s.n > ctas * kSortPerCta) ctas *= 2;
  return launch_next(sort_tokens_kernel<false>, dim3(unsigned(ctas)), kSortThreads, kSortSmem, ctas, s, st,
                     "token sort kernel launch");
}

// The three launches; what refuses them comes before the first.
template <typename G, typename T, int V>
fsp_status launch_rows(const SortArgs& sort, RowArgs& a, cudaStream_t st) {
  // the widest of 32, 64 and 128 threads that leaves the fewest columns over
  const int64_t vectors = (a.dim + V - 1) / V;
  auto padded = [&](int64_t c) { return (vectors + c - 1) / c * c; };
  a.cols = kRowThreads;
  for (int c : {64, 32})
    if (padded(c) < padded(a.cols)) a.cols = c;
  a.col_ctas = int((a.dim + int64_t(a.cols) * V - 1) / (int64_t(a.cols) * V));
  const int64_t chunks = (int64_t(a.n) + kChunk - 1) / kChunk;
  const int per_cta = kRowThreads / a.cols;
  a.sum_ctas = (chunks + per_cta - 1) / per_cta * a.col_ctas;
  constexpr int kJoinV = V > 4 ? 4 : V;
  const int64_t join_cols = (a.dim + 32 * kJoinV - 1) / (32 * kJoinV);
  const int64_t words = a.accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
  const bool late = chunks >= kLateChunks && size_t(a.vocab) * size_t(a.dim) * sizeof(T) >= kLateBytes;
  a.zero_ctas = late ? 0 : words;
  a.join_zeros = late ? uint32_t((words + join_cols - 1) / join_cols) : 0u;
  const int64_t ctas = a.sum_ctas + a.zero_ctas, join_ctas = a.join_zeros + (chunks + kJoinWarps - 1) / kJoinWarps;
  if (ctas > INT32_MAX || join_ctas > INT32_MAX || join_cols > 65535)
    return fail(FSP_EUNSUPPORTED, "too many tokens times columns");
  fsp_status s = launch_sort(sort, st);
  if (s == FSP_OK)
    s = launch_next(sum_rows_kernel<G, T, V>, dim3(unsigned(ctas)), kRowThreads, 0, 1, a, st, "embedding gradient (sum) kernel launch");
  if (s != FSP_OK || chunks <= 1) return s;
  return launch_next(join_rows_kernel<T, kJoinV, V>, dim3(unsigned(join_ctas), unsigned(join_cols)), kJoinThreads, 0, 1, a, st,
                     "embedding gradient (join) kernel launch");
}

template <typename G, typename T>
fsp_status launch_rows_v(const SortArgs& sort, RowArgs& a, int v, cudaStream_t st) {
  return v == 8 ? launch_rows<G, T, 8>(sort, a, st) : v == 4 ? launch_rows<G, T, 4>(sort, a, st) : launch_rows<G, T, 1>(sort, a, st);
}

fsp_status backward(const void* tokens, int32_t index_bytes, int64_t n, const void* grad, int32_t gd, int64_t dim,
                    int64_t gs, void* weight, int32_t wd, int64_t vocab, int64_t ws, float scale, int64_t padding_idx,
                    int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  fsp_status s = check_sizes(vocab, dim, n);
  if (s == FSP_OK) s = check_tokens(tokens, index_bytes, n);
  if (s == FSP_OK) s = check_matrix(grad, n, dim, gs, gd, "grad_out");
  if (s == FSP_OK) s = check_matrix(weight, vocab, dim, ws, wd, "grad_weight");
  if (s != FSP_OK) return s;
  if (vocab == 0 || dim == 0 || (n == 0 && accumulate)) return FSP_OK;
  const Workspace w = workspace_of(vocab, dim, n);
  if (!workspace) return fail(FSP_EINVAL, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(workspace) % 16) return fail(FSP_EINVAL, "workspace is not 16-byte aligned");
  if (workspace_bytes < w.bytes) return fail(FSP_EINVAL, "workspace is smaller than fsp_embedding_backward_workspace_bytes");
  s = check_allocation(workspace, w.bytes, "workspace");
  if (s != FSP_OK) return s;
  const struct {
    const void* p;
    size_t bytes;
    const char* name;
  } bufs[] = {{weight, span_bytes(vocab, dim, ws, wd), "grad_weight"},
              {workspace, w.bytes, "workspace"},
              {grad, span_bytes(n, dim, gs, gd), "grad_out"},
              {tokens, size_t(n) * size_t(index_bytes), "tokens"}};
  for (int i = 0; i < 2; ++i)   // what is written
    for (int j = i + 1; j < 4; ++j)
      if (overlap(bufs[i].p, bufs[i].bytes, bufs[j].p, bufs[j].bytes))
        return fail(FSP_EINVAL, std::string(bufs[i].name) + " overlaps " + bufs[j].name);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* base = reinterpret_cast<char*>(round256(reinterpret_cast<uintptr_t>(workspace)));
  SortArgs sa{};
  sa.tokens = tokens;
  sa.a = reinterpret_cast<uint2*>(base + w.a);
  sa.b = reinterpret_cast<uint2*>(base + w.b);
  sa.present = reinterpret_cast<uint32_t*>(base + w.present);
  sa.totals = reinterpret_cast<uint32_t*>(base + w.totals);
  sa.vocab = vocab;
  sa.padding_idx = padding_idx;
  sa.n = int(n);
  sa.index_bytes = index_bytes;
  sa.n_words = int((vocab + 31) / 32);
  int bits = 1;   // of the largest key, vocab
  while ((vocab >> bits) != 0) ++bits;
  sa.passes = (bits + kDigitBits - 1) / kDigitBits;
  sa.bits = (bits + sa.passes - 1) / sa.passes;
  RowArgs a{};
  a.items = sa.passes & 1 ? sa.a : sa.b;
  a.present = sa.present;
  a.grad = grad;
  a.weight = weight;
  a.parts = reinterpret_cast<float*>(base + w.parts);
  a.vocab = vocab;
  a.dim = dim;
  a.grad_stride = gs;
  a.weight_stride = ws;
  a.scale = scale;
  a.n = int(n);
  a.accumulate = accumulate != 0;
  int v = 1;
  for (int k : {8, 4})
    if (v == 1 && dim % k == 0 && rows_fit(grad, gs, gd, k) && rows_fit(weight, ws, wd, k)) v = k;
  using B = __nv_bfloat16;
  if (gd == FSP_DTYPE_F32)
    return wd == FSP_DTYPE_F32 ? launch_rows_v<float, float>(sa, a, v, st) : launch_rows_v<float, B>(sa, a, v, st);
  return wd == FSP_DTYPE_F32 ? launch_rows_v<B, float>(sa, a, v, st) : launch_rows_v<B, B>(sa, a, v, st);
}

}  // namespace

cudaError_t take_token_error(unsigned* bits) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_token_error, sizeof(*bits));
  const unsigned zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_token_error, &zero, sizeof(zero));
  return e;
}

}  // namespace fsp

extern "C" fsp_status fsp_embedding(const void* weight, int32_t weight_dtype, int64_t vocab, int64_t dim,
                                    int64_t weight_stride, const void* tokens, int32_t index_bytes, int64_t n_tokens,
                                    float scale, void* out, int32_t out_dtype, int64_t out_stride, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::lookup(weight, weight_dtype, vocab, dim, weight_stride, tokens, index_bytes, n_tokens, scale, out,
                       out_dtype, out_stride, cuda_stream);
  });
}

extern "C" fsp_status fsp_embedding_backward_workspace_bytes(int64_t vocab, int64_t dim, int64_t n_tokens,
                                                             size_t* bytes) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (!bytes) return fsp::fail(FSP_EINVAL, "bytes is NULL");
    const fsp_status s = fsp::check_sizes(vocab, dim, n_tokens);
    if (s == FSP_OK) *bytes = fsp::workspace_of(vocab, dim, n_tokens).bytes;
    return s;
  });
}

extern "C" fsp_status fsp_embedding_backward(const void* tokens, int32_t index_bytes, int64_t n_tokens,
                                             const void* grad_out, int32_t grad_dtype, int64_t dim,
                                             int64_t grad_stride, void* grad_weight, int32_t weight_dtype,
                                             int64_t vocab, int64_t weight_stride, float scale, int64_t padding_idx,
                                             int32_t accumulate, void* workspace, size_t workspace_bytes,
                                             void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::backward(tokens, index_bytes, n_tokens, grad_out, grad_dtype, dim, grad_stride, grad_weight,
                         weight_dtype, vocab, weight_stride, scale, padding_idx, accumulate, workspace,
                         workspace_bytes, cuda_stream);
  });
}
