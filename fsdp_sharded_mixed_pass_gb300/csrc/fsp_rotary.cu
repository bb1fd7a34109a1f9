// Rotary positions (sm_103a): the first `rotary_dim` elements of each head as pairs (a, b),
// turned by the angle of their token's position t and their pair's frequency f_j,
//
//   a' = scale (a cos(t f_j) - b sin(t f_j)),  b' = scale (b cos(t f_j) + a sin(t f_j));
//
// the gradient is the same with the angle negated.
//
// Bound: HBM (131072 tokens of 12 bf16 heads of 64 61 us, 0.97 of the measured copy; 16384 of 24
// heads of 128 within a projection's rows 34 us, 0.87).  A frequency is held in units of 2^-64
// turn per position, rounded once, so t f_j modulo a turn is one 64-bit product that wraps, off by at
// most |t| 2^-65 turn (2^-34 at position 2^31, where a 32-bit angle's last place is 2^-32), without
// arithmetic in 64-bit floating point.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fsp_rows.cuh"

namespace fsp {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTensors = 2;
constexpr int64_t kMostHeads = 1 << 20, kMostHeadDim = 1 << 16;

struct Tensor {
  const void* x;
  void* out;
  int64_t x_stride[3], out_stride[3];   // batch, token, head
  int heads;
  int rest;                             // elements past the rotated ones to copy (0 in place)
};

struct RotaryArgs {
  Tensor t[kMostTensors];
  const void* positions;
  const uint64_t* phases;
  int64_t positions_stride;   // between batches
  int64_t n_threads, tokens;
  float scale;
  int index_bytes;
  int turning;                // threads along the rotated part of a head
  int units;                  // and along all of it
  int splits;                 // threads along the heads of a token
  int heads;                  // of both tensors
  int rotary_dim;
  int run_step, second;       // elements from unit to unit of the rotated part, and from its first run to its second
  bool inverse;
};

// Sine and cosine of an angle in units of 2^-32 turn.  The nearest quarter is taken off in
// whole numbers; what is left, r in [-pi/4, pi/4], goes through the Taylor series up to r^9 / 9!
// and r^10 / 10! (what follows is below 2^-28 and 2^-32 of the result).
__device__ __forceinline__ void sine_cosine(uint32_t angle, float* sine, float* cosine) {
  const uint32_t quarter = (angle + 0x20000000u) >> 30;
  const float r = float(int32_t(angle - (quarter << 30))) * 1.46291807926715968e-9f;   // pi / 2^31
  const float q = r * r;
  float s = __fmaf_rn(q, 1.f / 362880.f, -1.f / 5040.f), c = __fmaf_rn(q, -1.f / 3628800.f, 1.f / 40320.f);
  s = __fmaf_rn(q, s, 1.f / 120.f);
  c = __fmaf_rn(q, c, -1.f / 720.f);
  s = __fmaf_rn(q, s, -1.f / 6.f);
  c = __fmaf_rn(q, c, 1.f / 24.f);
  s = __fmaf_rn(r * q, s, r);
  c = __fmaf_rn(q, c, -0.5f);
  c = __fmaf_rn(q, c, 1.f);
  // quarters 1 and 3 swap the two; the sine is negative in 2 and 3, the cosine in 1 and 2
  const float a = quarter & 1u ? c : s, b = quarter & 1u ? s : c;
  *sine = __uint_as_float(__float_as_uint(a) ^ ((quarter & 2u) << 30));
  *cosine = __uint_as_float(__float_as_uint(b) ^ (((quarter + 1u) & 2u) << 30));
}

// (spelt out, so that every layout and width rounds alike)
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float p = __fmaf_rn(a, c, -__fmul_rn(b, s));
  b = __fmaf_rn(b, c, __fmul_rn(a, s));
  a = p;
}

// A thread: one unit of every splits-th head of one token, so that its sines and cosines are
// computed once.  A unit is kAccesses accesses - kRuns = 2: the pairs of a run of V elements
// with another one, kRuns = 1: V / 2 pairs of neighbours - as far apart as there are units, or
// as many runs of V elements that are copied.  Heads of odd sizes take narrow accesses, several
// a thread: what counts is how many bytes are in flight.  The loads of kHeads heads come before
// their stores.  (Measured at accesses of eight elements: four CTAs per SM for bf16 neighbours 61 us,
// unbounded 64, 131072 x 12 heads of 64; three for halves 40 us, two, as their registers allow, 34,
// 16384 x 24 heads of 128.  Narrower neighbours have the bound without a measurement; those of four
// elements, two accesses a thread, spill 18 bytes for it.)
template <typename T, int V, int kRuns, int kAccesses, int kHeads>
__global__ void __launch_bounds__(kThreads, kRuns == 1 && sizeof(T) == 2 ? 4 : 1) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int kPairs = V * kRuns / 2;
  launch_dependents();
  grid_dependency_wait();
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.n_threads) return;
  int unit, split;
  int64_t token, batch, at;
  if (a.n_threads <= UINT32_MAX) {   // (32-bit divisions)
    uint32_t k = uint32_t(i);
    unit = int(k % uint32_t(a.units));
    k /= uint32_t(a.units);
    split = int(k % uint32_t(a.splits));
    k /= uint32_t(a.splits);
    token = k;
    batch = k / uint32_t(a.tokens);
    at = k % uint32_t(a.tokens);
  } else {
    int64_t k = i;
    unit = int(k % a.units);
    k /= a.units;
    split = int(k % a.splits);
    token = k / a.splits;
    batch = token / a.tokens;
    at = token % a.tokens;
  }
  const bool turns = unit < a.turning;
  // the unit's first access of its part of a head, the part's units and accesses
  const int first = turns ? unit : unit - a.turning, units = turns ? a.turning : a.units - a.turning;
  float c[kAccesses][kPairs], s[kAccesses][kPairs];
  if (turns) {
    const int64_t index = batch * a.positions_stride + at;
    const int64_t pos = a.index_bytes == 8 ? static_cast<const int64_t*>(a.positions)[index] : static_cast<const int32_t*>(a.positions)[index];
#pragma unroll
    for (int m = 0; m < kAccesses; ++m)
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const int pair = min((first + m * units) * kPairs + j, a.rotary_dim / 2 - 1);
        sine_cosine(uint32_t(uint64_t(pos) * a.phases[pair] >> 32), &s[m][j], &c[m][j]);
        c[m][j] *= a.scale;
        s[m][j] *= a.inverse ? -a.scale : a.scale;
      }
  }
  const T *from0, *from1;
  T *to0, *to1;
  auto place = [&](const Tensor& t, const T*& from, T*& to) {
    const int begin = turns ? first * a.run_step : a.rotary_dim + first * V;
    from = static_cast<const T*>(t.x) + batch * t.x_stride[0] + at * t.x_stride[1] + begin;
    to = static_cast<T*>(t.out) + batch * t.out_stride[0] + at * t.out_stride[1] + begin;
  };
  place(a.t[0], from0, to0);
  place(a.t[1], from1, to1);
  // kHeads heads from h on, or as many as are left
  auto some = [&](auto turning, auto all_there, int h) {
    constexpr bool kTurn = decltype(turning)::value, kAll = decltype(all_there)::value;
    constexpr int kUsed = kTurn ? kRuns : 1;
    const int gap = units * (kTurn ? a.run_step : V);
    alignas(32) T x[kHeads][kAccesses][kUsed][V];
    T* to[kHeads];
    bool there[kHeads][kAccesses];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int head = h + k * a.splits, later = head - a.t[0].heads;
      const T* from = later < 0 ? from0 + head * a.t[0].x_stride[2] : from1 + later * a.t[1].x_stride[2];
      to[k] = later < 0 ? to0 + head * a.t[0].out_stride[2] : to1 + later * a.t[1].out_stride[2];
      const int accesses = kTurn ? a.rotary_dim / (V * kRuns) : (later < 0 ? a.t[0].rest : a.t[1].rest) / V;
#pragma unroll
      for (int m = 0; m < kAccesses; ++m) {
        there[k][m] = (kAll || head < a.heads) && ((kTurn && kAccesses == 1) || first + m * units < accesses);
        if (there[k][m]) {
#pragma unroll
          for (int n = 0; n < kUsed; ++n) load_raw<T, V>(from + m * gap + n * a.second, x[k][m][n]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
#pragma unroll
      for (int m = 0; m < kAccesses; ++m) {
        if constexpr (kTurn) {
          float f[kRuns][V];
#pragma unroll
          for (int n = 0; n < kRuns; ++n)
#pragma unroll
            for (int j = 0; j < V; ++j) f[n][j] = widen(x[k][m][n][j]);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) {
            if constexpr (kRuns == 2)
              turn(f[0][j], f[1][j], c[m][j], s[m][j]);
            else
              turn(f[0][2 * j], f[0][2 * j + 1], c[m][j], s[m][j]);
          }
          if (there[k][m]) {
#pragma unroll
            for (int n = 0; n < kRuns; ++n) store_vec<T, V>(to[k] + m * gap + n * a.second, f[n]);
          }
        } else if (there[k][m]) {
          store_raw<T, V>(to[k] + m * gap, x[k][m][0]);   // (the bits themselves)
        }
      }
  };
  auto all = [&](auto turning) {
    int h = split;
    for (; h + (kHeads - 1) * a.splits < a.heads; h += kHeads * a.splits) some(turning, std::true_type{}, h);
    if (h < a.heads) some(turning, std::false_type{}, h);
  };
  if (turns)
    all(std::true_type{});
  else
    all(std::false_type{});
}

// ---- host -----------------------------------------------------------------------------

// One of a call's strided buffers: elements at sum of index[d] * stride[d] + 0 ... head_dim - 1.
struct View {
  const void* p;
  int64_t extent[3], stride[3], head_dim;
  int64_t size;   // bytes of an element
  std::string name;
};

int64_t span_of(const View& v) {   // elements from the first to past the last
  int64_t last = v.head_dim;
  for (int d = 0; d < 3; ++d) last += (v.extent[d] - 1) * v.stride[d];
  return last;
}

bool same_view(const View& v, const View& w) {
  bool same = v.p == w.p && v.head_dim == w.head_dim && v.size == w.size;
  for (int d = 0; d < 3; ++d)
    same = same && v.extent[d] == w.extent[d] && (v.extent[d] == 1 || v.stride[d] == w.stride[d]);
  return same;
}

// Whether no element of v is one of w: their spans do not meet, or both repeat with a common
// stride m and lie in different parts of it (query and key heads within one projection's rows).
bool disjoint(const View& v, const View& w) {
  if (!overlap(v.p, size_t(span_of(v) * v.size), w.p, size_t(span_of(w) * w.size))) return true;
  if (v.size != w.size) return false;
  for (int k = 0; k < 6; ++k) {
    const View& from = k < 3 ? v : w;
    const int64_t m = from.stride[k % 3];
    if (from.extent[k % 3] == 1 || m == 0) continue;   // (0: an input that repeats a head)
    auto part = [&](const View& x) {   // elements that it covers of a period; 0: it has none
      int64_t n = x.head_dim;
      for (int d = 0; d < 3; ++d) {
        if (x.extent[d] == 1) continue;
        if (x.stride[d] < m)
          n += (x.extent[d] - 1) * x.stride[d];
        else if (x.stride[d] % m)
          return int64_t(0);
      }
      return n <= m ? n : int64_t(0);
    };
    const int64_t nv = part(v), nw = part(w);
    if (!nv || !nw) continue;
    const int64_t period = m * v.size;
    int64_t d = int64_t((reinterpret_cast<intptr_t>(w.p) - reinterpret_cast<intptr_t>(v.p)) % period);
    if (d < 0) d += period;
    if (nv * v.size <= d && d + nw * w.size <= period) return true;
  }
  return false;
}

// Whether every element of v has a place of its own.
bool distinct(const View& v) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return v.stride[a] < v.stride[b]; });
  int64_t reach = v.head_dim;
  for (int d : order) {
    if (v.extent[d] == 1) continue;
    if (v.stride[d] < reach) return false;
    reach += (v.extent[d] - 1) * v.stride[d];
  }
  return true;
}

fsp_status check_view(const View& v) {
  for (int d = 0; d < 3; ++d)
    if (v.stride[d] < 0 || v.stride[d] > (int64_t(1) << 57) / v.extent[d])
      return fail(FSP_EINVAL, v.name + "'s strides are out of range");
  if (!v.p) return fail(FSP_EINVAL, v.name + " is NULL");
  if (reinterpret_cast<uintptr_t>(v.p) % size_t(v.size)) return fail(FSP_EINVAL, v.name + " is not aligned to its elements");
  return FSP_OK;
}

bool fits(const View& v, int elems) {
  bool ok = reinterpret_cast<uintptr_t>(v.p) % size_t(elems * v.size) == 0;
  for (int d = 0; d < 3; ++d) ok = ok && (v.extent[d] == 1 || v.stride[d] % elems == 0);
  return ok;
}

// Accesses of a thread, of V elements each, where a launch has enough threads without; and the
// heads whose loads it has in flight.
template <typename T>
constexpr int accesses(int v) {
  return v == 8 ? 1 : v == 4 ? 2 : v == 2 ? 4 : sizeof(T) == 4 ? 4 : 2;
}
template <typename T>
constexpr int heads(int v, int runs, int accesses) {
  return v * runs * accesses * int(sizeof(T)) > 64 ? 2 : 4;
}

template <typename T, int V, int kRuns>
fsp_status launch_rotary(const RotaryArgs& a, bool several, cudaStream_t st) {
  constexpr int kMany = accesses<T>(V);
  const int64_t ctas = (a.n_threads + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return fail(FSP_EUNSUPPORTED, "too many tokens");
  void (*kernel)(RotaryArgs) = several ? rotary_kernel<T, V, kRuns, kMany, heads<T>(V, kRuns, kMany)> : rotary_kernel<T, V, kRuns, 1, heads<T>(V, kRuns, 1)>;
  return launch_next(kernel, dim3(unsigned(ctas)), kThreads, 0, 1, a, st, "rotary kernel launch");
}

template <typename T>
fsp_status launch_width(const RotaryArgs& a, int v, int runs, bool several, cudaStream_t st) {
  if (runs == 1)
    return v == 8 ? launch_rotary<T, 8, 1>(a, several, st) : v == 4 ? launch_rotary<T, 4, 1>(a, several, st) : launch_rotary<T, 2, 1>(a, several, st);
  return v == 8   ? launch_rotary<T, 8, 2>(a, several, st)
         : v == 4 ? launch_rotary<T, 4, 2>(a, several, st)
         : v == 2 ? launch_rotary<T, 2, 2>(a, several, st)
                  : launch_rotary<T, 1, 2>(a, several, st);
}

// A token's heads are spread over threads until a launch has this many (16 + 8 heads of 128,
// us, with 152 x 768 and 152 x 384: 1024 tokens 7.3 and 5.9, 4096 tokens 12.2 and 13.5: one number,
// which costs some thousands of tokens what it gains a thousand).
constexpr int64_t kEnoughThreads = 152 * 384;
// From this many threads of one access each on they take several (20000 tokens, 12 bf16 heads
// of 146, 60 turned in pairs: 63 us with one, 38 with four).
constexpr int64_t kSeveralThreads = 152 * 1536;

fsp_status rotary(const fsp_rotary_tensor* tensors, int32_t n, int32_t dtype, int64_t batch, int64_t tokens,
                  const void* positions, int32_t index_bytes, int64_t positions_stride, const uint64_t* phases,
                  int64_t rotary_dim, int32_t layout, float scale, int32_t inverse, void* stream) {
  if (n < 1 || n > kMostTensors || !tensors) return fail(FSP_EINVAL, "one or two tensors are rotated by a call");
  if (!known(dtype)) return fail(FSP_EINVAL, "unknown dtype");
  if (batch < 0 || tokens < 0) return fail(FSP_EINVAL, "batch and tokens must be >= 0");
  if (index_bytes != 4 && index_bytes != 8) return fail(FSP_EINVAL, "index_bytes must be 4 or 8");
  if (layout != FSP_ROTARY_HALF && layout != FSP_ROTARY_INTERLEAVED) return fail(FSP_EINVAL, "unknown layout");
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > kMostHeadDim) return fail(FSP_EINVAL, "rotary_dim must be even, from 2 to 65536");
  if (!(std::fabs(scale) <= 3.4e38f)) return fail(FSP_EINVAL, "scale must be finite");
  if (positions_stride != 0 && (positions_stride < tokens || (batch > 0 && positions_stride > (int64_t(1) << 57) / batch))) return fail(FSP_EINVAL, "positions_stride must be 0 or at least tokens, and in range");
  if (tokens > 0 && batch > (int64_t(1) << 40) / tokens) return fail(FSP_EUNSUPPORTED, "too many tokens");
  RotaryArgs a{};
  View views[2 * kMostTensors];   // x, out of each tensor that holds elements
  int n_views = 0, k = 0;
  for (int i = 0; i < n; ++i) {
    const fsp_rotary_tensor& t = tensors[i];
    const std::string of = n > 1 ? " of tensor " + std::to_string(i) : std::string();
    if (t.heads < 0 || t.heads > kMostHeads || t.head_dim < 0 || t.head_dim > kMostHeadDim)
      return fail(FSP_EINVAL, "heads" + of + " must be from 0 to 2^20 and head_dim from 0 to 2^16");
    if (t.head_dim < rotary_dim) return fail(FSP_EINVAL, "head_dim" + of + " is smaller than rotary_dim");
    if (batch == 0 || tokens == 0 || t.heads == 0) continue;
    for (int out = 0; out < 2; ++out) {
      View& v = views[n_views++];
      v = View{out ? t.out : t.x, {batch, tokens, t.heads}, {}, t.head_dim, int64_t(size_of(dtype)), (out ? "out" : "x") + of};
      std::copy_n(out ? t.out_strides : t.x_strides, 3, v.stride);
      const fsp_status s = check_view(v);
      if (s != FSP_OK) return s;
      if (out && !distinct(v)) return fail(FSP_EINVAL, v.name + ": elements share a place");
    }
    Tensor& d = a.t[k++];
    d.x = t.x;
    d.out = t.out;
    std::copy_n(t.x_strides, 3, d.x_stride);
    std::copy_n(t.out_strides, 3, d.out_stride);
    d.heads = int(t.heads);
    d.rest = same_view(views[n_views - 2], views[n_views - 1]) ? 0 : int(t.head_dim - rotary_dim);
    a.heads += d.heads;
  }
  if (n_views == 0) return FSP_OK;
  const size_t position_bytes = (size_t(positions_stride) * size_t(batch - 1) + size_t(tokens)) * size_t(index_bytes);
  if (!positions || !phases) return fail(FSP_EINVAL, "positions or phases is NULL");
  if (reinterpret_cast<uintptr_t>(positions) % size_t(index_bytes)) return fail(FSP_EINVAL, "positions is not aligned to its elements");
  if (reinterpret_cast<uintptr_t>(phases) % 8) return fail(FSP_EINVAL, "phases is not 8-byte aligned");
  for (int i = 1; i < n_views; i += 2) {
    const View& out = views[i];
    const size_t bytes = size_t(span_of(out) * out.size);
    if (overlap(out.p, bytes, positions, position_bytes) || overlap(out.p, bytes, phases, size_t(rotary_dim) * 4))
      return fail(FSP_EINVAL, out.name + " overlaps positions or phases");
    for (int j = 0; j < n_views; ++j)
      if (j != i && !disjoint(out, views[j]) && !(j == i - 1 && same_view(out, views[j])))
        return fail(FSP_EINVAL, out.name + " overlaps " + views[j].name);
  }
  fsp_status s = check_allocation(positions, position_bytes, "positions");
  if (s == FSP_OK) s = check_allocation(phases, size_t(rotary_dim) * 4, "phases");
  for (int i = 0; i < n_views && s == FSP_OK; ++i)
    s = check_allocation(views[i].p, size_t(span_of(views[i]) * views[i].size), views[i].name.c_str());
  if (s != FSP_OK) return s;
  // the widest accesses at which every head, half and rest begins
  const bool half = layout == FSP_ROTARY_HALF;
  auto fit = [&](int k) {
    bool ok = rotary_dim % (half ? 2 * k : k) == 0;
    for (int i = 0; i < n_views; ++i) ok = ok && fits(views[i], k) && views[i].head_dim % k == 0;
    return ok;
  };
  const int v = fit(8) ? 8 : fit(4) ? 4 : fit(2) ? 2 : 1;
  const int runs = half || v == 1 ? 2 : 1;
  a.positions = positions;
  a.phases = phases;
  a.positions_stride = positions_stride;
  a.tokens = tokens;
  a.scale = scale;
  a.index_bytes = index_bytes;
  auto units = [&](int per_unit) {
    auto of = [&](int64_t elements) { return int((elements + int64_t(v) * per_unit - 1) / (int64_t(v) * per_unit)); };
    a.turning = of(rotary_dim / runs);
    a.units = a.turning + of(std::max(a.t[0].rest, a.t[1].rest));
  };
  units(1);
  const bool several = batch * tokens * a.units >= kSeveralThreads;
  if (several) units(dtype == FSP_DTYPE_F32 ? accesses<float>(v) : accesses<__nv_bfloat16>(v));
  a.rotary_dim = int(rotary_dim);
  a.run_step = half ? v : v * runs;
  a.second = half ? int(rotary_dim / 2) : 1;
  a.inverse = inverse != 0;
  const int64_t alone = batch * tokens * a.units;
  a.splits = int(std::clamp<int64_t>(kEnoughThreads / alone, 1, a.heads));
  a.n_threads = alone * a.splits;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == FSP_DTYPE_F32 ? launch_width<float>(a, v, runs, several, st) : launch_width<__nv_bfloat16>(a, v, runs, several, st);
}

}  // namespace
}  // namespace fsp

namespace fsp {
namespace {

// f / (2 pi) in units of 2^-64 turn, without whole turns, rounded to the nearest (and off by 2^-11 of a
// unit at most before that).  |f| = M 2^e with M of 53 bits below 2^64: M times the bits of 1 / (2 pi) from
// weight 2^-(e + 1) on, the first 64 of which count units and the next 64 parts of one; what is above them
// gives whole turns.
uint64_t phase_of(double f) {
  // 1 / (2 pi), 192 bits after the point (pi by Machin's formula in whole numbers)
  constexpr uint64_t kPerRadian[4] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull, 0};
  auto bits = [&](int from) -> uint64_t {   // 64 of them
    if (from <= -64) return 0;
    if (from < 0) return kPerRadian[0] >> -from;
    const int i = from / 64, k = from % 64;
    return k ? kPerRadian[i] << k | kPerRadian[i + 1] >> (64 - k) : kPerRadian[i];
  };
  int e;
  const uint64_t m = uint64_t(std::ldexp(std::frexp(std::fabs(f), &e), 53));
  e -= 53;   // at most 11
  const unsigned __int128 parts = static_cast<unsigned __int128>(m) * bits(e + 64) + (uint64_t(1) << 63);
  const uint64_t phase = m * bits(e) + uint64_t(parts >> 64);
  return f < 0 ? 0 - phase : phase;
}

}  // namespace
}  // namespace fsp

extern "C" fsp_status fsp_rotary_phases(const double* frequencies, int64_t n, uint64_t* phases) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (n < 0 || (n > 0 && (!frequencies || !phases))) return fsp::fail(FSP_EINVAL, "n is negative or a pointer NULL");
    for (int64_t j = 0; j < n; ++j) {
      if (!(std::fabs(frequencies[j]) < 18446744073709551616.0)) return fsp::fail(FSP_EINVAL, "a frequency is not finite, or 2^64 or above");
      phases[j] = fsp::phase_of(frequencies[j]);
    }
    return FSP_OK;
  });
}

extern "C" fsp_status fsp_rotary(const fsp_rotary_tensor* tensors, int32_t n, int32_t dtype, int64_t batch, int64_t tokens,
                                 const void* positions, int32_t index_bytes, int64_t positions_stride,
                                 const uint64_t* phases, int64_t rotary_dim, int32_t layout, float scale, int32_t inverse,
                                 void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::rotary(tensors, n, dtype, batch, tokens, positions, index_bytes, positions_stride, phases, rotary_dim,
                       layout, scale, inverse, cuda_stream);
  });
}
