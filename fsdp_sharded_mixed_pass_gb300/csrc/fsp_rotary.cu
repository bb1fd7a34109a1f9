// Rotary positions (sm_103a): the first `rotary_dim` elements of each head as pairs (a, b),
// turned by the angle of their token's position t and their pair's frequency f_j,
//
//   a' = scale (a cos(t f_j) - b sin(t f_j)),  b' = scale (b cos(t f_j) + a sin(t f_j));
//
// the gradient is the same with the angle negated.
//
// Bound: HBM.  A frequency is held in units of 2^-64 turn per position, so t f_j modulo a
// turn is one 64-bit product that wraps: as exact at position 2^31 as at position 1, without
// arithmetic in 64-bit floating point.
#include <algorithm>
#include <cmath>

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
  int groups;                 // threads along a head
  int splits;                 // threads along the heads of a token
  int heads;                  // of both tensors
  int rotary_dim;
  bool inverse;
};

// (spelt out, so that every layout and width rounds alike)
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float p = __fmaf_rn(a, c, -__fmul_rn(b, s));
  b = __fmaf_rn(b, c, __fmul_rn(a, s));
  a = p;
}

// A thread: P pairs of every splits-th head of one token.  kHalf: pair j is elements j and
// j + rotary_dim / 2, otherwise 2 j and 2 j + 1.  V: elements of an access.
template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  constexpr int P = kHalf ? V : (V > 1 ? V / 2 : 1);
  launch_dependents();
  grid_dependency_wait();
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.n_threads) return;
  const int group = int(i % a.groups);
  const int64_t rest = i / a.groups;
  const int split = int(rest % a.splits);
  const int64_t token = rest / a.splits, batch = token / a.tokens, at = token - batch * a.tokens;
  const int64_t index = batch * a.positions_stride + at;
  const int64_t pos = a.index_bytes == 8 ? static_cast<const int64_t*>(a.positions)[index] : static_cast<const int32_t*>(a.positions)[index];
  float c[P], s[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int pair = group * P + j;
    // turns, as a signed fraction of 2^32 (below half a unit of 2^-31 half turns is cut off)
    const int32_t part = pair < a.rotary_dim / 2 ? int32_t(uint64_t(pos) * a.phases[pair] >> 32) : 0;
    sincospif(float(part) * 0x1p-31f, &s[j], &c[j]);
    c[j] *= a.scale;
    s[j] *= a.inverse ? -a.scale : a.scale;
  }
  for (int h = split; h < a.heads; h += a.splits) {
    const bool second = h >= a.t[0].heads;
    const Tensor& t = second ? a.t[1] : a.t[0];
    const int head = second ? h - a.t[0].heads : h;
    const T* x = static_cast<const T*>(t.x) + batch * t.x_stride[0] + at * t.x_stride[1] + head * t.x_stride[2];
    T* out = static_cast<T*>(t.out) + batch * t.out_stride[0] + at * t.out_stride[1] + head * t.out_stride[2];
    if constexpr (kHalf) {
      const int first = group * P;
      if (first < a.rotary_dim / 2) {
        float u[V], v[V];
        load_vec<T, V>(x + first, u);
        load_vec<T, V>(x + a.rotary_dim / 2 + first, v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          turn(u[j], v[j], c[j], s[j]);
        }
        store_vec<T, V>(out + first, u);
        store_vec<T, V>(out + a.rotary_dim / 2 + first, v);
      }
    } else {
      const int first = group * 2 * P;
      if (first < a.rotary_dim) {
        float u[2 * P];
        if constexpr (V == 1) {
          u[0] = widen(x[first]);
          u[1] = widen(x[first + 1]);
        } else {
          load_vec<T, V>(x + first, u);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          turn(u[2 * j], u[2 * j + 1], c[j], s[j]);
        }
        if constexpr (V == 1) {
          out[first] = narrow<T>(u[0]);
          out[first + 1] = narrow<T>(u[1]);
        } else {
          store_vec<T, V>(out + first, u);
        }
      }
    }
    for (int k = group * V; k < t.rest; k += a.groups * V) {
      alignas(32) float f[V];
      load_vec<T, V>(x + a.rotary_dim + k, f);
      store_vec<T, V>(out + a.rotary_dim + k, f);
    }
  }
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
    if (from.extent[k % 3] == 1) continue;
    const int64_t m = from.stride[k % 3];
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

template <typename T, int V>
fsp_status launch_rotary(const RotaryArgs& a, bool half, cudaStream_t st) {
  const int64_t ctas = (a.n_threads + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return fail(FSP_EUNSUPPORTED, "too many tokens");
  return launch_next(half ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>, dim3(unsigned(ctas)), kThreads, 0, 1, a, st,
                     "rotary kernel launch");
}

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
  // accesses of eight elements where every head, half and rest begins at a multiple of them
  const bool half = layout == FSP_ROTARY_HALF;
  bool vec = rotary_dim % (half ? 16 : 8) == 0;
  for (int i = 0; i < n_views; ++i) vec = vec && fits(views[i], 8) && views[i].head_dim % 8 == 0;
  const int pairs = vec ? (half ? 8 : 4) : 1;
  a.positions = positions;
  a.phases = phases;
  a.positions_stride = positions_stride;
  a.tokens = tokens;
  a.scale = scale;
  a.index_bytes = index_bytes;
  a.groups = int(rotary_dim / 2 / pairs);
  a.splits = std::min(a.heads, 4);
  a.rotary_dim = int(rotary_dim);
  a.inverse = inverse != 0;
  a.n_threads = batch * tokens * a.splits * a.groups;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == FSP_DTYPE_F32) return vec ? launch_rotary<float, 8>(a, half, st) : launch_rotary<float, 1>(a, half, st);
  return vec ? launch_rotary<__nv_bfloat16, 8>(a, half, st) : launch_rotary<__nv_bfloat16, 1>(a, half, st);
}

}  // namespace
}  // namespace fsp

extern "C" fsp_status fsp_rotary_phases(const double* frequencies, int64_t n, uint64_t* phases) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (n < 0 || (n > 0 && (!frequencies || !phases))) return fsp::fail(FSP_EINVAL, "n is negative or a pointer NULL");
    for (int64_t j = 0; j < n; ++j) {
      if (!std::isfinite(frequencies[j])) return fsp::fail(FSP_EINVAL, "a frequency is not finite");
      // turns per position, without the whole ones
      const double turns = std::fmod(frequencies[j] / 6.283185307179586476925, 1.0);
      const uint64_t part = uint64_t(std::ldexp(std::fabs(turns), 64));
      phases[j] = turns < 0 ? 0 - part : part;
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
