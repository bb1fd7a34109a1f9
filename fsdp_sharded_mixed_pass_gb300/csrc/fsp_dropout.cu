// Dropout from a counter-based generator, onto a residual stream (sm_103a).
//
//   T = round(65536 p), y_i = (u_i < T ? 0 : x_i 65536 / (65536 - T)) + residual_i
//
// u_i: the i-th 16 bits of Philox-4x32 with ten rounds (J. K. Salmon, M. A. Moraes,
// R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), keyed
// by the seed, its counter (i / 8, call).  The mask is a function of (seed, call, i) and is
// never stored: the gradient is the same function of dy, without the residual.
//
// Bound: HBM.  Sixteen bits an element, so that ten rounds (a block of four words) serve
// eight elements.
#include <type_traits>

#include "fsp_rows.cuh"

namespace fsp {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 8;   // elements that a block of the generator serves

struct DropoutArgs {
  const void* x;
  const void* residual;
  void* out;
  const int64_t* call_dev;   // NULL: `call`
  int64_t n, dim, x_stride, residual_stride, out_stride;
  int64_t call;
  uint32_t key[2];
  uint32_t dropped;          // of 65536
  float scale;
};

__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t u = uint64_t(0xD2511F53u) * c.x, v = uint64_t(0xCD9E8D57u) * c.z;
    c = make_uint4(uint32_t(v >> 32) ^ c.y ^ k0, uint32_t(v), uint32_t(u >> 32) ^ c.w ^ k1, uint32_t(u));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

struct None {};   // no residual

template <bool kAdd>
__device__ __forceinline__ float one(float x, float scale, float residual, bool keep) {
  if constexpr (kAdd) return keep ? __fmaf_rn(x, scale, residual) : residual;
  return keep ? x * scale : 0.f;   // (a select: what is dropped may be infinite or NaN)
}

// One thread: a block of the generator.  kVec: its elements are one access each (of a flat
// buffer, or within a row); otherwise element by element.
template <typename X, typename R, typename O, bool kVec>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutArgs a) {
  constexpr bool kAdd = !std::is_same_v<R, None>;
  launch_dependents();
  grid_dependency_wait();
  const int64_t b = int64_t(blockIdx.x) * kThreads + threadIdx.x, i0 = b * kBlock;
  if (i0 >= a.n) return;
  const int64_t call = a.call_dev ? *a.call_dev : a.call;
  const uint4 w4 = philox(make_uint4(uint32_t(b), uint32_t(b >> 32), uint32_t(call), uint32_t(uint64_t(call) >> 32)), a.key[0], a.key[1]);
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  auto keep = [&](int j) { return (j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu) >= a.dropped; };
  const int64_t row = i0 / a.dim, col = i0 - row * a.dim;
  if (kVec && i0 + kBlock <= a.n) {
    float f[kBlock], r[kBlock] = {};
    load_vec<X, kBlock>(static_cast<const X*>(a.x) + row * a.x_stride + col, f);
    if constexpr (kAdd) load_vec<R, kBlock>(static_cast<const R*>(a.residual) + row * a.residual_stride + col, r);
#pragma unroll
    for (int j = 0; j < kBlock; ++j) f[j] = one<kAdd>(f[j], a.scale, r[j], keep(j));
    store_vec<O, kBlock>(static_cast<O*>(a.out) + row * a.out_stride + col, f);
    return;
  }
  int64_t y = row, c = col;
#pragma unroll
  for (int j = 0; j < kBlock; ++j) {
    if (i0 + j >= a.n) break;
    float r = 0.f;
    if constexpr (kAdd) r = widen(static_cast<const R*>(a.residual)[y * a.residual_stride + c]);
    const float f = one<kAdd>(widen(static_cast<const X*>(a.x)[y * a.x_stride + c]), a.scale, r, keep(j));
    static_cast<O*>(a.out)[y * a.out_stride + c] = narrow<O>(f);
    if (++c == a.dim) {
      c = 0;
      ++y;
    }
  }
}

template <typename X, typename R, typename O>
fsp_status launch_dropout(const DropoutArgs& a, bool vec, cudaStream_t st) {
  const int64_t ctas = ((a.n + kBlock - 1) / kBlock + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return fail(FSP_EUNSUPPORTED, "too many elements");
  return launch_next(vec ? dropout_kernel<X, R, O, true> : dropout_kernel<X, R, O, false>, dim3(unsigned(ctas)), kThreads, 0, 1, a, st,
                     "dropout kernel launch");
}

template <typename X, typename O>
fsp_status launch_residual(const DropoutArgs& a, int32_t rd, bool vec, cudaStream_t st) {
  if (!a.residual) return launch_dropout<X, None, O>(a, vec, st);
  return rd == FSP_DTYPE_F32 ? launch_dropout<X, float, O>(a, vec, st) : launch_dropout<X, __nv_bfloat16, O>(a, vec, st);
}

fsp_status dropout(const void* x, int32_t xd, int64_t rows, int64_t dim, int64_t xs, double p, uint64_t seed, int64_t call,
                   const int64_t* call_dev, const void* residual, int32_t rd, int64_t rs, void* out, int32_t od, int64_t os,
                   void* stream) {
  if (rows < 0 || dim < 0) return fail(FSP_EINVAL, "rows and dim must be >= 0");
  if (!(p >= 0.0 && p <= 1.0)) return fail(FSP_EINVAL, "p must be within 0 and 1");
  fsp_status s = check_form(x, rows, dim, xs, xd, "x");
  if (s == FSP_OK && residual) s = check_form(residual, rows, dim, rs, rd, "residual");
  if (s == FSP_OK) s = check_form(out, rows, dim, os, od, "out");
  if (s == FSP_OK && reinterpret_cast<uintptr_t>(call_dev) % 8) s = fail(FSP_EINVAL, "call_dev is not 8-byte aligned");
  if (s != FSP_OK || rows == 0 || dim == 0) return s;
  const Operand to = rows_operand(out, rows, dim, os, od, "out");
  const Operand ins[] = {rows_operand(x, rows, dim, xs, xd, "x"), rows_operand(residual, rows, dim, rs, rd, "residual"),
                         {call_dev, call_dev ? size_t(8) : 0, "call_dev"}};
  s = check_operands(&to, 1, ins, 3);
  if (s != FSP_OK) return s;
  DropoutArgs a{x, residual, out, call_dev, rows * dim, dim, xs, rs, os, call, {uint32_t(seed), uint32_t(seed >> 32)}, 0, 0.f};
  a.dropped = uint32_t(p * 65536.0 + 0.5);
  a.scale = a.dropped < 65536u ? float(65536.0 / double(65536u - a.dropped)) : 0.f;
  // rows without gaps are one flat row
  if (rows == 1 || (xs == dim && os == dim && (!residual || rs == dim))) a.dim = a.n;
  const bool aligned = rows_fit(x, 0, xd, kBlock) && rows_fit(out, 0, od, kBlock) && (!residual || rows_fit(residual, 0, rd, kBlock));
  const bool vec = aligned && (a.dim == a.n || (dim % kBlock == 0 && rows_fit(x, xs, xd, kBlock) && rows_fit(out, os, od, kBlock) &&
                                                (!residual || rows_fit(residual, rs, rd, kBlock))));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (xd == FSP_DTYPE_F32)
    return od == FSP_DTYPE_F32 ? launch_residual<float, float>(a, rd, vec, st) : launch_residual<float, B>(a, rd, vec, st);
  return od == FSP_DTYPE_F32 ? launch_residual<B, float>(a, rd, vec, st) : launch_residual<B, B>(a, rd, vec, st);
}

}  // namespace
}  // namespace fsp

extern "C" fsp_status fsp_dropout(const void* x, int32_t x_dtype, int64_t rows, int64_t dim, int64_t x_stride, double p,
                                  uint64_t seed, int64_t call, const int64_t* call_dev, const void* residual,
                                  int32_t residual_dtype, int64_t residual_stride, void* out, int32_t out_dtype,
                                  int64_t out_stride, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::dropout(x, x_dtype, rows, dim, x_stride, p, seed, call, call_dev, residual, residual_dtype,
                        residual_stride, out, out_dtype, out_stride, cuda_stream);
  });
}
