// Dropout from a counter-based generator, onto a residual stream (sm_103a).
//
//   T = round(65536 p), y_i = (u_i < T ? 0 : x_i 65536 / (65536 - T)) + residual_i
//
// u_i: the i-th 16 bits of Philox-4x32 with ten rounds (J. K. Salmon, M. A. Moraes,
// R. O. Dror, D. E. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011), keyed
// by the seed, its counter (i / 8, call).  The mask is a function of (seed, call, i) and is
// never stored: the gradient is the same function of dy, without the residual.
//
// Bound: HBM (2^26 bf16 elements onto a residual 57 us, 1.03 of the measured copy; without one 44
// us, 0.90, where issue slots count too).  Sixteen bits an element, so that ten rounds (a block of
// four words) serve eight elements; with 32 the generator alone would take as long as the memory.
#include <type_traits>

#include "fsp_rows.cuh"

namespace fsp {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 8;   // elements that a block of the generator serves
constexpr int kRounds = 10;

struct DropoutArgs {
  const void* x;
  const void* residual;
  void* out;
  const int64_t* call_dev;   // NULL: `call`
  int64_t n, dim, x_stride, residual_stride, out_stride;
  int64_t call;
  uint32_t key[kRounds][2];  // of each round
  uint32_t dropped;          // T
  float scale;
};

__device__ __forceinline__ void philox(uint32_t (&c)[4], const DropoutArgs& a) {
#pragma unroll
  for (int round = 0; round < kRounds; ++round) {
    const uint64_t u = uint64_t(0xD2511F53u) * c[0], v = uint64_t(0xCD9E8D57u) * c[2];
    c[0] = uint32_t(v >> 32) ^ c[1] ^ a.key[round][0];
    c[2] = uint32_t(u >> 32) ^ c[3] ^ a.key[round][1];
    c[1] = uint32_t(v);
    c[3] = uint32_t(u);
  }
}

struct None {};   // no residual

template <bool kAdd>
__device__ __forceinline__ float one(float x, float scale, float residual, bool keep) {
  if constexpr (kAdd) return keep ? __fmaf_rn(x, scale, residual) : residual;
  return keep ? x * scale : 0.f;   // (a select: what is dropped may be infinite or NaN)
}

enum Shape { kFlat, kRows, kAny };   // blocks that are one access each: of a flat buffer, or within its rows; any other

// A thread: kPer blocks of the generator, kThreads apart.  The loads of all of them come first
// and none waits for the generator.  (CTAs that stay and prefetch: 2^26 bf16 elements 50 to 57
// us, with a residual 64 to 79.)
template <typename X, typename R, typename O, Shape kShape, int kPer>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutArgs a) {
  constexpr bool kAdd = !std::is_same_v<R, None>;
  using RT = std::conditional_t<kAdd, R, float>;
  launch_dependents();
  grid_dependency_wait();
  const int64_t first = int64_t(blockIdx.x) * (kThreads * kPer) + threadIdx.x;
  const int64_t call = a.call_dev ? *a.call_dev : a.call;
  const X* x = static_cast<const X*>(a.x);
  const RT* residual = static_cast<const RT*>(a.residual);
  O* out = static_cast<O*>(a.out);
  // element i's place, by a row stride
  auto place = [&](int64_t i, int64_t stride) { return kShape == kFlat ? i : i / a.dim * stride + i % a.dim; };
  alignas(32) X xs[kPer][kBlock];
  alignas(32) RT rs[kPer][kBlock];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i0 = (first + k * kThreads) * kBlock;
    if (kShape != kAny && i0 + kBlock <= a.n) {
      load_raw<X, kBlock>(x + place(i0, a.x_stride), xs[k]);
      if constexpr (kAdd) load_raw<RT, kBlock>(residual + place(i0, a.residual_stride), rs[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t b = first + k * kThreads, i0 = b * kBlock;
    if (i0 >= a.n) return;
    uint32_t w[4] = {uint32_t(b), uint32_t(uint64_t(b) >> 32), uint32_t(call), uint32_t(uint64_t(call) >> 32)};
    philox(w, a);
    auto keep = [&](int j) { return (j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu) >= a.dropped; };
    if (kShape != kAny && i0 + kBlock <= a.n) {
      float f[kBlock];
#pragma unroll
      for (int j = 0; j < kBlock; ++j) f[j] = one<kAdd>(widen(xs[k][j]), a.scale, kAdd ? widen(rs[k][j]) : 0.f, keep(j));
      store_vec<O, kBlock>(out + place(i0, a.out_stride), f);
    } else {
#pragma unroll
      for (int j = 0; j < kBlock; ++j) {
        const int64_t i = i0 + j;
        if (i >= a.n) break;
        float r = 0.f;
        if constexpr (kAdd) r = widen(residual[place(i, a.residual_stride)]);
        out[place(i, a.out_stride)] = narrow<O>(one<kAdd>(widen(x[place(i, a.x_stride)]), a.scale, r, keep(j)));
      }
    }
  }
}

// With a residual a thread takes four blocks from this many elements on (bf16, us, one block
// and four: 2^22 5.7 and 6.1, 2^23 9.6 and 9.3, 2^24 17.2 and 15.9, 2^26 63.0 and 57.2); without
// one a block (2^24 12.4 and 13.8, 2^26 44.0 and 46.0).
constexpr int64_t kManyElements = int64_t(1) << 23;

template <typename X, typename R, typename O, Shape kShape, int kPer>
fsp_status launch_blocks(const DropoutArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.n + kBlock - 1) / kBlock, ctas = (blocks + kThreads * kPer - 1) / (kThreads * kPer);
  if (ctas > INT32_MAX) return fail(FSP_EUNSUPPORTED, "too many elements");
  return launch_next(dropout_kernel<X, R, O, kShape, kPer>, dim3(unsigned(ctas)), kThreads, 0, 1, a, st, "dropout kernel launch");
}

template <typename X, typename R, typename O>
fsp_status launch_dropout(const DropoutArgs& a, Shape shape, cudaStream_t st) {
  if (shape == kAny) return launch_blocks<X, R, O, kAny, 1>(a, st);
  if constexpr (!std::is_same_v<R, None>)
    if (a.n >= kManyElements) return shape == kFlat ? launch_blocks<X, R, O, kFlat, 4>(a, st) : launch_blocks<X, R, O, kRows, 4>(a, st);
  return shape == kFlat ? launch_blocks<X, R, O, kFlat, 1>(a, st) : launch_blocks<X, R, O, kRows, 1>(a, st);
}

template <typename X, typename O>
fsp_status launch_residual(const DropoutArgs& a, int32_t rd, Shape shape, cudaStream_t st) {
  if (!a.residual) return launch_dropout<X, None, O>(a, shape, st);
  return rd == FSP_DTYPE_F32 ? launch_dropout<X, float, O>(a, shape, st) : launch_dropout<X, __nv_bfloat16, O>(a, shape, st);
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
  DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.out = out;
  a.call_dev = call_dev;
  a.n = rows * dim;
  a.dim = dim;
  a.x_stride = xs;
  a.residual_stride = rs;
  a.out_stride = os;
  a.call = call;
  uint32_t key[2] = {uint32_t(seed), uint32_t(seed >> 32)};
  for (auto& k : a.key) {
    k[0] = key[0];
    k[1] = key[1];
    key[0] += 0x9E3779B9u;
    key[1] += 0xBB67AE85u;
  }
  a.dropped = uint32_t(p * 65536.0 + 0.5);
  a.scale = a.dropped < 65536u ? float(65536.0 / double(65536u - a.dropped)) : 0.f;
  const bool flat = rows == 1 || (xs == dim && os == dim && (!residual || rs == dim));   // no gaps between the rows
  auto fits = [&](int64_t fx, int64_t fo, int64_t fr) {
    return rows_fit(x, fx, xd, kBlock) && rows_fit(out, fo, od, kBlock) && (!residual || rows_fit(residual, fr, rd, kBlock));
  };
  const Shape shape = flat && fits(0, 0, 0) ? kFlat : dim % kBlock == 0 && fits(xs, os, rs) ? kRows : kAny;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (xd == FSP_DTYPE_F32)
    return od == FSP_DTYPE_F32 ? launch_residual<float, float>(a, rd, shape, st) : launch_residual<float, B>(a, rd, shape, st);
  return od == FSP_DTYPE_F32 ? launch_residual<B, float>(a, rd, shape, st) : launch_residual<B, B>(a, rd, shape, st);
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
