// Matrices in 8-bit floating point with a scale per block of 128 along the
// summed axis, and their product (sm_103a).
//
//   s = 2^e, e = min{e: 448 s >= max|x|};  code = e4m3(x / s)
//   C = sum_k (code_a s_a) (code_b s_b), summed in fp32
//
// A power of two loses no bit of a value, so the codes and the sum are those
// that exact arithmetic on the inputs gives, up to the order of the fp32 sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cfloat>
#include <map>
#include <mutex>
#include <string>
#include <utility>

#include "fsp_host.h"
#include "fsp_internal.h"
#include "fsp_ops.h"

namespace fsp {
namespace {

constexpr int kTileBytes = 128 * 128;              // 128 rows x one block of codes
constexpr int kScaleBytes = 128 * 4;               // 128 rows x four blocks' scales

}  // namespace
}  // namespace fsp

#include "fsp_fp8_mma.cuh"

namespace fsp {
namespace {

// Where a matrix's parts lie (the layout fsp_ops.h states).
struct Fp8Layout {
  int64_t row_tiles, blocks, pieces;   // rows / 128, cols / 128, cols / 512, rounded up
  int64_t scale_offset, bytes;
};
__host__ __device__ __forceinline__ Fp8Layout layout_of(int64_t rows, int64_t cols) {
  Fp8Layout l;
  l.row_tiles = (rows + 127) / 128;
  l.blocks = (cols + 127) / 128;
  l.pieces = (cols + 511) / 512;
  l.scale_offset = l.row_tiles * l.blocks * kTileBytes;
  l.bytes = l.scale_offset + l.row_tiles * l.pieces * kScaleBytes;
  return l;
}
// Row r's 16-byte piece p (of 8) within a tile; row r's scale of block k within a piece.
__host__ __device__ __forceinline__ int code_at(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }
__host__ __device__ __forceinline__ int scale_at(int r, int k) { return (r & 31) * 16 + (r >> 5) * 4 + k; }

// ---- quantisation ------------------------------------------------------------------

constexpr int kQuantThreads = 256;

struct QuantArgs {
  const void* x;
  uint8_t* out;
  int64_t rows, cols, stride;
  Fp8Layout l;
  int64_t row_tile;   // of 128 rows, that x's first row begins
};

// The biased exponent of a block's scale from the bits of its largest
// magnitude: p - 8 for f 2^p with f <= 1.75 (448 = 1.75 x 2^8), else p - 7.
__device__ __forceinline__ int scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255;
  const int b = int(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(b, 0);   // 2^-127 at least (a zero or subnormal largest value too)
}
// 1 / s of a scale byte below 255: 2^(127 - byte), a normal number.
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float(uint32_t(254 - min(byte, 253)) << 23); }

__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ uint4 codes16(const float* x, float inv) {
  return make_uint4(codes4(x, inv), codes4(x + 4, inv), codes4(x + 8, inv), codes4(x + 12, inv));
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// V elements of a row from column c, as they are stored; zeros past the last one.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int64_t c, int64_t cols, bool vec, T* x) {
  if (vec && c + V <= cols) {
#pragma unroll
    for (int k = 0; k < V * int(sizeof(T)) / 16; ++k) reinterpret_cast<uint4*>(x)[k] = reinterpret_cast<const uint4*>(row + c)[k];
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = c + j < cols ? row[c + j] : T(0.f);
  }
}

// The bits of the largest magnitude of V values, as fp32; NaN above all.  bf16: two
// at a time, their magnitudes order as 16-bit numbers.
template <typename T, int V>
__device__ __forceinline__ uint32_t largest(const T* x) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) top = __vmaxu2(top, w[j] & 0x7fff7fffu);
    return max(top << 16, top & 0xffff0000u);
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    return top;
  }
}

// Blocks along the rows of x: a warp per row and four blocks, eight lanes of
// 16 elements per block, two rows at a time; the rows of a CTA follow each other,
// so that each of the four tiles that it writes gets one run of bytes.
constexpr int kRowsPerWarp = 2;
constexpr int kRowsPerCta = kRowsPerWarp * kQuantThreads / 32;

template <typename T>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const __grid_constant__ QuantArgs a, bool vec) {
  launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t piece = blockIdx.x;
  const int64_t row0 = int64_t(blockIdx.y) * kRowsPerCta + (threadIdx.x >> 5) * kRowsPerWarp;
  const int64_t block = piece * 4 + (lane >> 3);
  alignas(16) T x[kRowsPerWarp][16];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i)
    if (row0 + i < a.rows)
      load_row<T, 16>(static_cast<const T*>(a.x) + (row0 + i) * a.stride, piece * 512 + lane * 16, a.cols, vec, x[i]);
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) {
    const int64_t row = row0 + i;
    if (row >= a.rows) return;   // the whole warp
    uint32_t top = largest<T, 16>(x[i]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int s = scale_byte(top);
    const int r = int(row & 127);
    const int64_t tile = a.row_tile + (row >> 7);
    float f[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = widen(x[i][j]);
    if (block < a.l.blocks)
      *reinterpret_cast<uint4*>(a.out + (tile * a.l.blocks + block) * kTileBytes + code_at(r, lane & 7)) =
          codes16(f, inverse_scale(s));
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) word |= uint32_t(__shfl_sync(0xffffffffu, s, k * 8)) << (8 * k);
    if (lane == 0)
      *reinterpret_cast<uint32_t*>(a.out + a.l.scale_offset + (tile * a.l.pieces + piece) * kScaleBytes +
                                   scale_at(r, 0)) = word;
  }
}

// Blocks along the columns of x (the transpose's rows), and where `out` is given
// those along its rows too: a CTA per 128 x 128 tile, read once into shared
// memory.  Rows: 16 lanes of eight elements each, on the way in.  Columns: a
// thread takes two neighbouring columns and a quarter of their block; its codes
// go back through shared memory, laid out as the transpose's tile, so that the
// tile is written as one run of 16 KB.
template <typename T>
struct ColsSmem {
  static constexpr int kPitch = 128 + 16 / int(sizeof(T));   // elements
  T x[128][kPitch];
  uint32_t tops[4][128];
};
static_assert(sizeof(ColsSmem<__nv_bfloat16>) >= kTileBytes, "the codes take the tile's place");

template <typename T>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 4 : 2)
    quantize_cols_kernel(const __grid_constant__ QuantArgs a, uint8_t* out, Fp8Layout l, bool vec) {
  extern __shared__ __align__(16) unsigned char raw[];
  launch_dependents();
  grid_dependency_wait();
  ColsSmem<T>& sm = *reinterpret_cast<ColsSmem<T>*>(raw);
  const int tid = threadIdx.x;
  const int64_t c0 = int64_t(blockIdx.x) * 128, r0 = int64_t(blockIdx.y) * 128;
  {
    const int c = (tid & 15) * 8, first = tid >> 4;
    const bool rows = out != nullptr;
    alignas(16) T x[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + first + 16 * i;
      if (row < a.rows) {
        load_row<T, 8>(static_cast<const T*>(a.x) + row * a.stride, c0 + c, a.cols, vec, x[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = T(0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = first + 16 * i;
#pragma unroll
      for (int k = 0; k < int(sizeof(T)) / 2; ++k)
        reinterpret_cast<uint4*>(&sm.x[r][c])[k] = reinterpret_cast<const uint4*>(x[i])[k];
      if (rows) {
        uint32_t top = largest<T, 8>(x[i]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (r0 + r < a.rows) {
          const int s = scale_byte(top);
          const float inv = inverse_scale(s);
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = widen(x[i][j]);
          *reinterpret_cast<uint2*>(out + (int64_t(blockIdx.y) * l.blocks + blockIdx.x) * kTileBytes + code_at(r, c >> 4) +
                                    (c & 8)) = make_uint2(codes4(f, inv), codes4(f + 4, inv));
          if (c == 0)
            out[l.scale_offset + (int64_t(blockIdx.y) * l.pieces + (blockIdx.x >> 2)) * kScaleBytes +
                scale_at(r, int(blockIdx.x & 3))] = uint8_t(s);
        }
      }
    }
  }
  __syncthreads();
  const int c = (tid & 63) * 2, q = tid >> 6;   // two columns, a quarter of their block
  alignas(8) T two[32][2];
  uint32_t top[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<uint2*>(two[j]) = *reinterpret_cast<const uint2*>(&sm.x[q * 32 + j][c]);
    else
      *reinterpret_cast<uint32_t*>(two[j]) = *reinterpret_cast<const uint32_t*>(&sm.x[q * 32 + j][c]);
  }
  if constexpr (sizeof(T) == 2) {
    uint32_t both = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) both = __vmaxu2(both, *reinterpret_cast<const uint32_t*>(two[j]) & 0x7fff7fffu);
    top[0] = both << 16;
    top[1] = both & 0xffff0000u;
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) top[k] = max(top[k], __float_as_uint(two[j][k]) & 0x7fffffffu);
  }
  sm.tops[q][c] = top[0];
  sm.tops[q][c + 1] = top[1];
  __syncthreads();   // (every value of the tile is in registers: the codes may take its place)
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = c + k;   // of the transpose's tile
    const int s = scale_byte(max(max(sm.tops[0][r], sm.tops[1][r]), max(sm.tops[2][r], sm.tops[3][r])));
    const float inv = inverse_scale(s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = widen(two[16 * h + j][k]);
      *reinterpret_cast<uint4*>(raw + code_at(r, 2 * q + h)) = codes16(f, inv);
    }
    if (q == 0 && c0 + r < a.cols)
      a.out[a.l.scale_offset + (int64_t(blockIdx.x) * a.l.pieces + (blockIdx.y >> 2)) * kScaleBytes +
            scale_at(r, int(blockIdx.y & 3))] = uint8_t(s);
  }
  __syncthreads();
  uint4* dst = reinterpret_cast<uint4*>(a.out + (int64_t(blockIdx.x) * a.l.blocks + blockIdx.y) * kTileBytes);
  const int n = int(min(int64_t(128), a.cols - c0)) * 8;   // 16-byte pieces of the rows that exist
#pragma unroll
  for (int i = 0; i < kTileBytes / 16 / kQuantThreads; ++i) {
    const int at = i * kQuantThreads + tid;
    if (at < n) dst[at] = reinterpret_cast<const uint4*>(raw)[at];
  }
}

__device__ __forceinline__ float scale_value(uint8_t b) {
  return __uint_as_float(b == 255 ? 0x7fffffffu : b ? uint32_t(b) << 23 : 0x00400000u);
}
__device__ __forceinline__ float code_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__global__ void __launch_bounds__(kQuantThreads) values_kernel(const uint8_t* q, int64_t rows, int64_t cols,
                                                               Fp8Layout l, float* out) {
  const int64_t i = int64_t(blockIdx.x) * kQuantThreads + threadIdx.x;
  if (i >= rows * cols) return;
  const int64_t row = i / cols, col = i % cols;
  const int r = int(row & 127), k = int(col & 127);
  const int64_t tile = row >> 7, block = col >> 7;
  const uint8_t code = q[(tile * l.blocks + block) * kTileBytes + code_at(r, k >> 4) + (k & 15)];
  const uint8_t s = q[l.scale_offset + (tile * l.pieces + (block >> 2)) * kScaleBytes + scale_at(r, int(block & 3))];
  out[i] = code_value(code) * scale_value(s);
}

// ---- few rows times a matrix ----------------------------------------------------------
//
// Up to four rows of x: the product is bound by the bytes of w, read once, and a
// tensor-core tile would be mostly empty.  A CTA quantises x for itself (its codes'
// values go to shared memory as fp32) and takes 16 rows of w at a time; its eight
// warps share out the blocks of k.  A lane holds one 16-byte piece of a block
// for four rows of w (rows r, r + 4, ...), so that a warp's load is 512 bytes of
// a tile in a run, and x's 16 values serve four rows.  The eight lanes of a row,
// then the eight warps, are added in a fixed order.
//
// A sum of 16 values of x times codes of w is below 2^22 of x's scale, and w's scale
// comes after it: with a scale of x above 2^104 the sum could leave fp32's range where
// what it stands for does not.  The values of such a block are kept 2^16 smaller and
// w's scale takes the factor.  A CTA without such a block runs a form without factors
// (4 x 5632 x 4096 30 us; with a factor at every block 33).
constexpr int kFewThreads = 256;
constexpr int kFewRows = 16;             // of w, per CTA and turn
constexpr int64_t kFewSmem = 64 * 1024;  // of x's values, at most

struct FewArgs {
  const void* x;
  const uint8_t* w;
  void* y;
  int64_t cols, x_stride, n, y_stride;
  Fp8Layout l;   // of w
  int rows;
};

__device__ __forceinline__ void values16(uint4 c, float* f) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
}

// All rows of w of this CTA; kFactors: with the factors of x's blocks.
template <int M, typename O, bool kFactors>
__device__ __forceinline__ void few_rows_of_w(const FewArgs& a, float* xv) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t width = a.l.blocks * 128;
  float* factors = xv + M * width;
  float* part = factors + M * a.l.blocks;
  const int sub = lane >> 3, p = lane & 7;
  for (int64_t n0 = int64_t(blockIdx.x) * kFewRows; n0 < a.n; n0 += int64_t(gridDim.x) * kFewRows) {
    const int64_t tile = n0 >> 7;
    const int r0 = int(n0 & 127) + sub;
    float acc[4][M];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m) acc[i][m] = 0.f;
    for (int64_t block = warp; block < a.l.blocks; block += kFewThreads / 32) {
      const uint8_t* src = a.w + (tile * a.l.blocks + block) * kTileBytes;
      const uint8_t* scales = a.w + a.l.scale_offset + (tile * a.l.pieces + (block >> 2)) * kScaleBytes;
      uint4 c[4];
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = *reinterpret_cast<const uint4*>(src + code_at(r0 + 4 * i, p));
        s[i] = scale_value(scales[scale_at(r0 + 4 * i, int(block & 3))]);
      }
      float x[M][16];
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(&x[m][4 * j]) = *reinterpret_cast<const float4*>(xv + m * width + block * 128 + p * 16 + 4 * j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[16], sum[M];
        values16(c[i], f);
#pragma unroll
        for (int m = 0; m < M; ++m) sum[m] = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int m = 0; m < M; ++m) sum[m] = fmaf(f[j], x[m][j], sum[m]);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          float t = s[i];
          if constexpr (kFactors) {
            // (beyond fp32 its largest number serves: any sum but 0 times that is infinite, and 0 stays 0)
            t *= factors[m * a.l.blocks + block];
            if (t > FLT_MAX) t = FLT_MAX;
          }
          acc[i][m] = fmaf(sum[m], t, acc[i][m]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < M; ++m) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) acc[i][m] += __shfl_xor_sync(0xffffffffu, acc[i][m], o);
        if (p == 0) part[(warp * kFewRows + sub + 4 * i) * M + m] = acc[i][m];
      }
    __syncthreads();
    const int r = threadIdx.x / M, m = threadIdx.x % M;
    if (r < kFewRows && n0 + r < a.n && m < a.rows) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kFewThreads / 32; ++w) sum += part[(w * kFewRows + r) * M + m];
      O* y = static_cast<O*>(a.y) + m * a.y_stride + n0 + r;
      if constexpr (sizeof(O) == 4)
        *y = sum;
      else
        *y = __float2bfloat16_rn(sum);
    }
    __syncthreads();
  }
}
// Out of line: beside it in one function the usual form was slower (1 x 151936 x 1024 46 us, so 40).
template <int M, typename O>
__device__ __noinline__ void few_rows_with_factors(const FewArgs& a, float* xv) {
  few_rows_of_w<M, O, true>(a, xv);
}

// (One row: registers for four CTAs per SM, with three 1 x 151936 x 1024 takes 51 us.)
template <int M, typename T, typename O>
__global__ void __launch_bounds__(kFewThreads, M == 1 ? 4 : 2) few_rows_kernel(const __grid_constant__ FewArgs a) {
  extern __shared__ float xv[];   // [M][blocks * 128], then [M][blocks] factors, then [8 warps][16][M]
  launch_dependents();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t width = a.l.blocks * 128;
  float* factors = xv + M * width;
  bool huge = false;
  for (int64_t b = warp; b < a.l.blocks * M; b += kFewThreads / 32) {
    const int64_t m = b / a.l.blocks, block = b % a.l.blocks, c = block * 128 + lane * 4;
    const T* row = static_cast<const T*>(a.x) + m * a.x_stride;
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = m < a.rows && c + j < a.cols ? widen(row[c + j]) : 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
    const int s = scale_byte(__reduce_max_sync(0xffffffffu, top));
    const uint32_t codes = codes4(f, inverse_scale(s));
    const bool far = s > 127 + 104 && s < 255;
    const float scale = scale_value(uint8_t(far ? s - 16 : s));
    float4 v;
    v.x = code_value(uint8_t(codes)) * scale;
    v.y = code_value(uint8_t(codes >> 8)) * scale;
    v.z = code_value(uint8_t(codes >> 16)) * scale;
    v.w = code_value(uint8_t(codes >> 24)) * scale;
    *reinterpret_cast<float4*>(xv + m * width + c) = v;
    if (lane == 0) factors[b] = far ? 65536.f : 1.f;
    huge = huge || far;
  }
  huge = __syncthreads_or(huge);
  if (huge)
    few_rows_with_factors<M, O>(a, xv);
  else
    few_rows_of_w<M, O, false>(a, xv);
}

// ---- host ----------------------------------------------------------------------------

size_t size_of(int32_t dtype) { return dtype == FSP_DTYPE_F32 ? 4 : 2; }
constexpr int64_t kMaxDim = int64_t(1) << 30;

fsp_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FSP_OK : fail(FSP_ECUDA, cuda_msg(what, e));
}

// Launches with programmatic stream serialisation: the CTAs of a pass's next kernel
// are there when the one before it ends (every kernel here waits for that before
// it touches a buffer).
template <typename... P, typename... A>
fsp_status launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const char* what, A... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  return e == cudaSuccess ? FSP_OK : fail(FSP_ECUDA, cuda_msg(what, e));
}

fsp_status check_dims(std::initializer_list<int64_t> dims) {
  for (int64_t d : dims)
    if (d < 0 || d > kMaxDim) return fail(FSP_EINVAL, "a size is out of range");
  return FSP_OK;
}

fsp_status check_codes(const void* p, const char* name) {
  if (!p) return fail(FSP_EINVAL, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % 16) return fail(FSP_EINVAL, std::string(name) + " is not 16-byte aligned");
  return FSP_OK;
}

bool overlap(const void* p, int64_t pb, const void* q, int64_t qb) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + uintptr_t(qb) && b < a + uintptr_t(pb);
}

// A buffer of a call: NULL or 0 bytes where the call has none.
struct Range {
  const void* p;
  int64_t bytes;
  const char* name;
};
// The first `written` of the ranges against each other and all the others, then
// that each lies in a live allocation.
fsp_status check_ranges(const Range* r, int n, int written) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(r[i].p, r[i].bytes, r[j].p, r[j].bytes))
        return fail(FSP_EINVAL, std::string(r[i].name) + " overlaps " + r[j].name);
  for (int i = 0; i < n; ++i)
    if (r[i].p && r[i].bytes > 0) {
      const fsp_status s = check_allocation(r[i].p, size_t(r[i].bytes), r[i].name);
      if (s != FSP_OK) return s;
    }
  return FSP_OK;
}

template <typename T>
fsp_status run_quantize(const QuantArgs& in, void* out, void* out_t, bool vec, cudaStream_t st) {
  QuantArgs a = in;
  const Fp8Layout l = layout_of(a.rows, a.cols);
  if (out_t) {
    constexpr int kSmem = int(sizeof(ColsSmem<T>));
    const fsp_status ok = allow_kernel(reinterpret_cast<const void*>(&quantize_cols_kernel<T>), kSmem);
    if (ok != FSP_OK) return ok;
    a.out = static_cast<uint8_t*>(out_t);
    a.l = layout_of(a.cols, a.rows);
    if (a.l.blocks > 65535) return fail(FSP_EUNSUPPORTED, "the matrix is too large");
    return launch_next(quantize_cols_kernel<T>, dim3(unsigned(a.l.row_tiles), unsigned(a.l.blocks)), kQuantThreads, kSmem, st,
                       "transposing quantisation kernel launch", a, static_cast<uint8_t*>(out), l, vec);
  }
  a.out = static_cast<uint8_t*>(out);
  a.l = l;
  const int64_t ctas = (a.rows + kRowsPerCta - 1) / kRowsPerCta;
  // (the grid's second dimension holds 65535: taller matrices in several launches)
  constexpr int64_t kMost = 65535 / 8 * 8;
  for (int64_t done = 0; done < ctas; done += kMost) {
    QuantArgs part = a;
    part.x = static_cast<const T*>(a.x) + done * kRowsPerCta * a.stride;
    part.rows = std::min(a.rows - done * kRowsPerCta, kMost * kRowsPerCta);
    part.row_tile = done * kRowsPerCta / 128;
    const fsp_status s = launch_next(quantize_rows_kernel<T>, dim3(unsigned(a.l.pieces), unsigned(std::min(kMost, ctas - done))),
                                     kQuantThreads, 0, st, "quantisation kernel launch", part, vec);
    if (s != FSP_OK) return s;
  }
  return FSP_OK;
}

fsp_status check_matrix(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, const char* name) {
  if (dtype != FSP_DTYPE_F32 && dtype != FSP_DTYPE_BF16) return fail(FSP_EINVAL, std::string("unknown dtype of ") + name);
  if (stride < cols || (rows > 0 && stride > (int64_t(1) << 58) / rows))
    return fail(FSP_EINVAL, std::string(name) + "'s rows overlap or their stride is out of range");
  if (rows == 0 || cols == 0) return FSP_OK;
  if (!p) return fail(FSP_EINVAL, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % size_of(dtype))
    return fail(FSP_EINVAL, std::string(name) + " is not aligned to its elements");
  return FSP_OK;
}
int64_t span(int64_t rows, int64_t cols, int64_t stride, int32_t dtype) {
  return rows > 0 && cols > 0 ? ((rows - 1) * stride + cols) * int64_t(size_of(dtype)) : 0;
}

// On checked arguments: rows and cols above 0.
fsp_status quantize_checked(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, void* out, void* out_t,
                            cudaStream_t st) {
  QuantArgs a{};
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.stride = stride;
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && size_t(stride) * size_of(dtype) % 16 == 0;
  return dtype == FSP_DTYPE_F32 ? run_quantize<float>(a, out, out_t, vec, st)
                                : run_quantize<__nv_bfloat16>(a, out, out_t, vec, st);
}

fsp_status quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, void* out, void* out_t,
                    void* stream) {
  fsp_status s = check_dims({rows, cols});
  if (s == FSP_OK && rows > 0 && cols > 0 && !out && !out_t) return fail(FSP_EINVAL, "out and out_t are both NULL");
  if (s == FSP_OK) s = check_matrix(x, dtype, rows, cols, stride, "x");
  if (s != FSP_OK || rows == 0 || cols == 0) return s;
  const Fp8Layout l = layout_of(rows, cols), lt = layout_of(cols, rows);
  if (out) s = check_codes(out, "out");
  if (s == FSP_OK && out_t) s = check_codes(out_t, "out_t");
  if (s != FSP_OK) return s;
  const Range ranges[] = {{out, l.bytes, "out"}, {out_t, lt.bytes, "out_t"}, {x, span(rows, cols, stride, dtype), "x"}};
  s = check_ranges(ranges, 3, 2);
  if (s != FSP_OK) return s;
  return quantize_checked(x, dtype, rows, cols, stride, out, out_t, static_cast<cudaStream_t>(stream));
}

fsp_status values(const void* q, int64_t rows, int64_t cols, float* out, void* stream) {
  fsp_status s = check_dims({rows, cols});
  if (s != FSP_OK || rows == 0 || cols == 0) return s;
  const Fp8Layout l = layout_of(rows, cols);
  s = check_codes(q, "q");
  if (s == FSP_OK) s = check_matrix(out, FSP_DTYPE_F32, rows, cols, cols, "out");
  if (s != FSP_OK) return s;
  const Range ranges[] = {{out, rows * cols * 4, "out"}, {q, l.bytes, "q"}};
  s = check_ranges(ranges, 2, 1);
  if (s != FSP_OK) return s;
  const int64_t ctas = (rows * cols + kQuantThreads - 1) / kQuantThreads;
  if (ctas > INT32_MAX) return fail(FSP_EUNSUPPORTED, "the matrix is too large");
  values_kernel<<<unsigned(ctas), kQuantThreads, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const uint8_t*>(q), rows,
                                                                                          cols, l, out);
  return launched("8-bit values kernel launch");
}

// Whether `rows` rows of `cols` values go through few_rows_kernel.
constexpr int64_t kFewMost = 4;
bool few(int64_t rows, int64_t cols) { return rows <= kFewMost && rows * ((cols + 127) / 128 * 128) * 4 <= kFewSmem; }

template <int M, typename T, typename O>
fsp_status launch_few_of(const FewArgs& a, cudaStream_t st) {
  constexpr int kMost = int(kFewSmem) * 2 + int(kFewSmem) / 64 + 8 * kFewRows * 4 * M;   // (three rows run in the kernel of four)
  fsp_status ok = allow_kernel(reinterpret_cast<const void*>(&few_rows_kernel<M, T, O>), kMost);
  int sms = 0;
  if (ok == FSP_OK) ok = sm_count(&sms);
  if (ok != FSP_OK) return ok;
  const size_t smem = size_t(M) * size_t(a.l.blocks) * (512 + 4) + 8 * kFewRows * 4 * M;
  // x is quantised once per CTA: at most eight CTAs per SM, which then take turns
  const int64_t ctas = std::min<int64_t>((a.n + kFewRows - 1) / kFewRows, int64_t(sms) * 8);
  return launch_next(few_rows_kernel<M, T, O>, dim3(unsigned(ctas)), kFewThreads, smem, st,
                     "8-bit linear (few rows) kernel launch", a);
}
template <typename T, typename O>
fsp_status launch_few(const FewArgs& a, cudaStream_t st) {
  return a.rows == 1 ? launch_few_of<1, T, O>(a, st) : a.rows == 2 ? launch_few_of<2, T, O>(a, st) : launch_few_of<4, T, O>(a, st);
}

template <int BN, bool kSwap, typename T>
fsp_status launch_product_of(const MmArgs& g, cudaStream_t st) {
  constexpr int kSmem = MmCfg<BN>::kSmem;
  fsp_status ok = allow_kernel(reinterpret_cast<const void*>(&fp8_product_kernel<BN, kSwap, T>), kSmem);
  int sms = 0;
  if (ok == FSP_OK) ok = sm_count(&sms);
  if (ok != FSP_OK) return ok;
  const unsigned grid = unsigned(std::min<int64_t>(sms, g.tiles_p * g.tiles_q));
  return launch_next(fp8_product_kernel<BN, kSwap, T>, dim3(grid), kMmThreads, kSmem, st, "8-bit product kernel launch", g);
}

template <int BN, bool kSwap>
fsp_status launch_product(MmArgs& g, int32_t dtype, cudaStream_t st) {
  g.tiles_q = (g.nq + BN - 1) / BN;
  return dtype == FSP_DTYPE_F32 ? launch_product_of<BN, kSwap, float>(g, st)
                                : launch_product_of<BN, kSwap, __nv_bfloat16>(g, st);
}

// Pairs of CTAs that can run at one time: a pair's SMs share a GPC, so this can be
// fewer than half of the SMs, and a pair that had to wait for others to finish
// would double a launch's time.
template <typename T>
fsp_status resident_pairs(int* pairs) {
  static std::mutex mu;
  static std::map<int, int> known;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FSP_ECUDA, cuda_msg("cudaGetDevice", e));
  fsp_status s = allow_kernel(reinterpret_cast<const void*>(&fp8_pair_kernel<T>), PairCfg::kSmem);
  if (s == FSP_OK) s = sm_count(&sms);
  if (s != FSP_OK) return s;
  std::lock_guard<std::mutex> lock(mu);
  int& n = known[dev];
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(sms / 2 * 2));
    cfg.blockDim = dim3(PairCfg::kThreads);
    cfg.dynamicSmemBytes = PairCfg::kSmem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, fp8_pair_kernel<T>, &cfg);
    if (e != cudaSuccess || n < 1) {
      n = 0;
      return fail(FSP_ECUDA, cuda_msg("cudaOccupancyMaxActiveClusters", e));
    }
  }
  *pairs = n;
  return FSP_OK;
}

// `n` tiles of `rows` x 128 bytes, one after the other from `base`, as a tensor whose
// box is a tile.
fsp_status tile_map(const uint8_t* base, int64_t n, int rows, CUtensorMap* map) {
  static const auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(driver_function("cuTensorMapEncodeTiled"));
  if (!encode) return fail(FSP_ECUDA, "cannot resolve cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {128, cuuint64_t(rows), cuuint64_t(n)}, strides[2] = {128, cuuint64_t(rows) * 128};
  const cuuint32_t box[3] = {128, cuuint32_t(rows), 1}, steps[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FSP_OK : fail(FSP_ECUDA, "cuTensorMapEncodeTiled: error " + std::to_string(int(r)));
}

template <typename T>
fsp_status launch_pairs_of(const MmArgs& g, cudaStream_t st) {
  int pairs = 0;
  PairArgs a{};
  a.g = g;
  const int64_t rows_p = (g.np + 127) / 128, rows_q = (g.nq + 127) / 128;
  fsp_status s = resident_pairs<T>(&pairs);
  // (tile numbers fit 32 bits: 2^31 tiles of 16 KB are more than any device holds)
  if (s == FSP_OK) s = tile_map(g.p, rows_p * g.blocks, 128, &a.p);
  if (s == FSP_OK) s = tile_map(g.q, rows_q * g.blocks, 128, &a.q);
  if (s == FSP_OK) s = tile_map(g.p + g.p_scales, rows_p * g.pieces, 4, &a.p_scales);
  if (s == FSP_OK) s = tile_map(g.q + g.q_scales, rows_q * g.pieces, 4, &a.q_scales);
  if (s != FSP_OK) return s;
  const unsigned grid = unsigned(2 * std::min<int64_t>(pairs, g.tiles_p * g.tiles_q));
  return launch_next(fp8_pair_kernel<T>, dim3(grid), PairCfg::kThreads, PairCfg::kSmem, st, "8-bit product kernel launch", a);
}

fsp_status launch_pairs(MmArgs& g, int32_t dtype, cudaStream_t st) {
  g.tiles_p = (g.np + PairCfg::kTile - 1) / PairCfg::kTile;
  g.tiles_q = (g.nq + PairCfg::kTile - 1) / PairCfg::kTile;
  return dtype == FSP_DTYPE_F32 ? launch_pairs_of<float>(g, st) : launch_pairs_of<__nv_bfloat16>(g, st);
}

// On checked arguments: m, n and k above 0.
fsp_status matmul_checked(const void* a, const void* b, int64_t m, int64_t n, int64_t k, void* c, int32_t dtype,
                          int64_t c_stride, bool accumulate, cudaStream_t st) {
  const Fp8Layout la = layout_of(m, k), lb = layout_of(n, k);
  // Up to 128 rows of a: b's rows fill the 128 rows of the tiles, a's their columns.
  const bool swap = m <= 128;
  MmArgs g{};
  g.p = static_cast<const uint8_t*>(swap ? b : a);
  g.q = static_cast<const uint8_t*>(swap ? a : b);
  g.c = c;
  g.np = swap ? n : m;
  g.nq = swap ? m : n;
  g.blocks = la.blocks;
  g.pieces = la.pieces;
  g.p_scales = (swap ? lb : la).scale_offset;
  g.q_scales = (swap ? la : lb).scale_offset;
  g.c_stride = c_stride;
  g.accumulate = accumulate;
  g.vec = reinterpret_cast<uintptr_t>(c) % 16 == 0 && size_t(c_stride) * size_of(dtype) % 16 == 0;
  g.tiles_p = (g.np + kTileP - 1) / kTileP;
  if (m <= 16) return launch_product<16, true>(g, dtype, st);
  if (m <= 32) return launch_product<32, true>(g, dtype, st);
  if (m <= 64) return launch_product<64, true>(g, dtype, st);
  if (m <= 128) return launch_product<128, true>(g, dtype, st);
  // The narrowest tiles that give every SM at most one: a product too small to fill
  // the pairs spreads over more SMs (1024 x 2048 x 2048: tiles of 128 8.0 us, pairs
  // 8.7; 333 x 1001 x 777: tiles of 64 5.0, of 128 6.1, pairs 7.5), a larger one
  // gains from them (2048 x 2048 x 2048: pairs 9.3, tiles of 128 13.2).
  int sms = 0;
  const fsp_status s = sm_count(&sms);
  if (s != FSP_OK) return s;
  if (g.tiles_p * ((n + 63) / 64) <= sms) return launch_product<64, false>(g, dtype, st);
  if (g.tiles_p * ((n + 127) / 128) <= sms) return launch_product<128, false>(g, dtype, st);
  return launch_pairs(g, dtype, st);
}

fsp_status sum_of_nothing(int64_t m, int64_t n, void* c, int32_t dtype, int64_t c_stride, cudaStream_t st) {
  const cudaError_t e = cudaMemset2DAsync(c, size_t(c_stride) * size_of(dtype), 0, size_t(n) * size_of(dtype), size_t(m), st);
  return e == cudaSuccess ? FSP_OK : fail(FSP_ECUDA, cuda_msg("cudaMemset2DAsync", e));
}

fsp_status matmul(const void* a, const void* b, int64_t m, int64_t n, int64_t k, void* c, int32_t dtype,
                  int64_t c_stride, int32_t accumulate, void* stream) {
  fsp_status s = check_dims({m, n, k});
  if (s != FSP_OK) return s;
  if (accumulate && dtype == FSP_DTYPE_BF16) return fail(FSP_EUNSUPPORTED, "accumulate adds to fp32 only");
  s = check_matrix(c, dtype, m, n, c_stride, "c");
  if (s != FSP_OK || m == 0 || n == 0) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (k == 0) {
    const Range ranges[] = {{c, span(m, n, c_stride, dtype), "c"}};
    s = check_ranges(ranges, 1, 1);
    return s != FSP_OK || accumulate ? s : sum_of_nothing(m, n, c, dtype, c_stride, st);
  }
  const Fp8Layout la = layout_of(m, k), lb = layout_of(n, k);
  s = check_codes(a, "a");
  if (s == FSP_OK) s = check_codes(b, "b");
  if (s != FSP_OK) return s;
  const Range ranges[] = {{c, span(m, n, c_stride, dtype), "c"}, {a, la.bytes, "a"}, {b, lb.bytes, "b"}};
  s = check_ranges(ranges, 3, 1);
  if (s != FSP_OK) return s;
  return matmul_checked(a, b, m, n, k, c, dtype, c_stride, accumulate != 0, st);
}

// ---- the linear layer ---------------------------------------------------------------

int64_t round256(int64_t x) { return (x + 255) / 256 * 256; }

int64_t forward_workspace(int64_t rows, int64_t in, int64_t out) {
  return rows == 0 || in == 0 || out == 0 || few(rows, in) ? 0 : round256(layout_of(rows, in).bytes);
}
int64_t backward_workspace(int64_t rows, int64_t in, int64_t out) {
  if (rows == 0 || in == 0 || out == 0) return 0;
  return round256(layout_of(rows, out).bytes) + round256(layout_of(out, rows).bytes) + round256(layout_of(in, rows).bytes);
}

fsp_status check_workspace(const void* p, size_t bytes, int64_t want) {
  if (want == 0) return FSP_OK;
  if (!p) return fail(FSP_EINVAL, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(p) % 16) return fail(FSP_EINVAL, "workspace is not 16-byte aligned");
  if (bytes < size_t(want)) return fail(FSP_EINVAL, "workspace is smaller than fsp_fp8_linear_workspace_bytes");
  return FSP_OK;
}

fsp_status linear(const void* x, int32_t xd, int64_t rows, int64_t in, int64_t xs, const void* w, int64_t out, void* y,
                  int32_t yd, int64_t ys, void* workspace, size_t workspace_bytes, void* stream) {
  fsp_status s = check_dims({rows, in, out});
  if (s == FSP_OK) s = check_matrix(x, xd, rows, in, xs, "x");
  if (s == FSP_OK) s = check_matrix(y, yd, rows, out, ys, "y");
  if (s != FSP_OK || rows == 0 || out == 0) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Fp8Layout lw = layout_of(out, in);
  const int64_t want = forward_workspace(rows, in, out);
  if (in > 0) s = check_codes(w, "w");
  if (s == FSP_OK) s = check_workspace(workspace, workspace_bytes, want);
  if (s != FSP_OK) return s;
  const Range ranges[] = {{y, span(rows, out, ys, yd), "y"},
                          {workspace, want, "workspace"},
                          {x, span(rows, in, xs, xd), "x"},
                          {w, lw.bytes, "w"}};
  s = check_ranges(ranges, 4, 2);
  if (s != FSP_OK) return s;
  if (in == 0) return sum_of_nothing(rows, out, y, yd, ys, st);
  if (few(rows, in)) {
    const FewArgs a{x, static_cast<const uint8_t*>(w), y, in, xs, out, ys, lw, int(rows)};
    using B = __nv_bfloat16;
    if (xd == FSP_DTYPE_F32) return yd == FSP_DTYPE_F32 ? launch_few<float, float>(a, st) : launch_few<float, B>(a, st);
    return yd == FSP_DTYPE_F32 ? launch_few<B, float>(a, st) : launch_few<B, B>(a, st);
  }
  s = quantize_checked(x, xd, rows, in, xs, workspace, nullptr, st);
  return s != FSP_OK ? s : matmul_checked(workspace, w, rows, out, in, y, yd, ys, false, st);
}

fsp_status linear_backward(const void* x, int32_t xd, int64_t xs, const void* dy, int32_t dyd, int64_t dys, int64_t rows,
                           int64_t in, int64_t out, const void* wt, void* dx, int32_t dxd, int64_t dxs, float* dw,
                           int64_t dws, bool accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  fsp_status s = check_dims({rows, in, out});
  if (s == FSP_OK) s = check_matrix(dy, dyd, rows, out, dys, "grad_y");
  if (s == FSP_OK && dw) s = check_matrix(x, xd, rows, in, xs, "x");
  if (s == FSP_OK && dx) s = check_matrix(dx, dxd, rows, in, dxs, "grad_x");
  if (s == FSP_OK && dw) s = check_matrix(dw, FSP_DTYPE_F32, out, in, dws, "grad_w");
  if (s != FSP_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0 || in == 0 || out == 0) {   // one of the products may still be a sum of nothing
    const Range ranges[] = {{dx, dx ? span(rows, in, dxs, dxd) : 0, "grad_x"},
                            {dw, dw ? span(out, in, dws, FSP_DTYPE_F32) : 0, "grad_w"}};
    s = check_ranges(ranges, 2, 2);
    if (s == FSP_OK && dx && rows > 0 && in > 0) s = sum_of_nothing(rows, in, dx, dxd, dxs, st);
    if (s == FSP_OK && dw && !accumulate && out > 0 && in > 0) s = sum_of_nothing(out, in, dw, FSP_DTYPE_F32, dws, st);
    return s;
  }
  if (!dx && !dw) return FSP_OK;
  const Fp8Layout lw = layout_of(in, out);
  const int64_t want = backward_workspace(rows, in, out);
  if (dx) s = check_codes(wt, "wt");
  if (s == FSP_OK) s = check_workspace(workspace, workspace_bytes, want);
  if (s != FSP_OK) return s;
  const Range ranges[] = {{dx, dx ? span(rows, in, dxs, dxd) : 0, "grad_x"},
                          {dw, dw ? span(out, in, dws, FSP_DTYPE_F32) : 0, "grad_w"},
                          {workspace, want, "workspace"},
                          {dy, span(rows, out, dys, dyd), "grad_y"},
                          {x, dw ? span(rows, in, xs, xd) : 0, "x"},
                          {wt, dx ? lw.bytes : 0, "wt"}};
  s = check_ranges(ranges, 6, 3);
  if (s != FSP_OK) return s;
  char* q = static_cast<char*>(workspace);
  char* qt = q + round256(layout_of(rows, out).bytes);
  char* xt = qt + round256(layout_of(out, rows).bytes);
  s = quantize_checked(dy, dyd, rows, out, dys, dx ? q : nullptr, dw ? qt : nullptr, st);
  if (s == FSP_OK && dw) s = quantize_checked(x, xd, rows, in, xs, nullptr, xt, st);
  if (s == FSP_OK && dx) s = matmul_checked(q, wt, rows, in, out, dx, dxd, dxs, false, st);
  if (s == FSP_OK && dw) s = matmul_checked(qt, xt, out, in, rows, dw, FSP_DTYPE_F32, dws, accumulate, st);
  return s;
}

}  // namespace

cudaError_t take_fp8_error(unsigned* bits) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_fp8_error, sizeof(*bits));
  const unsigned zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_fp8_error, &zero, sizeof(zero));
  return e;
}

}  // namespace fsp

extern "C" fsp_status fsp_fp8_bytes(int64_t rows, int64_t cols, size_t* bytes, size_t* scale_offset) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (!bytes || !scale_offset) return fsp::fail(FSP_EINVAL, "bytes or scale_offset is NULL");
    const fsp_status s = fsp::check_dims({rows, cols});
    if (s != FSP_OK) return s;
    const fsp::Fp8Layout l = fsp::layout_of(rows, cols);
    *bytes = size_t(l.bytes);
    *scale_offset = size_t(l.scale_offset);
    return FSP_OK;
  });
}

extern "C" fsp_status fsp_fp8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                                       void* out, void* out_t, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::quantize(x, dtype, rows, cols, stride, out, out_t, cuda_stream);
  });
}

extern "C" fsp_status fsp_fp8_values(const void* q, int64_t rows, int64_t cols, float* out, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::values(q, rows, cols, out, cuda_stream);
  });
}

extern "C" fsp_status fsp_fp8_matmul(const void* a, const void* b, int64_t m, int64_t n, int64_t k, void* c,
                                     int32_t dtype, int64_t c_stride, int32_t accumulate, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::matmul(a, b, m, n, k, c, dtype, c_stride, accumulate, cuda_stream);
  });
}

extern "C" fsp_status fsp_fp8_linear(const void* x, int32_t x_dtype, int64_t rows, int64_t in_features, int64_t x_stride,
                                     const void* w, int64_t out_features, void* y, int32_t y_dtype, int64_t y_stride,
                                     void* workspace, size_t workspace_bytes, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::linear(x, x_dtype, rows, in_features, x_stride, w, out_features, y, y_dtype, y_stride, workspace,
                       workspace_bytes, cuda_stream);
  });
}

extern "C" fsp_status fsp_fp8_linear_backward(const void* x, int32_t x_dtype, int64_t x_stride, const void* grad_y,
                                              int32_t grad_y_dtype, int64_t grad_y_stride, int64_t rows,
                                              int64_t in_features, int64_t out_features, const void* wt, void* grad_x,
                                              int32_t grad_x_dtype, int64_t grad_x_stride, float* grad_w,
                                              int64_t grad_w_stride, int32_t accumulate, void* workspace,
                                              size_t workspace_bytes, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::linear_backward(x, x_dtype, x_stride, grad_y, grad_y_dtype, grad_y_stride, rows, in_features,
                                out_features, wt, grad_x, grad_x_dtype, grad_x_stride, grad_w, grad_w_stride,
                                accumulate != 0, workspace, workspace_bytes, cuda_stream);
  });
}

extern "C" fsp_status fsp_fp8_linear_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features,
                                                     int32_t backward, size_t* bytes) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (!bytes) return fsp::fail(FSP_EINVAL, "bytes is NULL");
    const fsp_status s = fsp::check_dims({rows, in_features, out_features});
    if (s == FSP_OK)
      *bytes = size_t(backward ? fsp::backward_workspace(rows, in_features, out_features)
                               : fsp::forward_workspace(rows, in_features, out_features));
    return s;
  });
}
