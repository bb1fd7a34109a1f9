// AdamW over a list of tensors (sm_103a): one launch updates every tensor,
// with fp32 states or with 8-bit states in blocks of 256.
//
//   g = coef G;  m' = b1 m + (1 - b1) g;  v' = b2 v + (1 - b2) g^2;
//   p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
//
// 8-bit states of a block (s its largest |m'|, or v'):
//   m = s q |q| / 127^2, q = sgn(m') rint(127 sqrt(|m'| / s));
//   v = s (q / 255)^4,   q = rint(255 (v' / s)^(1/4)), at least 1 where v' > 0.
// The roots spread the codes over the magnitudes a block holds: neighbouring
// codes of m differ by 2 / q of the value, of v by 4 / q (1.6 % at the block's
// largest), and the smallest v above 0 is 2.4e-10 of the largest.
//
// Bound: HBM.  Per element G (2 or 4 B), p read and written (8), the bf16 copy
// (2 where asked for), the states read and written (16, or 4 + 16/256).
//
// Layout: a CTA takes one tile of up to kListTile elements of one tensor (the
// block scheduler hands tiles out in order, so the traffic stays in one window
// of the buffers).  A warp takes the 256 elements of one block, a lane elements
// 4 l .. 4 l + 3 of each half, so that every access of a warp is one run of 512
// (fp32), 256 (bf16) or 128 bytes (codes) and a block's largest value is one
// reduction over the warp.
#pragma once

#include "fsp_host.h"
#include "fsp_kernels.cuh"
#include "fsp_list.h"

namespace fsp {

constexpr int kListThreads = 256;
static_assert(kListTile == kListThreads / 32 * kListBlock, "one block per warp");

// Codes and back.  Every step is a separately rounded operation, so that the
// codes are a function of the values that any IEEE implementation reproduces.
constexpr float kInv127 = float(1.0 / 127.0), kInv255 = float(1.0 / 255.0);

__device__ __forceinline__ float m_of_code(int q, float s) {
  const float x = __fmul_rn(float(q), kInv127);
  return __fmul_rn(s, __fmul_rn(x, fabsf(x)));
}
__device__ __forceinline__ float v_of_code(unsigned q, float s) {
  float x = __fmul_rn(float(q), kInv255);
  x = __fmul_rn(x, x);
  return __fmul_rn(s, __fmul_rn(x, x));
}
__device__ __forceinline__ int code_of_m(float m, float s) {
  if (!(s > 0.f)) return 0;
  const int q = __float2int_rn(__fmul_rn(__fsqrt_rn(__fdiv_rn(fabsf(m), s)), 127.f));
  return m < 0.f ? -q : q;
}
__device__ __forceinline__ unsigned code_of_v(float v, float s) {
  if (!(s > 0.f)) return 0u;
  const unsigned q = __float2uint_rn(__fmul_rn(__fsqrt_rn(__fsqrt_rn(__fdiv_rn(v, s))), 255.f));
  return v > 0.f && q == 0u ? 1u : q;
}

// The largest |x| of the warp's block: magnitudes order as their bit patterns,
// NaN above infinity, so a NaN anywhere is what comes back.
__device__ __forceinline__ float block_largest(const float* x) {
  unsigned top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
  return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

// Four consecutive elements at base + i (i counted in elements): one vector
// access where the tensor's pointers allow it, else element by element with
// `n` of the four inside the tensor.
__device__ __forceinline__ void load4(const void* base, bool bf16, bool vec, int64_t i, int n, float* x) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (vec && n == 4) {
      const uint2 b = __ldcs(reinterpret_cast<const uint2*>(p));
      x[0] = __uint_as_float(b.x << 16);
      x[1] = __uint_as_float(b.x & 0xffff0000u);
      x[2] = __uint_as_float(b.y << 16);
      x[3] = __uint_as_float(b.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = j < n ? __uint_as_float(uint32_t(__ldcs(p + j)) << 16) : 0.f;
    }
  } else {
    const float* p = static_cast<const float*>(base) + i;
    if (vec && n == 4) {
      const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
      x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = j < n ? __ldcs(p + j) : 0.f;
    }
  }
}

__device__ __forceinline__ void store4(void* base, bool bf16, bool vec, int64_t i, int n, const float* x) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    if (vec && n == 4) {
      __stcs(reinterpret_cast<uint2*>(p), pack_bf16x4(make_float4(x[0], x[1], x[2], x[3])));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) __stcs(p + j, bf16_bits(x[j]));
    }
  } else {
    float* p = static_cast<float*>(base) + i;
    if (vec && n == 4) {
      __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) __stcs(p + j, x[j]);
    }
  }
}

// The update of one element whose states will be rounded to 8 bits: m' and v'
// with every product rounded on its own (their codes are then reproducible),
// p' as adamw()'s fp32 evaluation (the states' 1.6 % steps leave nothing for
// its float-pair refinement to keep).
__device__ __forceinline__ void adamw_coarse(float g, float& p, float& m, float& v, const Coeffs& c) {
  m = __fadd_rn(__fmul_rn(m, c.beta1), __fmul_rn(g, c.one_minus_beta1_hi));
  v = __fadd_rn(__fmul_rn(v, c.beta2), __fmul_rn(__fmul_rn(g, g), c.one_minus_beta2_hi));
  const float r = rcp_approx(__fmaf_rn(sqrt_approx(v), c.isb_hi, c.eps));
  p = __fsub_rn(__fmul_rn(p, c.decay_hi), __fmul_rn(c.step_hi, __fmul_rn(m, r)));
}

__device__ __forceinline__ Coeffs list_coeffs(const ListArgs& a) {
  if (!a.step_dev) return a.c;
  int64_t t = *a.step_dev;
  if (t < 1) {
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_fsp_device_error, kErrStepIndex);
    t = 1;
  }
  Coeffs c = a.c;
  bias_scalars(c, a.lr, t);
  return c;
}

template <bool k8Bit>
__global__ void __launch_bounds__(kListThreads) adamw_list_kernel(const __grid_constant__ ListArgs a) {
  const ListTile tile = a.tiles[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int begin = warp * kListBlock;   // this warp's block in the tile
  if (begin >= tile.len) return;
  const bool pb = tile.flags & kListParamBf16, gb = tile.flags & kListGradBf16, vec = tile.flags & kListVec;
  const int64_t slot = tile.state_off + begin;
  const int i0 = begin + lane * 4, i1 = i0 + kListBlock / 2;
  const int n0 = min(4, max(0, tile.len - i0)), n1 = min(4, max(0, tile.len - i1));
  float g[8], p[8], m[8], v[8];
  load4(tile.grad, gb, vec, i0, n0, g);
  load4(tile.grad, gb, vec, i1, n1, g + 4);
  load4(tile.param, pb, vec, i0, n0, p);
  load4(tile.param, pb, vec, i1, n1, p + 4);
  char4* mq = nullptr;
  uchar4* vq = nullptr;
  float *mf = nullptr, *vf = nullptr;
  if (k8Bit) {
    mq = reinterpret_cast<char4*>(static_cast<int8_t*>(a.m) + slot) + lane;
    vq = reinterpret_cast<uchar4*>(static_cast<uint8_t*>(a.v) + slot) + lane;
    const float ms = a.m_scale[slot / kListBlock], vs = a.v_scale[slot / kListBlock];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const char4 cm = mq[32 * h];
      const uchar4 cv = vq[32 * h];
      const int n = h ? n1 : n0;
      const int qm[4] = {cm.x, cm.y, cm.z, cm.w};
      const unsigned qv[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[4 * h + j] = j < n ? m_of_code(qm[j], ms) : 0.f;
        v[4 * h + j] = j < n ? v_of_code(qv[j], vs) : 0.f;
      }
    }
  } else {
    mf = static_cast<float*>(a.m) + slot - begin;
    vf = static_cast<float*>(a.v) + slot - begin;
    load4(mf, false, true, i0, n0, m);
    load4(mf, false, true, i1, n1, m + 4);
    load4(vf, false, true, i0, n0, v);
    load4(vf, false, true, i1, n1, v + 4);
  }
  const float coef = a.grad_scale ? *a.grad_scale : 1.f;
  const Coeffs c = list_coeffs(a);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = __fmul_rn(g[j], coef);
    if (k8Bit)
      adamw_coarse(gj, p[j], m[j], v[j], c);
    else
      adamw(gj, p[j], m[j], v[j], c);
  }
  store4(tile.param, pb, vec, i0, n0, p);
  store4(tile.param, pb, vec, i1, n1, p + 4);
  if (tile.copy) {
    store4(tile.copy, true, vec, i0, n0, p);
    store4(tile.copy, true, vec, i1, n1, p + 4);
  }
  if (k8Bit) {
    // past the tensor's end g, m and v are 0: they stay out of the largest value
    // (unless coef is not finite, which every element of the block then shows)
    const float ms = block_largest(m), vs = block_largest(v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* x = m + 4 * h;
      const float* y = v + 4 * h;
      char4 cm = make_char4(code_of_m(x[0], ms), code_of_m(x[1], ms), code_of_m(x[2], ms), code_of_m(x[3], ms));
      uchar4 cv = make_uchar4(code_of_v(y[0], vs), code_of_v(y[1], vs), code_of_v(y[2], vs), code_of_v(y[3], vs));
      const int n = h ? n1 : n0;
      if (n == 4) {
        mq[32 * h] = cm;
        vq[32 * h] = cv;
      } else {
        const signed char qm[4] = {cm.x, cm.y, cm.z, cm.w};
        const unsigned char qv[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) {
            reinterpret_cast<signed char*>(mq + 32 * h)[j] = qm[j];
            reinterpret_cast<unsigned char*>(vq + 32 * h)[j] = qv[j];
          }
      }
    }
    if (lane == 0) {
      a.m_scale[slot / kListBlock] = ms;
      a.v_scale[slot / kListBlock] = vs;
    }
  } else {
    store4(mf, false, true, i0, n0, m);
    store4(mf, false, true, i1, n1, m + 4);
    store4(vf, false, true, i0, n0, v);
    store4(vf, false, true, i1, n1, v + 4);
  }
}

// fp32 states <-> 8-bit states of whole blocks: a warp per block, grid over
// all blocks of the state buffers.
__global__ void __launch_bounds__(kListThreads) list_state_values_kernel(const int8_t* m8, const uint8_t* v8,
                                                                         const float* ms, const float* vs, float* m,
                                                                         float* v, int64_t n_blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t b = int64_t(blockIdx.x) * (kListThreads / 32) + (threadIdx.x >> 5);
  if (b >= n_blocks) return;
  const float s = ms[b], t = vs[b];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b * kListBlock + h * (kListBlock / 2) + lane * 4;
    const char4 cm = *reinterpret_cast<const char4*>(m8 + i);
    const uchar4 cv = *reinterpret_cast<const uchar4*>(v8 + i);
    __stcs(reinterpret_cast<float4*>(m + i),
           make_float4(m_of_code(cm.x, s), m_of_code(cm.y, s), m_of_code(cm.z, s), m_of_code(cm.w, s)));
    __stcs(reinterpret_cast<float4*>(v + i),
           make_float4(v_of_code(cv.x, t), v_of_code(cv.y, t), v_of_code(cv.z, t), v_of_code(cv.w, t)));
  }
}

__global__ void __launch_bounds__(kListThreads) list_state_load_kernel(const float* m, const float* v, int8_t* m8,
                                                                       uint8_t* v8, float* ms, float* vs,
                                                                       int64_t n_blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t b = int64_t(blockIdx.x) * (kListThreads / 32) + (threadIdx.x >> 5);
  if (b >= n_blocks) return;
  float x[8], y[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b * kListBlock + h * (kListBlock / 2) + lane * 4;
    load4(m, false, true, i, 4, x + 4 * h);
    load4(v, false, true, i, 4, y + 4 * h);
  }
  const float s = block_largest(x), t = block_largest(y);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b * kListBlock + h * (kListBlock / 2) + lane * 4;
    const float* xh = x + 4 * h;
    const float* yh = y + 4 * h;
    *reinterpret_cast<char4*>(m8 + i) =
        make_char4(code_of_m(xh[0], s), code_of_m(xh[1], s), code_of_m(xh[2], s), code_of_m(xh[3], s));
    *reinterpret_cast<uchar4*>(v8 + i) =
        make_uchar4(code_of_v(yh[0], t), code_of_v(yh[1], t), code_of_v(yh[2], t), code_of_v(yh[3], t));
  }
  if (lane == 0) {
    ms[b] = s;
    vs[b] = t;
  }
}

// ---- launches (host) --------------------------------------------------------------

fsp_status launch_adamw_list(const ListArgs& a, bool eight_bit, int64_t n_tiles, void* stream) {
  if (n_tiles > INT32_MAX) return fail(FSP_EUNSUPPORTED, "more than 2^31 work tiles");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (eight_bit)
    adamw_list_kernel<true><<<unsigned(n_tiles), kListThreads, 0, st>>>(a);
  else
    adamw_list_kernel<false><<<unsigned(n_tiles), kListThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FSP_OK : fail(FSP_ECUDA, cuda_msg("AdamW list kernel launch", e));
}

fsp_status launch_list_state(bool load, void* m8, void* v8, float* ms, float* vs, float* m, float* v, int64_t len,
                             void* stream) {
  const int64_t n = len / kListBlock;
  const int64_t ctas = (n + kListThreads / 32 - 1) / (kListThreads / 32);
  if (ctas > INT32_MAX) return fail(FSP_EUNSUPPORTED, "more than 2^31 work tiles");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (load)
    list_state_load_kernel<<<unsigned(ctas), kListThreads, 0, st>>>(m, v, static_cast<int8_t*>(m8),
                                                                    static_cast<uint8_t*>(v8), ms, vs, n);
  else
    list_state_values_kernel<<<unsigned(ctas), kListThreads, 0, st>>>(static_cast<int8_t*>(m8),
                                                                      static_cast<uint8_t*>(v8), ms, vs, m, v, n);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FSP_OK : fail(FSP_ECUDA, cuda_msg("AdamW state kernel launch", e));
}

}  // namespace fsp
