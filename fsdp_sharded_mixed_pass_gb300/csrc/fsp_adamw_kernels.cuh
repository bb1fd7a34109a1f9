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
//
// A list with many tiles per SM goes through a ring of stages that bulk copies
// fill and drain instead (adamw_ring_kernel, below): the same tiles, a warp per
// block, with the copies of the next tiles in flight meanwhile.
#pragma once

#include "fsp_host.h"
#include "fsp_kernels.cuh"
#include "fsp_list.h"

namespace fsp {

constexpr int kListThreads = 256;
static_assert(kListTile == kListThreads / 32 * kListBlock, "one block per warp");

// ---- 8-bit states, two elements at a time ----------------------------------------
//
// The arithmetic runs on pairs of floats (one instruction for two products or
// sums, each rounded as its own).  Every step of a code is a separately rounded
// operation, so that codes are a function of the values that any IEEE
// implementation reproduces.

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 abs2(float2 x) { return make_float2(fabsf(x.x), fabsf(x.y)); }

// Code bytes 2 h, 2 h + 1 of a word as floats: the byte becomes the low bits of
// 2^23, whose ulp is 1.
__device__ __forceinline__ float2 bytes2(uint32_t w, int h, float offset) {
  const float lo = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540u | unsigned(2 * h)));
  const float hi = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540u | unsigned(2 * h + 1)));
  return __fadd2_rn(make_float2(lo, hi), both(-offset));
}
constexpr float kInv127 = float(1.0 / 127.0), kInv255 = float(1.0 / 255.0);
// What four codes stand for in a block of scale s.
__device__ __forceinline__ void m_of_codes(uint32_t q, float s, float2* m) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 x = __fmul2_rn(bytes2(q ^ 0x80808080u, h, 8388608.f + 128.f), both(kInv127));
    m[h] = __fmul2_rn(both(s), __fmul2_rn(x, abs2(x)));
  }
}
__device__ __forceinline__ void v_of_codes(uint32_t q, float s, float2* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 x = __fmul2_rn(bytes2(q, h, 8388608.f), both(kInv255));
    x = __fmul2_rn(x, x);
    v[h] = __fmul2_rn(both(s), __fmul2_rn(x, x));
  }
}

__device__ __forceinline__ int exact_code_of_m(float m, float s) {   // of |m|
  return __float2int_rn(__fmul_rn(__fsqrt_rn(__fdiv_rn(fabsf(m), s)), 127.f));
}
__device__ __forceinline__ int exact_code_of_v(float v, float s) {
  return __float2int_rn(__fmul_rn(__fsqrt_rn(__fsqrt_rn(__fdiv_rn(v, s))), 255.f));
}
__device__ __forceinline__ float sqrt_approx_ftz(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A block's scale and its reciprocal for the quick evaluation (NaN where that
// could leave the range of fp32: such a block takes the exact one throughout).
struct BlockScale {
  float s, inv;
};
__device__ __forceinline__ BlockScale block_scale(float s) {
  return {s, s > 0x1p-100f && s < 0x1p100f ? rcp_approx(s) : __int_as_float(0x7fffffff)};
}

// rint(r) for |r| < 2^22 as the low bits of r + 3 2^22, whose ulp is 1.
constexpr float kRintMagic = 12582912.f;
// The quick evaluations err by at most 2^-13 codes (below); nearer to a tie than
// 2^-12 an element takes the exact one, so every code is the exact one's.
constexpr float kNearTie = 0.5f - 0x1p-12f;

// The rounded value's low bits in t's, and whether no rounding is near a tie.
__device__ __forceinline__ bool rint2(float2 r, float2& t) {
  t = __fadd2_rn(r, both(kRintMagic));
  const float2 f = __fadd2_rn(t, both(-kRintMagic));
  const float2 e = __fadd2_rn(r, make_float2(-f.x, -f.y));
  return fabsf(e.x) <= kNearTie && fabsf(e.y) <= kNearTie;
}
__device__ __forceinline__ uint32_t low_bytes(const float2* t) {
  const uint32_t lo = __byte_perm(__float_as_uint(t[0].x), __float_as_uint(t[0].y), 0x0040u);
  const uint32_t hi = __byte_perm(__float_as_uint(t[1].x), __float_as_uint(t[1].y), 0x0040u);
  return __byte_perm(lo, hi, 0x5410u);
}

// The codes of four elements, the first in the low byte.  Approximate roots: with
// x' = |m| inv (two roundings and rcp_approx: relative error below 2^-21.4) the
// approximate root errs by 2^-22 and half of that, 127 x' by 2^-24 more: together
// below 2^-21 of a code of at most 127, or 2^-14.  v: two roots and a quarter of
// x's error, below 2^-21 of at most 255, or 2^-13.
__device__ __forceinline__ uint32_t codes_of_m(const float2* m, BlockScale b) {
  if (!(b.s > 0.f)) return 0u;
  float2 t[2];
  bool sure = true;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 x = __fmul2_rn(m[h], both(b.inv));
    const float2 r = __fmul2_rn(make_float2(copysignf(sqrt_approx_ftz(fabsf(x.x)), x.x), copysignf(sqrt_approx_ftz(fabsf(x.y)), x.y)),
                                both(127.f));
    sure = rint2(r, t[h]) && sure;
  }
  uint32_t w = low_bytes(t);
  if (!sure) {
    w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = j & 1 ? m[j >> 1].y : m[j >> 1].x;
      const int q = exact_code_of_m(x, b.s);
      w |= uint32_t((x < 0.f ? -q : q) & 0xff) << (8 * j);
    }
  }
  return w;
}
__device__ __forceinline__ uint32_t codes_of_v(const float2* v, BlockScale b) {
  if (!(b.s > 0.f)) return 0u;
  float2 t[2];
  bool sure = true;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 x = __fmul2_rn(v[h], both(b.inv));
    const float2 r = __fmul2_rn(make_float2(sqrt_approx_ftz(sqrt_approx_ftz(x.x)), sqrt_approx_ftz(sqrt_approx_ftz(x.y))), both(255.f));
    sure = rint2(r, t[h]) && sure;
    // above 0 but rounded to 0: code 1
    sure = sure && !(r.x < 0.5f && v[h].x > 0.f) && !(r.y < 0.5f && v[h].y > 0.f);
  }
  uint32_t w = low_bytes(t);
  if (!sure) {
    w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = j & 1 ? v[j >> 1].y : v[j >> 1].x;
      w |= uint32_t(x > 0.f ? max(exact_code_of_v(x, b.s), 1) : 0) << (8 * j);
    }
  }
  return w;
}

// The largest |x| of the warp's block, NaN where one is: magnitudes order as
// their bit patterns, NaN above infinity.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float block_largest(const float2* x) {
  float top = max_nan(fabsf(x[0].x), fabsf(x[0].y));
#pragma unroll
  for (int j = 1; j < 4; ++j) top = max_nan(top, max_nan(fabsf(x[j].x), fabsf(x[j].y)));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// ---- element access ---------------------------------------------------------------

// Four consecutive elements at base + i (i counted in elements): one vector
// access where the tensor's pointers allow it, else element by element with
// `n` of the four inside the tensor.
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// Streaming loads, volatile: they stay behind the wait for the launch before.
__device__ __forceinline__ float4 stream4(const float* p) {
  float4 x;
  asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "l"(p));
  return x;
}
__device__ __forceinline__ uint2 stream4(const uint16_t* p) {
  uint2 x;
  asm volatile("ld.global.cs.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t stream4(const uint8_t* p) {
  uint32_t x;
  asm volatile("ld.global.cs.b32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

__device__ __forceinline__ void load4(const void* base, bool bf16, bool vec, int64_t i, int n, float2* x) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (vec && n == 4) {
      const uint2 b = stream4(p);
      x[0] = make_float2(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u));
      x[1] = make_float2(__uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[h] = make_float2(2 * h < n ? bf16_value(p[2 * h]) : 0.f, 2 * h + 1 < n ? bf16_value(p[2 * h + 1]) : 0.f);
    }
  } else {
    const float* p = static_cast<const float*>(base) + i;
    if (vec && n == 4) {
      const float4 f = stream4(p);
      x[0] = make_float2(f.x, f.y);
      x[1] = make_float2(f.z, f.w);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) x[h] = make_float2(2 * h < n ? p[2 * h] : 0.f, 2 * h + 1 < n ? p[2 * h + 1] : 0.f);
    }
  }
}

__device__ __forceinline__ void store4(void* base, bool bf16, bool vec, int64_t i, int n, const float2* x) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    if (vec && n == 4) {
      __stcs(reinterpret_cast<uint2*>(p), pack_bf16x4(make_float4(x[0].x, x[0].y, x[1].x, x[1].y)));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (2 * h < n) __stcs(p + 2 * h, bf16_bits(x[h].x));
        if (2 * h + 1 < n) __stcs(p + 2 * h + 1, bf16_bits(x[h].y));
      }
    }
  } else {
    float* p = static_cast<float*>(base) + i;
    if (vec && n == 4) {
      __stcs(reinterpret_cast<float4*>(p), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (2 * h < n) __stcs(p + 2 * h, x[h].x);
        if (2 * h + 1 < n) __stcs(p + 2 * h + 1, x[h].y);
      }
    }
  }
}

// The update of two elements whose states will be rounded to 8 bits: m' and v'
// with every product rounded on its own (their codes are then reproducible),
// p' in fp32 as adamw()'s first evaluation (the states' 1.6 % steps leave
// nothing for its float-pair refinement to keep).
__device__ __forceinline__ void adamw_coarse(float2 g, float2& p, float2& m, float2& v, const Coeffs& c) {
  m = __fmul2_rn(m, both(c.beta1));
  v = __fmul2_rn(v, both(c.beta2));
  const float2 gm = __fmul2_rn(g, both(c.one_minus_beta1_hi));
  const float2 gv = __fmul2_rn(__fmul2_rn(g, g), both(c.one_minus_beta2_hi));
  m = make_float2(__fadd_rn(m.x, gm.x), __fadd_rn(m.y, gm.y));   // (a sum of pairs would be fused with its product)
  v = make_float2(__fadd_rn(v.x, gv.x), __fadd_rn(v.y, gv.y));
  const float2 d = __ffma2_rn(make_float2(sqrt_approx(v.x), sqrt_approx(v.y)), both(c.isb_hi), both(c.eps));
  const float2 u = __fmul2_rn(m, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
  p = __ffma2_rn(p, both(c.decay_hi), __fmul2_rn(u, both(-c.step_hi)));
}

// The update's scalars.  Thread 0 of block 0 reports a device-resident update index
// below 1 (taken as 1): here, or where it does not come here (kReport false) on its own.
template <bool kReport>
__device__ __forceinline__ Coeffs list_coeffs(const ListArgs& a) {
  if (!a.step_dev) return a.c;
  int64_t t = *a.step_dev;
  if (t < 1) {
    if (kReport && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_fsp_device_error, kErrStepIndex);
    t = 1;
  }
  Coeffs c = a.c;
  bias_scalars(c, a.lr, t);
  return c;
}

// One block as a lane holds it: elements 4 l .. 4 l + 3 of each half.
struct ListBlock {
  float2 g[4], p[4];
  float2 m[4], v[4];          // fp32 states
  uint32_t qm[2], qv[2];      // 8-bit states
  float ms, vs;
};

template <bool k8Bit>
__device__ __forceinline__ void load_block(const ListArgs& a, const ListTile& t, int begin, int lane, ListBlock& b) {
  const bool pb = t.flags & kListParamBf16, gb = t.flags & kListGradBf16, vec = t.flags & kListVec;
  const int64_t slot = t.state_off + begin;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = begin + h * (kListBlock / 2) + lane * 4, n = min(4, max(0, t.len - i));
    load4(t.grad, gb, vec, i, n, b.g + 2 * h);
    load4(t.param, pb, vec, i, n, b.p + 2 * h);
    if (k8Bit) {
      const uint32_t in = n == 4 ? ~0u : (1u << (8 * n)) - 1u;   // nothing past the tensor's end
      b.qm[h] = stream4(static_cast<const uint8_t*>(a.m) + slot + 4 * (32 * h + lane)) & in;
      b.qv[h] = stream4(static_cast<const uint8_t*>(a.v) + slot + 4 * (32 * h + lane)) & in;
    } else {
      load4(static_cast<const float*>(a.m) + t.state_off, false, true, i, n, b.m + 2 * h);
      load4(static_cast<const float*>(a.v) + t.state_off, false, true, i, n, b.v + 2 * h);
    }
  }
  if (k8Bit) {
    b.ms = a.m_scale[slot / kListBlock];
    b.vs = a.v_scale[slot / kListBlock];
  }
}

template <bool k8Bit>
__device__ __forceinline__ void update_block(const ListArgs& a, const ListTile& t, const Coeffs& c, float coef, int begin,
                                             int lane, ListBlock& b) {
  const bool pb = t.flags & kListParamBf16, vec = t.flags & kListVec;
  const int64_t slot = t.state_off + begin;
  if (k8Bit) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m_of_codes(b.qm[h], b.ms, b.m + 2 * h);
      v_of_codes(b.qv[h], b.vs, b.v + 2 * h);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __fmul2_rn(b.g[j], both(coef));
    if (k8Bit) {
      adamw_coarse(x, b.p[j], b.m[j], b.v[j], c);
    } else {
      adamw(x.x, b.p[j].x, b.m[j].x, b.v[j].x, c);
      adamw(x.y, b.p[j].y, b.m[j].y, b.v[j].y, c);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = begin + h * (kListBlock / 2) + lane * 4, n = min(4, max(0, t.len - i));
    store4(t.param, pb, vec, i, n, b.p + 2 * h);
    if (t.copy) store4(t.copy, true, vec, i, n, b.p + 2 * h);
    if (!k8Bit) {
      store4(static_cast<float*>(a.m) + t.state_off, false, true, i, n, b.m + 2 * h);
      store4(static_cast<float*>(a.v) + t.state_off, false, true, i, n, b.v + 2 * h);
    }
  }
  if (k8Bit) {
    // past the tensor's end g, m and v are 0: they stay out of the largest value
    // (unless coef is not finite, which every element of the block then shows)
    const BlockScale ms = block_scale(block_largest(b.m)), vs = block_scale(block_largest(b.v));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t qm = codes_of_m(b.m + 2 * h, ms), qv = codes_of_v(b.v + 2 * h, vs);
      uint32_t* pm = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.m) + slot) + 32 * h + lane;
      uint32_t* pv = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.v) + slot) + 32 * h + lane;
      const int n = min(4, max(0, t.len - (begin + h * (kListBlock / 2) + lane * 4)));
      if (n == 4) {
        __stcs(pm, qm);
        __stcs(pv, qv);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) {
            reinterpret_cast<uint8_t*>(pm)[j] = uint8_t(qm >> (8 * j));
            reinterpret_cast<uint8_t*>(pv)[j] = uint8_t(qv >> (8 * j));
          }
      }
    }
    if (lane == 0) {
      a.m_scale[slot / kListBlock] = ms.s;
      a.v_scale[slot / kListBlock] = vs.s;
    }
  }
}

template <bool k8Bit>
__global__ void __launch_bounds__(kListThreads, k8Bit ? 5 : 4) adamw_list_kernel(const __grid_constant__ ListArgs a) {
  launch_dependents();
  const ListTile tile = a.tiles[blockIdx.x];   // (a table that no kernel writes)
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int begin = warp * kListBlock;   // this warp's block in the tile
  if (begin >= tile.len) return;
  ListBlock b;
  load_block<k8Bit>(a, tile, begin, lane, b);
  update_block<k8Bit>(a, tile, list_coeffs<true>(a), a.grad_scale ? *a.grad_scale : 1.f, begin, lane, b);
}

// ---- long lists: a ring of stages in shared memory ---------------------------------
//
// One CTA per SM.  A producer warp takes tiles (in order from a counter, or with a
// fixed stride) and streams each one's gradient, parameter and states into a stage
// with bulk asynchronous copies (its scales with 4-byte asynchronous copies: they
// have no 16-byte alignment); two teams of eight consumer warps take the stages in
// turn, a block per warp, and leave the results in place; a storer thread writes
// them back with bulk stores and frees the stage.  Warps then wait for shared memory
// only, and loads are in flight whatever the arithmetic does.  A tile that bulk
// copies cannot move (a tensor off 16-byte alignment, the last odd elements of one)
// gets an empty stage, and the team does it from global memory.
//
// Measured (GB300): fp32 states, bf16 gradients and copies, 360.7 M elements 1442 us
// = 7.0 TB/s (one CTA per tile 1640-1730); 8-bit states, 541.1 M elements 1434 us =
// 6.1 TB/s (2000).

constexpr int kTeamWarps = kListTile / kListBlock;

template <bool k8Bit>
struct Ring {
  static constexpr int kStateBytes = kListTile * (k8Bit ? 1 : 4);
  static constexpr int kGrad = 0, kParam = kListTile * 4, kM = 2 * kListTile * 4, kV = kM + kStateBytes;
  static constexpr int kCopy = kV + kStateBytes, kScale = kCopy + kListTile * 2;   // kScale: [2][kTeamWarps] floats
  static constexpr int kStage = kScale + (k8Bit ? 128 : 0);
  static constexpr bool kCounter = !k8Bit;
  static constexpr int kTeams = 2;
  static constexpr int kThreads = 64 + 32 * kTeamWarps * kTeams;
  static constexpr int kStages = k8Bit ? 8 : 6;
  static constexpr int kLag = 1;   // stages whose stores may still be reading
  static_assert(kStages % kTeams == 0, "a team's stages come round with the ring");
  static constexpr int kHeaders = 256;                  // after the barriers
  static constexpr int kBase = kHeaders + kStages * 64; // 64 bytes per header
  static constexpr int kSmem = (kBase + 127) / 128 * 128 + kStages * kStage;
  static_assert(kStage % 128 == 0 && kSmem <= 232448, "shared memory of the ring");
  static_assert(sizeof(ListTile) <= 64, "header");
};

__device__ __forceinline__ bool bulk_tile(const ListTile& t) { return (t.flags & kListBulk) && t.len % 16 == 0; }

__device__ __forceinline__ void copy4_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives at `bar` once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// All but the N newest groups of bulk stores have read their shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read_but() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Four elements of a stage's array from element i.
__device__ __forceinline__ void stage_load4(const unsigned char* base, bool bf16, int i, float2* x) {
  if (bf16) {
    const uint2 b = *reinterpret_cast<const uint2*>(base + 2 * i);
    x[0] = make_float2(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u));
    x[1] = make_float2(__uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
  } else {
    const float4 f = *reinterpret_cast<const float4*>(base + 4 * i);
    x[0] = make_float2(f.x, f.y);
    x[1] = make_float2(f.z, f.w);
  }
}
__device__ __forceinline__ void stage_store4(unsigned char* base, bool bf16, int i, const float2* x) {
  const float4 f = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
  if (bf16)
    *reinterpret_cast<uint2*>(base + 2 * i) = pack_bf16x4(f);
  else
    *reinterpret_cast<float4*>(base + 4 * i) = f;
}

// mbar_wait by a whole warp, whose lanes agree on whether it ran out.
__device__ __forceinline__ bool mbar_wait_all(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 255u) == 0 && __any_sync(0xffffffffu, global_ns() - t0 > kWaitLimitNs)) return false;
  }
  return false;
}

// One block of a stage, in place.
template <bool k8Bit>
__device__ __forceinline__ void update_stage(const ListArgs& a, const ListTile& t, const Coeffs& c, float coef, int begin,
                                             int lane, unsigned char* stage) {
  using R = Ring<k8Bit>;
  const bool pb = t.flags & kListParamBf16, gb = t.flags & kListGradBf16;
  float2 g[4], p[4], m[4], v[4];
  const int block = begin / kListBlock;
  float* scales = reinterpret_cast<float*>(stage + R::kScale);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = begin + h * (kListBlock / 2) + lane * 4;
    const bool in = i < t.len;   // (a multiple of 16: all four or none)
    stage_load4(stage + R::kGrad, gb, i, g + 2 * h);
    stage_load4(stage + R::kParam, pb, i, p + 2 * h);
    if (k8Bit) {
      m_of_codes(in ? *reinterpret_cast<const uint32_t*>(stage + R::kM + i) : 0u, scales[block], m + 2 * h);
      v_of_codes(in ? *reinterpret_cast<const uint32_t*>(stage + R::kV + i) : 0u, scales[kTeamWarps + block], v + 2 * h);
    } else {
      stage_load4(stage + R::kM, false, i, m + 2 * h);
      stage_load4(stage + R::kV, false, i, v + 2 * h);
    }
    if (!in) g[2 * h] = g[2 * h + 1] = both(0.f);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __fmul2_rn(g[j], both(coef));
    if (k8Bit) {
      adamw_coarse(x, p[j], m[j], v[j], c);
    } else {
      adamw(x.x, p[j].x, m[j].x, v[j].x, c);
      adamw(x.y, p[j].y, m[j].y, v[j].y, c);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = begin + h * (kListBlock / 2) + lane * 4;
    stage_store4(stage + R::kParam, pb, i, p + 2 * h);
    if (t.copy) stage_store4(stage + R::kCopy, true, i, p + 2 * h);
    if (!k8Bit) {
      stage_store4(stage + R::kM, false, i, m + 2 * h);
      stage_store4(stage + R::kV, false, i, v + 2 * h);
    }
  }
  if (k8Bit) {
    const BlockScale ms = block_scale(block_largest(m)), vs = block_scale(block_largest(v));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = begin + h * (kListBlock / 2) + lane * 4;
      *reinterpret_cast<uint32_t*>(stage + R::kM + i) = codes_of_m(m + 2 * h, ms);
      *reinterpret_cast<uint32_t*>(stage + R::kV + i) = codes_of_v(v + 2 * h, vs);
    }
    if (lane == 0) {
      const int64_t at = (t.state_off + begin) / kListBlock;
      a.m_scale[at] = ms.s;
      a.v_scale[at] = vs.s;
    }
  }
}

template <bool k8Bit>
__global__ void __launch_bounds__(Ring<k8Bit>::kThreads, 1) adamw_ring_kernel(const __grid_constant__ ListArgs a) {
  using R = Ring<k8Bit>;
  constexpr int S = R::kStages;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t bars = smem_addr(smem);
  const uint32_t full = bars, computed = full + 8 * S, empty = computed + 8 * S;
  unsigned char* const stages = smem + (R::kBase + 127) / 128 * 128;
  auto header = [&](int s) { return reinterpret_cast<ListTile*>(smem + R::kHeaders + 64 * s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, k8Bit ? 33 : 1);   // the bulk copies, and each lane's copies of scales
      mbar_init(computed + 8 * s, kTeamWarps);
      mbar_init(empty + 8 * s, 1);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 0 && blockIdx.x == 0 && a.step_dev && *a.step_dev < 1) atomicOr(&g_fsp_device_error, kErrStepIndex);
  __syncthreads();

  if (warp == 0) {
    // ---- producer: the whole warp, lane 0 issues the bulk copies ----
    auto fetch = [&](int64_t i) {
      ListTile t{};
      if (i < a.n_tiles)
        t = a.tiles[i];
      else
        t.len = -1;   // no more work
      return t;
    };
    // Tile numbers.  fp32 states: in order from the counter, kPerClaim at a time and
    // claimed two claims ahead (in lane 0, until they are handed round: the round trip,
    // about 1 us, is most of a tile's time).  8-bit states move half the bytes per
    // tile, and there a fixed stride is ahead.
    constexpr int kPerClaim = 2;
    unsigned long long next = 0, second = 0;
    auto claim = [&] { return lane == 0 ? atomicAdd(a.counter, 1ull) : 0ull; };
    int64_t at_number = R::kCounter ? 0 : int64_t(blockIdx.x);
    int used = kPerClaim;
    auto number = [&] {
      if constexpr (R::kCounter) {
        if (used == kPerClaim) {
          at_number = int64_t(__shfl_sync(0xffffffffu, next, 0)) * kPerClaim;
          next = second;
          second = claim();
          used = 0;
        }
        return at_number + used++;
      } else {
        const int64_t n = at_number;
        at_number += gridDim.x;
        return n;
      }
    };
    if constexpr (R::kCounter) {
      next = claim();
      second = claim();
    }
    // (descriptors two tiles ahead)
    ListTile tile = fetch(number()), ahead = fetch(number());
    int s = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    int ends = 0;
    while (true) {
      const ListTile later = fetch(number());
      if (!mbar_wait_all(empty + 8 * s, phase ^ 1u)) {   // (the lanes agree: they go on as a warp)
        if (lane == 0) atomicOr(&g_fsp_device_error, kErrProducerWait);
        break;
      }
      const uint32_t bar = full + 8 * s;
      unsigned char* stage = stages + s * R::kStage;
      const uint32_t at = smem_addr(stage);
      const bool bulk = tile.len > 0 && bulk_tile(tile);
      if (lane == 0) *header(s) = tile;
      if (k8Bit && bulk && lane < 2 * kTeamWarps) {
        const int block = lane % kTeamWarps;
        const float* src = (lane < kTeamWarps ? a.m_scale : a.v_scale) + tile.state_off / kListBlock + block;
        if (block * kListBlock < tile.len) copy4_async(at + R::kScale + 4 * lane, src);
      }
      if (k8Bit) arrive_after_copies(bar);
      if (lane == 0) {
        const uint32_t n = uint32_t(bulk ? tile.len : 0);
        const uint32_t gb = n * (tile.flags & kListGradBf16 ? 2 : 4), pb = n * (tile.flags & kListParamBf16 ? 2 : 4);
        const uint32_t sb = n * (k8Bit ? 1 : 4);
        mbar_arrive_expect_tx(bar, gb + pb + 2 * sb);
        if (bulk) {
          const int64_t off = tile.state_off * (k8Bit ? 1 : 4);
          bulk_load(at + R::kGrad, tile.grad, gb, bar);
          bulk_load(at + R::kParam, tile.param, pb, bar);
          bulk_load(at + R::kM, static_cast<const char*>(a.m) + off, sb, bar);
          bulk_load(at + R::kV, static_cast<const char*>(a.v) + off, sb, bar);
        }
      }
      __syncwarp();
      ++issued;
      if (++s == S) s = 0, phase ^= 1u;
      if (tile.len < 0 && ++ends == R::kTeams) break;   // each team gets an end
      if (tile.len >= 0) tile = ahead, ahead = later;
    }
    for (int64_t i = issued > S ? issued - S : 0; i < issued; ++i)   // what is in flight lands
      if (!mbar_wait(full + 8 * uint32_t(i % S), uint32_t(i / S) & 1u)) break;
  } else if (warp == 1) {
    // ---- storer ----
    if (lane == 0) {
      int s = 0, ends = 0;
      uint32_t phase = 0, stored = 0;
      while (ends < R::kTeams) {
        if (!mbar_wait(computed + 8 * s, phase)) {
          atomicOr(&g_fsp_device_error, kErrConsumerWait);
          break;
        }
        const ListTile t = *header(s);
        if (t.len < 0) ++ends;
        if (t.len > 0 && bulk_tile(t)) {
          const uint32_t at = smem_addr(stages + s * R::kStage), n = uint32_t(t.len);
          const int64_t off = t.state_off * (k8Bit ? 1 : 4);
          bulk_store(t.param, at + R::kParam, n * (t.flags & kListParamBf16 ? 2 : 4));
          if (t.copy) bulk_store(t.copy, at + R::kCopy, n * 2);
          bulk_store(static_cast<char*>(a.m) + off, at + R::kM, n * (k8Bit ? 1 : 4));
          bulk_store(static_cast<char*>(a.v) + off, at + R::kV, n * (k8Bit ? 1 : 4));
        }
        bulk_commit();
        // a stage is free once its stores have read it: kLag stages later, so that
        // stores follow each other without waiting
        bulk_wait_read_but<R::kLag>();
        if (stored >= R::kLag) mbar_arrive(empty + 8 * uint32_t((stored - R::kLag) % S));
        ++stored;
        if (++s == S) s = 0, phase ^= 1u;
      }
      // (nothing waits for the last kLag stages: the producer issues no more)
      bulk_wait_all();
    }
  } else {
    // ---- consumers: team k takes stages k, k + kTeams, ... ----
    const int team = (warp - 2) / kTeamWarps, begin = (warp - 2) % kTeamWarps * kListBlock;
    const float coef = a.grad_scale ? *a.grad_scale : 1.f;
    const Coeffs c = list_coeffs<false>(a);
    int s = team;
    uint32_t phase = 0;
    while (true) {
      if (!mbar_wait_all(full + 8 * s, phase)) {
        if (lane == 0) atomicOr(&g_fsp_device_error, kErrConsumerWait);
        break;
      }
      const ListTile t = *header(s);
      if (begin < t.len) {
        if (bulk_tile(t)) {
          update_stage<k8Bit>(a, t, c, coef, begin, lane, stages + s * R::kStage);
        } else {
          ListBlock b;
          load_block<k8Bit>(a, t, begin, lane, b);
          update_block<k8Bit>(a, t, c, coef, begin, lane, b);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(computed + 8 * s);
      if (t.len < 0) break;
      s += R::kTeams;
      if (s >= S) s -= S, phase ^= 1u;
    }
  }
  __syncwarp();
  __syncthreads();
  // the last CTA to finish leaves the counter at 0 for the next launch
  if (R::kCounter && threadIdx.x == 0) {
    __threadfence();   // this thread made the CTA's claims: they are all in the counter
    if (atomicAdd(a.counter + 1, 1ull) == gridDim.x - 1) {
      __threadfence();
      a.counter[0] = 0;
      a.counter[1] = 0;
    }
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
    float2 x[2];
    m_of_codes(*reinterpret_cast<const uint32_t*>(m8 + i), s, x);
    store4(m, false, true, i, 4, x);
    v_of_codes(*reinterpret_cast<const uint32_t*>(v8 + i), t, x);
    store4(v, false, true, i, 4, x);
  }
}

__global__ void __launch_bounds__(kListThreads) list_state_load_kernel(const float* m, const float* v, int8_t* m8,
                                                                       uint8_t* v8, float* ms, float* vs,
                                                                       int64_t n_blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t b = int64_t(blockIdx.x) * (kListThreads / 32) + (threadIdx.x >> 5);
  if (b >= n_blocks) return;
  float2 x[4], y[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b * kListBlock + h * (kListBlock / 2) + lane * 4;
    load4(m, false, true, i, 4, x + 2 * h);
    load4(v, false, true, i, 4, y + 2 * h);
  }
  const BlockScale s = block_scale(block_largest(x)), t = block_scale(block_largest(y));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t i = b * kListBlock + h * (kListBlock / 2) + lane * 4;
    *reinterpret_cast<uint32_t*>(m8 + i) = codes_of_m(x + 2 * h, s);
    *reinterpret_cast<uint32_t*>(v8 + i) = codes_of_v(y + 2 * h, t);
  }
  if (lane == 0) {
    ms[b] = s.s;
    vs[b] = t.s;
  }
}

}  // namespace fsp
