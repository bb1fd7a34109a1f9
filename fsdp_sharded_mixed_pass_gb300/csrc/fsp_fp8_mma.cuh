// The product of two 8-bit block-scaled matrices on the tensor cores (sm_103a):
//
//   D[p][q] = sum_k (P[p][k] s_P[p][k / 128]) (Q[q][k] s_Q[q][k / 128])
//
// tcgen05.mma kind::mxf8f6f4 multiplies e4m3 codes and applies an 8-bit
// exponent per row and 32 elements of k inside the tensor core, so a scale per
// 128 costs nothing: its byte is named for all four instructions of a block.
//
// Two kernels.  fp8_product_kernel, for products of few tiles, a persistent CTA per
// SM with six warps:
//   warp 0     producer: bulk copies of the operands' tiles (stored in the order
//              that shared memory wants them, so each is one run of bytes) and
//              of their scales into a ring of stages, a block of 128 of k each;
//   warp 1     issues the copies of a stage's scales to tensor memory and its
//              four MMAs; owns the tensor memory;
//   warps 2-5  read a finished accumulator (32 lanes of tensor memory each),
//              round it and write C, while the next tile is being summed in the
//              other accumulator.
// fp8_pair_kernel, for all others, two CTAs (SMs) per 256 x 256 tile: below.
// Every mbarrier wait gives up after about 2 s, records a bit in the error word
// and ends its role; the CTA then lets its copies land and frees its memory.
//
// Bound: the tensor cores (3.8 PFLOP/s taken as twice the measured bf16 rate), and
// for short k the epilogue beside them.  Measured, launches back to back in a graph:
// 8192^3 304-313 us = 3510-3620 TFLOP/s (box to box), 8192 x 5632 x 2048 58.6 us = 3225,
// 8192 x 2048 x 5632 57 us, 4096 x 151936 x 1024 431-445 us = 2860-2960.

#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace fsp {
namespace {

constexpr unsigned kErrProduct = 32u;   // a wait of the product kernel ran out
__device__ unsigned int g_fp8_error = 0;

// ---- PTX ----------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// kPair: what is waited for may come from the other CTA of a cluster.
template <bool kPair>
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
// False once about 2 s have passed.
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (mbar_try<false>(bar, parity)) return true;
    if ((i & 255u) == 0) {
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (t - t0 > 2000000000ull) break;
    }
  }
  atomicOr(&g_fp8_error, kErrProduct);
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < 4; ++i)
    if (mbar_try<false>(bar, parity)) return true;
  return mbar_wait_slow(bar, parity);
}
// The same by a whole warp, whose lanes agree on whether it ran out (what they do next
// elects one of them, or wants them all).
template <bool kPair>
__device__ __noinline__ bool mbar_wait_slow_all(uint32_t bar, uint32_t parity) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (__all_sync(0xffffffffu, mbar_try<kPair>(bar, parity))) return true;
    if ((i & 255u) == 0) {
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (__any_sync(0xffffffffu, t - t0 > 2000000000ull)) break;
    }
  }
  if ((threadIdx.x & 31) == 0) atomicOr(&g_fp8_error, kErrProduct);
  return false;
}
template <bool kPair = false>
__device__ __forceinline__ bool mbar_wait_all(uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_try<kPair>(bar, parity))) return true;
  return mbar_wait_slow_all<kPair>(bar, parity);
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// One lane of a converged warp.  The warps that issue MMAs and copies run their
// loops whole, so that addresses and descriptors live in uniform registers, and
// elect a lane for the instructions themselves (with the whole loop inside a
// single-lane branch a block of k took 717 cycles to issue, above its MMAs' 512).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Programmatic dependent launch: let the next launch on the stream that allows
// it be scheduled; wait until the launches this grid depends on have completed.
// Loads after the wait are ordinary or volatile ones: what a compiler takes for a
// load of constant memory (__ldg and the like) it may move ahead of the wait.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void scale_copy(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                           bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(uint32_t(add))
      : "memory");
}
// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors.  Operands: rows of 128 bytes in the 128-byte
// swizzle, eight rows (1024 bytes) apart from the next eight.  Scales: 32 rows of
// 16 bytes, no swizzle, eight rows (128 bytes) apart from the next eight.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return uint64_t((addr & 0x3ffffu) >> 4) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
         uint64_t(2) << 61;
}
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return uint64_t((addr & 0x3ffffu) >> 4) | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
}

// A producer's last stages (it would fill stage s next, with parity `phase`), before the
// CTA's memory is given back: the commits that free them have arrived - nobody else
// waits for these, and one still on its way would land in the memory of whatever runs
// here next - and with them the copies that the products read.  Where a wait runs out,
// the copies in flight land (`counts`: they count at this CTA's barriers).  kPair: by a
// whole warp of a pair's CTA, else by one thread.
template <int S, bool kPair = false>
__device__ __forceinline__ void wait_last_stages(uint32_t full, uint32_t empty, int s, uint32_t phase, bool counts = true) {
  auto wait = [](uint32_t bar, uint32_t parity) { return kPair ? mbar_wait_all<true>(bar, parity) : mbar_wait(bar, parity); };
  bool ok = true;
#pragma unroll 1
  for (int j = 0; j < S && ok; ++j) ok = wait(empty + 8 * j, j < s ? phase : phase ^ 1u);   // (a stage never filled: passes)
#pragma unroll 1
  for (int j = 0; j < S && !ok && counts; ++j)
    if (!wait(full + 8 * j, j < s ? phase : phase ^ 1u)) break;
}

// ---- the kernel ----------------------------------------------------------------------

constexpr int kMmThreads = 192;
constexpr int kTileP = 128;
constexpr int kGroupP = 32;   // tiles of P walked before the next tile of Q

struct MmArgs {
  const uint8_t* p;
  const uint8_t* q;
  void* c;
  int64_t np, nq;             // rows of P and Q
  int64_t blocks;             // of 128 along k
  int64_t pieces;             // of 512 along k (scales)
  int64_t p_scales, q_scales; // byte offsets of the scales
  int64_t c_stride;
  int64_t tiles_p, tiles_q;
  int accumulate;
  int vec;                    // C's rows are 16-byte aligned
};

// The epilogue's part of shared memory, per warp: 16 rows of 128 bytes.
constexpr int kStagePitch = 128 + 16;             // bytes of a row: eight lanes' 16-byte stores meet no bank twice
constexpr int kWarpStage = 16 * kStagePitch;

// BN: rows of Q per tile, a part of a stored tile of 128.
template <int BN>
struct MmCfg {
  static constexpr int kScaleCols = 8;                              // tensor memory columns of a stage's scales: 4 of P, 4 of Q
  static constexpr int kStageBytes = kTileP * 128 + BN * 128 + 1024;
  static constexpr int kEpilogue = 4 * kWarpStage;
  static constexpr int kFixed = 1024 + 256 + kEpilogue;             // alignment, barriers, epilogue
  static constexpr int kFit = (232448 - kFixed) / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kAccCols = BN < 32 ? 32 : BN;
  static constexpr int kScaleBase = 2 * kAccCols;
  static constexpr int kColsUsed = kScaleBase + kStages * kScaleCols;
  static constexpr int kCols = kColsUsed <= 128 ? 128 : kColsUsed <= 256 ? 256 : 512;
  static constexpr int kSmem = kFixed + kStages * kStageBytes;
  static_assert(kColsUsed <= 512, "tensor memory");
  static_assert(128 % BN == 0 && BN % 16 == 0, "tile of Q");
};

struct TileAt {
  int64_t p, q;
};
// Tiles of P in groups, all of a group before the next tile of Q: the CTAs that
// run at one time share few tiles of each operand.
__device__ __forceinline__ TileAt tile_at(const MmArgs& g, int64_t t) {
  const int64_t per_group = kGroupP * g.tiles_q;
  const int64_t group = t / per_group, rest = t - group * per_group;
  const int64_t size = min(int64_t(kGroupP), g.tiles_p - group * kGroupP);
  return {group * kGroupP + rest % size, rest / size};
}

__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Rows p0 .. p0 + 31 (a lane each), columns q0 .. q0 + kCols - 1 of C from registers,
// through this warp's part of shared memory, 16 rows at a time, so that rows are
// written in whole lines: 128 bytes, 64 columns of bf16 or 32 of fp32.
template <typename T>
constexpr int kLineCols = 128 / int(sizeof(T));

template <typename T>
__device__ __forceinline__ void write_lines(const MmArgs& g, const uint32_t* x, unsigned char* stage, int lane, int64_t p0,
                                            int64_t q0) {
  constexpr int kCols = kLineCols<T>;
  T* const c = static_cast<T*>(g.c) + p0 * g.c_stride + q0;
  const int rows = int(min(int64_t(32), g.np - p0)), cols = int(min(int64_t(kCols), g.nq - q0));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h * 16 >= rows) break;
    if (lane >> 4 == h) {
      uint4* mine = reinterpret_cast<uint4*>(stage + (lane & 15) * kStagePitch);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (sizeof(T) == 4)
          mine[j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        else
          mine[j] = make_uint4(pack_bf16(x[8 * j], x[8 * j + 1]), pack_bf16(x[8 * j + 2], x[8 * j + 3]),
                               pack_bf16(x[8 * j + 4], x[8 * j + 5]), pack_bf16(x[8 * j + 6], x[8 * j + 7]));
      }
    }
    __syncwarp();
    if (g.vec && cols == kCols) {
      const int r = lane >> 3, v = lane & 7;   // four rows of eight 16-byte vectors at a time
      uint4* dst = reinterpret_cast<uint4*>(c + (h * 16 + r) * g.c_stride) + v;
      const int64_t step = g.c_stride * int(sizeof(T)) / 4;   // four rows, in vectors
#pragma unroll
      for (int i = 0; i < 16; i += 4, dst += step) {
        if (h * 16 + i + r >= rows) break;
        uint4 y = *reinterpret_cast<const uint4*>(stage + (i + r) * kStagePitch + v * 16);
        if constexpr (sizeof(T) == 4) {
          if (g.accumulate) {
            const float4 o = *reinterpret_cast<const float4*>(dst);
            y = make_uint4(__float_as_uint(__uint_as_float(y.x) + o.x), __float_as_uint(__uint_as_float(y.y) + o.y),
                           __float_as_uint(__uint_as_float(y.z) + o.z), __float_as_uint(__uint_as_float(y.w) + o.w));
          }
        }
        *dst = y;
      }
    } else {
      const int n = min(16, rows - h * 16);
#pragma unroll
      for (int v0 = 0; v0 < kCols; v0 += 32) {   // a lane per element
        const int v = v0 + lane;
        if (v >= cols) continue;
        T* dst = c + int64_t(h * 16) * g.c_stride + v;
#pragma unroll 4
        for (int i = 0; i < n; ++i, dst += g.c_stride) {
          T y = *reinterpret_cast<const T*>(stage + i * kStagePitch + v * int(sizeof(T)));
          if constexpr (sizeof(T) == 4) {
            if (g.accumulate) y += *dst;
          }
          *dst = y;
        }
      }
    }
    __syncwarp();
  }
}
// 64 columns from registers.
template <typename T>
__device__ __forceinline__ void write_block(const MmArgs& g, const uint32_t* acc, unsigned char* stage, int lane, int64_t p0,
                                            int64_t q0) {
#pragma unroll
  for (int k = 0; k < 64; k += kLineCols<T>)
    if (p0 < g.np && q0 + k < g.nq) write_lines<T>(g, acc + k, stage, lane, p0, q0 + k);
}

template <int BN, bool kSwap, typename T>
__global__ void __launch_bounds__(kMmThreads, 1) fp8_product_kernel(const __grid_constant__ MmArgs g) {
  using Cfg = MmCfg<BN>;
  constexpr int S = Cfg::kStages;
  extern __shared__ unsigned char raw[];
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* smem = raw + (base - smem_addr(raw));
  const uint32_t at_p = base, at_q = at_p + S * kTileP * 128, at_sp = at_q + S * BN * 128;
  const uint32_t at_sq = at_sp + S * 512, at_epi = at_sq + S * 512;
  const uint32_t bars = at_epi + Cfg::kEpilogue;
  const uint32_t full = bars, empty = full + 8 * S, acc_full = empty + 8 * S, acc_empty = acc_full + 16;
  const uint32_t drained = acc_empty + 16, slot = drained + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, 4);
    }
    mbar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 1) tmem_alloc(slot, Cfg::kCols);
  fence_before();
  __syncthreads();
  fence_after();
  launch_dependents();
  grid_dependency_wait();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - base));
  const int64_t tiles = g.tiles_p * g.tiles_q;
  const int blocks = int(g.blocks);

  if (warp == 0 && lane == 0) {
    // ---- producer ----
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const TileAt tile = tile_at(g, t);
      const int64_t q0 = tile.q * BN, q_tile = q0 >> 7;
      const uint8_t* src_p = g.p + tile.p * g.blocks * kTileBytes;
      const uint8_t* src_q = g.q + q_tile * g.blocks * kTileBytes + (q0 & 127) * 128;
      const uint8_t* src_sp = g.p + g.p_scales + tile.p * g.pieces * kScaleBytes;
      const uint8_t* src_sq = g.q + g.q_scales + q_tile * g.pieces * kScaleBytes;
      for (int k = 0; k < blocks; ++k) {
        if (!(ok = mbar_wait(empty + 8 * s, phase ^ 1u))) break;
        const uint32_t bar = full + 8 * s;
        const int64_t piece = int64_t(k >> 2) * kScaleBytes;
        mbar_expect(bar, Cfg::kStageBytes);
        bulk_load(at_p + s * kTileP * 128, src_p + int64_t(k) * kTileBytes, kTileP * 128, bar);
        bulk_load(at_q + s * BN * 128, src_q + int64_t(k) * kTileBytes, BN * 128, bar);
        bulk_load(at_sp + s * 512, src_sp + piece, 512, bar);
        bulk_load(at_sq + s * 512, src_sq + piece, 512, bar);
        if (++s == S) s = 0, phase ^= 1u;
      }
    }
    wait_last_stages<S>(full, empty, s, phase);
  } else if (warp == 1) {
    // ---- scales and MMAs ----
    const uint32_t idesc = uint32_t(BN >> 3) << 17 | 1u << 23 | uint32_t(kTileP >> 4) << 24;
    const uint64_t desc_p = operand_desc(at_p), desc_q = operand_desc(at_q);
    const uint64_t desc_sp = scale_desc(at_sp), desc_sq = scale_desc(at_sq);
    int s = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const uint32_t sq_shift = uint32_t((tile_at(g, t).q * BN) & 127) / 32;   // columns of the scales before q0
      if (!(ok = mbar_wait_all(acc_empty + 8 * buf, acc_phase ^ 1u))) break;
      fence_after();
      const uint32_t d = tmem + buf * Cfg::kAccCols;
      for (int k = 0; k < blocks; ++k) {
        if (!(ok = mbar_wait_all(full + 8 * s, phase))) break;
        fence_after();
        const uint32_t sp = tmem + Cfg::kScaleBase + s * Cfg::kScaleCols, sq = sp + 4;
        const uint32_t id = idesc | uint32_t(k & 3) << 4 | uint32_t(k & 3) << 29;   // which byte of a row's four
        const uint64_t dp = desc_p + uint64_t(s * (kTileP * 128 / 16)), dq = desc_q + uint64_t(s * (BN * 128 / 16));
        if (elect_one()) {
          scale_copy(sp, desc_sp + uint64_t(s * 32));
          scale_copy(sq, desc_sq + uint64_t(s * 32));
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_scaled(d, dp + 2 * i, dq + 2 * i, id, sp, sq + sq_shift, (k | i) != 0);
          mma_commit(empty + 8 * s);
        }
        __syncwarp();
        if (++s == S) s = 0, phase ^= 1u;
      }
      if (elect_one()) mma_commit(acc_full + 8 * buf);   // (on a wait that ran out too: what was issued completes)
      __syncwarp();
      buf ^= 1;
      if (buf == 0) acc_phase ^= 1u;
    }
    if (elect_one()) mma_commit(drained);   // nothing issued here runs on when the tensor memory is given back
    __syncwarp();
    mbar_wait_all(drained, 0);
  } else if (warp >= 2) {
    // ---- epilogue ----
    const int quarter = warp & 3;   // the tensor memory lanes this warp may read
    unsigned char* stage = smem + (at_epi - base) + (warp - 2) * kWarpStage;
    int buf = 0;
    uint32_t phase = 0;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
      const TileAt tile = tile_at(g, t);
      if (!mbar_wait_all(acc_full + 8 * buf, phase)) break;
      fence_after();
      const uint32_t d = tmem + buf * Cfg::kAccCols + (uint32_t(quarter * 32) << 16);
      const int64_t p0 = tile.p * kTileP + quarter * 32, q0 = tile.q * BN;
      if constexpr (kSwap) {
        // a lane holds one row of P: 32 lanes are 32 neighbours of a row of C
        T* c = static_cast<T*>(g.c) + p0 + lane;
#pragma unroll
        for (int j0 = 0; j0 < BN; j0 += 16) {
          uint32_t acc[16];
          tmem_load16(d + j0, acc);
          tmem_wait_loads();
          if (p0 + lane < g.np) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (q0 + j0 + j >= g.nq) break;
              T* dst = c + (q0 + j0 + j) * g.c_stride;
              if constexpr (sizeof(T) == 4)
                *dst = g.accumulate ? *dst + __uint_as_float(acc[j]) : __uint_as_float(acc[j]);
              else
                *dst = __float2bfloat16_rn(__uint_as_float(acc[j]));
            }
          }
          __syncwarp();
        }
      } else {
        static_assert(BN % 64 == 0 || kSwap, "whole blocks of 64 columns");
#pragma unroll 1
        for (int j0 = 0; j0 < BN; j0 += 64) {
          uint32_t acc[64];
          tmem_load32(d + j0, acc);
          tmem_load32(d + j0 + 32, acc + 32);
          tmem_wait_loads();
          write_block<T>(g, acc, stage, lane, p0, q0 + j0);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * buf);
      buf ^= 1;
      if (buf == 0) phase ^= 1u;
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 1) tmem_free(tmem, Cfg::kCols);
}


// ---- pairs of CTAs ---------------------------------------------------------------------
//
// Large products: two SMs work on one 256 x 256 tile (cta_group::2).  Each CTA
// loads 128 rows of P and 128 rows of Q, and the tensor cores of both read both
// halves of Q, so a byte loaded is used for twice as many products.  The leader
// (rank 0 of the cluster) issues the MMAs of both.  The copies of both count at the
// leader's barrier, which tensor copies with cta_group::2 can do (a bulk copy signals
// its own CTA only): the MMAs then wait for what they read itself, with no thread of
// the other CTA to pass the word on.  Every wait here acquires at cluster scope.
//
// Tensor memory: two accumulators of 256 columns and the scales do not fit into
// 512 columns, so the accumulators overlap by the scales' 24 columns.  The
// epilogue reads the overlapping block of an accumulator first and gives it
// back; the next tile's sum starts then, into the other accumulator.  Scales are
// copied once per four blocks of k into one of two slots.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// Arrives at a barrier of the other CTA.  Relaxed: what it reports, reads of tensor
// memory, is ordered by the tcgen05 fences on both sides.
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Tile `t` of a map (its box at coordinates 0, 0, t) into this CTA's shared memory; its
// bytes count at the barrier of the pair's leader.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int32_t t, uint32_t leader_bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(0), "r"(t), "r"(leader_bar)
      : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar) {   // arrives at `bar` of both CTAs
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"(uint16_t(3))
               : "memory");
}
__device__ __forceinline__ void pair_commit_here(uint32_t bar) {   // ... of this CTA alone
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void pair_scale_copy(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(uint32_t(add))
      : "memory");
}

struct PairCfg {
  static constexpr int kTile = 256;                     // of P and of Q
  static constexpr int kOperand = 128 * 128;            // bytes of one operand's stage in one CTA
  static constexpr int kScales = 3 * 512;               // a stage's scales: 128 rows of P, 256 of Q
  static constexpr int kWarps = 8;                      // of the epilogue, two per quarter of the rows
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kEpilogue = kWarps * kWarpStage;
  static constexpr int kStages = 6;
  static constexpr int kSmem = 1024 + 256 + kEpilogue + kStages * (2 * kOperand + kScales);
  static constexpr int kScaleCols = 12;
  static constexpr int kScaleBase = 512 - 2 * kScaleCols;
  static constexpr int kSecond = kScaleBase - 256;      // first column of the second accumulator
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(256 - kSecond <= 64, "the overlap lies within one block of 64 columns of either accumulator");
  // a slot of scales is waited for by the barrier of a stage five blocks back, which
  // must not have come round again
  static_assert(kStages >= 5, "stages");
};

// The operands as tensors of tiles: 128 rows x 128 bytes of codes, 4 x 128 bytes of scales.
struct PairArgs {
  MmArgs g;
  CUtensorMap p, q, p_scales, q_scales;
};

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg::kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ PairArgs a) {
  using Cfg = PairCfg;
  const MmArgs& g = a.g;
  constexpr int S = Cfg::kStages;
  extern __shared__ unsigned char raw[];
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  unsigned char* smem = raw + (base - smem_addr(raw));
  const uint32_t at_p = base, at_q = at_p + S * Cfg::kOperand, at_s = at_q + S * Cfg::kOperand;
  const uint32_t at_epi = at_s + S * Cfg::kScales;
  const uint32_t bars = at_epi + Cfg::kEpilogue;
  const uint32_t full = bars, empty = full + 8 * S, acc_full = empty + 8 * S, acc_part = acc_full + 16;
  const uint32_t drained = acc_part + 16, slot = drained + 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);   // the leader's: both CTAs' copies (the other's is not used)
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_part + 8 * b, 2 * Cfg::kWarps);
    }
    mbar_init(drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 1) asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
  fence_before();
  __syncthreads();
  cluster_sync_all();
  fence_after();
  launch_dependents();
  grid_dependency_wait();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + (slot - base));
  const int64_t tiles = g.tiles_p * g.tiles_q;
  const int64_t step = gridDim.x >> 1;
  const int blocks = int(g.blocks);

  if (warp == 0) {
    // ---- producer: this CTA's 128 rows of each operand ----
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int64_t p_tiles = (g.np + 127) >> 7, q_tiles = (g.nq + 127) >> 7;
    const uint32_t leader_full = in_cta(full, 0);
    for (int64_t t = blockIdx.x >> 1; t < tiles && ok; t += step) {
      const TileAt tile = tile_at(g, t);
      const int64_t p_first = tile.p * 2, q_first = tile.q * 2, p_tile = p_first + rank, q_tile = q_first + rank;
      const bool has_p = p_tile < p_tiles, has_q = q_tile < q_tiles;   // rows past the matrices are not loaded
      const uint32_t halves_p = p_first + 1 < p_tiles ? 2 : 1, halves_q = q_first + 1 < q_tiles ? 2 : 1;
      // both CTAs': codes, and each one's rows of P and all of Q of the scales
      const uint32_t bytes = (halves_p + halves_q) * uint32_t(Cfg::kOperand);
      const uint32_t scale_bytes = 512u * (halves_p + 2 * halves_q);
      const int32_t at_tile_p = int32_t(p_tile * g.blocks), at_tile_q = int32_t(q_tile * g.blocks);
      const int32_t piece_p = int32_t(p_tile * g.pieces), piece_q = int32_t(q_first * g.pieces);
      for (int k = 0; k < blocks; ++k) {
        if (!(ok = mbar_wait_all<true>(empty + 8 * s, phase ^ 1u))) break;
        const uint32_t bar = leader_full + 8 * s;
        const bool scales = (k & 3) == 0;
        if (elect_one()) {
          if (rank == 0) mbar_expect(full + 8 * s, bytes + (scales ? scale_bytes : 0u));
          if (has_p) pair_load(at_p + s * Cfg::kOperand, &a.p, at_tile_p + k, bar);
          if (has_q) pair_load(at_q + s * Cfg::kOperand, &a.q, at_tile_q + k, bar);
          if (scales) {
            const uint32_t dst = at_s + s * Cfg::kScales;
            if (has_p) pair_load(dst, &a.p_scales, piece_p + (k >> 2), bar);
            for (uint32_t j = 0; j < halves_q; ++j)
              pair_load(dst + 512 * (1 + j), &a.q_scales, piece_q + int32_t(j * g.pieces) + (k >> 2), bar);
          }
        }
        __syncwarp();
        if (++s == S) s = 0, phase ^= 1u;
      }
    }
    wait_last_stages<S, true>(full, empty, s, phase, rank == 0);
  } else if (warp == 1 && rank == 0) {
    // ---- leader: scales and MMAs of both CTAs ----
    const uint32_t idesc = uint32_t(Cfg::kTile >> 3) << 17 | 1u << 23 | uint32_t(Cfg::kTile >> 4) << 24;
    const uint64_t desc_p = operand_desc(at_p), desc_q = operand_desc(at_q), desc_s = scale_desc(at_s);
    int s = 0, n = 0;   // n: tiles so far
    uint32_t phase = 0, group = 0;
    // the barrier and parity that show the last block reading each slot of scales complete
    uint32_t bar0 = 0, par0 = 0, bar1 = 0, par1 = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x >> 1; t < tiles && ok; t += step, ++n) {
      // the columns that this tile's accumulator shares with the one before it have been read
      if (n > 0 && !(ok = mbar_wait_all<true>(acc_part + 8 * ((n - 1) & 1), uint32_t((n - 1) >> 1) & 1u))) break;
      fence_after();
      const uint32_t d = tmem + (n & 1 ? Cfg::kSecond : 0);
      uint32_t sp = 0;
      for (int k = 0; k < blocks; ++k) {
        if (!(ok = mbar_wait_all<true>(full + 8 * s, phase))) break;
        if ((k & 3) == 0) {
          if (group >= 2 && !(ok = mbar_wait_all<true>(group & 1 ? bar1 : bar0, group & 1 ? par1 : par0))) break;
          sp = tmem + Cfg::kScaleBase + (group & 1) * Cfg::kScaleCols;
        }
        fence_after();
        const uint32_t id = idesc | uint32_t(k & 3) << 4 | uint32_t(k & 3) << 29;
        const uint64_t dp = desc_p + uint64_t(s * (Cfg::kOperand / 16)), dq = desc_q + uint64_t(s * (Cfg::kOperand / 16));
        const uint64_t ds = desc_s + uint64_t(s * (Cfg::kScales / 16));
        if (elect_one()) {
          if ((k & 3) == 0) {
            pair_scale_copy(sp, ds);
            pair_scale_copy(sp + 4, ds + 32);
            pair_scale_copy(sp + 8, ds + 64);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) pair_mma(d, dp + 2 * i, dq + 2 * i, id, sp, sp + 4, (k | i) != 0);
          pair_commit(empty + 8 * s);
        }
        __syncwarp();
        if ((k & 3) == 3 || k + 1 == blocks) {   // the slot's last block
          if (group & 1)
            bar1 = empty + 8 * s, par1 = phase;
          else
            bar0 = empty + 8 * s, par0 = phase;
          ++group;
        }
        if (++s == S) s = 0, phase ^= 1u;
      }
      if (elect_one()) pair_commit(acc_full + 8 * (n & 1));
      __syncwarp();
    }
    if (elect_one()) pair_commit_here(drained);   // (the other CTA's epilogue and producer wait for the commits to them)
    __syncwarp();
    mbar_wait_all<true>(drained, 0);
  } else if (warp >= 2) {
    // ---- epilogue: this CTA's 128 rows ----
    const int quarter = warp & 3, half = (warp - 2) >> 2;   // rows; alternate blocks of 64 columns
    unsigned char* stage = smem + (at_epi - base) + (warp - 2) * kWarpStage;
    int n = 0;
    for (int64_t t = blockIdx.x >> 1; t < tiles; t += step, ++n) {
      const TileAt tile = tile_at(g, t);
      const int buf = n & 1;
      if (!mbar_wait_all<true>(acc_full + 8 * buf, uint32_t(n >> 1) & 1u)) break;
      fence_after();
      const uint32_t d = tmem + (buf ? Cfg::kSecond : 0) + (uint32_t(quarter * 32) << 16);
      const int64_t p0 = tile.p * Cfg::kTile + rank * 128 + quarter * 32, q0 = tile.q * Cfg::kTile;
#pragma unroll 1
      for (int j = 64 * half; j < Cfg::kTile; j += 128) {
        // the first accumulator's last block, the second one's first, are what the other needs next
        const int j0 = buf ? j : 192 - j;
        uint32_t acc[64];
        tmem_load32(d + j0, acc);
        tmem_load32(d + j0 + 32, acc + 32);
        tmem_wait_loads();
        if (j < 128) {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(in_cta(acc_part + 8 * buf, 0));
        }
        write_block<T>(g, acc, stage, lane, p0, q0 + j0);
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  // Neither CTA's memory is read or signalled by the other any more: each has waited for
  // every commit that arrives at its barriers (producer: the stages', epilogue: the
  // accumulators', leader: drained), and the epilogue's arrivals come before this.
  cluster_sync_all();
  fence_after();
  if (warp == 1) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

}  // namespace
}  // namespace fsp
