// What the operators on rows of fp32 or bf16 elements share (embedding, layer norm,
// dropout, rotary positions): programmatic launches, element access, and the host's
// checks of matrices.  Not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "fsp_host.h"
#include "fsp_internal.h"
#include "fsp_ops.h"

namespace fsp {

// Programmatic dependent launch: let the next launch on the stream that allows
// it be scheduled; wait until the launches this grid depends on have completed.
// Loads after the wait are ordinary or volatile ones: what a compiler takes for a
// load of constant memory (__ldg and the like) it may move ahead of the wait.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- element access -----------------------------------------------------------

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V elements at p as one access of V * sizeof(T) bytes (4 to 32; p aligned to
// that), or element by element for V = 1.  32 bytes are one access of a whole sector:
// as two of 16 bytes, a warp's stores half-filled every sector twice.
template <typename T, int V>
__device__ __forceinline__ void load_raw(const T* p, T* x) {
  constexpr int kBytes = int(sizeof(T)) * V;
  uint32_t* w = reinterpret_cast<uint32_t*>(x);
  if constexpr (V == 1) {
    x[0] = p[0];
  } else if constexpr (kBytes == 32) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
  } else if constexpr (kBytes == 16) {
    *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p);
  } else if constexpr (kBytes == 8) {
    *reinterpret_cast<uint2*>(x) = *reinterpret_cast<const uint2*>(p);
  } else {
    static_assert(kBytes == 4);
    *w = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  alignas(32) T x[V];
  load_raw<T, V>(p, x);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] = widen(x[j]);
}

template <typename T, int V>
__device__ __forceinline__ void store_raw(T* p, const T* t) {
  constexpr int kBytes = int(sizeof(T)) * V;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(t);
  if constexpr (V == 1) {
    p[0] = t[0];
  } else if constexpr (kBytes == 32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else if constexpr (kBytes == 16) {
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(t));
  } else if constexpr (kBytes == 8) {
    __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(t));
  } else {
    static_assert(kBytes == 4);
    __stcs(reinterpret_cast<uint32_t*>(p), *w);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  alignas(32) T t[V];
#pragma unroll
  for (int j = 0; j < V; ++j) t[j] = narrow<T>(f[j]);
  store_raw<T, V>(p, t);
}

// ---- host ----------------------------------------------------------------------------

inline size_t size_of(int32_t dtype) { return dtype == FSP_DTYPE_F32 ? 4 : 2; }
inline bool known(int32_t dtype) { return dtype == FSP_DTYPE_F32 || dtype == FSP_DTYPE_BF16; }
inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Bytes from a matrix's first to past its last element.
inline size_t span_bytes(int64_t rows, int64_t cols, int64_t stride, int32_t dtype) {
  return rows > 0 && cols > 0 ? (size_t(rows - 1) * size_t(stride) + size_t(cols)) * size_of(dtype) : 0;
}

// A matrix's arguments, without asking whether its memory is there.
inline fsp_status check_form(const void* p, int64_t rows, int64_t cols, int64_t stride, int32_t dtype, const char* name) {
  if (!known(dtype)) return fail(FSP_EINVAL, std::string("unknown dtype of ") + name);
  if (stride < cols || (rows > 0 && stride > (int64_t(1) << 58) / rows))
    return fail(FSP_EINVAL, std::string(name) + "'s rows overlap or their stride is out of range");
  if (!span_bytes(rows, cols, stride, dtype)) return FSP_OK;
  if (!p) return fail(FSP_EINVAL, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % size_of(dtype)) return fail(FSP_EINVAL, std::string(name) + " is not aligned to its elements");
  return FSP_OK;
}

inline fsp_status check_matrix(const void* p, int64_t rows, int64_t cols, int64_t stride, int32_t dtype, const char* name) {
  const fsp_status s = check_form(p, rows, cols, stride, dtype, name);
  const size_t bytes = span_bytes(rows, cols, stride, dtype);
  return s != FSP_OK || !bytes ? s : check_allocation(p, bytes, name);
}

inline bool overlap(const void* p, size_t pb, const void* q, size_t qb) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return pb && qb && a < b + qb && b < a + pb;
}

// One of a call's buffers (bytes 0: it has none).
struct Operand {
  const void* p;
  size_t bytes;
  const char* name;
  int64_t stride = 0;   // above 0: of rows that a result may take the place of
  int32_t dtype = -1;
  size_t row_bytes = 0;
};
inline Operand rows_operand(const void* p, int64_t rows, int64_t cols, int64_t stride, int32_t dtype, const char* name) {
  return {p, p ? span_bytes(rows, cols, stride, dtype) : 0, name, stride, dtype, size_t(cols) * size_of(dtype)};
}

// Whether a and b meet: their spans do, and they are not columns of their own within the
// same rows.
inline bool meet(const Operand& a, const Operand& b) {
  if (!overlap(a.p, a.bytes, b.p, b.bytes)) return false;
  if (a.stride <= 0 || b.stride <= 0) return true;
  const size_t pitch = size_t(a.stride) * size_of(a.dtype);
  if (pitch != size_t(b.stride) * size_of(b.dtype)) return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const size_t at = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;   // b's first column, from a's
  return at < a.row_bytes || at + b.row_bytes > pitch;
}

// What a call writes overlaps nothing, unless it takes the place of an input's rows exactly;
// then that all of it lies in live allocations.
inline fsp_status check_operands(const Operand* out, int n_out, const Operand* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (meet(out[i], out[j]))
        return fail(FSP_EINVAL, std::string(out[i].name) + " overlaps " + out[j].name);
    for (int j = 0; j < n_in; ++j) {
      const bool same = out[i].stride > 0 && out[i].p == in[j].p && out[i].stride == in[j].stride && out[i].dtype == in[j].dtype;
      if (!same && meet(out[i], in[j]))
        return fail(FSP_EINVAL, std::string(out[i].name) + " overlaps " + in[j].name);
    }
  }
  for (int i = 0; i < n_out + n_in; ++i) {
    const Operand& o = i < n_out ? out[i] : in[i - n_out];
    const fsp_status s = o.bytes ? check_allocation(o.p, o.bytes, o.name) : FSP_OK;
    if (s != FSP_OK) return s;
  }
  return FSP_OK;
}

// Whether rows of V elements may be accessed as vectors.
inline bool rows_fit(const void* p, int64_t stride, int32_t dtype, int v) {
  const size_t bytes = size_t(v) * size_of(dtype);
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && size_t(stride) * size_of(dtype) % bytes == 0;
}

// Launches with programmatic stream serialisation (every kernel here waits for the
// launch before it ahead of its first access), a cluster of `cluster` CTAs.
template <typename A>
fsp_status launch_next(void (*kernel)(A), dim3 grid, int threads, size_t smem, int cluster, const A& args, cudaStream_t st,
                       const char* what) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
  return e == cudaSuccess ? FSP_OK : fail(FSP_ECUDA, cuda_msg(what, e));
}

}  // namespace fsp
