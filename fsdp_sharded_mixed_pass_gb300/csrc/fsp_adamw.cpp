// Host side of AdamW over a list of tensors: the registered list and its work
// tiles, argument checks and the C entry points.  The kernels are in
// fsp_adamw_kernels.cuh.
#include <cuda_runtime_api.h>

#include <algorithm>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "fsp_host.h"
#include "fsp_list.h"

struct fsp_adamw_list {
  int device = -1;
  int64_t state_len = 0;
  std::vector<int64_t> offsets;
  fsp::ListTile* tiles = nullptr;   // device, with the launches' two counters behind them
  int64_t n_tiles = 0, bulk_tiles = 0;
  // every registered tensor as [begin, end) device addresses, sorted by begin
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
};

namespace fsp {
namespace {

size_t size_of(int32_t dtype) { return dtype == FSP_DTYPE_F32 ? 4 : 2; }

void free_list(fsp_adamw_list* l) {
  if (!l) return;
  if (l->tiles) {
    int prev = -1;
    const bool have_prev = cudaGetDevice(&prev) == cudaSuccess;
    if (cudaSetDevice(l->device) == cudaSuccess) cudaFree(l->tiles);
    if (have_prev) cudaSetDevice(prev);
  }
  delete l;
}

struct ListOwner {   // frees a half-made list on every early return
  fsp_adamw_list* l;
  ~ListOwner() { free_list(l); }
};

fsp_status create_list(int32_t n, const int64_t* numels, void* const* params, const int32_t* pd,
                       const void* const* grads, const int32_t* gd, void* const* copies, fsp_adamw_list** out) {
  if (!out) return fail(FSP_EINVAL, "out is NULL");
  *out = nullptr;
  if (n < 0) return fail(FSP_EINVAL, "n must be >= 0");
  if (n > 0 && (!numels || !params || !pd || !grads || !gd)) return fail(FSP_EINVAL, "an argument array is NULL");
  ListOwner own{new fsp_adamw_list()};
  fsp_adamw_list* l = own.l;
  std::vector<ListTile> tiles;
  struct Span {
    uintptr_t begin, end;
    std::string name;
  };
  std::vector<Span> spans;
  for (int32_t i = 0; i < n; ++i) {
    const std::string at = "[" + std::to_string(i) + "]";
    if (numels[i] < 0 || numels[i] > (int64_t(1) << 44)) return fail(FSP_EINVAL, "numels" + at + " out of range");
    if ((pd[i] != FSP_DTYPE_F32 && pd[i] != FSP_DTYPE_BF16) || (gd[i] != FSP_DTYPE_F32 && gd[i] != FSP_DTYPE_BF16))
      return fail(FSP_EINVAL, "unknown dtype of tensor " + std::to_string(i));
    l->offsets.push_back(l->state_len);
    const int64_t len = numels[i];
    if (len == 0) continue;
    const struct {
      const void* ptr;
      size_t esz;
      const char* name;
    } bufs[] = {{params[i], size_of(pd[i]), "params"},
                {grads[i], size_of(gd[i]), "grads"},
                {copies ? copies[i] : nullptr, 2, "copies"}};
    bool vec = true, bulk = true;
    for (const auto& b : bufs) {
      if (!b.ptr) {
        if (b.name[0] == 'c') continue;
        return fail(FSP_EINVAL, b.name + at + " is NULL");
      }
      const uintptr_t p = reinterpret_cast<uintptr_t>(b.ptr);
      if (p % b.esz != 0) return fail(FSP_EINVAL, b.name + at + " is not aligned to its elements");
      vec = vec && p % (4 * b.esz) == 0;
      bulk = bulk && p % 16 == 0;
      spans.push_back({p, p + size_t(len) * b.esz, b.name + at});
    }
    const int32_t flags = (pd[i] == FSP_DTYPE_BF16 ? kListParamBf16 : 0) | (gd[i] == FSP_DTYPE_BF16 ? kListGradBf16 : 0) |
                          (vec ? kListVec : 0) | (bulk ? kListBulk : 0);
    for (int64_t k = 0; k < len; k += kListTile) {
      ListTile t{};
      t.param = static_cast<char*>(params[i]) + size_t(k) * size_of(pd[i]);
      t.grad = static_cast<const char*>(grads[i]) + size_t(k) * size_of(gd[i]);
      t.copy = copies && copies[i] ? static_cast<uint16_t*>(copies[i]) + k : nullptr;
      t.state_off = l->state_len + k;
      t.len = int32_t(std::min<int64_t>(kListTile, len - k));
      t.flags = flags;
      tiles.push_back(t);
      l->bulk_tiles += bulk ? 1 : 0;
    }
    l->state_len += (len + kListBlock - 1) / kListBlock * kListBlock;
  }
  std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.begin < y.begin; });
  for (size_t k = 1; k < spans.size(); ++k)
    if (spans[k - 1].end > spans[k].begin) return fail(FSP_EINVAL, spans[k - 1].name + " overlaps " + spans[k].name);
  for (const Span& s : spans) {
    const fsp_status st = check_allocation(reinterpret_cast<const void*>(s.begin), s.end - s.begin, s.name.c_str());
    if (st != FSP_OK) return st;
    l->spans.emplace_back(s.begin, s.end);
  }
  l->n_tiles = int64_t(tiles.size());
  if (!tiles.empty()) {
    cudaError_t e = cudaGetDevice(&l->device);
    if (e != cudaSuccess) return fail(FSP_ECUDA, cuda_msg("cudaGetDevice", e));
    const size_t bytes = tiles.size() * sizeof(ListTile);
    e = cudaMalloc(reinterpret_cast<void**>(&l->tiles), bytes + 2 * sizeof(unsigned long long));
    if (e != cudaSuccess) {
      cudaGetLastError();
      l->tiles = nullptr;
      return fail(FSP_ENOMEM, cuda_msg("cudaMalloc (list tiles)", e));
    }
    e = cudaMemset(l->tiles + tiles.size(), 0, 2 * sizeof(unsigned long long));
    if (e == cudaSuccess) e = upload_table(l->tiles, tiles.data(), bytes);
    if (e != cudaSuccess) return fail(FSP_ECUDA, cuda_msg("uploading the list tiles", e));
  }
  own.l = nullptr;
  *out = l;
  return FSP_OK;
}

bool overlaps_list(const fsp_adamw_list* l, const void* ptr, size_t bytes) {
  if (!bytes) return false;
  const uintptr_t b = reinterpret_cast<uintptr_t>(ptr), e = b + bytes;
  auto it = std::lower_bound(l->spans.begin(), l->spans.end(), std::make_pair(e, uintptr_t(0)));
  return it != l->spans.begin() && std::prev(it)->second > b;
}

struct NamedBuf {
  const void* ptr;
  size_t bytes;
  size_t align;
  const char* name;
};

// NULL, alignment, overlap (with each other and the list's tensors) and
// residence of the buffers of a call; a list without elements has none.
fsp_status check_buffers(const fsp_adamw_list* l, const NamedBuf* bufs, int n) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(FSP_ECUDA, cuda_msg("cudaGetDevice", e));
  if (dev != l->device) return fail(FSP_EINVAL, "the list was created on another device");
  for (int i = 0; i < n; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(bufs[i].ptr);
    if (!a) return fail(FSP_EINVAL, std::string(bufs[i].name) + " is NULL");
    if (a % bufs[i].align)
      return fail(FSP_EINVAL, std::string(bufs[i].name) + " is not " + std::to_string(bufs[i].align) + "-byte aligned");
    if (overlaps_list(l, bufs[i].ptr, bufs[i].bytes))
      return fail(FSP_EINVAL, std::string(bufs[i].name) + " overlaps a registered tensor");
    for (int j = 0; j < i; ++j) {
      const uintptr_t b = reinterpret_cast<uintptr_t>(bufs[j].ptr);
      if (a < b + bufs[j].bytes && b < a + bufs[i].bytes)
        return fail(FSP_EINVAL, std::string(bufs[j].name) + " overlaps " + bufs[i].name);
    }
  }
  for (int i = 0; i < n; ++i) {
    const fsp_status s = check_allocation(bufs[i].ptr, bufs[i].bytes, bufs[i].name);
    if (s != FSP_OK) return s;
  }
  return FSP_OK;
}

fsp_status step_list(const fsp_adamw_list* l, int32_t sd, void* m, void* v, float* ms, float* vs,
                     const fsp_adamw_hparams* hp, int64_t step, int64_t* step_dev, int32_t advance,
                     const float* grad_scale, void* stream) {
  if (!l) return fail(FSP_EINVAL, "list is NULL");
  if (sd != FSP_STATE_F32 && sd != FSP_STATE_8BIT) return fail(FSP_EINVAL, "unknown state dtype");
  const bool eight = sd == FSP_STATE_8BIT;
  if (!eight && (ms || vs)) return fail(FSP_EINVAL, "fp32 states take no scales");
  const fsp_status hs = check_hparams(hp, step_dev ? 1 : step);
  if (hs != FSP_OK) return hs;
  const size_t sbytes = size_t(l->state_len) * (eight ? 1 : 4), cbytes = size_t(l->state_len / kListBlock) * 4;
  NamedBuf bufs[6] = {{m, sbytes, 16, "exp_avg"}, {v, sbytes, 16, "exp_avg_sq"}};
  int nb = 2;
  if (eight) {
    bufs[nb++] = {ms, cbytes, 4, "exp_avg_scale"};
    bufs[nb++] = {vs, cbytes, 4, "exp_avg_sq_scale"};
  }
  if (step_dev) bufs[nb++] = {step_dev, 8, 8, "step_dev"};
  if (grad_scale) bufs[nb++] = {grad_scale, 4, 4, "grad_scale"};
  if (l->n_tiles > 0) {
    fsp_status s = check_buffers(l, bufs, nb);
    if (s != FSP_OK) return s;
    StepArgs sa{};
    set_coeffs(sa, hp, step_dev ? 1 : step);
    ListArgs a{};
    a.tiles = l->tiles;
    a.n_tiles = l->n_tiles;
    a.bulk_tiles = l->bulk_tiles;
    a.counter = reinterpret_cast<unsigned long long*>(l->tiles + l->n_tiles);
    a.m = m;
    a.v = v;
    a.m_scale = ms;
    a.v_scale = vs;
    a.grad_scale = grad_scale;
    a.step_dev = step_dev;
    a.lr = sa.lr;
    a.c = sa.c;
    s = launch_adamw_list(a, eight, stream);
    if (s != FSP_OK) return s;
  } else if (step_dev) {
    const fsp_status s = check_allocation(step_dev, 8, "step_dev");
    if (s != FSP_OK) return s;
  }
  return step_dev && advance ? advance_step(step_dev, stream) : FSP_OK;
}

fsp_status state_list(bool load, const fsp_adamw_list* l, const void* m8, const void* v8, const float* ms,
                      const float* vs, const float* m, const float* v, void* stream) {
  if (!l) return fail(FSP_EINVAL, "list is NULL");
  if (l->n_tiles == 0) return FSP_OK;
  const size_t n = size_t(l->state_len), c = n / kListBlock * 4;
  const NamedBuf bufs[6] = {{m8, n, 16, "exp_avg"},
                            {v8, n, 16, "exp_avg_sq"},
                            {ms, c, 4, "exp_avg_scale"},
                            {vs, c, 4, "exp_avg_sq_scale"},
                            {m, n * 4, 16, load ? "exp_avg_in" : "exp_avg_out"},
                            {v, n * 4, 16, load ? "exp_avg_sq_in" : "exp_avg_sq_out"}};
  const fsp_status s = check_buffers(l, bufs, 6);
  if (s != FSP_OK) return s;
  return launch_list_state(load, const_cast<void*>(m8), const_cast<void*>(v8), const_cast<float*>(ms),
                           const_cast<float*>(vs), const_cast<float*>(m), const_cast<float*>(v), l->state_len, stream);
}

}  // namespace
}  // namespace fsp

extern "C" fsp_status fsp_adamw_list_create(int32_t n, const int64_t* numels, void* const* params,
                                            const int32_t* param_dtypes, const void* const* grads,
                                            const int32_t* grad_dtypes, void* const* copies, fsp_adamw_list** out) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::create_list(n, numels, params, param_dtypes, grads, grad_dtypes, copies, out);
  });
}

extern "C" fsp_status fsp_adamw_list_info(const fsp_adamw_list* list, int64_t* state_len, int64_t* offsets) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    if (!list || !state_len) return fsp::fail(FSP_EINVAL, "list or state_len is NULL");
    *state_len = list->state_len;
    if (offsets) std::copy(list->offsets.begin(), list->offsets.end(), offsets);
    return FSP_OK;
  });
}

extern "C" void fsp_adamw_list_destroy(fsp_adamw_list* list) { fsp::free_list(list); }

extern "C" fsp_status fsp_adamw_list_step(const fsp_adamw_list* list, int32_t state_dtype, void* exp_avg,
                                          void* exp_avg_sq, float* exp_avg_scale, float* exp_avg_sq_scale,
                                          const fsp_adamw_hparams* hp, int64_t step, int64_t* step_dev,
                                          int32_t advance, const float* grad_scale, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::step_list(list, state_dtype, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, hp, step, step_dev,
                          advance, grad_scale, cuda_stream);
  });
}

extern "C" fsp_status fsp_adamw_list_state_values(const fsp_adamw_list* list, const void* exp_avg,
                                                  const void* exp_avg_sq, const float* exp_avg_scale,
                                                  const float* exp_avg_sq_scale, float* exp_avg_out,
                                                  float* exp_avg_sq_out, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::state_list(false, list, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, exp_avg_out,
                           exp_avg_sq_out, cuda_stream);
  });
}

extern "C" fsp_status fsp_adamw_list_state_load(const fsp_adamw_list* list, const float* exp_avg_in,
                                                const float* exp_avg_sq_in, void* exp_avg, void* exp_avg_sq,
                                                float* exp_avg_scale, float* exp_avg_sq_scale, void* cuda_stream) {
  return fsp::guard([&]() -> fsp_status {
    fsp::clear_error();
    return fsp::state_list(true, list, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, exp_avg_in, exp_avg_sq_in,
                           cuda_stream);
  });
}
