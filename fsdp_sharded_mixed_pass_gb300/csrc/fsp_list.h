// AdamW over a list of tensors: what its host side (fsp_adamw.cpp) and its
// kernels (fsp_adamw_kernels.cuh) share.  Not part of the C ABI.
#pragma once

#include <cstdint>

#include "fsp_args.h"
#include "fsp_ops.h"

namespace fsp {

constexpr int kListBlock = FSP_ADAMW_BLOCK;   // elements that share a scale
constexpr int kListTile = 2048;               // most elements of one work tile

constexpr int32_t kListParamBf16 = 1, kListGradBf16 = 2;
constexpr int32_t kListVec = 4;    // param, grad and copy aligned to four elements
constexpr int32_t kListBulk = 8;   // ... to 16 bytes

// `len` elements of one tensor: its pointers at the tile's first element (a
// multiple of kListBlock from the tensor's start) and the states' slot there.
struct ListTile {
  void* param;
  const void* grad;
  uint16_t* copy;   // or nullptr
  int64_t state_off;
  int32_t len;
  int32_t flags;
};
static_assert(sizeof(ListTile) == 40, "list tile layout");

struct ListArgs {
  const ListTile* tiles;
  int64_t n_tiles, bulk_tiles;   // bulk_tiles: of tensors with kListBulk
  unsigned long long* counter;   // two words, 0 between launches: tiles handed out, CTAs that are done
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  const float* grad_scale;   // or nullptr: 1
  const int64_t* step_dev;   // update index t in device memory (nullptr: t is folded into c)
  float lr;                  // kept to rebuild c's t-dependent scalars from *step_dev
  Coeffs c;
};

// (n_tiles > 0)
fsp_status launch_adamw_list(const ListArgs& a, bool eight_bit, void* stream);
// fp32 states (len slots) into codes and scales (load), or back.
fsp_status launch_list_state(bool load, void* m8, void* v8, float* ms, float* vs, float* m, float* v, int64_t len,
                             void* stream);

}  // namespace fsp
