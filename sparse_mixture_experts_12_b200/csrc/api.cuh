// Host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <stdint.h>

#include <initializer_list>
#include <utility>

#include "kernels.cuh"

#define MOE_API extern "C" __attribute__((visibility("default")))

#define MOE_TRY(expr)                        \
  do {                                       \
    moe_status_t s_ = (expr);                \
    if (s_ != MOE_OK) return s_;             \
  } while (0)
#define MOE_CUDA(expr) MOE_TRY(::moe::cuda_status(expr))

namespace moe {

inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool expert_choice(const moe_cfg_t &c) { return c.routing == MOE_ROUTING_EXPERT_CHOICE; }

// host upper bound on sum_g ceil(rows_g / kRowTile)
inline int m_tiles_ub(long long rows, int groups) {
  long long ub = ceil_div((int)rows, kRowTile) + groups;
  if (ub > rows) ub = rows;
  return (int)ub;
}

// rows of the expert-contiguous buffers (x_perm, h, y_perm): T*k (token choice) or
// E*C (expert choice)
long long expert_rows(const moe_cfg_t &c);

moe_status_t check_cfg(const moe_cfg_t *c);
// every pointer in the list: non-null required unless allowed, 16-byte aligned
moe_status_t check_ptrs(std::initializer_list<std::pair<const void *, bool>> ps);
moe_status_t check_expert_weights(const moe_cfg_t *c, const moe_weights_t *w);
moe_status_t check_shared_weights(const moe_cfg_t *c, const moe_weights_t *w);

}  // namespace moe
