// Shared by the cache and attention kernels: checks of the cache's fields and
// the request bookkeeping that every kernel reads from device memory.
#pragma once

#include "exl3_host.cuh"

namespace exl3 {
namespace kv {

inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

inline exl3_status check_cache(const exl3_kv_cache* c) {
  if (c == nullptr) return EXL3_ERR_NULL;
  if (!page_size_ok(c->page_size) || (c->head_dim != 64 && c->head_dim != 128) || c->kv_heads < 1 || c->pages < 1)
    return EXL3_ERR_SHAPE;
  // (page, head) pairs are numbered in 31 bits
  if (static_cast<long long>(c->pages) * c->kv_heads > 0x7FFFFFFFLL) return EXL3_ERR_SHAPE;
  if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr) return EXL3_ERR_NULL;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4))
    return EXL3_ERR_ALIGN;
  return EXL3_OK;
}

// Strides of [tokens][heads][dim] halves: whole tokens apart, 16-byte loads.
inline exl3_status check_stride(long long stride, int heads, int dim) {
  if (stride < static_cast<long long>(heads) * dim || (stride & 7) != 0) return EXL3_ERR_SHAPE;
  return EXL3_OK;
}

}  // namespace kv
}  // namespace exl3
