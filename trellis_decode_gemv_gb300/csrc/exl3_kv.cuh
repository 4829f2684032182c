// Shared by the cache and attention kernels: checks of the cache's fields and
// the request bookkeeping that every kernel reads from device memory.
#pragma once

#include "exl3_host.cuh"

namespace exl3 {

// Two binary32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

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
