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

// Kernels that may begin where the blocks of the kernel before them end, and let the next one
// do the same (it waits in turn): between large calls that saves the gap of a launch, 2 us of 43.
// Nothing is read or written before.
__device__ __forceinline__ void chained_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename P>
inline exl3_status launch_chained(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t stream, const P& params) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, params) != cudaSuccess) return EXL3_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? EXL3_OK : EXL3_ERR_CUDA;
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

// The place of a ring's head, whatever number the caller keeps (rings may have more than 2^30 places).
__device__ __forceinline__ int ring_head(int state, int capacity) {
  if (capacity <= 0) return 0;
  const int r = state % capacity;
  return r < 0 ? r + capacity : r;
}

// `rows` rows of `len` bytes, `stride` bytes apart, that a call reads or writes.
struct Span {
  const void* at;
  long long rows, len, stride;
};
inline Span halves(const void* at, long long rows, long long n, long long stride) { return {at, rows, 2 * n, 2 * (rows > 1 ? stride : n)}; }
inline Span bytes(const void* at, long long len) { return {at, 1, len, len}; }
// Whether any of their bytes are the same.  (Rows of different strides that lie between one
// another count as that.)
inline bool meet(const Span& a, const Span& b) {
  if (a.at == nullptr || b.at == nullptr || a.len == 0 || b.len == 0) return false;
  const long long d = static_cast<long long>(reinterpret_cast<uintptr_t>(b.at)) - static_cast<long long>(reinterpret_cast<uintptr_t>(a.at));
  if (d >= (a.rows - 1) * a.stride + a.len || -d >= (b.rows - 1) * b.stride + b.len) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  // row i of a and row j of b: d - a.len < (i - j) * stride < d + b.len
  const long long s = a.rows > 1 ? a.stride : b.stride, low = d - a.len;
  long long k = low >= 0 ? low / s + 1 : -((s - 1 - low) / s) + 1;
  if (k < 1 - b.rows) k = 1 - b.rows;
  return k < a.rows && k * s < d + b.len;
}

// Strides of [tokens][heads][dim] halves: whole tokens apart, 16-byte loads.
inline exl3_status check_stride(long long stride, int heads, int dim) {
  if (stride < static_cast<long long>(heads) * dim || (stride & 7) != 0) return EXL3_ERR_SHAPE;
  return EXL3_OK;
}

}  // namespace kv
}  // namespace exl3
