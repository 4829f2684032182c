// exl3_attention: attention of each request's newest tokens over its paged 8-bit
// cache.
#include <math.h>

#include "exl3_kv.cuh"

namespace exl3 {
namespace attn {
namespace {

struct AttnParams {
  exl3_kv_cache c;
  const __half* q;
  long long q_stride;
  const int32_t* q_start;
  const int32_t* seq_len;
  const int32_t* table;
  __half* out;
  long long out_stride;
  float* lse;
  float scale;
  int q_heads, requests, tokens, stride;
};

constexpr int kWarps = 4;

// One CTA per (token, head); its warps share the keys, each with an online
// softmax of its own, joined at the end.  A lane holds D / 32 elements.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) row_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  const int t = blockIdx.x;
  const int h = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (t >= p.q_start[p.requests] || t < p.q_start[0]) return;
  int lo = 0, hi = p.requests;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int size = p.c.page_size;
  const long long most = static_cast<long long>(p.stride) * size;
  const long long seq = min(static_cast<long long>(max(p.seq_len[lo], 0)), most);
  const long long last = seq - (p.q_start[lo + 1] - t);  // this row's own position
  const int kvh = h / (p.q_heads / p.c.kv_heads);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __half2float(p.q[static_cast<size_t>(t) * p.q_stride + h * D + lane * E + e]);
    o[e] = 0.f;
  }
  for (long long j = warp; j <= last; j += kWarps) {
    const int page = p.table[static_cast<size_t>(lo) * p.stride + j / size];
    const bool in = page >= 0 && page < p.c.pages;
    const size_t block = in ? static_cast<size_t>(page) * p.c.kv_heads + kvh : 0;
    const size_t at = (block * size + j % size) * D + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * static_cast<float>(p.c.k[at + e]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= in ? p.c.k_scale[block] * p.scale : 0.f;
    const float vs = in ? p.c.v_scale[block] : 0.f;
    const float top = fmaxf(m, s);
    const float base = top == -INFINITY ? 0.f : top;
    const float keep = expf(m - base);
    const float w = expf(s - base);
    m = top;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * vs * static_cast<float>(p.c.v[at + e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) sum += sl[w] * expf(sm[w] - base);
  for (int i = threadIdx.x; i < D; i += 32 * kWarps) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += so[w][i] * expf(sm[w] - base);
    p.out[static_cast<size_t>(t) * p.out_stride + h * D + i] = __float2half_rn(last >= 0 ? v / sum : 0.f);
  }
  if (p.lse != nullptr && threadIdx.x == 0)
    p.lse[static_cast<size_t>(t) * p.q_heads + h] = last >= 0 ? base + logf(sum) : -INFINITY;
}

}  // namespace
}  // namespace attn
}  // namespace exl3

using namespace exl3;

extern "C" size_t exl3_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_new) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128) || max_new < 1)
    return 0;
  return 256;
}

extern "C" exl3_status exl3_attention(const exl3_kv_cache* cache, const exl3_half* q, long long q_stride, int q_heads,
                                      const int32_t* q_start, const int32_t* seq_len, int requests, int tokens,
                                      int max_new, const int32_t* block_table, int table_stride, float scale,
                                      exl3_half* out, long long out_stride, float* lse, void* workspace,
                                      size_t workspace_bytes, exl3_stream_t stream) {
  exl3_status st = kv::check_cache(cache);
  if (st != EXL3_OK) return st;
  if (q_heads < 1 || q_heads > 65535 || q_heads % cache->kv_heads != 0 || table_stride < 1) return EXL3_ERR_SHAPE;
  if ((st = kv::check_stride(q_stride, q_heads, cache->head_dim)) != EXL3_OK ||
      (st = kv::check_stride(out_stride, q_heads, cache->head_dim)) != EXL3_OK)
    return st;
  if (requests < 0 || requests > EXL3_MAX_REQUESTS || tokens < 0 || max_new < 1) return EXL3_ERR_BATCH;
  if (requests == 0 || tokens == 0) return EXL3_OK;
  if (q == nullptr || q_start == nullptr || seq_len == nullptr || block_table == nullptr || out == nullptr)
    return EXL3_ERR_NULL;
  if (!aligned16(q) || !aligned16(out) || !kv::aligned_to(q_start, 4) || !kv::aligned_to(seq_len, 4) ||
      !kv::aligned_to(block_table, 4) || !kv::aligned_to(lse, 4) || !aligned16(workspace))
    return EXL3_ERR_ALIGN;
  if (workspace == nullptr ||
      workspace_bytes < exl3_attention_workspace_bytes(q_heads, cache->kv_heads, cache->head_dim, max_new))
    return EXL3_ERR_WORKSPACE;
  attn::AttnParams p{*cache, reinterpret_cast<const __half*>(q), q_stride, q_start, seq_len, block_table,
                     reinterpret_cast<__half*>(out), out_stride, lse, scale, q_heads, requests, tokens, table_stride};
  const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(q_heads));
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (cache->head_dim == 64)
    attn::row_kernel<64><<<grid, 32 * attn::kWarps, 0, cs>>>(p);
  else
    attn::row_kernel<128><<<grid, 32 * attn::kWarps, 0, cs>>>(p);
  return launch_status();
}
