// exl3_attention: attention of each request's newest tokens over its paged 8-bit
// cache.
#include "exl3_attn.cuh"

namespace exl3 {
namespace attn {

exl3_status cache_map(CUtensorMap* map, const int8_t* base, const exl3_kv_cache& c, int rows) {
  const EncodeTiledFn encode = encode_tiled();
  if (encode == nullptr) return EXL3_ERR_CUDA;
  const cuuint64_t d = static_cast<cuuint64_t>(c.head_dim), size = static_cast<cuuint64_t>(c.page_size);
  const cuuint64_t dims[3] = {d, size, static_cast<cuuint64_t>(c.pages) * static_cast<cuuint64_t>(c.kv_heads)};
  const cuuint64_t strides[2] = {d, d * size};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(rows), 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(base), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE,
                            c.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EXL3_OK : EXL3_ERR_CUDA;
}

exl3_status query_map(CUtensorMap* map, const AttnParams& p, int head_dim, int tokens) {
  const EncodeTiledFn encode = encode_tiled();
  if (encode == nullptr) return EXL3_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(p.q_heads),
                              static_cast<cuuint64_t>(p.tokens)};
  const cuuint64_t strides[2] = {2ull * head_dim, 2ull * p.q_stride};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(p.q), dims, strides, box, estr,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? EXL3_OK : EXL3_ERR_CUDA;
}

}  // namespace attn
}  // namespace exl3

using namespace exl3;

extern "C" size_t exl3_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_new) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128) || max_new < 1)
    return 0;
  const size_t step = 2 * attn::kMaxCtas * attn::step_slot_floats(head_dim);
  const size_t prompt = 2 * attn::kMaxPromptCtas * attn::prompt_slot_floats(head_dim);
  const bool few = static_cast<long long>(max_new) * (q_heads / kv_heads) <= attn::kStepRows;
  return attn::head_bytes() + (few ? step : step + prompt) * sizeof(float);
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
  attn::AttnParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.q_start = q_start;
  p.seq_len = seq_len;
  p.table = block_table;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.out = reinterpret_cast<__half*>(out);
  p.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.c = scale * attn::kLog2e;
  p.q_heads = q_heads;
  p.kv_heads = cache->kv_heads;
  p.group = q_heads / cache->kv_heads;
  p.requests = requests;
  p.tokens = tokens;
  p.table_stride = table_stride;
  p.pages = cache->pages;
  while ((1 << p.page_shift) < cache->page_size) ++p.page_shift;
  // keys are numbered in 31 bits
  p.most = static_cast<long long>(table_stride) << p.page_shift;
  if (p.most > 0x7FFFFF00LL) p.most = 0x7FFFFF00LL;
  p.stall = debug_stall();
  p.status = static_cast<uint32_t*>(workspace);
  p.arrived = reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(workspace) + 256);
  p.split = reinterpret_cast<attn::SplitItem*>(p.arrived + attn::kCounters);
  p.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + attn::head_bytes());
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool step = static_cast<long long>(max_new) * p.group <= attn::kStepRows;
  const bool both = !step && requests > 1;
  if (step || both) {
    p.rows_lo = 1;
    p.rows_hi = step ? 0x7FFFFFFF : attn::kStepRows;
    p.followed = both;
    if ((st = attn::launch_step(p, *cache, (step ? max_new : 1) * p.group > 8, cs)) != EXL3_OK || step) return st;
  }
  p.rows_lo = both ? attn::kStepRows + 1 : 1;
  p.rows_hi = 0x7FFFFFFF;
  p.partial += 2 * attn::kMaxCtas * attn::step_slot_floats(cache->head_dim);
  return attn::launch_prompt(p, *cache, both, cs);
}
