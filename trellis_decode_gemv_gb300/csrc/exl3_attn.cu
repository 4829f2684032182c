// exl3_attention: attention of each request's newest tokens over its paged 8-bit
// cache.  exl3_attention_shared: the same for groups of requests behind a prefix,
// whose keys are read once for all of a group.
//
// A call with prefixes numbers its work like one without: the prefixes come as requests
// before the requests, with the rows of all their group and no mask, and a
// request's own keys begin behind its prefix.  Both kernels then leave a row's sums (m, l
// and the numerators, binary32) in place of its result, and a third one puts the two
// parts together.  A prefix counts up to a multiple of a unit of the kernel that goes on
// behind it, so no unit is cut at its lower end; the keys behind that are the
// request's own.
#include <algorithm>

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

namespace exl3 {
namespace attn {
namespace {

// The checks and parameters that calls with and without prefixes have in common.
exl3_status prepare(AttnParams& p, const exl3_kv_cache* cache, const exl3_half* q, long long q_stride, int q_heads,
                    const int32_t* q_start, const int32_t* seq_len, int requests, int tokens, int max_new,
                    const int32_t* block_table, int table_stride, float scale, exl3_half* out, long long out_stride, float* lse,
                    void* workspace) {
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
  p.c = scale * kLog2e;
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
  p.split = reinterpret_cast<SplitItem*>(p.arrived + kCounters);
  p.partial = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + head_bytes());
  return EXL3_OK;
}

bool few_rows(int tokens, int group) { return static_cast<long long>(tokens) * group <= kStepRows; }

// Where the sums of a call with prefixes lie in its workspace, and its bytes.
struct SharedLayout {
  size_t part, ml, end;
};
SharedLayout shared_layout(int q_heads, int kv_heads, int head_dim, int max_new, int max_group, int tokens) {
  const int group = q_heads / kv_heads;
  const size_t step = 2 * kMaxCtas * step_slot_floats(head_dim), prompt = 2 * kMaxPromptCtas * prompt_slot_floats(head_dim);
  const bool few = few_rows(max_new, group) && few_rows(max_group, group);
  const size_t rows = 2 * static_cast<size_t>(tokens) * q_heads;
  SharedLayout x;
  x.part = align256(head_bytes() + (few ? step : step + prompt) * sizeof(float));
  x.ml = x.part + rows * head_dim * sizeof(float);
  x.end = x.ml + rows * sizeof(float2);
  return x;
}

// A row's result from its sums over the prefix and over its own keys, 8 columns a
// thread.  Rows of no request are left alone.
constexpr int kMergeThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ AttnParams p) {
  const int t = blockIdx.x;
  int b = -1, hi = p.requests + 1;   // the last request that begins at t or before
  while (hi - b > 1) {
    const int mid = (b + hi) >> 1;
    if (p.q_start[mid] <= t) b = mid; else hi = mid;
  }
  const bool live = b >= 0 && b < p.requests;
  Req r{0, 0, 0, 0, 0, 0, 0};
  if (live) r = load_req<true>(p, p.groups + b);
  const int h = static_cast<int>(blockIdx.y) * (8 * kMergeThreads / D) + static_cast<int>(threadIdx.x) / (D / 8);
  const int c = static_cast<int>(threadIdx.x) % (D / 8);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live || h >= p.q_heads || t < r.t0 || t - r.t0 >= r.n) return;
  const bool sees = r.late + (t - r.t0) + 1 > 0;
  const size_t at = static_cast<size_t>(t) * p.q_heads + h;
  const size_t own = static_cast<size_t>(p.tokens) * p.q_heads + at;
  const float2 mo = __ldcg(p.part_ml + own);
  const float2 mp = r.k0 > 0 ? __ldcg(p.part_ml + at) : make_float2(-INFINITY, 0.f);
  const float4* po = reinterpret_cast<const float4*>(p.part + own * D) + 2 * c;
  const float4* pp = reinterpret_cast<const float4*>(p.part + at * D) + 2 * c;
  float4 x[2], y[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    x[e] = __ldcg(po + e);
    y[e] = r.k0 > 0 ? __ldcg(pp + e) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float top = fmaxf(mo.x, mp.x);
  const float base = top == -INFINITY ? 0.f : top;
  const float fo = ex2(mo.x - base), fp = ex2(mp.x - base);
  const float sum = mo.y * fo + mp.y * fp;
  const float inv = inverse_sum(sum, sees);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float v[4] = {x[e].x * fo + y[e].x * fp, x[e].y * fo + y[e].y * fp, x[e].z * fo + y[e].z * fp, x[e].w * fo + y[e].w * fp};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 q = __floats2half2_rn(sees ? v[2 * i] * inv : 0.f, sees ? v[2 * i + 1] * inv : 0.f);
      w[2 * e + i] = *reinterpret_cast<const uint32_t*>(&q);
    }
  }
  *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(t) * p.out_stride + static_cast<size_t>(h) * D + 8 * c) =
      make_uint4(w[0], w[1], w[2], w[3]);
  if (p.lse != nullptr && c == 0) p.lse[at] = sees ? kLn2 * base + logf(sum) : -INFINITY;
}

template <int D>
exl3_status launch_merge(const AttnParams& p, cudaStream_t cs) {
  constexpr int kHeads = 8 * kMergeThreads / D;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tokens), static_cast<unsigned>((p.q_heads + kHeads - 1) / kHeads));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, merge_kernel<D>, p) != cudaSuccess) return EXL3_ERR_CUDA;
  return launch_status();
}

}  // namespace
}  // namespace attn
}  // namespace exl3

extern "C" exl3_status exl3_attention(const exl3_kv_cache* cache, const exl3_half* q, long long q_stride, int q_heads,
                                      const int32_t* q_start, const int32_t* seq_len, int requests, int tokens,
                                      int max_new, const int32_t* block_table, int table_stride, float scale,
                                      exl3_half* out, long long out_stride, float* lse, void* workspace,
                                      size_t workspace_bytes, exl3_stream_t stream) {
  attn::AttnParams p{};
  exl3_status st = attn::prepare(p, cache, q, q_stride, q_heads, q_start, seq_len, requests, tokens, max_new, block_table,
                                 table_stride, scale, out, out_stride, lse, workspace);
  if (st != EXL3_OK || requests == 0 || tokens == 0) return st;
  if (workspace == nullptr ||
      workspace_bytes < exl3_attention_workspace_bytes(q_heads, cache->kv_heads, cache->head_dim, max_new))
    return EXL3_ERR_WORKSPACE;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const bool step = attn::few_rows(max_new, p.group);
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

extern "C" size_t exl3_attention_shared_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_new, int max_group,
                                                        int tokens) {
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (head_dim != 64 && head_dim != 128) || max_new < 1 ||
      max_group < 1 || tokens < 1)
    return 0;
  return attn::shared_layout(q_heads, kv_heads, head_dim, max_new, max_group, tokens).end;
}

extern "C" exl3_status exl3_attention_shared(const exl3_kv_cache* cache, const exl3_half* q, long long q_stride, int q_heads,
                                             const int32_t* q_start, const int32_t* seq_len, int requests, int tokens,
                                             int max_new, const int32_t* block_table, int table_stride,
                                             const int32_t* group_start, const int32_t* prefix_len, int groups, int max_group,
                                             float scale, exl3_half* out, long long out_stride, float* lse, void* workspace,
                                             size_t workspace_bytes, exl3_stream_t stream) {
  attn::AttnParams p{};
  exl3_status st = attn::prepare(p, cache, q, q_stride, q_heads, q_start, seq_len, requests, tokens, max_new, block_table,
                                 table_stride, scale, out, out_stride, lse, workspace);
  if (st != EXL3_OK) return st;
  if (groups < 0 || groups > EXL3_MAX_REQUESTS || requests + groups > EXL3_MAX_REQUESTS || max_group < 1) return EXL3_ERR_BATCH;
  if (requests == 0 || tokens == 0) return EXL3_OK;
  if (group_start == nullptr || (groups > 0 && prefix_len == nullptr)) return EXL3_ERR_NULL;
  if (!kv::aligned_to(group_start, 4) || !kv::aligned_to(prefix_len, 4)) return EXL3_ERR_ALIGN;
  const attn::SharedLayout at = attn::shared_layout(q_heads, cache->kv_heads, cache->head_dim, max_new, max_group, tokens);
  if (workspace == nullptr || workspace_bytes < at.end) return EXL3_ERR_WORKSPACE;
  p.group_start = group_start;
  p.prefix_len = prefix_len;
  p.groups = groups;
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + at.part);
  p.part_ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) + at.ml);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  // The few-rows kernel takes the requests if they all have few rows, and the prefixes that
  // have few; the other kernel the rest.
  const bool own_few = attn::few_rows(max_new, p.group), prefix_few = attn::few_rows(max_group, p.group);
  const bool both = !own_few || !prefix_few;
  p.align = own_few ? attn::step_unit(cache->head_dim) : attn::kPromptUnit;
  p.rows_lo = p.prefix_lo = 1;
  p.rows_hi = own_few ? 0x7FFFFFFF : attn::kStepRows;
  p.prefix_hi = prefix_few ? 0x7FFFFFFF : attn::kStepRows;
  p.followed = 1;
  const int most = std::max(own_few ? max_new : 1, prefix_few ? max_group : 1);
  if ((st = attn::launch_step(p, *cache, most * p.group > 8, cs)) != EXL3_OK) return st;
  attn::AttnParams m = p;
  if (both) {
    m.rows_lo = own_few ? 0x7FFFFFFF : attn::kStepRows + 1;
    m.prefix_lo = prefix_few ? 0x7FFFFFFF : attn::kStepRows + 1;
    m.rows_hi = own_few ? 0 : 0x7FFFFFFF;
    m.prefix_hi = prefix_few ? 0 : 0x7FFFFFFF;
    m.partial += 2 * attn::kMaxCtas * attn::step_slot_floats(cache->head_dim);
    if ((st = attn::launch_prompt(m, *cache, true, cs)) != EXL3_OK) return st;
  }
  return cache->head_dim == 64 ? attn::launch_merge<64>(p, cs) : attn::launch_merge<128>(p, cs);
}
