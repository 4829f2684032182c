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

// Bytes of keys and values that the tables can hold, up to which a call does not look for
// shared ones: what it would save is soon read, and what it takes besides are a second kernel, or
// two.  One: 8 requests behind 2011 tokens (38 MB) 14.7 us, 14.5 without; behind 3000 (54 MB) 14.8 and
// 16.2; two behind 8000 (34 MB) 19.9 and 17.0, behind 16000 (67 MB) 20.1 and 21.6.  Two: 64 requests behind 500 tokens (107 MB) 29.3 and 22.9, behind
// 1000 (172 MB) 30.1 and 32.0; 16 behind 1000 (43 MB) 25.4 and 15.0.
constexpr double kWorthOne = 48e6, kWorthBoth = 160e6;

bool few_rows(int tokens, int group) { return static_cast<long long>(tokens) * group <= kStepRows; }

// Where what a call with prefixes needs besides lies in its workspace, and its bytes.
struct SharedLayout {
  size_t split, flag, where, part, ml, end;
};
SharedLayout shared_layout(int q_heads, int kv_heads, int head_dim, int max_new, int max_group, int tokens) {
  const int group = q_heads / kv_heads;
  const size_t step = 2 * kMaxCtas * step_slot_floats(head_dim), prompt = 2 * kMaxPromptCtas * prompt_slot_floats(head_dim);
  const bool few = few_rows(max_new, group) && few_rows(max_group, group);
  const size_t rows = static_cast<size_t>(tokens) * q_heads;
  SharedLayout x;
  x.split = align256(head_bytes() + (few ? step : step + prompt) * sizeof(float));
  x.flag = align256(x.split + (kMaxCtas + kMaxPromptCtas) * sizeof(SharedSplit));
  x.where = align256(x.flag + rows * sizeof(uint32_t));
  x.part = align256(x.where + rows * sizeof(uint32_t));
  x.ml = x.part + 2 * rows * head_dim * sizeof(float);
  x.end = x.ml + 2 * rows * sizeof(float2);
  return x;
}

// A row's result from its sums over the prefix and over its own keys, either of which may lie
// in parts, one for each range that the item was spread over.  A warp takes 64 columns of
// four neighbouring rows (of the heads of one key/value head), eight lanes a row: whole
// sectors of either kernel's slots, the many-rows one's, four columns of all rows after one another, and
// the other's, row after row.  (A warp a row read half sectors of the former: 64 requests behind 32000
// tokens 70 us.)  The parts come in the order of the keys, eight at a time, m and l a part a
// lane.  What a row needs besides the other kernels have left beside its sums: finding
// its request anew took 1.5 us.  Rows of no request are left alone.
constexpr int kMergeThreads = 128;
constexpr int kMergeRows = 4;
constexpr int kMergeLanes = 32 / kMergeRows;   // of a row; parts at a time

// A row's sums over its prefix or its own keys: of part i columns 0..3 lie at x + slot *
// max(2 i - 1, 0) floats, the others four by four `step` floats apart, m and l like x.
struct Parts {
  const float *x, *m;
  int count, slot, step, to_l;
};

template <int D>
__device__ __forceinline__ Parts parts_of(const AttnParams& p, bool own, uint32_t code, bool any, size_t at, long long row) {
  const int c = static_cast<int>(min(code, static_cast<uint32_t>(kMaxCtas + kMaxPromptCtas))) - 1;
  Parts x;
  x.count = any ? 1 : 0;
  x.slot = 0;
  x.step = 4;
  x.to_l = 1;
  if (c < 0) {
    const size_t part = (own ? static_cast<size_t>(p.tokens) * p.q_heads : 0) + at;
    x.x = p.part + part * D;
    x.m = &p.part_ml[part].x;
    return x;
  }
  // bounded, whatever the lists were
  const SharedSplit s = p.shared_split[c];
  const bool step = c < kMaxCtas;
  const int range = step ? c : c - kMaxCtas, rows = step ? p.step_tile : 256;
  if (any) x.count = max(1, min(s.last, (step ? kMaxCtas : kMaxPromptCtas) - 1) - range + 1);
  const int in = static_cast<int>(max(0LL, min(row - s.first, static_cast<long long>(rows - 1))));
  x.slot = rows * (D + 2);
  const float* slot = p.partial + (step ? 0 : 2 * kMaxCtas * step_slot_floats(D)) + static_cast<size_t>(2 * range + 1) * x.slot;
  if (step) {
    x.x = slot + in * D;
    x.m = slot + rows * D + in;
    x.to_l = rows;
  } else {
    slot += (in >> 7) * (prompt_slot_floats(D) / 2);
    x.x = slot + (in & 127) * 4;
    x.step = 4 * 128;
    x.m = slot + D * 128 + (in & 127);
    x.to_l = 128;
  }
  return x;
}

template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kHalves = D / 64;   // warps of a row
  const int lane = threadIdx.x & 31, in_row = lane % kMergeLanes;
  const long long unit = static_cast<long long>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const int half = static_cast<int>(unit % kHalves);
  const long long row = unit / kHalves * kMergeRows + lane / kMergeLanes;   // token * group + head of the group
  const long long t = row / p.group;
  const int h = static_cast<int>(blockIdx.y) * p.group + static_cast<int>(row - t * p.group);
  const size_t at = static_cast<size_t>(t) * p.q_heads + h;
  // the requests' tokens: all between the first one's and the last one's
  const Lists lists(p);
  const bool live = t >= first_token(p, lists, 0) && t < first_token(p, lists, p.requests);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // (the next call may not begin yet: its blocks took 4 us of SMs from these)
  if (!__any_sync(0xFFFFFFFFu, live)) return;
  const uint32_t flag = live ? __ldcg(p.flag + at) : 0u, where = live ? __ldcg(p.where + at) : 0u;
  const bool sees = (flag & kSees) != 0u;
  const Parts a = parts_of<D>(p, false, where, live && (flag & kHasPrefix) != 0u, at, row);
  const Parts b = parts_of<D>(p, true, flag >> 2, live, at, row);
  const int parts = a.count + b.count;
  const int most = __reduce_max_sync(0xFFFFFFFFu, parts);
  const int quad = half * 16 + in_row;   // and quad + 8
  float top = -INFINITY, sum = 0.f;
  float4 acc[2] = {};
#pragma unroll 1
  for (int i0 = 0; i0 < most; i0 += kMergeLanes) {
    float4 v[kMergeLanes][2];
#pragma unroll
    for (int i = 0; i < kMergeLanes; ++i) {
      const int n = i0 + i;
      const bool first = n < a.count;
      const float* from = (first ? a.x : b.x) + static_cast<size_t>(first ? a.slot : b.slot) * max(2 * (first ? n : n - a.count) - 1, 0);
      const int step = first ? a.step : b.step;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        v[i][e] = n < parts ? __ldcg(reinterpret_cast<const float4*>(from + static_cast<size_t>(quad + 8 * e) * step))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    const int n = i0 + in_row;
    if (n < parts) {
      const bool first = n < a.count;
      const float* from = (first ? a.m : b.m) + static_cast<size_t>(first ? a.slot : b.slot) * max(2 * (first ? n : n - a.count) - 1, 0);
      m = __ldcg(from);
      l = __ldcg(from + (first ? a.to_l : b.to_l));
    }
    float next = fmaxf(top, m);
#pragma unroll
    for (int d = 1; d < kMergeLanes; d <<= 1) next = fmaxf(next, __shfl_xor_sync(0xFFFFFFFFu, next, d));
    const float base = next == -INFINITY ? 0.f : next;
    const float f = ex2(m - base), keep = ex2(top - base);
    float s = l * f;
#pragma unroll
    for (int d = 1; d < kMergeLanes; d <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    sum = sum * keep + s;
    top = next;
#pragma unroll
    for (int e = 0; e < 2; ++e) acc[e] = make_float4(acc[e].x * keep, acc[e].y * keep, acc[e].z * keep, acc[e].w * keep);
#pragma unroll
    for (int i = 0; i < kMergeLanes; ++i) {
      const float w = __shfl_sync(0xFFFFFFFFu, f, i, kMergeLanes);
      if (i0 + i < parts) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          acc[e] = make_float4(fmaf(v[i][e].x, w, acc[e].x), fmaf(v[i][e].y, w, acc[e].y), fmaf(v[i][e].z, w, acc[e].z),
                               fmaf(v[i][e].w, w, acc[e].w));
      }
    }
  }
  if (!live) return;
  const float inv = inverse_sum(sum, sees);
  __half* to = p.out + t * p.out_stride + static_cast<size_t>(h) * D;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const __half2 x = __floats2half2_rn(sees ? acc[e].x * inv : 0.f, sees ? acc[e].y * inv : 0.f);
    const __half2 y = __floats2half2_rn(sees ? acc[e].z * inv : 0.f, sees ? acc[e].w * inv : 0.f);
    *reinterpret_cast<uint2*>(to + 4 * (quad + 8 * e)) = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  }
  if (p.lse != nullptr && in_row == 0 && half == 0) p.lse[at] = sees ? kLn2 * (top == -INFINITY ? 0.f : top) + logf(sum) : -INFINITY;
}

template <int D>
exl3_status launch_merge(const AttnParams& p, cudaStream_t cs) {
  const long long rows = static_cast<long long>(p.tokens) * p.group;
  const long long warps = (rows + kMergeRows - 1) / kMergeRows * (D / 64);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32)), static_cast<unsigned>(p.kv_heads));
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
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  p.shared_split = reinterpret_cast<attn::SharedSplit*>(ws + at.split);
  p.flag = reinterpret_cast<uint32_t*>(ws + at.flag);
  p.where = reinterpret_cast<uint32_t*>(ws + at.where);
  p.part = reinterpret_cast<float*>(ws + at.part);
  p.part_ml = reinterpret_cast<float2*>(ws + at.ml);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  // The few-rows kernel takes the requests if they all have few rows, and the prefixes that
  // have few; the other kernel the rest, first, so that its blocks begin on SMs of their own.
  const bool own_few = attn::few_rows(max_new, p.group), prefix_few = attn::few_rows(max_group, p.group);
  p.both = !own_few || !prefix_few;
  if (2.0 * requests * static_cast<double>(p.most) * cache->kv_heads * cache->head_dim <= (p.both ? attn::kWorthBoth : attn::kWorthOne))
    return exl3_attention(cache, q, q_stride, q_heads, q_start, seq_len, requests, tokens, max_new, block_table, table_stride, scale,
                          out, out_stride, lse, workspace, workspace_bytes, stream);
  p.align = own_few ? attn::step_unit(cache->head_dim) : attn::kPromptUnit;
  p.rows_hi = own_few ? 0x7FFFFFFF : attn::kStepRows;
  p.prefix_hi = prefix_few ? 0x7FFFFFFF : attn::kStepRows;
  p.followed = 1;
  p.sms = device_sm_count();
  const bool wide = std::max(own_few ? max_new : 1, prefix_few ? max_group : 1) * p.group > 8;
  p.step_shift = wide ? 4 : 3;
  p.step_tile = 1 << p.step_shift;
  if (p.both) {
    attn::AttnParams many = p;
    many.many = 1;
    many.partial += 2 * attn::kMaxCtas * attn::step_slot_floats(cache->head_dim);
    if ((st = attn::launch_prompt(many, *cache, false, cs)) != EXL3_OK) return st;
  }
  if ((st = attn::launch_step(p, *cache, wide, cs)) != EXL3_OK) return st;
  return cache->head_dim == 64 ? attn::launch_merge<64>(p, cs) : attn::launch_merge<128>(p, cs);
}
