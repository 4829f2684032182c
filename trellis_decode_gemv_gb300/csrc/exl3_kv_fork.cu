// Forks of requests over the paged cache: exl3_kv_fork (block tables from parent
// rows, pages that nobody holds any more) and exl3_kv_copy (the partly filled pages
// that forks do not share, in all layers).
#include <cooperative_groups.h>

#include "exl3_kv.cuh"

namespace exl3 {
namespace kv {
namespace {

namespace cg = cooperative_groups;

// ---- fork ----------------------------------------------------------------------

constexpr int kForkThreads = 1024;
constexpr int kFewThreads = 256;   // up to as many rows and requests
constexpr int kForkCluster = 8;
constexpr int kMostClusters = 16;
constexpr int kAtOnce = 4;   // entries of a table that a lane has on their way
constexpr int kNobody = 0x7FFFFFFF;

struct ForkParams {
  const int32_t* parent;
  const int32_t* ctx_len;
  int32_t* ring;
  const int32_t* state;
  int32_t* state_out;
  const int32_t* table;
  int32_t* ctx_out;
  int32_t* table_out;
  int32_t* copy_from;
  int32_t* copy_to;
  int32_t* copy_tokens;
  unsigned char* gone;   // [pages rounded up to 16] held before, by a request that no row continues
  unsigned char* kept;   // [the same] held after
  uint32_t* arrived;     // clusters whose bytes are set
  int rows, requests, page_shift, pages, capacity, stride;
};

__device__ __forceinline__ int warp_inclusive(int v) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (static_cast<int>(threadIdx.x & 31) >= d) v += o;
  }
  return v;
}

// Exclusive prefix of `v` over the block's threads, the total in `total`.
__device__ __forceinline__ int fork_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int inc = warp_inclusive(v);
  __syncthreads();   // the sums' readers of the scan before
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  const int sums = warp_inclusive(lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0);
  total = __shfl_sync(0xFFFFFFFFu, sums, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, sums, (warp + 31) & 31);
  return inc - v + (warp > 0 ? before : 0);
}

// Tokens of a request: at most what its row of the table holds.
__device__ __forceinline__ int tokens_of(const ForkParams& p, int b) {
  const long long most = static_cast<long long>(p.stride) << p.page_shift;
  return static_cast<int>(min(static_cast<long long>(max(p.ctx_len[b], 0)), most));
}

// Place `by` <= cap behind `head` < cap in the ring.
__device__ __forceinline__ int wrapped(int head, int by, int cap) {
  const uint32_t at = static_cast<uint32_t>(head) + static_cast<uint32_t>(by);
  return static_cast<int>(at >= static_cast<uint32_t>(cap) ? at - static_cast<uint32_t>(cap) : at);
}

__device__ __forceinline__ int flags_of(uint32_t gone, uint32_t kept) { return __popc(gone & ~kept & 0x01010101u); }

// One launch.  Every block goes over all rows for itself (the first row of each
// parent, then the ranks of the rows that need a page: a few KB that stay in
// L2), so that the rows' tables, which are most of the bytes, need no hand-over.
// Where a request ends, each entry of the old table sets a byte for its page (held by a
// request that ends, or by one that goes on), and the cluster of blocks that is done last
// counts, and appends in ascending order, the pages with the one and not the other, a range of
// them for each of its blocks; none waits for another cluster.  Plain stores of the same byte need
// no atomics; the bytes are zero again when the call ends.  Calls in a graph: 16 requests of 125
// pages into 64 rows 3.3 us where none ends and 7.3 where one does, the latency of a dozen
// dependent steps; 500 of up to 125 pages into 509 rows 11, of up to 500 pages 25 (65 where one block
// appends what all have marked, 33 with one cluster for all of it).
__global__ void __launch_bounds__(kForkThreads) __cluster_dims__(kForkCluster, 1, 1)
    fork_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int32_t fork_smem[];
  int32_t* first = fork_smem;                // [requests] its first row
  int32_t* rank = fork_smem + p.requests;    // [rows] pages taken before it, -1: it needs none
  __shared__ int warp_sums[kForkThreads / 32];
  __shared__ int counts[kForkCluster];       // pages that go back, of the cluster's blocks
  __shared__ int last;
  chained_begin();
  const int threads = static_cast<int>(blockDim.x);
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int cap = p.capacity;
  const int head = ring_head(p.state[0], cap);
  const int count = min(max(p.state[1], 0), cap);
  const int size = 1 << p.page_shift;
  const uint32_t stride = static_cast<uint32_t>(p.stride);   // (places up to 128 past its end fit in 32 bits)

  for (int b = tid; b < p.requests; b += threads) first[b] = kNobody;
  __syncthreads();
  for (int i = tid; i < p.rows; i += threads) {
    const int b = p.parent[i];
    if (b >= 0 && b < p.requests) atomicMin(&first[b], i);
  }
  __syncthreads();
  const int per = (p.rows + threads - 1) / threads;
  const int i0 = min(tid * per, p.rows), i1 = min(i0 + per, p.rows);
  int mine = 0, need_total;
  for (int i = i0; i < i1; ++i) {
    const int b = p.parent[i];
    const bool need = b >= 0 && b < p.requests && first[b] != i && (tokens_of(p, b) & (size - 1)) != 0;
    rank[i] = need ? mine : -1;
    mine += need ? 1 : 0;
  }
  const int before = fork_scan(mine, warp_sums, need_total);
  for (int i = i0; i < i1; ++i)
    if (rank[i] >= 0) rank[i] += before;
  // whether any request that holds pages ends: the same answer in every block
  bool ends = false;
  for (int b = tid; b < p.requests; b += threads) ends |= first[b] == kNobody && tokens_of(p, b) > 0;
  ends = __syncthreads_or(ends) != 0;
  const int taken = min(need_total, count);

  // rows of the new table, a warp each
  const int warps = static_cast<int>(gridDim.x) * (threads / 32);
  const int warp = static_cast<int>(blockIdx.x) * (threads / 32) + (tid >> 5);
  for (int i = warp; i < p.rows; i += warps) {
    const int b = p.parent[i];
    const bool live = b >= 0 && b < p.requests;
    const int r = rank[i];
    const int c = live && r < count ? tokens_of(p, b) : 0;
    const uint32_t full = static_cast<uint32_t>(c) >> p.page_shift;
    const int part = c & (size - 1);
    const int32_t* old = p.table + static_cast<size_t>(live ? b : 0) * p.stride;
    const int fresh = r >= 0 && c > 0 ? p.ring[wrapped(head, r, cap)] : -1;   // a rank below `count`: cap is not 0
    int32_t* to = p.table_out + static_cast<size_t>(i) * p.stride;
    const uint32_t copied = full + (part > 0 && r < 0 ? 1 : 0);
    for (uint32_t j = lane; j < stride; j += 32 * kAtOnce) {
      int v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) v[k] = j + 32 * k < copied ? old[j + 32 * k] : -1;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (j + 32 * k < stride) to[j + 32 * k] = j + 32 * k == full && r >= 0 && c > 0 ? fresh : v[k];
    }
    if (lane == 0) {
      const bool copy = r >= 0 && c > 0;
      p.ctx_out[i] = c;
      p.copy_from[i] = copy ? old[full] : -1;
      p.copy_to[i] = copy ? fresh : -1;
      p.copy_tokens[i] = copy ? part : 0;
    }
  }

  int back_total = 0;
  if (ends) {
    // (from the last warp on: the first ones have a row)
    for (int b = warps - 1 - warp; b < p.requests; b += warps) {
      unsigned char* flags = first[b] == kNobody ? p.gone : p.kept;
      const int held = static_cast<int>((static_cast<uint32_t>(tokens_of(p, b)) + size - 1) >> p.page_shift);
      const int32_t* old = p.table + static_cast<size_t>(b) * p.stride;
      for (int j = lane; j < held; j += 32 * kAtOnce) {
        int v[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) v[k] = j + 32 * k < held ? old[j + 32 * k] : -1;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (v[k] >= 0 && v[k] < p.pages) flags[v[k]] = 1;
      }
    }
    for (int i = static_cast<int>(blockIdx.x) * threads + tid; i < taken; i += static_cast<int>(gridDim.x) * threads) {
      const int pg = p.ring[wrapped(head, i, cap)];
      if (pg >= 0 && pg < p.pages) p.kept[pg] = 1;
    }
    cg::cluster_group cluster = cg::this_cluster();
    const int me = static_cast<int>(cluster.block_rank());
    __threadfence();
    cluster.sync();
    if (me == 0 && tid == 0) {
      const int done = atomicAdd(p.arrived, 1u) == gridDim.x / kForkCluster - 1 ? 1 : 0;
      if (done) *p.arrived = 0u;
      for (int i = 0; i < kForkCluster; ++i) *cluster.map_shared_rank(&last, i) = done;
    }
    cluster.sync();
    if (last == 0) return;
    __threadfence();
    // the bytes in sixteens: a range of them for every block, and of that for every thread
    const int words = (p.pages - 1) / 16 + 1;
    const int share = (words - 1) / kForkCluster + 1;
    const int w0 = min(me * share, words), w1 = min(w0 + share, words);
    const int each = (w1 - w0 + threads - 1) / threads;
    const int a = min(w0 + tid * each, w1), e = min(a + each, w1);
    uint4* gone = reinterpret_cast<uint4*>(p.gone);
    uint4* kept = reinterpret_cast<uint4*>(p.kept);
    int found = 0, of_block;
#pragma unroll 4
    for (int w = a; w < e; ++w) {
      const uint4 g = __ldcg(gone + w), k = __ldcg(kept + w);
      found += flags_of(g.x, k.x) + flags_of(g.y, k.y) + flags_of(g.z, k.z) + flags_of(g.w, k.w);
    }
    int at = fork_scan(found, warp_sums, of_block);
    if (tid < kForkCluster) *cluster.map_shared_rank(&counts[me], tid) = of_block;
    cluster.sync();
#pragma unroll
    for (int i = 0; i < kForkCluster; ++i) {
      at += i < me ? counts[i] : 0;
      back_total += counts[i];
    }
    // behind what is left in the ring: the places of the pages that were taken, which every cluster has read, are free
    const int left = count - taken, rest = wrapped(head, taken, cap);
    for (int w = a; w < e; ++w) {
      const uint4 g = __ldcg(gone + w), k = __ldcg(kept + w);
      const uint32_t bits[4] = {g.x & ~k.x, g.y & ~k.y, g.z & ~k.z, g.w & ~k.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        for (uint32_t m = bits[i] & 0x01010101u; m != 0u; m &= m - 1, ++at)
          if (at < cap - left)
            p.ring[wrapped(rest, left + at, cap)] = 16 * w + 4 * i + ((__ffs(static_cast<int>(m)) - 1) >> 3);
      __stcg(gone + w, make_uint4(0u, 0u, 0u, 0u));
      __stcg(kept + w, make_uint4(0u, 0u, 0u, 0u));
    }
  }
  if (tid == 0 && (ends ? blockIdx.x % kForkCluster == 0 : blockIdx.x == 0)) {
    p.state_out[0] = cap > 0 ? wrapped(head, taken, cap) : 0;
    p.state_out[1] = count - taken + min(back_total, cap - count + taken);
    p.state_out[2] = need_total - taken;
  }
}

size_t fork_flags(int pages) { return (static_cast<size_t>(pages) + 15) & ~static_cast<size_t>(15); }

// ---- copy ----------------------------------------------------------------------

// A warp takes the tokens of one page and head, of the keys or the values of one
// layer, eight 16-byte vectors a lane in flight; a block a pair's keys or values in one layer.
// Bytes bound it.  The caches come by value, so a captured call needs no array that
// outlives it.
constexpr int kCopyThreads = 128;

template <int LAYERS>
struct CopyParams {
  struct Cache {
    int8_t* x[2];       // keys, values
    float* scale[2];
  } c[LAYERS];
  const int32_t* from;
  const int32_t* to;
  const int32_t* tokens;
  int pages, kv_heads, page_size, head_dim;
};

template <int LAYERS>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams<LAYERS> p) {
  chained_begin();
  const int pair = blockIdx.x;
  const int from = p.from[pair], to = p.to[pair];
  const int tokens = min(max(p.tokens[pair], 0), p.page_size);
  if (from < 0 || from >= p.pages || to < 0 || to >= p.pages || from == to) return;
  const typename CopyParams<LAYERS>::Cache& c = p.c[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const int vecs = tokens * p.head_dim / 16;
  const size_t of_head = static_cast<size_t>(p.page_size) * p.head_dim;
  const int side = blockIdx.z;
  for (int head = threadIdx.x >> 5; head < p.kv_heads; head += kCopyThreads / 32) {
    const size_t src = static_cast<size_t>(from) * p.kv_heads + head, dst = static_cast<size_t>(to) * p.kv_heads + head;
    const uint4* a = reinterpret_cast<const uint4*>(c.x[side] + src * of_head);
    uint4* b = reinterpret_cast<uint4*>(c.x[side] + dst * of_head);
    if (lane == 0) c.scale[side][dst] = c.scale[side][src];
    for (int v0 = lane; v0 < vecs; v0 += 256) {
      uint4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v0 + 32 * k < vecs) v[k] = a[v0 + 32 * k];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v0 + 32 * k < vecs) b[v0 + 32 * k] = v[k];
    }
  }
}

template <int LAYERS>
exl3_status launch_copy(const exl3_kv_cache* caches, int layers, const int32_t* from, const int32_t* to, const int32_t* tokens,
                        int pairs, cudaStream_t cs) {
  CopyParams<LAYERS> p{};
  for (int i = 0; i < layers; ++i) p.c[i] = {{caches[i].k, caches[i].v}, {caches[i].k_scale, caches[i].v_scale}};
  p.from = from;
  p.to = to;
  p.tokens = tokens;
  p.pages = caches->pages;
  p.kv_heads = caches->kv_heads;
  p.page_size = caches->page_size;
  p.head_dim = caches->head_dim;
  return launch_chained(copy_kernel<LAYERS>, dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(layers), 2), kCopyThreads, 0, cs, p);
}

}  // namespace
}  // namespace kv
}  // namespace exl3

using namespace exl3;

extern "C" size_t exl3_kv_fork_workspace_bytes(int pages) { return pages < 1 ? 0 : 2 * kv::fork_flags(pages) + 16; }

extern "C" exl3_status exl3_kv_fork(const int32_t* parent, int rows, const int32_t* ctx_len, int requests, int page_size,
                                    int pages, int32_t* free_pages, int free_capacity, const int32_t* free_state,
                                    int32_t* free_state_out, const int32_t* block_table, int table_stride, int32_t* ctx_out,
                                    int32_t* table_out, int32_t* copy_from, int32_t* copy_to, int32_t* copy_tokens,
                                    void* workspace, size_t workspace_bytes, exl3_stream_t stream) {
  if (rows < 0 || rows > EXL3_MAX_REQUESTS || requests < 0 || requests > EXL3_MAX_REQUESTS) return EXL3_ERR_BATCH;
  if (!kv::page_size_ok(page_size) || pages < 1 || table_stride < 1 || free_capacity < 0) return EXL3_ERR_SHAPE;
  if (free_state == nullptr || free_state_out == nullptr || (requests > 0 && (ctx_len == nullptr || block_table == nullptr)) ||
      (rows > 0 && (parent == nullptr || ctx_out == nullptr || table_out == nullptr || copy_from == nullptr ||
                    copy_to == nullptr || copy_tokens == nullptr)) ||
      (free_capacity > 0 && free_pages == nullptr))
    return EXL3_ERR_NULL;
  for (const void* q : {static_cast<const void*>(parent), static_cast<const void*>(ctx_len), static_cast<const void*>(free_pages),
                        static_cast<const void*>(free_state), static_cast<const void*>(free_state_out),
                        static_cast<const void*>(block_table), static_cast<const void*>(ctx_out),
                        static_cast<const void*>(table_out), static_cast<const void*>(copy_from),
                        static_cast<const void*>(copy_to), static_cast<const void*>(copy_tokens)})
    if (!kv::aligned_to(q, 4)) return EXL3_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < exl3_kv_fork_workspace_bytes(pages)) return EXL3_ERR_WORKSPACE;
  if (!aligned16(workspace)) return EXL3_ERR_ALIGN;
  const long long word = sizeof(int32_t), table = word * table_stride;
  const kv::Span all[] = {   // what is written first
      kv::bytes(free_state_out, 3 * word),
      kv::bytes(free_pages, word * free_capacity),
      kv::bytes(workspace, static_cast<long long>(exl3_kv_fork_workspace_bytes(pages))),
      kv::bytes(rows > 0 ? ctx_out : nullptr, word * rows),
      kv::bytes(rows > 0 ? table_out : nullptr, table * rows),
      kv::bytes(rows > 0 ? copy_from : nullptr, word * rows),
      kv::bytes(rows > 0 ? copy_to : nullptr, word * rows),
      kv::bytes(rows > 0 ? copy_tokens : nullptr, word * rows),
      kv::bytes(free_state, 2 * word),
      kv::bytes(rows > 0 ? parent : nullptr, word * rows),
      kv::bytes(requests > 0 ? ctx_len : nullptr, word * requests),
      kv::bytes(requests > 0 ? block_table : nullptr, table * requests)};
  constexpr int kSpans = sizeof(all) / sizeof(all[0]), kWritten = kSpans - 4;
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kSpans; ++j)
      if (kv::meet(all[i], all[j])) return EXL3_ERR_SHAPE;
  kv::ForkParams p{};
  p.parent = parent;
  p.ctx_len = ctx_len;
  p.ring = free_pages;
  p.state = free_state;
  p.state_out = free_state_out;
  p.table = block_table;
  p.ctx_out = ctx_out;
  p.table_out = table_out;
  p.copy_from = copy_from;
  p.copy_to = copy_to;
  p.copy_tokens = copy_tokens;
  p.gone = static_cast<unsigned char*>(workspace);
  p.kept = p.gone + kv::fork_flags(pages);
  p.arrived = reinterpret_cast<uint32_t*>(p.kept + kv::fork_flags(pages));
  p.rows = rows;
  p.requests = requests;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.pages = pages;
  p.capacity = free_capacity;
  p.stride = table_stride;
  const size_t smem = sizeof(int32_t) * (static_cast<size_t>(requests) + rows);
  static std::atomic<unsigned long long> allowed{0};
  if (smem > 47 * 1024 && !allow_smem(kv::fork_kernel, sizeof(int32_t) * 2 * EXL3_MAX_REQUESTS, allowed)) return EXL3_ERR_CUDA;
  // a warp for each row and each request
  const int threads = rows <= kv::kFewThreads && requests <= kv::kFewThreads ? kv::kFewThreads : kv::kForkThreads;
  const int warps = kv::kForkCluster * threads / 32;
  const int want = (rows + requests + warps - 1) / warps;
  const int clusters = want < 1 ? 1 : want > kv::kMostClusters ? kv::kMostClusters : want;
  return launch_chained(kv::fork_kernel, dim3(static_cast<unsigned>(clusters * kv::kForkCluster)), threads, smem,
                        reinterpret_cast<cudaStream_t>(stream), p);
}

extern "C" exl3_status exl3_kv_copy(const exl3_kv_cache* caches, int layers, const int32_t* from, const int32_t* to,
                                    const int32_t* tokens, int pairs, exl3_stream_t stream) {
  if (layers < 0 || layers > EXL3_MAX_LAYERS || pairs < 0) return EXL3_ERR_BATCH;
  if (layers > 0 && caches == nullptr) return EXL3_ERR_NULL;
  for (int i = 0; i < layers; ++i) {
    const exl3_status st = kv::check_cache(caches + i);
    if (st != EXL3_OK) return st;
    if (caches[i].pages != caches->pages || caches[i].kv_heads != caches->kv_heads ||
        caches[i].page_size != caches->page_size || caches[i].head_dim != caches->head_dim)
      return EXL3_ERR_SHAPE;
  }
  if (layers == 0 || pairs == 0) return EXL3_OK;
  if (from == nullptr || to == nullptr || tokens == nullptr) return EXL3_ERR_NULL;
  if (!kv::aligned_to(from, 4) || !kv::aligned_to(to, 4) || !kv::aligned_to(tokens, 4)) return EXL3_ERR_ALIGN;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return layers <= 64 ? kv::launch_copy<64>(caches, layers, from, to, tokens, pairs, cs)
                      : kv::launch_copy<EXL3_MAX_LAYERS>(caches, layers, from, to, tokens, pairs, cs);
}
