// The paged 8-bit key/value cache: exl3_kv_plan (block tables and slot maps
// from the requests' lengths) and exl3_kv_append (quantization of new keys and
// values into their pages).
#include "exl3_kv.cuh"

namespace exl3 {
namespace kv {
namespace {

// ---- plan ----------------------------------------------------------------------

constexpr int kPlanThreads = 256;
constexpr int kPlanTokensPerCta = 1024;

struct PlanParams {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* ring;
  const int32_t* state;
  int32_t* state_out;
  int32_t* table;
  int32_t* seq_len;
  int32_t* q_start;
  int64_t* slot;
  int32_t* position;
  int requests, tokens, page_shift, capacity, stride;
};

// Exclusive prefix of `v` over the CTA's threads; the total in `total`.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const long long s = warp_sums[w];
    before += w < warp ? s : 0;
    total += s;
  }
  __syncthreads();
  return before + inc - v;
}

struct Request {
  long long ctx, add;   // cached and new tokens
  long long have, want; // pages before and after
  bool done;
};

__device__ __forceinline__ Request request_of(const PlanParams& p, int b) {
  Request r;
  const int c = p.ctx_len[b];
  const int n = p.new_len[b];
  r.ctx = c > 0 ? c : 0;
  r.add = n > 0 ? n : 0;
  r.done = n < 0;
  const long long round = (1LL << p.page_shift) - 1;
  r.have = (r.ctx + round) >> p.page_shift;
  r.want = (r.ctx + r.add + round) >> p.page_shift;
  return r;
}

// Every CTA scans all requests (the whole input is a few KB that stay in L2,
// and one launch without a hand-over between CTAs is what a step's latency
// wants), keeps the running sums in shared memory and handles its share of the
// tokens; CTA 0 writes the per-request outputs.  A page that a token opens is
// entered into the table by that token, so no CTA waits for another.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* starts = plan_smem;                   // [requests + 1], cut to `tokens`
  int32_t* first = plan_smem + p.requests + 1;   // [requests] pages taken before, -1: refused
  __shared__ long long sums[kPlanThreads / 32];
  const int tid = threadIdx.x;
  const int per = (p.requests + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.requests);
  const int b1 = min(b0 + per, p.requests);
  const int cap = p.capacity;
  const int head = cap > 0 ? ((p.state[0] % cap) + cap) % cap : 0;
  const int count = min(max(p.state[1], 0), cap);

  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += request_of(p, b).add;
  long long ends = block_scan(mine, sums, total);
  long long need_mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b);
    starts[b] = static_cast<int32_t>(min(ends, static_cast<long long>(p.tokens)));
    ends += r.add;
    const bool fits = !r.done && r.want <= p.stride && ends <= p.tokens;
    first[b] = fits ? static_cast<int32_t>(r.want - r.have) : -1;  // the need, until the second scan
    need_mine += fits ? r.want - r.have : 0;
  }
  if (tid == 0) starts[p.requests] = static_cast<int32_t>(min(total, static_cast<long long>(p.tokens)));
  long long need_total;
  long long before = block_scan(need_mine, sums, need_total);
  long long taken_mine = 0;
  for (int b = b0; b < b1; ++b) {
    const int need = first[b];
    const bool got = need == 0 || (need > 0 && before + need <= count);
    first[b] = got ? static_cast<int32_t>(min(before, 0x7FFFFFFFLL)) : -1;
    if (need > 0) {
      before += need;
      taken_mine += got ? need : 0;
    }
  }
  __syncthreads();
  const int used = starts[p.requests];

  // tokens
  const int page = 1 << p.page_shift;
  for (int t = blockIdx.x * kPlanThreads + tid; t < p.tokens; t += gridDim.x * kPlanThreads) {
    long long slot = -1;
    int pos = -1;
    if (t < used) {
      int lo = 0, hi = p.requests;  // the last b with starts[b] <= t and a token of its own
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid;
      }
      const Request r = request_of(p, lo);
      const long long at = r.ctx + (t - starts[lo]);
      pos = static_cast<int>(at);
      if (first[lo] >= 0) {
        const long long idx = at >> p.page_shift;
        int32_t* cell = p.table + static_cast<size_t>(lo) * p.stride + idx;
        int pg;
        if (idx < r.have) {
          pg = *cell;
        } else {
          pg = p.ring[(head + first[lo] + (idx - r.have)) % cap];
          if ((at & (page - 1)) == 0) *cell = pg;
        }
        slot = static_cast<long long>(pg) * page + (at & (page - 1));
      }
    }
    p.slot[t] = slot;
    p.position[t] = pos;
  }

  // per-request outputs; the pages of finished requests
  if (blockIdx.x == 0) {
    for (int b = tid; b < p.requests; b += kPlanThreads) {
      const Request r = request_of(p, b);
      p.seq_len[b] = r.done ? 0 : static_cast<int32_t>(first[b] >= 0 ? r.ctx + r.add : r.ctx);
      p.q_start[b] = starts[b];
    }
    if (tid == 0) p.q_start[p.requests] = used;
  }
  long long back_mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(p, b);
    back_mine += r.done ? min(r.have, static_cast<long long>(p.stride)) : 0;
  }
  long long back_total, taken_total;
  long long to = block_scan(back_mine, sums, back_total);
  block_scan(taken_mine, sums, taken_total);
  const long long room = cap - count;
  if (back_total > 0) {
    // `first` is free now: where a finished request's pages go
    for (int b = b0; b < b1; ++b) {
      const Request r = request_of(p, b);
      first[b] = r.done ? static_cast<int32_t>(min(to, 0x7FFFFFFFLL)) : -1;
      to += r.done ? min(r.have, static_cast<long long>(p.stride)) : 0;
    }
    __syncthreads();
    for (int b = blockIdx.x; b < p.requests; b += gridDim.x) {
      if (first[b] < 0) continue;
      const long long n = min(request_of(p, b).have, static_cast<long long>(p.stride));
      for (long long j = tid; j < n && first[b] + j < room; j += kPlanThreads)
        p.ring[(static_cast<long long>(head) + count + first[b] + j) % cap] =
            p.table[static_cast<size_t>(b) * p.stride + j];
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.state_out[0] = cap > 0 ? static_cast<int32_t>((head + taken_total) % cap) : 0;
    p.state_out[1] = static_cast<int32_t>(count - taken_total + min(back_total, room));
    p.state_out[2] = static_cast<int32_t>(min(need_total - taken_total, 0x7FFFFFFFLL));
  }
}

// ---- append ----------------------------------------------------------------------

constexpr int kAppendThreads = 128;

struct AppendParams {
  exl3_kv_cache c;
  const __half* x[2];  // keys, values
  long long stride[2];
  const int64_t* slot;
  int tokens;
  int page_shift;
};

// q = the nearest integer to the binary32 quotient x / s.
__device__ __forceinline__ int quantize(float x, float s) {
  return s > 0.f ? __float2int_rn(__fdiv_rn(x, s)) : 0;
}

// One CTA per (token, head): the CTA of a run's first token (a run: the tokens of
// this call that go into one page) handles the run.
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  const int t0 = blockIdx.x;
  const int h = blockIdx.y;
  const int tid = threadIdx.x;
  const int size = 1 << p.page_shift;
  const int dim = p.c.head_dim;
  const long long slots = static_cast<long long>(p.c.pages) << p.page_shift;
  const long long s0 = p.slot[t0];
  if (s0 < 0 || s0 >= slots) return;
  const int off = static_cast<int>(s0 & (size - 1));
  if (t0 > 0 && off != 0 && p.slot[t0 - 1] == s0 - 1) return;
  __shared__ int ends;
  __shared__ uint32_t top;
  if (tid == 0) ends = size - off;
  __syncthreads();
  for (int j = tid; j < size - off; j += kAppendThreads)
    if (t0 + j >= p.tokens || p.slot[t0 + j] != s0 + j) atomicMin(&ends, j);
  __syncthreads();
  const int n = ends;
  const long long page = s0 >> p.page_shift;
  const size_t block = static_cast<size_t>(page) * p.c.kv_heads + h;
  for (int which = 0; which < 2; ++which) {
    const __half* x = p.x[which] + static_cast<size_t>(t0) * p.stride[which] + static_cast<size_t>(h) * dim;
    int8_t* q = (which == 0 ? p.c.k : p.c.v) + block * size * dim;
    float* scale = (which == 0 ? p.c.k_scale : p.c.v_scale) + block;
    if (tid == 0) top = 0;
    __syncthreads();
    uint32_t m = 0;  // |x| as binary16 bits order as numbers do
    for (int i = tid; i < n * dim; i += kAppendThreads) {
      const int r = i / dim;
      m = max(m, static_cast<uint32_t>(__half_as_ushort(x[static_cast<size_t>(r) * p.stride[which] + (i - r * dim)])) & 0x7FFFu);
    }
    atomicMax(&top, m);
    const float old = off > 0 ? *scale : 0.f;
    __syncthreads();
    float fresh = __fdiv_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(top))), 127.f);
    fresh = top >= 0x7C00u || old != old ? __int_as_float(0x7FC00000) : fmaxf(old, fresh);
    if (fresh != old) {
      const float ratio = fresh > 0.f ? __fdiv_rn(old, fresh) : 0.f;
      for (int i = tid; i < off * dim; i += kAppendThreads)
        q[i] = static_cast<int8_t>(__float2int_rn(__fmul_rn(static_cast<float>(q[i]), ratio)));
    }
    for (int i = tid; i < n * dim; i += kAppendThreads) {
      const int r = i / dim;
      q[off * dim + i] = static_cast<int8_t>(
          quantize(__half2float(x[static_cast<size_t>(r) * p.stride[which] + (i - r * dim)]), fresh));
    }
    __syncthreads();
    if (tid == 0) *scale = fresh;
    __syncthreads();
  }
}

int log2_page(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

}  // namespace
}  // namespace kv
}  // namespace exl3

using namespace exl3;

extern "C" exl3_status exl3_kv_plan(const int32_t* ctx_len, const int32_t* new_len, int requests, int tokens,
                                    int page_size, int32_t* free_pages, int free_capacity,
                                    const int32_t* free_state, int32_t* free_state_out, int32_t* block_table,
                                    int table_stride, int32_t* seq_len, int32_t* q_start, int64_t* slot,
                                    int32_t* position, exl3_stream_t stream) {
  if (requests < 0 || requests > EXL3_MAX_REQUESTS || tokens < 0) return EXL3_ERR_BATCH;
  if (!kv::page_size_ok(page_size) || table_stride < 1 || free_capacity < 0) return EXL3_ERR_SHAPE;
  if (free_state == nullptr || free_state_out == nullptr || q_start == nullptr ||
      (requests > 0 && (ctx_len == nullptr || new_len == nullptr || block_table == nullptr || seq_len == nullptr)) ||
      (tokens > 0 && (slot == nullptr || position == nullptr)) || (free_capacity > 0 && free_pages == nullptr))
    return EXL3_ERR_NULL;
  for (const void* q : {static_cast<const void*>(ctx_len), static_cast<const void*>(new_len),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_state),
                        static_cast<const void*>(free_state_out), static_cast<const void*>(block_table),
                        static_cast<const void*>(seq_len), static_cast<const void*>(q_start),
                        static_cast<const void*>(position)})
    if (!kv::aligned_to(q, 4)) return EXL3_ERR_ALIGN;
  if (!kv::aligned_to(slot, 8)) return EXL3_ERR_ALIGN;
  kv::PlanParams p{ctx_len, new_len, free_pages, free_state, free_state_out, block_table, seq_len, q_start,
                   slot,    position, requests,  tokens,     kv::log2_page(page_size), free_capacity, table_stride};
  const size_t smem = sizeof(int32_t) * (2 * static_cast<size_t>(requests) + 1);
  if (smem > 48 * 1024 - 256 &&
      cudaFuncSetAttribute(kv::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
          cudaSuccess)
    return EXL3_ERR_CUDA;
  const int sms = device_sm_count();
  const int want = (tokens + kv::kPlanTokensPerCta - 1) / kv::kPlanTokensPerCta;
  const int grid = want < 1 ? 1 : want > sms ? sms : want;
  kv::plan_kernel<<<grid, kv::kPlanThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}

extern "C" exl3_status exl3_kv_append(const exl3_kv_cache* cache, const exl3_half* k, long long k_stride,
                                      const exl3_half* v, long long v_stride, const int64_t* slot, int tokens,
                                      exl3_stream_t stream) {
  exl3_status st = kv::check_cache(cache);
  if (st != EXL3_OK) return st;
  if (tokens < 0) return EXL3_ERR_BATCH;
  if ((st = kv::check_stride(k_stride, cache->kv_heads, cache->head_dim)) != EXL3_OK ||
      (st = kv::check_stride(v_stride, cache->kv_heads, cache->head_dim)) != EXL3_OK)
    return st;
  if (tokens == 0) return EXL3_OK;
  if (k == nullptr || v == nullptr || slot == nullptr) return EXL3_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !kv::aligned_to(slot, 8)) return EXL3_ERR_ALIGN;
  if (cache->kv_heads > 65535) return EXL3_ERR_SHAPE;
  kv::AppendParams p{*cache,
                     {reinterpret_cast<const __half*>(k), reinterpret_cast<const __half*>(v)},
                     {k_stride, v_stride},
                     slot,
                     tokens,
                     kv::log2_page(cache->page_size)};
  kv::append_kernel<<<dim3(static_cast<unsigned>(tokens), static_cast<unsigned>(cache->kv_heads)), kv::kAppendThreads,
                      0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}
