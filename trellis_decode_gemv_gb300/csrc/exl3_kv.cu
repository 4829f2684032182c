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
// entered into the table by that token, so no CTA waits for another.  64 requests:
// 3.7 us, 200 with 25 K tokens: 7.5 us, the chain of loads, scans and one search.
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
  const int head = ring_head(p.state[0], cap);
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
          pg = p.ring[(static_cast<long long>(head) + first[lo] + (idx - r.have)) % cap];
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

// One CTA per (window of tokens, head): the runs (the tokens of this call that go
// into one page) that begin in the window, one after the other; half of the threads
// take the keys, half the values.  A run's values are read once, 16 bytes a lane, and
// stay in registers between the maximum and the rounding: a side of a page is at most
// 64 threads with up to 16 rows each, not more threads with fewer, which spent as much
// again on addresses and the run.  Prompts of 25 K tokens, 8 heads of 128: 34 us, 154 MB
// at 4.5 TB/s (50 MB of it written), 16.0 M instructions in 46% of the issue cycles.
// Neither the bytes (23 us) nor the instructions bind it alone: each block is one chain
// of slots, values and stores, and 128 registers a thread leave 16 warps an SM to hide it.
template <int SIZE>
constexpr int append_threads() { return SIZE < 32 ? 64 : 2 * SIZE; }

struct AppendParams {
  exl3_kv_cache c;
  const __half* x[2];  // keys, values
  long long stride[2];
  const int64_t* slot;
  int tokens;
  int window;          // tokens, a power of two, at most a page
};

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Eight values to the nearest integers to their binary32 quotients by s.  The quotient
// lies between the products with 1 / s a little enlarged and a little reduced (by
// 2^-21, more than the three roundings together); where both round to the same
// integer so does it, and only next to a tie the division is needed.
__device__ __forceinline__ uint2 quantize8(const uint4& v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float more = inv * (1.f + 0x1p-21f), less = inv * (1.f - 0x1p-21f);
  const uint64_t hi = pair(more, more), lo = pair(less, less);
  const uint64_t magic = pair(12582912.f, 12582912.f);   // 1.5 * 2^23: a sum's last bits are the integer
  uint32_t q[8], differ = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    const uint64_t x = pair(f.x, f.y);
    const uint64_t a = add2(mul2(x, hi), magic), b = add2(mul2(x, lo), magic);
    q[2 * i] = static_cast<uint32_t>(a);
    q[2 * i + 1] = static_cast<uint32_t>(a >> 32);
    differ |= (q[2 * i] ^ static_cast<uint32_t>(b)) | (q[2 * i + 1] ^ static_cast<uint32_t>(b >> 32));
  }
  if (differ != 0u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      q[2 * i] = static_cast<uint32_t>(__float2int_rn(__fdiv_rn(f.x, s)));
      q[2 * i + 1] = static_cast<uint32_t>(__float2int_rn(__fdiv_rn(f.y, s)));
    }
  }
  return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

template <int D, int SIZE>
__global__ void __launch_bounds__(append_threads<SIZE>()) append_kernel(const AppendParams p) {
  constexpr int kAppendThreads = append_threads<SIZE>();
  constexpr int kSideThreads = kAppendThreads / 2;
  constexpr int kLanes = D / 8;                       // lanes of a row
  constexpr int kRowsAtOnce = kSideThreads / kLanes;  // 8 or 16
  constexpr int kMost = SIZE / kRowsAtOnce;           // rows of a lane
  constexpr int kSideWarps = kSideThreads / 32;
  static_assert(kMost >= 1 && 2 * SIZE <= kAppendThreads, "a window and the page that its last run reaches into");
  __shared__ long long slots[kAppendThreads];         // of the tokens from the window's first on
  __shared__ uint32_t joined[kAppendThreads / 32 + 1];// bit t: token t follows token t - 1 in its page
  __shared__ uint32_t tops[2][kAppendThreads / 32];
  const int tid = threadIdx.x;
  const int side = tid / kSideThreads;                // keys, values
  const int st = tid % kSideThreads;
  const long long total = static_cast<long long>(p.c.pages) * SIZE;
  const int w0 = static_cast<int>(blockIdx.x) * p.window;
  const int h = blockIdx.y;
  const long long stride = p.stride[side];
  const __half* x = p.x[side] + static_cast<size_t>(w0) * stride + static_cast<size_t>(h) * D + (st % kLanes) * 8;
  const int here = min(p.window, p.tokens - w0);
  {
    const int t = w0 + tid;
    const long long s = t < p.tokens ? p.slot[t] : -1;
    const long long before = t > 0 && t <= p.tokens ? p.slot[t - 1] : -1;
    slots[tid] = s;
    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, s >= 0 && before == s - 1 && (s & (SIZE - 1)) != 0);
    if ((tid & 31) == 0) joined[tid >> 5] = bits;
    if (tid == 0) joined[kAppendThreads / 32] = 0u;
  }
  __syncthreads();
  int parity = 0;
  for (int i = 0, n; i < here; i += n) {
    // the tokens from i on that share its page
    n = 1;
    {
      int at = i + 1;
      uint32_t word = ~joined[at >> 5] & (0xFFFFFFFFu << (at & 31));
      while (word == 0u) {   // ends: the last word is zero, and a page before it
        at = (at | 31) + 1;
        word = ~joined[at >> 5];
      }
      n = (at & ~31) + __ffs(static_cast<int>(word)) - 1 - i;
    }
    const long long s0 = slots[i];
    if (s0 < 0 || s0 >= total) continue;
    if ((joined[i >> 5] >> (i & 31)) & 1u) continue;   // the run began before this window: its CTA takes it
    const int off = static_cast<int>(s0 & (SIZE - 1));
    const size_t block = static_cast<size_t>(s0 / SIZE) * p.c.kv_heads + h;
    int8_t* page = (side == 0 ? p.c.k : p.c.v) + block * SIZE * D;
    float* scale = (side == 0 ? p.c.k_scale : p.c.v_scale) + block;
    const float old = off > 0 ? *scale : 0.f;
    const __half* row = x + static_cast<size_t>(i + st / kLanes) * stride;
    uint4 v[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      v[k] = st / kLanes + k * kRowsAtOnce < n ? __ldg(reinterpret_cast<const uint4*>(row + static_cast<size_t>(k * kRowsAtOnce) * stride))
                                               : make_uint4(0u, 0u, 0u, 0u);
    __half2 most = __float2half2_rn(0.f);
#pragma unroll
    for (int k = 0; k < kMost; ++k) {
      const __half2* w = reinterpret_cast<const __half2*>(&v[k]);
      most = __hmax2_nan(most, __hmax2_nan(__hmax2_nan(__habs2(w[0]), __habs2(w[1])), __hmax2_nan(__habs2(w[2]), __habs2(w[3]))));
    }
    // |x| as binary16 bits order as numbers do, infinity and NaN above them
    uint32_t m = *reinterpret_cast<const uint32_t*>(&most) & 0x7FFF7FFFu;
    m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
    if ((tid & 31) == 0) tops[parity][tid >> 5] = m;
    __syncthreads();
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kSideWarps; ++k) top = max(top, tops[parity][side * kSideWarps + k]);
    parity ^= 1;   // the next run's maxima do not meet this one's readers
    float fresh = __fdiv_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(top))), 127.f);
    const bool bad = top >= 0x7C00u || old != old;
    fresh = bad ? __int_as_float(0x7FC00000) : fmaxf(old, fresh);
    const float inv = fresh > 1e-30f ? __frcp_rn(fresh) : 0.f;   // below, every new value is 0
    if (off > 0 && fresh != old) {
      // the page's earlier tokens under the larger scale
      const float ratio = fresh > 0.f ? __fdiv_rn(old, fresh) : 0.f;
      for (int k = st; k < off * (D / 4); k += kSideThreads) {
        char4* at = reinterpret_cast<char4*>(page) + k;
        char4 q = *at;
        q.x = static_cast<signed char>(__float2int_rn(__fmul_rn(static_cast<float>(q.x), ratio)));
        q.y = static_cast<signed char>(__float2int_rn(__fmul_rn(static_cast<float>(q.y), ratio)));
        q.z = static_cast<signed char>(__float2int_rn(__fmul_rn(static_cast<float>(q.z), ratio)));
        q.w = static_cast<signed char>(__float2int_rn(__fmul_rn(static_cast<float>(q.w), ratio)));
        *at = q;
      }
    }
    int8_t* to = page + (off + st / kLanes) * D + (st % kLanes) * 8;
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      if (st / kLanes + k * kRowsAtOnce < n)
        *reinterpret_cast<uint2*>(to + k * kRowsAtOnce * D) = bad ? make_uint2(0u, 0u) : quantize8(v[k], fresh, inv);
    if (st == 0) *scale = fresh;
  }
}

template <int D>
void launch_append(const AppendParams& p, dim3 grid, cudaStream_t cs) {
  switch (p.c.page_size) {
    case 16: append_kernel<D, 16><<<grid, append_threads<16>(), 0, cs>>>(p); break;
    case 32: append_kernel<D, 32><<<grid, append_threads<32>(), 0, cs>>>(p); break;
    case 64: append_kernel<D, 64><<<grid, append_threads<64>(), 0, cs>>>(p); break;
    default: append_kernel<D, 128><<<grid, append_threads<128>(), 0, cs>>>(p); break;
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
  static std::atomic<unsigned long long> allowed{0};
  constexpr size_t kMost = sizeof(int32_t) * (2 * EXL3_MAX_REQUESTS + 1);
  if (smem > 48 * 1024 - 256 && !allow_smem(kv::plan_kernel, kMost, allowed)) return EXL3_ERR_CUDA;
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
                     1};
  // Windows of a page where that leaves enough CTAs for the SMs (prompts), down to
  // single tokens where it does not (a step's tokens, each in a page of its own).
  p.window = cache->page_size;
  const long long enough = 8LL * device_sm_count();
  while (p.window > 1 && static_cast<long long>(tokens) * cache->kv_heads < enough * p.window) p.window >>= 1;
  const dim3 grid(static_cast<unsigned>((tokens + p.window - 1) / p.window), static_cast<unsigned>(cache->kv_heads));
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (cache->head_dim == 64)
    kv::launch_append<64>(p, grid, cs);
  else
    kv::launch_append<128>(p, grid, cs);
  return launch_status();
}
