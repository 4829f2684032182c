// Attention of a few query rows per key/value head (single tokens, drafted tokens):
// every cached byte is read once and used by at most 16 rows, so the cache's
// bytes per second are the bound, and what the kernel must do besides is to turn
// every byte into a binary16 MMA operand (1.25 to 1.5 instructions a byte) with
// enough copies in flight.
//
// Three consumer warps and one producer warp.  A unit is 4 KB of K and of V of an
// item (32 or 64 keys), one tensor copy each (or one per page, if those are smaller), into
// a ring of stages; unit i of the CTA's range goes to stage i % kStages and to
// consumer i % 3.  The producer walks the range ahead of the consumers: page
// numbers and scales of up to 32 units at a time, the copies, and each item's
// query rows (bulk copies) into a two-deep ring of their own, so nothing that
// waits for memory is left to the consumers.
//
// A consumer computes S^T = K Q^T and O^T += V^T P^T with m16n8k16 MMAs: the 16
// side is keys, then head dimensions, the 8 side the query rows (one or two
// tiles of 8), so that four or eight heads of a group do not fill half of a
// 16-row operand with nothing.  K is operand A of the first product: a lane's
// bytes of a key row are contiguous (the order of the head dimension in the
// products is free, Q is laid out the same).  V^T is operand A of the second:
// lane (g, t) reads the 16 bytes g of keys 2t, 2t+1, 2t+8, 2t+9, and the byte
// permutes that widen them also pair the keys.  P^T comes from S^T by one 8x8
// transposition (movmatrix).  The tensor copies swizzle 16-byte pieces, so both
// reads are free of bank conflicts for D = 128.
//
// Measured (64 requests of 4096 keys, 32 heads over 8): D = 128 94 us, 5.7 TB/s of
// keys and values, read once (543.7 MB of DRAM traffic for 541); D = 64 58 us, 4.6
// TB/s.  Instructions issue in 42% of the cycles, so it is neither they nor the
// bytes alone: 9 consumer warps an SM (168 registers, three CTAs) hide their own
// latencies only in part.  One request of 131K keys takes 56 us where its 268.6 MB
// need 40; the 57 partial results of each head added 10 us when the last arrival joined
// them all, and add about 5 in two steps.  Tiles of 16 rows want more registers than
// three CTAs an SM leave: with two (242 registers, six consumer warps in place of
// nine) one request of 32 K keys and 16 rows takes 26.7 us in place of 32.3, 16 of up
// to 4000 24.6 and not 28.9.
#include "exl3_attn.cuh"

namespace exl3 {
namespace attn {
namespace {

// Keys of a unit: 4 KB of K and of V, whatever the head dimension (32 keys of 64
// elements are too little for what a unit costs besides: 68 us for 64 requests of
// 4096 keys and 8 heads, where 64 keys take 57).
template <int D>
constexpr int unit_keys() { return 4096 / D; }
constexpr int kQSlots = 2;
constexpr int kJoinOnce = 24;   // partial results that are joined in one step
constexpr int kJoinBarrier = 1;

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kConsumers = 3;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  static constexpr int kCtasPerSm = NT == 1 ? 3 : 2;
  static constexpr int kStages = 6;
  static_assert(kStages % kConsumers == 0, "each stage belongs to one consumer, so that no parity wait skips a phase");
  static constexpr int kUnit = unit_keys<D>();
  static constexpr int kGroups = kUnit / 16;             // of 16 keys, one scale each
  static constexpr int kHalfBytes = kUnit * D;           // K or V of a unit
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kPartStride = D + 4;
};

template <int kConsumers>
__device__ __forceinline__ void join_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(kJoinBarrier), "n"(32 * kConsumers) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int NT>
__device__ __forceinline__ int req_tiles(const Req& r) { return (r.rows + 8 * NT - 1) / (8 * NT); }
template <int D>
__device__ __forceinline__ int req_blocks(const Req& r) { return max(1, (r.seq + unit_keys<D>() - 1) / unit_keys<D>()); }

// Ranges are cut in equal parts of units plus kItemCost for each item (its Q, the
// join of the warps).  An item of at most kWhole units is not split: a boundary that
// falls into it moves to its nearer end.  Measured on 1 to 200 requests of 300 to
// 131 K keys; with an item counted as one unit 200 requests of up to 600 keys took
// 45 us, with four 35; with kWhole 24 a single request of 517 keys 10.2, with 12 8.7.
constexpr int kItemCost = 4;
constexpr int kWhole = 12;
// Units that are worth a range of their own: with 8 in place of 4 33 requests of up to
// 2011 keys took 12.1 us in place of 11.4, 8 of 1024 11.8 and not 11.0, but one of 2000 10.3
// and not 11.1.
constexpr int kLeast = 4;

// What a request's items cost together, and the ranges that they are worth.
template <int D, int NT>
__device__ __forceinline__ void req_cost(const AttnParams& p, const Req& r, long long& cost, long long& ranges) {
  const int blocks = req_blocks<D>(r);
  const long long items = static_cast<long long>(req_tiles<NT>(r)) * p.kv_heads;
  cost += items * (blocks + kItemCost);
  ranges += items * (blocks <= kWhole ? 1 : (blocks + kLeast - 1) / kLeast);
}

// A boundary between ranges: unit `lo` of item `item` of request `b`; c0, c1 the first
// and last range that the item is spread over.
struct Edge {
  int b, item, lo, c0, c1;
};

// The boundary at cost u, in request b, whose items begin at cost `before`.
template <int D>
__device__ __forceinline__ Edge edge_at(const Req& r, int b, long long u, long long before, long long total, int ctas) {
  const int blocks = req_blocks<D>(r);
  const int each = blocks + kItemCost;
  Edge e;
  e.b = b;
  e.item = static_cast<int>((u - before) / each);
  const long long start = before + static_cast<long long>(e.item) * each;
  const int off = static_cast<int>(u - start);
  e.lo = blocks <= kWhole ? (2 * off < each ? 0 : blocks) : max(0, off - kItemCost);
  e.c0 = range_of(total, start + kItemCost, ctas);
  e.c1 = range_of(total, start + each - 1, ctas);
  return e;
}

// The items of a range, one after the other.  Each lane of a warp holds one
// request; every warp walks by itself.
template <int D, int NT>
struct Walker {
  const AttnParams& p;
  int base, b;        // request of lane 0, current request
  Req mine;
  int item;
  int end_b, end_item, end_lo;
  // current segment
  Req r;
  int blocks, tiles, head, tile, lo, hi;

  // `lanes` holds the requests from `first` on
  __device__ __forceinline__ Walker(const AttnParams& params, const Edge& from, const Edge& to, int first, const Req& lanes)
      : p(params), base(first), b(from.b), mine(lanes), item(from.item), end_b(to.b), end_item(to.item), end_lo(to.lo), lo(from.lo) {
    fetch();
    if (lo == blocks) advance();
    place();
  }
  __device__ __forceinline__ void fetch() {
    const int src = b - base;
    r.t0 = __shfl_sync(0xFFFFFFFFu, mine.t0, src);
    r.n = __shfl_sync(0xFFFFFFFFu, mine.n, src);
    r.rows = __shfl_sync(0xFFFFFFFFu, mine.rows, src);
    r.seq = __shfl_sync(0xFFFFFFFFu, mine.seq, src);
    blocks = req_blocks<D>(r);
    tiles = req_tiles<NT>(r);
  }
  __device__ __forceinline__ void place() {
    head = tiles > 1 ? item / tiles : item;
    tile = item - head * max(tiles, 1);
    hi = b > end_b || (b == end_b && item > end_item) ? lo : b == end_b && item == end_item ? min(blocks, end_lo) : blocks;
  }
  __device__ __forceinline__ void advance() {
    lo = 0;
    if (++item >= tiles * p.kv_heads) {
      item = 0;
      do {
        if (++b - base == 32) {
          base = b;
          mine = load_req(p, base + (threadIdx.x & 31));
        }
        fetch();
      } while (r.rows == 0 && b < p.requests);
    }
  }
  __device__ __forceinline__ bool more() const { return hi > lo; }
  __device__ __forceinline__ void next() {
    advance();
    place();
  }
};

template <int D, int NT>
struct Shared {
  using C = Cfg<D, NT>;
  unsigned char ring[C::kStages][C::kStageBytes];  // first: 1024-byte aligned
  __half q[kQSlots][C::kRows * D];
  static constexpr int kConsumers = C::kConsumers, kThreads = C::kThreads;
  float part[kConsumers][8][C::kPartStride];
  float pm[kConsumers][8], pl[kConsumers][8];
  float4 scale[C::kStages][C::kGroups];   // per 16 keys: PageScale
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t q_full[kQSlots], q_empty[kQSlots];
  long long warp_sum[kThreads / 32], warp_ranges[kThreads / 32];
  Edge edge[2];
  uint32_t abort, last;
};

// The consumers' sums of a row, 4 columns of it: with the row's maximum and sum.
template <int D, int NT>
__device__ __forceinline__ float4 join_warps(const Shared<D, NT>& sh, int row, int q4, float& top, float& sum) {
  constexpr int kConsumers = Cfg<D, NT>::kConsumers;
  top = -INFINITY;
#pragma unroll
  for (int k = 0; k < kConsumers; ++k) top = fmaxf(top, sh.pm[k][row]);
  const float base = top == -INFINITY ? 0.f : top;
  sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kConsumers; ++k) {
    const float f = ex2(sh.pm[k][row] - base);
    const float4 v = *reinterpret_cast<const float4*>(&sh.part[k][row][4 * q4]);
    sum += sh.pl[k][row] * f;
    acc.x += v.x * f;
    acc.y += v.y * f;
    acc.z += v.z * f;
    acc.w += v.w * f;
  }
  return acc;
}

// 4 columns of row `rr` of a request's item, finished.
template <int D>
__device__ __forceinline__ void store_out(const AttnParams& p, const Req& r, int head, int rr, int q4, const float4& acc, float top,
                                          float sum) {
  const int tok = rr / p.group;
  const int h = head * p.group + (rr - tok * p.group);
  const bool sees = r.seq - r.n + tok + 1 > 0;
  const float inv = inverse_sum(sum, sees);
  const __half2 ha = __floats2half2_rn(sees ? acc.x * inv : 0.f, sees ? acc.y * inv : 0.f);
  const __half2 hb = __floats2half2_rn(sees ? acc.z * inv : 0.f, sees ? acc.w * inv : 0.f);
  *reinterpret_cast<uint2*>(p.out + static_cast<size_t>(r.t0 + tok) * p.out_stride + static_cast<size_t>(h) * D + 4 * q4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&ha), *reinterpret_cast<const uint32_t*>(&hb));
  if (p.lse != nullptr && q4 == 0)
    p.lse[static_cast<size_t>(r.t0 + tok) * p.q_heads + h] = sees ? kLn2 * (top == -INFINITY ? 0.f : top) + logf(sum) : -INFINITY;
}

// 4 columns of a row of a partial result.
template <int D, int ROWS>
__device__ __forceinline__ void leave(float* slot, int row, int q4, const float4& acc, float top, float sum) {
  __stcg(reinterpret_cast<float4*>(slot + row * D) + q4, acc);
  if (q4 == 0) {
    __stcg(slot + ROWS * D + row, top);
    __stcg(slot + ROWS * D + ROWS + row, sum);
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, Cfg<D, NT>::kCtasPerSm)
    step_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<D, NT>;
  constexpr int kRows = C::kRows;
  constexpr int kConsumers = C::kConsumers, kThreads = C::kThreads;
  constexpr int kStages = C::kStages;
  constexpr int kUnit = C::kUnit;
  constexpr int kGroups = C::kGroups;
  constexpr int KS = D / 16;  // k-steps of the first product, m-tiles of the second
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Shared<D, NT>& sh = *reinterpret_cast<Shared<D, NT>*>(smem_raw);
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const int cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 2);   // the copies, the scales
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kQSlots; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], kConsumers);
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  if (p.followed) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // This CTA's range.  Up to 32 requests every warp finds it by itself.
  Edge from, to;
  int ctas, first = 0;
  Req lanes;
  if (p.requests <= 32) {
    const Req r = load_req(p, lane);
    lanes = r;
    long long cost = 0, ranges = 0;
    req_cost<D, NT>(p, r, cost, ranges);
    long long inc = cost;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += o;
      ranges += __shfl_xor_sync(0xFFFFFFFFu, ranges, d);
    }
    const long long total = __shfl_sync(0xFFFFFFFFu, inc, 31);
    ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), ranges));
    if (cta >= ctas) return;
    __syncthreads();   // the barriers
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long u = range_begin(total, cta + e, ctas);
      const int b = __popc(__ballot_sync(0xFFFFFFFFu, inc <= u));   // the request that holds u
      Req q;
      q.t0 = 0;
      q.n = 0;
      q.rows = 1;
      q.seq = __shfl_sync(0xFFFFFFFFu, r.seq, b & 31);
      const long long before = __shfl_sync(0xFFFFFFFFu, inc - cost, b & 31);
      Edge x{p.requests, 0, 0, 0, 0};
      if (b < 32) x = edge_at<D>(q, b, u, before, total, ctas);
      if (e == 0) from = x; else to = x;
    }
  } else {
    const int per = (p.requests + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.requests), b1 = min(b0 + per, p.requests);
    long long mine = 0, ranges = 0;
    for (int b = b0; b < b1; ++b) req_cost<D, NT>(p, load_req(p, b), mine, ranges);
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += o;
      ranges += __shfl_xor_sync(0xFFFFFFFFu, ranges, d);
    }
    if (lane == 31) {
      sh.warp_sum[warp] = inc;
      sh.warp_ranges[warp] = ranges;
    }
    if (tid == 0) sh.edge[1] = Edge{p.requests, 0, 0, 0, 0};   // the last range's end is in no item
    __syncthreads();
    long long total = 0, before = inc - mine, all_ranges = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < warp ? sh.warp_sum[w] : 0;
      total += sh.warp_sum[w];
      all_ranges += sh.warp_ranges[w];
    }
    ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), all_ranges));
    if (cta >= ctas) return;
    const long long u[2] = {range_begin(total, cta, ctas), range_begin(total, cta + 1, ctas)};
    if (u[1] >= before && u[0] < before + mine) {
      for (int b = b0; b < b1; ++b) {
        const Req r = load_req(p, b);
        long long n = 0, unused = 0;
        req_cost<D, NT>(p, r, n, unused);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (u[e] >= before && u[e] < before + n) sh.edge[e] = edge_at<D>(r, b, u[e], before, total, ctas);
        before += n;
      }
    }
    __syncthreads();
    from = sh.edge[0];
    to = sh.edge[1];
    first = from.b;
    lanes = load_req(p, first + lane);
  }
  Walker<D, NT> w(p, from, to, first, lanes);

  if (warp == kConsumers) {
    // ---- producer ------------------------------------------------------------------
    const int size = 1 << p.page_shift;
    const int copy_keys = min(size, kUnit);          // a unit is one copy, or one per page
    const uint32_t copy_bytes = static_cast<uint32_t>(copy_keys * D);
    uint32_t i = 0;       // unit of the range
    int seg = 0;
    bool ok = true;
    for (; w.more() && ok; w.next(), ++seg) {
      // query rows of the item
      const int qs = seg % kQSlots;
      if (seg >= kQSlots) ok = mbar_wait(&sh.q_empty[qs], static_cast<uint32_t>((seg / kQSlots) - 1) & 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
      const int row0 = w.tile * kRows;
      const int rows = min(kRows, w.r.rows - row0);
      if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[qs], static_cast<uint32_t>(rows) * D * 2);
      __syncwarp();
      const int tok0 = row0 / p.group;
      const int tok = tok0 + lane;   // at most 16 tokens have rows in a tile
      const int ra = max(row0, tok * p.group), rb = min(row0 + rows, (tok + 1) * p.group);
      if (ra < rb)
        bulk_g2s(&sh.q[qs][(ra - row0) * D],
                 p.q + static_cast<size_t>(w.r.t0 + tok) * p.q_stride + static_cast<size_t>(w.head * p.group + (ra - tok * p.group)) * D,
                 static_cast<uint32_t>(rb - ra) * D * 2, &sh.q_full[qs]);
      // units, 32 at a time: lane l looks up unit g0 + l
      const int32_t* row = p.table + static_cast<size_t>(w.b) * p.table_stride;
      for (int g0 = w.lo; g0 < w.hi && ok; g0 += 32) {
        const int mykey = (g0 + lane) * kUnit;
        int block[kGroups];                            // of the tensor map, per 16 keys
        float ks[kGroups], vs[kGroups];
        PageScale scale[kGroups];
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) {
          const int key = mykey + 16 * gr;
          int page = -1;
          if (g0 + lane < w.hi && key < w.r.seq) page = __ldg(row + (key >> p.page_shift));
          const bool in = page >= 0 && page < p.pages;   // a page outside the pool reads as zeros
          block[gr] = in ? page * p.kv_heads + w.head : p.pages * p.kv_heads;
          const size_t at = static_cast<size_t>(in ? block[gr] : 0);
          ks[gr] = in ? __ldg(p.k_scale + at) : 0.f;
          vs[gr] = in ? __ldg(p.v_scale + at) : 1.f;
        }
        const int n = p.stall == 0 ? min(32, w.hi - g0) : i == 0 ? 1 : 0;
        for (int j = 0; j < n; ++j, ++i) {
          const uint32_t st = i % kStages;
          const uint32_t use = i / kStages;
          if (use > 0) ok = mbar_wait(&sh.empty[st], (use - 1) & 1);
          if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
          if (lane == j) {
            // what lies past the request's keys is not copied: any int8 is finite, and P is 0 there
            const int left = min(kUnit, w.r.seq - mykey);
            const uint32_t parts = left > 0 ? static_cast<uint32_t>((left + copy_keys - 1) / copy_keys) : 0u;
            mbar_arrive_expect_tx(&sh.full[st], 2 * copy_bytes * parts);
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) {
              const int key = 16 * gr;
              if ((key & (copy_keys - 1)) != 0 || key >= left) continue;
              unsigned char* dst = sh.ring[st] + key * D;
              tensor_g2s(dst, &kmap, (mykey + key) & (size - 1), block[gr], &sh.full[st]);
              tensor_g2s(dst + C::kHalfBytes, &vmap, (mykey + key) & (size - 1), block[gr], &sh.full[st]);
            }
          }
          if (j == 0) {   // the first copies do not wait for the scales
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) scale[gr] = page_scale(p, ks[gr], vs[gr]);
          }
          if (lane == j) {
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr) sh.scale[st][gr] = make_float4(scale[gr].c, scale[gr].lv, scale[gr].iv, 0.f);
            mbar_arrive(&sh.full[st]);
          }
          __syncwarp();
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&sh.abort, 1u);
    // Wait (bounded) for the copies in flight.
    for (uint32_t k = 0; k < kStages && k < i; ++k) mbar_wait(&sh.full[(i - 1 - k) % kStages], ((i - 1 - k) / kStages) & 1);
    for (int k = 0; k < kQSlots && k < seg; ++k) mbar_wait(&sh.q_full[(seg - 1 - k) % kQSlots], static_cast<uint32_t>((seg - 1 - k) / kQSlots) & 1);
    return;
  }

  // ---- consumers --------------------------------------------------------------------
  const int g = lane >> 2;
  const int t = lane & 3;
  bool ok = true;
  uint32_t i = 0;   // unit of the range at the segment's start
  for (int seg = 0; w.more(); w.next(), ++seg) {
    const int qs = seg % kQSlots;
    if (ok) ok = mbar_wait(&sh.q_full[qs], (seg / kQSlots) & 1) && *reinterpret_cast<volatile uint32_t*>(&sh.abort) == 0u;
    ok = __all_sync(0xFFFFFFFFu, ok);
    const int row0 = w.tile * kRows;
    // Q as operand B: lane (g, t) holds row g's elements E t .. E t + E - 1, E = D / 4
    uint32_t qf[NT][KS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4* src = reinterpret_cast<const uint4*>(&sh.q[qs][(nt * 8 + g) * D + t * (D / 4)]);
#pragma unroll
      for (int k = 0; k < KS / 2; ++k) {
        const uint4 v = src[k];
        qf[nt][2 * k][0] = v.x;
        qf[nt][2 * k][1] = v.y;
        qf[nt][2 * k + 1][0] = v.z;
        qf[nt][2 * k + 1][1] = v.w;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_empty[qs]);
    // keys that this lane's rows (8 nt + 2t, + 1) see; the least of the tile
    const int seen0 = w.r.seq - w.r.n;
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) lim[nt][e] = seen0 + (row0 + nt * 8 + 2 * t + e) / p.group + 1;
    const int lim_min = seen0 + row0 / p.group + 1;

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    const int skip = static_cast<int>((warp + kConsumers - i % kConsumers) % kConsumers);
    for (int blk = w.lo + skip; blk < w.hi; blk += kConsumers) {
      const uint32_t at = i + static_cast<uint32_t>(blk - w.lo);
      const uint32_t st = at % kStages;
      if (ok) ok = mbar_wait(&sh.full[st], (at / kStages) & 1) && *reinterpret_cast<volatile uint32_t*>(&sh.abort) == 0u;
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) {
        if (lane == 0) atomicOr(&sh.abort, 1u);
        break;
      }
      const unsigned char* kb = sh.ring[st];
      const unsigned char* vb = kb + C::kHalfBytes;
      float s[kGroups][NT][4];   // scores
#pragma unroll
      for (int hf = 0; hf < kGroups; ++hf) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[hf][nt][e] = 0.f;
        const int r0 = hf * 16 + g;
#pragma unroll
        for (int pc = 0; pc < D / 64; ++pc) {   // 16-byte pieces of a lane's share of a row
          uint4 a, b;
          if constexpr (D == 128) {
            const int off = ((2 * t + pc) ^ g) * 16;
            a = *reinterpret_cast<const uint4*>(kb + r0 * D + off);
            b = *reinterpret_cast<const uint4*>(kb + (r0 + 8) * D + off);
          } else {
            const int off = (t ^ ((g >> 1) & 3)) * 16;
            a = *reinterpret_cast<const uint4*>(kb + r0 * D + off);
            b = *reinterpret_cast<const uint4*>(kb + (r0 + 8) * D + off);
          }
          const uint32_t aw[4] = {a.x ^ 0x80808080u, a.y ^ 0x80808080u, a.z ^ 0x80808080u, a.w ^ 0x80808080u};
          const uint32_t bw[4] = {b.x ^ 0x80808080u, b.y ^ 0x80808080u, b.z ^ 0x80808080u, b.w ^ 0x80808080u};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = cvt_lo(aw[k]), a1 = cvt_lo(bw[k]), a2 = cvt_hi(aw[k]), a3 = cvt_hi(bw[k]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(s[hf][nt], a0, a1, a2, a3, qf[nt][4 * pc + k][0], qf[nt][4 * pc + k][1]);
          }
        }
      }
      // x = c ks s + log2 vs, masked
      float4 sc[kGroups];
#pragma unroll
      for (int hf = 0; hf < kGroups; ++hf) sc[hf] = sh.scale[st][hf];
      const int key0 = blk * kUnit;
      const bool mask = key0 + kUnit > lim_min;
      bool over = false;
#pragma unroll
      for (int hf = 0; hf < kGroups; ++hf)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = fmaf(s[hf][nt][e], sc[hf].x, sc[hf].y);
            if (mask && key0 + hf * 16 + g + (e >> 1) * 8 >= lim[nt][e & 1]) x = -INFINITY;
            s[hf][nt][e] = x;
            over |= x > room_above(m[nt][e & 1]);
          }
      if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = -INFINITY;
#pragma unroll
            for (int hf = 0; hf < kGroups; ++hf) top = fmaxf(top, fmaxf(s[hf][nt][e], s[hf][nt][e + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            // a row moves its own maximum only: what the other rows of the tile hold (nothing
            // of any request, past the item's rows) does not change its bits
            const bool moves = top > room_above(m[nt][e]);
            const float next = top - kBelow;
            const float keep = moves ? ex2(m[nt][e] - next) : 1.f;   // 0 from a maximum of -inf
            if (moves) m[nt][e] = next;
            l[nt][e] *= keep;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[nt][k][e] *= keep;
              o[nt][k][e + 2] *= keep;
            }
          }
      }
      uint32_t pb[kGroups][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float base0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
        const float base1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int hf = 0; hf < kGroups; ++hf) {
          const float p0 = ex2(s[hf][nt][0] - base0), p1 = ex2(s[hf][nt][1] - base1);
          const float p2 = ex2(s[hf][nt][2] - base0), p3 = ex2(s[hf][nt][3] - base1);
          l[nt][0] = fmaf(p0 + p2, sc[hf].z, l[nt][0]);
          l[nt][1] = fmaf(p1 + p3, sc[hf].z, l[nt][1]);
          const __half2 lo = __floats2half2_rn(p0, p1), up = __floats2half2_rn(p2, p3);
          pb[hf][nt][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
          pb[hf][nt][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&up));
        }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int hf = 0; hf < kGroups; ++hf) {
        constexpr int W = D / 32;  // words of a lane's share of a key
        uint32_t v[4][W];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int r = hf * 16 + 2 * t + (kk & 1) + (kk >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vb + r * D + ((g ^ (r & 7)) * 16));
            v[kk][0] = x.x ^ 0x80808080u;
            v[kk][1] = x.y ^ 0x80808080u;
            v[kk][2] = x.z ^ 0x80808080u;
            v[kk][3] = x.w ^ 0x80808080u;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vb + r * D + (((g >> 1) ^ ((r >> 1) & 3)) * 16) + (g & 1) * 8);
            v[kk][0] = x.x ^ 0x80808080u;
            v[kk][1] = x.y ^ 0x80808080u;
          }
        }
        if (hf == kGroups - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[st]);  // the stage is in registers
        }
#pragma unroll
        for (int wd = 0; wd < W; ++wd) {
          const uint32_t x01 = __byte_perm(v[0][wd], v[1][wd], 0x5140), x23 = __byte_perm(v[0][wd], v[1][wd], 0x7362);
          const uint32_t y01 = __byte_perm(v[2][wd], v[3][wd], 0x5140), y23 = __byte_perm(v[2][wd], v[3][wd], 0x7362);
          {
            const uint32_t a0 = cvt_lo(x01), a1 = cvt_hi(x01), a2 = cvt_lo(y01), a3 = cvt_hi(y01);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][2 * wd], a0, a1, a2, a3, pb[hf][nt][0], pb[hf][nt][1]);
          }
          {
            const uint32_t a0 = cvt_lo(x23), a1 = cvt_hi(x23), a2 = cvt_lo(y23), a3 = cvt_hi(y23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][2 * wd + 1], a0, a1, a2, a3, pb[hf][nt][0], pb[hf][nt][1]);
          }
        }
      }
    }
    i += w.hi - w.lo;

    // ---- join the warps ---------------------------------------------------------
    const int rows = min(kRows, w.r.rows - row0);
    const bool whole = w.lo == 0 && w.hi == w.blocks;
    constexpr int kQuads = D / 4;  // a thread handles 4 elements of a row at a time
    float* slot = p.partial + static_cast<size_t>(2 * cta + (w.lo == 0 ? 1 : 0)) * (kRows * (D + 2));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {   // 8 rows at a time
      join_sync<kConsumers>();  // the readers of the rows before are done
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nt][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (g == 0) {
          sh.pm[warp][2 * t + e] = m[nt][e];
          sh.pl[warp][2 * t + e] = ok ? sum : unfinished();
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
          *reinterpret_cast<float2*>(&sh.part[warp][2 * t + e][g * KS * 2 + 2 * k]) = make_float2(o[nt][k][e], o[nt][k][e + 2]);
      }
      join_sync<kConsumers>();
      for (int x = tid; x < (rows - 8 * nt) * kQuads && x < 8 * kQuads; x += 32 * kConsumers) {
        const int row = x / kQuads;
        const int q4 = x - row * kQuads;
        float top, sum;
        const float4 acc = join_warps(sh, row, q4, top, sum);
        if (whole) {
          store_out<D>(p, w.r, w.head, row0 + 8 * nt + row, q4, acc, top, sum);
        } else {
          leave<D, kRows>(slot, 8 * nt + row, q4, acc, top, sum);
        }
      }
    }
    if (whole) continue;

    // ---- the item crosses ranges: the last to arrive joins --------------------------
    // Many ranges in two levels: the last of 8, 16 or 32 neighbours joins theirs into
    // the first one's slot, the last of those that joined puts the rest together.
    const int c0 = w.lo == 0 ? to.c0 : from.c0, c1 = w.lo == 0 ? to.c1 : from.c1;
    const int spread = c1 - c0 + 1;
    const bool two = spread > kJoinOnce;
    const int some = spread <= 64 ? 3 : spread <= 256 ? 4 : 5;   // its logarithm
    int k0 = c0, k1 = c1, step = 1;
    uint32_t* count = p.arrived + c0;
    if (two) {
      k0 += (cta - c0) >> some << some;
      k1 = min(k0 + (1 << some) - 1, c1);
      count = p.arrived + kMaxCtas + 2 * k0 + (k0 == c0 ? 1 : 0);
    }
    uint32_t others = static_cast<uint32_t>(k1 - k0);
    for (;;) {
      __threadfence();
      join_sync<kConsumers>();
      if (tid == 0) {
        const uint32_t before_me = atomicAdd(count, 1u);
        sh.last = before_me == others ? 1u : 0u;
        if (sh.last != 0u) *count = 0u;
      }
      join_sync<kConsumers>();
      if (sh.last == 0u) break;
      __threadfence();
      const bool rest = step > 1 || !two;   // nothing is left to join after this
      // Every warp adds up its share of the partial results, 8 rows at a time (a lane
      // holds 4 columns of several rows); then the warps are joined as above.
      constexpr size_t kSlot = static_cast<size_t>(kRows) * (D + 2);
      constexpr int kLanes = D / 4;              // lanes of a row
      constexpr int kAtOnce = 32 / kLanes;       // rows at a time
      constexpr int kMine = 8 / kAtOnce;         // rows of a lane
      const int q4 = lane % kLanes;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 8) {
        const int row_of = r0 + lane / kLanes;
        float top[kMine], sum[kMine];
        float4 acc[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          top[i] = -INFINITY;
          sum[i] = 0.f;
          acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 2
        for (int k = k0 + warp * step; k <= k1; k += kConsumers * step) {
          const float* s = p.partial + static_cast<size_t>(2 * k + (k == c0 ? 1 : 0)) * kSlot;
          float pm[kMine], pl[kMine];
          float4 v[kMine];
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const int row = i * kAtOnce + row_of;
            pm[i] = -INFINITY;
            pl[i] = 0.f;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rows) {
              pm[i] = __ldcg(s + kRows * D + row);
              pl[i] = __ldcg(s + kRows * D + kRows + row);
              v[i] = __ldcg(reinterpret_cast<const float4*>(s + row * D) + q4);
            }
          }
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const float up = fmaxf(top[i], pm[i]);
            const float base = up == -INFINITY ? 0.f : up;
            const float fa = ex2(top[i] - base), fb = ex2(pm[i] - base);
            top[i] = up;
            sum[i] = sum[i] * fa + pl[i] * fb;
            acc[i].x = acc[i].x * fa + v[i].x * fb;
            acc[i].y = acc[i].y * fa + v[i].y * fb;
            acc[i].z = acc[i].z * fa + v[i].z * fb;
            acc[i].w = acc[i].w * fa + v[i].w * fb;
          }
        }
        join_sync<kConsumers>();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int row = i * kAtOnce + lane / kLanes;
          *reinterpret_cast<float4*>(&sh.part[warp][row][4 * q4]) = acc[i];
          if (q4 == 0) {
            sh.pm[warp][row] = top[i];
            sh.pl[warp][row] = sum[i];
          }
        }
        join_sync<kConsumers>();
        for (int x = tid; x < (rows - r0) * kQuads && x < 8 * kQuads; x += 32 * kConsumers) {
          float mx, total;
          const int row = x / kQuads, col = x % kQuads;
          const float4 v = join_warps(sh, row, col, mx, total);
          if (rest)
            store_out<D>(p, w.r, w.head, row0 + r0 + row, col, v, mx, total);
          else
            leave<D, kRows>(p.partial + static_cast<size_t>(2 * k0 + (k0 == c0 ? 1 : 0)) * kSlot, r0 + row, col, v, mx, total);
        }
      }
      if (rest) break;
      k0 = c0;
      k1 = c1;
      step = 1 << some;
      count = p.arrived + c0;
      others = static_cast<uint32_t>((spread - 1) >> some);
    }
  }
  if (!ok && lane == 0) {
    atomicOr(&sh.abort, 1u);
    atomicOr(p.status, 1u);
  }
}

template <int D, int NT>
exl3_status launch(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  const size_t smem = sizeof(Shared<D, NT>);
  static std::atomic<unsigned long long> allowed{0};
  if (!allow_smem(step_kernel<D, NT>, smem, allowed)) return EXL3_ERR_CUDA;
  int ctas = device_sm_count() * C::kCtasPerSm;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  step_kernel<D, NT><<<ctas, C::kThreads, smem, stream>>>(p, kmap, vmap);
  return launch_status();
}

}  // namespace

exl3_status launch_step(const AttnParams& p, const exl3_kv_cache& c, bool wide, cudaStream_t stream) {
  CUtensorMap km, vm;
  exl3_status st;
  const int unit = c.head_dim == 64 ? unit_keys<64>() : unit_keys<128>();
  const int rows = c.page_size < unit ? c.page_size : unit;
  if ((st = cache_map(&km, c.k, c, rows)) != EXL3_OK || (st = cache_map(&vm, c.v, c, rows)) != EXL3_OK) return st;
  if (c.head_dim == 64) return wide ? launch<64, 2>(p, km, vm, stream) : launch<64, 1>(p, km, vm, stream);
  return wide ? launch<128, 2>(p, km, vm, stream) : launch<128, 1>(p, km, vm, stream);
}

}  // namespace attn
}  // namespace exl3
