// Attention of many query rows per key/value head (prompts and chunks of them) on
// the tensor cores: 4 D operations per row and key, so the MMAs are the bound.
//
// One persistent CTA per SM.  An item's tile is 256 rows (new tokens x heads of
// the group, token major, so that a group's heads share every key) as two MMA
// tiles of 128, A and B; a unit is 128 keys.  Per unit and MMA tile, with
// binary16 operands and binary32 sums in tensor memory:
//   S = Q K^T   (Q and K in shared memory, 128 x 128 x D),
//   P = 2^(x - m) in place of S, as operand A in tensor memory,
//   O += P V    (V in shared memory, 128 x D x 128).
// Tensor memory holds S/P and O of both tiles: 2 x (128 + D) columns.  While the
// softmax warps of one tile work, the MMAs of the other run.
//
// Warp roles (13 warps):
//   0-3, 4-7  softmax of tile A and B: a thread owns a row (its TMEM lane).  They
//             also bring the item's Q into shared memory and take O out.  S is
//             read twice (largest score, then P): 128 scores do not fit a
//             thread's registers beside the rest.  O is only rescaled when a
//             score passes the running maximum by 2^8, by these threads, between
//             the MMAs that add to it.
//   8-11      widening: int8 keys and values from global memory through registers
//             (the next unit's loads are in flight meanwhile) into binary16
//             operand images, two of K and two of V.  Both are [key][D] rows of
//             64-element, 128-byte pieces in the 128-byte swizzle: K is read as a
//             K-major operand, V as an MN-major one, so V needs no transposition.
//   12        MMA issue (one lane) and TMEM allocation.
// Pages may be smaller than a unit: scales are kept per 16 keys.
//
// Barriers: K and V images full/empty, scales full (four slots: a slot is
// rewritten only after the softmax of both tiles has used it), Q full, S full and
// P full per tile, O done per tile.  Every wait is bounded; on timeout the CTA
// sets its abort flag and the status word, every role stops waiting, the MMA lane
// waits (bounded) for its MMAs, TMEM is freed.
#include "exl3_attn.cuh"

namespace exl3 {
namespace attn {
namespace {

using tc::mma_commit;
using tc::tc_fence_after;
using tc::tc_fence_before;

constexpr int kTile = 128;             // rows of an MMA tile
constexpr int kItemRows = 2 * kTile;
constexpr int kKeys = 128;             // keys of a unit
constexpr int kGroups = kKeys / 16;    // scale groups of a unit
constexpr int kConvWarp0 = 8;
constexpr int kConvThreads = 128;
constexpr int kMmaWarp = 12;
constexpr int kThreads = 32 * 13;
constexpr int kTmemCols = 512;
constexpr int kTileBarrier = 1;        // + tile
constexpr int kScaleSlots = 4;

template <int D>
struct Cfg {
  static constexpr int kPieces = D / 64;               // 64-element pieces of a row
  static constexpr int kPieceBytes = 128 * 128;        // 128 rows of one piece
  static constexpr int kImageBytes = kPieces * kPieceBytes;
  static constexpr int kSmem = kImageBytes * 6 + 1024; // Q A, Q B, K x 2, V x 2; alignment
  static constexpr int kOCol = 2 * kKeys;
};

struct Control {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t c_full[kScaleSlots];
  uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], o_done[2], mma_done;
  float4 scale[kScaleSlots][kGroups];
  long long warp_sum[kThreads / 32];
  long long units;
  int first_b, first_tile, first_head, first_lo;
  uint32_t tmem_base, abort, last[2];
};

__device__ __forceinline__ bool aborted(const Control& c) { return *reinterpret_cast<const volatile uint32_t*>(&c.abort) != 0u; }

// A wait of a whole warp; false (for every lane) when it ran out or the CTA has given up.
__device__ __forceinline__ bool warp_wait(Control& c, uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity) && !aborted(c);
  if (__all_sync(0xFFFFFFFFu, ok)) return true;
  atomicOr(&c.abort, 1u);
  return false;
}

__device__ __forceinline__ void tile_sync(int tile) {
  asm volatile("bar.sync %0, %1;" ::"r"(kTileBarrier + tile), "n"(kTile) : "memory");
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[smem desc] x B[smem desc], kind::f16.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// Descriptor of an operand in the 128-byte swizzle: 8-row groups of 1024 bytes
// `sbo` apart (along the rows of a K-major operand, along K of an MN-major one),
// the 64-element pieces of an MN-major operand `lbo` apart.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return tc::smem_desc(addr, lbo, sbo) | (2ull << 61);
}

// D fp32, A and B fp16, M = 128; B MN-major if `transposed`.
constexpr uint32_t idesc(int n, bool transposed) {
  return (1u << 4) | (transposed ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ int row_tiles(const Req& r) { return (r.rows + kItemRows - 1) / kItemRows; }
// Units of row tile `rt`: up to the last key that its last row sees, at least one.
__device__ __forceinline__ int tile_units(const AttnParams& p, const Req& r, int rt) {
  const int last = (min((rt + 1) * kItemRows, r.rows) - 1) / p.group;
  const int end = r.seq - r.n + last + 1;
  return max(1, (end + kKeys - 1) / kKeys);
}

// The items of a range: row tiles in order, the heads of a row tile after one
// another.
struct Walker {
  const AttnParams& p;
  long long u, end;
  int b, rt, head, lo, hi, units;
  Req r;
  __device__ __forceinline__ Walker(const AttnParams& params, const Control& c, long long u0, long long u1)
      : p(params), u(u0), end(u1), b(c.first_b), rt(c.first_tile), head(c.first_head), lo(c.first_lo) {
    r = load_req(p, b);
    place();
  }
  __device__ __forceinline__ void place() {
    units = tile_units(p, r, rt);
    hi = static_cast<int>(min(static_cast<long long>(units), lo + (end - u)));
  }
  __device__ __forceinline__ bool more() const { return u < end; }
  __device__ __forceinline__ void next() {
    u += hi - lo;
    if (u >= end) return;
    lo = 0;
    if (++head == p.kv_heads) {
      head = 0;
      if (++rt == row_tiles(r)) {
        rt = 0;
        do {
          r = load_req(p, ++b);
        } while (r.rows == 0 && b < p.requests);
      }
    }
    place();
  }
};

// ---- prelude: units of all items, and where this CTA's range begins -----------------

__device__ __forceinline__ long long block_scan(Control& c, long long v, long long& total) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) c.warp_sum[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? c.warp_sum[w] : 0;
    total += c.warp_sum[w];
  }
  __syncthreads();
  return before + inc - v;
}

// `first` [requests]: row tiles before each request (room borrowed from the operand images).
__device__ __forceinline__ bool find_range(const AttnParams& p, Control& c, int32_t* first, int min_units, int& ctas,
                                           long long& u0, long long& u1) {
  const int tid = threadIdx.x;
  const int per = (p.requests + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.requests), b1 = min(b0 + per, p.requests);
  long long mine = 0, tiles;
  for (int b = b0; b < b1; ++b) mine += row_tiles(load_req(p, b));
  long long at = block_scan(c, mine, tiles);
  for (int b = b0; b < b1; ++b) {
    first[b] = static_cast<int32_t>(at);
    at += row_tiles(load_req(p, b));
  }
  __syncthreads();
  const int n = static_cast<int>(tiles);
  const int share = (n + kThreads - 1) / kThreads;
  const int x0 = min(tid * share, n), x1 = min(x0 + share, n);
  int lo = 0, hi = p.requests;   // the last request that begins at or before x0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x0) lo = mid; else hi = mid;
  }
  long long sum = 0;
  {
    int b = lo;
    Req r = load_req(p, b);
    for (int x = x0; x < x1; ++x) {
      while (x - first[b] >= row_tiles(r)) r = load_req(p, ++b);
      sum += static_cast<long long>(tile_units(p, r, x - first[b])) * p.kv_heads;
    }
  }
  long long units;
  long long before = block_scan(c, sum, units);
  ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), (units + min_units - 1) / min_units));
  const int cta = blockIdx.x;
  if (cta >= ctas) return false;
  u0 = range_begin(units, cta, ctas);
  u1 = range_begin(units, cta + 1, ctas);
  if (before <= u0 && u0 < before + sum) {
    int b = lo;
    Req r = load_req(p, b);
    for (int x = x0; x < x1; ++x) {
      while (x - first[b] >= row_tiles(r)) r = load_req(p, ++b);
      const int len = tile_units(p, r, x - first[b]);
      const long long all = static_cast<long long>(len) * p.kv_heads;
      if (u0 < before + all) {
        c.first_b = b;
        c.first_tile = x - first[b];
        c.first_head = static_cast<int>((u0 - before) / len);
        c.first_lo = static_cast<int>((u0 - before) - static_cast<long long>(c.first_head) * len);
        c.units = units;
        break;
      }
      before += all;
    }
  }
  __syncthreads();
  return true;
}

// ---- widening ------------------------------------------------------------------------

// The 16-byte pieces of a unit's K or V that a thread widens: piece `tid % (D/16)`
// of the rows tid / (D/16) + i * (128 / (D/16)).
template <int D>
struct Conv {
  static constexpr int kChunks = D / 16;
  static constexpr int kRowStep = kConvThreads / kChunks;
  static constexpr int kLoads = 128 / kRowStep;

  // From the pages of the unit: lane l % 8 of every warp holds the byte offset of group l's first key, -1: zeros.
  static __device__ __forceinline__ void load(const int8_t* base, long long group_at, int tid, uint4 (&v)[kLoads]) {
    const int c = tid % kChunks;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = tid / kChunks + i * kRowStep;
      const long long at = __shfl_sync(0xFFFFFFFFu, group_at, row >> 4);
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (at >= 0) v[i] = __ldg(reinterpret_cast<const uint4*>(base + at + (row & 15) * D + c * 16));
    }
  }
  static __device__ __forceinline__ void store(uint32_t image, int tid, const uint4 (&v)[kLoads]) {
    const int c = tid % kChunks;
    // the lanes of a row's second piece store their halves in the other order: no bank twice
    const int swap = D == 128 ? c >> 2 : 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = tid / kChunks + i * kRowStep;
      const uint32_t x = v[i].x ^ 0x80808080u, y = v[i].y ^ 0x80808080u, z = v[i].z ^ 0x80808080u, w = v[i].w ^ 0x80808080u;
      const uint32_t h[8] = {cvt_lo(x), cvt_hi(x), cvt_lo(y), cvt_hi(y), cvt_lo(z), cvt_hi(z), cvt_lo(w), cvt_hi(w)};
      const uint32_t at = image + static_cast<uint32_t>((c >> 2) * Cfg<D>::kPieceBytes + row * 128);
      const uint32_t first = static_cast<uint32_t>((2 * (c & 3) + swap) ^ (row & 7)) * 16;
      const uint32_t second = static_cast<uint32_t>((2 * (c & 3) + 1 - swap) ^ (row & 7)) * 16;
      st_shared_v4(at + first, swap ? h[4] : h[0], swap ? h[5] : h[1], swap ? h[6] : h[2], swap ? h[7] : h[3]);
      st_shared_v4(at + second, swap ? h[0] : h[4], swap ? h[1] : h[5], swap ? h[2] : h[6], swap ? h[3] : h[7]);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const AttnParams p, const int8_t* __restrict__ kbase, const int8_t* __restrict__ vbase, int min_units) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_dyn[];
  __shared__ Control ctl;
  unsigned char* smem_raw = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);  // swizzle atoms
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const int cta = blockIdx.x;
  const uint32_t images = smem_u32(smem_raw);   // Q A, Q B, K 0, K 1, V 0, V 1

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.k_full[i], kConvThreads / 32);
      mbar_init(&ctl.v_full[i], kConvThreads / 32);
      mbar_init(&ctl.k_empty[i], 1);
      mbar_init(&ctl.v_empty[i], 1);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], kTile / 32);
      mbar_init(&ctl.pv_done[i], 1);
      mbar_init(&ctl.o_done[i], 1);
      mbar_init(&ctl.q_full[i], kTile / 32);
    }
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(&ctl.c_full[i], 1);
    mbar_init(&ctl.mma_done, 1);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  int ctas;
  long long u0, u1;
  if (!find_range(p, ctl, reinterpret_cast<int32_t*>(smem_raw), min_units, ctas, u0, u1)) return;
  if (warp == kMmaWarp) tc::tmem_alloc(&ctl.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  Walker w(p, ctl, u0, u1);

  if (warp == kMmaWarp) {
    // ---- MMA issue ---------------------------------------------------------------------
    constexpr uint32_t kIdescS = idesc(kKeys, false), kIdescO = idesc(D, true);
    uint32_t n = 0;               // units of the range so far
    uint32_t used[2] = {0, 0};    // units of tile A, B so far
    uint32_t items[2] = {0, 0};   // items of tile A, B so far
    uint32_t pv[2] = {0, 0};      // waits on pv_done
    bool ok = true;
    auto scores = [&](uint32_t unit, int x) {
      if (lane == 0) {
        const uint64_t a = swizzled_desc(images + static_cast<uint32_t>(x) * C::kImageBytes, 16, 1024);
        const uint64_t b = swizzled_desc(images + (2 + (unit & 1)) * C::kImageBytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = static_cast<uint32_t>((k >> 2) * C::kPieceBytes + (k & 3) * 32) >> 4;
          mma_ss(tmem + static_cast<uint32_t>(x * kKeys), a + off, b + off, kIdescS, k > 0 ? 1u : 0u);
        }
        mma_commit(&ctl.s_full[x]);
      }
      __syncwarp();
    };
    for (; w.more() && ok; w.next()) {
      const int tiles = w.r.rows - w.rt * kItemRows > kTile ? 2 : 1;
      const int steps = w.hi - w.lo;
      for (int x = 0; x < tiles && ok; ++x) ok = warp_wait(ctl, &ctl.q_full[x], items[x]++ & 1);
      ok = ok && warp_wait(ctl, &ctl.k_full[n & 1], (n >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      for (int x = 0; x < tiles; ++x) scores(n, x);
      if (lane == 0) mma_commit(&ctl.k_empty[n & 1]);
      for (int j = 0; j < steps && ok; ++j) {
        const uint32_t unit = n + static_cast<uint32_t>(j);
        const bool more = j + 1 < steps;
        for (int x = 0; x < tiles; ++x) {
          if (x == 0) ok = warp_wait(ctl, &ctl.v_full[unit & 1], (unit >> 1) & 1);
          ok = ok && warp_wait(ctl, &ctl.p_full[x], used[x] & 1);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t b = swizzled_desc(images + (4 + (unit & 1)) * C::kImageBytes, C::kPieceBytes, 1024);
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              tc::mma_f16_ts(tmem + static_cast<uint32_t>(C::kOCol + x * D), tmem + static_cast<uint32_t>(x * kKeys + 8 * k),
                             b + static_cast<uint32_t>((k * 2048) >> 4), kIdescO, j > 0 || k > 0 ? 1u : 0u);
            if (x == tiles - 1) mma_commit(&ctl.v_empty[unit & 1]);
            mma_commit(more ? &ctl.pv_done[x] : &ctl.o_done[x]);
          }
          __syncwarp();
          if (more) {
            // the next scores go where P is: its product has to be complete
            if (x == 0) ok = warp_wait(ctl, &ctl.k_full[(unit + 1) & 1], ((unit + 1) >> 1) & 1);
            ok = ok && warp_wait(ctl, &ctl.pv_done[x], pv[x] & 1);
            if (!ok) break;
            ++pv[x];
            tc_fence_after();
            scores(unit + 1, x);
            if (x == tiles - 1 && lane == 0) mma_commit(&ctl.k_empty[(unit + 1) & 1]);
            __syncwarp();
          }
          ++used[x];
        }
      }
      n += static_cast<uint32_t>(steps);
    }
    if (lane == 0) mma_commit(&ctl.mma_done);
    __syncwarp();
    mbar_wait(&ctl.mma_done, 0);
  } else if (warp >= kConvWarp0) {
    // ---- widening ----------------------------------------------------------------------
    using V = Conv<D>;
    const int ct = tid - 32 * kConvWarp0;
    const int key16 = (lane & 7) * 16;
    // three units deep: page numbers, then offsets and scales, then the bytes
    bool live = w.more();
    int blk = w.lo;
    int page = -1, head = 0, token = 0;  // of the cursor's unit, this lane's 16 keys
    auto look_up = [&]() {
      page = -1;
      head = 0;
      if (live) {
        const int key = blk * kKeys + key16;
        head = w.head;
        if (key < w.r.seq) page = __ldg(p.table + static_cast<size_t>(w.b) * p.table_stride + (key >> p.page_shift));
        if (page >= p.pages) page = -1;
        // a page number outside the pool reads as zeros, as does what lies past the request
        if (page >= 0) token = key & ((1 << p.page_shift) - 1);
        if (++blk == w.hi) {
          w.next();
          live = w.more();
          blk = w.lo;
        }
      }
    };
    auto offset = [&]() -> long long {
      return page < 0 ? -1LL : (((static_cast<long long>(page) * p.kv_heads + head) << p.page_shift) + token) * D;
    };
    const uint32_t count = static_cast<uint32_t>(u1 - u0);
    uint4 kr[V::kLoads], vr[V::kLoads];
    look_up();
    long long at = offset();
    PageScale sc = page_scale(p, page, head);
    V::load(kbase, at, ct, kr);
    V::load(vbase, at, ct, vr);
    look_up();
    long long at1 = offset();
    PageScale sc1 = page_scale(p, page, head);
    look_up();
    for (uint32_t n = 0; n < count; ++n) {
      const int slot = n & 1;
      const uint32_t before = ((n >> 1) - 1) & 1;
      if (n >= 2 && !warp_wait(ctl, &ctl.k_empty[slot], before)) break;
      if (warp == kConvWarp0) {
        if (lane < kGroups) ctl.scale[n % kScaleSlots][lane] = make_float4(sc.c, sc.lv, sc.iv, 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.c_full[n % kScaleSlots]);
      }
      V::store(images + (2 + slot) * C::kImageBytes, ct, kr);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.k_full[slot]);
      V::load(kbase, at1, ct, kr);
      if (n >= 2 && !warp_wait(ctl, &ctl.v_empty[slot], before)) break;
      V::store(images + (4 + slot) * C::kImageBytes, ct, vr);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.v_full[slot]);
      V::load(vbase, at1, ct, vr);
      sc = sc1;
      at1 = offset();
      sc1 = page_scale(p, page, head);
      look_up();
    }
  } else {
    // ---- softmax -----------------------------------------------------------------------
    const int x = warp >> 2;
    const int r = tid & (kTile - 1);        // row of the tile = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + static_cast<uint32_t>(x * kKeys);
    const uint32_t o_at = tmem + lanes + static_cast<uint32_t>(C::kOCol + x * D);
    uint32_t n = 0, used = 0, items = 0;
    bool ok = true;
    for (; w.more(); w.next()) {
      const int rows = w.r.rows - w.rt * kItemRows - x * kTile;  // of this tile
      const int steps = w.hi - w.lo;
      if (rows <= 0) {
        n += static_cast<uint32_t>(steps);
        continue;
      }
      const int rr = w.rt * kItemRows + x * kTile + r;
      const int tok = rr / p.group;
      const int h = w.head * p.group + (rr - tok * p.group);
      const bool mine = r < rows;
      {  // this row of Q
        const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<size_t>(w.r.t0 + tok) * p.q_stride + static_cast<size_t>(h) * D);
        const uint32_t dst = images + static_cast<uint32_t>(x) * C::kImageBytes + static_cast<uint32_t>(r * 128);
#pragma unroll
        for (int half = 0; half < C::kPieces; ++half) {
          uint4 v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = mine ? src[half * 8 + c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            st_shared_v4(dst + static_cast<uint32_t>(half * C::kPieceBytes + ((c ^ (r & 7)) * 16)), v[c].x, v[c].y, v[c].z, v[c].w);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.q_full[x]);
      }
      const int lim = w.r.seq - w.r.n + tok + 1;            // keys that this row sees
      const int lim_min = __shfl_sync(0xFFFFFFFFu, lim, 0);
      const bool busy = (warp & 3) * 32 < rows;             // the warp has rows at all
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < steps; ++j, ++n, ++used) {
        ok = ok && warp_wait(ctl, &ctl.s_full[x], used & 1) && warp_wait(ctl, &ctl.c_full[n % kScaleSlots], (n / kScaleSlots) & 1);
        if (!ok) continue;
        if (busy) {
          tc_fence_after();
          const float4* sc = ctl.scale[n % kScaleSlots];
          const int key0 = (w.lo + j) * kKeys;
          const bool mask = key0 + kKeys > lim_min;
          const int left = lim - key0;     // keys of this unit that the row sees
          uint32_t a[32];
          // largest x = c ks s + log2 vs
          float top = -INFINITY;
#pragma unroll
          for (int ch = 0; ch < kKeys / 32; ++ch) {
            tmem_ld32(s_at + 32 * ch, a);
            tmem_ld_wait();
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
              const float4 f = sc[2 * ch + gr];
              if (mask) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (32 * ch + 16 * gr + e < left) top = fmaxf(top, fmaf(__uint_as_float(a[16 * gr + e]), f.x, f.y));
              } else {
                float best = __uint_as_float(a[16 * gr]) * f.x;
#pragma unroll
                for (int e = 1; e < 16; ++e) best = fmaxf(best, __uint_as_float(a[16 * gr + e]) * f.x);
                top = fmaxf(top, best + f.y);
              }
            }
          }
          if (j == 0) {
            m = top;
          } else {
            const bool over = top > m + kSlack;
            if (__any_sync(0xFFFFFFFFu, over)) {
              const float keep = over ? ex2(m - top) : 1.f;
              if (over) m = top;
              l *= keep;
#pragma unroll
              for (int ch = 0; ch < D / 32; ++ch) {
                tmem_ld32(o_at + 32 * ch, a);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * keep);
                tmem_st32(o_at + 32 * ch, a);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int ch = 0; ch < kKeys / 32; ++ch) {
            tmem_ld32(s_at + 32 * ch, a);
            tmem_ld_wait();
            uint32_t pk[16];
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
              const float4 f = sc[2 * ch + gr];
              const float lv = f.y - base;
              float sum = 0.f;
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float p0 = ex2(fmaf(__uint_as_float(a[16 * gr + e]), f.x, lv));
                float p1 = ex2(fmaf(__uint_as_float(a[16 * gr + e + 1]), f.x, lv));
                if (mask) {
                  if (32 * ch + 16 * gr + e >= left) p0 = 0.f;
                  if (32 * ch + 16 * gr + e + 1 >= left) p1 = 0.f;
                }
                sum += p0 + p1;
                const __half2 q = __floats2half2_rn(p0, p1);
                pk[8 * gr + e / 2] = *reinterpret_cast<const uint32_t*>(&q);
              }
              l = fmaf(sum, f.z, l);
            }
            tc::tmem_st16(s_at + 16 * ch, pk);
          }
          tc::tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[x]);
      }
      // ---- the item's sums: finished, or to be joined ---------------------------------
      ok = ok && warp_wait(ctl, &ctl.o_done[x], items & 1);
      ++items;
      if (ok) tc_fence_after();
      const bool whole = w.lo == 0 && w.hi == w.units;
      const bool sees = lim > 0;
      __half* dst = p.out + static_cast<size_t>(w.r.t0 + tok) * p.out_stride + static_cast<size_t>(h) * D;
      float* lse = p.lse == nullptr ? nullptr : p.lse + static_cast<size_t>(w.r.t0 + tok) * p.q_heads + h;
      constexpr size_t kTileFloats = static_cast<size_t>(kTile) * (D + 2);
      float* slot = p.partial + (static_cast<size_t>(2 * cta + (w.lo == 0 ? 1 : 0)) * 2 + x) * kTileFloats;
      const float inv = inverse_sum(l, sees);
      if (ok && busy) {
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t a[32];
          tmem_ld32(o_at + 32 * ch, a);
          tmem_ld_wait();
          if (whole) {
            if (mine) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t pk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float v0 = sees ? __uint_as_float(a[e + 2 * i]) * inv : 0.f;
                  const float v1 = sees ? __uint_as_float(a[e + 2 * i + 1]) * inv : 0.f;
                  const __half2 q = __floats2half2_rn(v0, v1);
                  pk[i] = *reinterpret_cast<const uint32_t*>(&q);
                }
                *reinterpret_cast<uint4*>(dst + 32 * ch + e) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              }
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              __stcg(reinterpret_cast<float4*>(slot) + static_cast<size_t>(8 * ch + e / 4) * kTile + r,
                     make_float4(__uint_as_float(a[e]), __uint_as_float(a[e + 1]), __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3])));
          }
        }
        tc_fence_before();
      }
      if (whole) {
        if (ok && mine && lse != nullptr) *lse = sees ? kLn2 * (m == -INFINITY ? 0.f : m) + logf(l) : -INFINITY;
        continue;
      }
      __stcg(slot + static_cast<size_t>(D) * kTile + r, m);
      __stcg(slot + static_cast<size_t>(D + 1) * kTile + r, l);
      const long long item_u = w.u - w.lo;
      const int c0 = range_of(ctl.units, item_u, ctas), c1 = range_of(ctl.units, item_u + w.units - 1, ctas);
      __threadfence();
      tile_sync(x);
      if (r == 0) {
        const bool last = atomicAdd(p.arrived + 2 * c0 + x, 1u) == static_cast<uint32_t>(c1 - c0);
        ctl.last[x] = last ? 1u : 0u;
        if (last) p.arrived[2 * c0 + x] = 0u;
      }
      tile_sync(x);
      const bool last = ctl.last[x] != 0u;
      tile_sync(x);  // before the flag is written again
      if (last && mine) {
      __threadfence();
      auto part = [&](int k) { return p.partial + (static_cast<size_t>(2 * k + (k == c0 ? 1 : 0)) * 2 + x) * kTileFloats; };
      float top = -INFINITY, sum = 0.f;
      for (int k = c0; k <= c1; ++k) top = fmaxf(top, __ldcg(part(k) + static_cast<size_t>(D) * kTile + r));
      const float base = top == -INFINITY ? 0.f : top;
      for (int k = c0; k <= c1; ++k)
        sum += __ldcg(part(k) + static_cast<size_t>(D + 1) * kTile + r) * ex2(__ldcg(part(k) + static_cast<size_t>(D) * kTile + r) - base);
      const float scale = inverse_sum(sum, sees);
#pragma unroll 1
      for (int ch = 0; ch < D / 16; ++ch) {
        float4 acc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = c0; k <= c1; ++k) {
          const float* q = part(k);
          const float f = ex2(__ldcg(q + static_cast<size_t>(D) * kTile + r) - base);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(q) + static_cast<size_t>(4 * ch + e) * kTile + r);
            acc[e].x = fmaf(v.x, f, acc[e].x);
            acc[e].y = fmaf(v.y, f, acc[e].y);
            acc[e].z = fmaf(v.z, f, acc[e].z);
            acc[e].w = fmaf(v.w, f, acc[e].w);
          }
        }
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __half2 q0 = __floats2half2_rn(sees ? acc[e].x * scale : 0.f, sees ? acc[e].y * scale : 0.f);
          const __half2 q1 = __floats2half2_rn(sees ? acc[e].z * scale : 0.f, sees ? acc[e].w * scale : 0.f);
          pk[2 * e] = *reinterpret_cast<const uint32_t*>(&q0);
          pk[2 * e + 1] = *reinterpret_cast<const uint32_t*>(&q1);
        }
        *reinterpret_cast<uint4*>(dst + 16 * ch) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<uint4*>(dst + 16 * ch + 8) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
      }
      if (lse != nullptr) *lse = sees ? kLn2 * base + logf(sum) : -INFINITY;
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && aborted(ctl)) atomicOr(p.status, 1u);
}

template <int D>
exl3_status launch(const AttnParams& p, const exl3_kv_cache& c, cudaStream_t stream) {
  if (cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) != cudaSuccess)
    return EXL3_ERR_CUDA;
  int ctas = device_sm_count();
  if (ctas > kMaxPromptCtas) ctas = kMaxPromptCtas;
  prompt_kernel<D><<<ctas, kThreads, Cfg<D>::kSmem, stream>>>(p, c.k, c.v, 2);
  return launch_status();
}

}  // namespace

exl3_status launch_prompt(const AttnParams& p, const exl3_kv_cache& c, cudaStream_t stream) {
  return c.head_dim == 64 ? launch<64>(p, c, stream) : launch<128>(p, c, stream);
}

}  // namespace attn
}  // namespace exl3
