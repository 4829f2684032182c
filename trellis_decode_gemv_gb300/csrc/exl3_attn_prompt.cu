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
// Warp roles (24 warps):
//   0         MMA issue (one lane) and TMEM allocation.
//   1         producer: page numbers and scales (two units ahead), tensor copies of
//             the int8 tiles.  Pages may be smaller than a unit: one copy per page,
//             scales per 16 keys.
//   2, 3      Q of the next item (A, B) into shared memory as soon as the last
//             scores of the current one are computed.
//   4-11, 12-19 softmax of tile A and B: two threads share a row (its TMEM lane), one
//             for each 64 keys of a unit and each half of O's columns; their warps
//             look by a barrier whether any score passes m by 2^15.9, and
//             only then exchange the rows' largest and rescale O, between the
//             MMAs that add to it.  They also take O out.
//   20-23     widening: int8 tiles in shared memory into binary16 operand images,
//             two of K and two of V.  Both are [key][D] rows of 64-element,
//             128-byte pieces in the 128-byte swizzle: K is read as a K-major
//             operand, V as an MN-major one, so V needs no transposition.
//
// Barriers: int8 K and V tiles full/empty, K and V images full, a unit's MMAs done
// (its images are free), scales full (four slots: a slot is rewritten only after
// the softmax of both tiles has used it), per tile Q full/empty, S full, P full (by
// half of the keys), product done, O done.  Every wait is bounded; on timeout the
// CTA sets its abort flag and the status word, every role stops waiting, the MMA
// lane waits (bounded) for its MMAs and the producer for its copies, TMEM is freed.
//
// Measured (2070 MHz, 32 heads over 8, D = 128; one launch): a prompt of 8192 tokens 464
// us, 1185 Tflop/s, the tensor pipe active for 51% of the cycles; four chunks of 512
// tokens after 32K 826 us, 1310 Tflop/s, 55%.  An MMA of 128 x 128 x 16 takes 64 clocks, so a
// unit's 32 take 2048 at D = 128, and a unit takes about 3800.  Two things bound it:
// a tile's S, softmax, P V one after another, because P lies in place of S and the
// next S must wait for the product; and shared memory, which feeds two operands of S,
// one of P V, the widening and its stores (about 2700 clocks a unit), and whose queue
// every wait and exchange stands in: three barriers polled at a time instead of one
// made the kernel 5% slower, the softmax warps polling S another 5%, widening by three
// warps in place of four, to leave the MMA warp's scheduler alone, 9%.  (Units of 64
// keys with two S a tile, which take the product out of the chain, were 1.5 times as
// slow: twice the MMAs and waits for the one thread that issues them.)  Small code
// matters: with the loops rolled (the 24 warps run five different ones) the
// instruction cache stopped missing, the most of the way from 1542 us to 898 for the
// prompt of 8192 when it was first measured.  128 scores a thread spill; a second MMA
// thread (1255 us where one took 911) and scores fetched ahead of their use (spills)
// were slower.
#include "exl3_attn.cuh"

namespace exl3 {
namespace attn {
namespace {

using tc::mma_commit;
using tc::tc_fence_after;
using tc::tc_fence_before;

constexpr int kTile = 128;             // rows of an MMA tile
constexpr int kItemRows = 2 * kTile;
constexpr int kKeys = kPromptUnit;     // keys of a unit
constexpr int kGroups = kKeys / 16;    // scale groups of a unit
constexpr int kMmaWarp = 0;
constexpr int kLoadWarp = 1;
constexpr int kQWarp0 = 2;
constexpr int kSoftmaxWarp0 = 4;
constexpr int kConvWarp0 = 20;
constexpr int kConvThreads = 128;
constexpr int kThreads = 32 * 24;
constexpr int kTmemCols = 512;
constexpr int kPairBarrier = 1;        // + 4 * tile + quarter: the two warps of 32 rows
constexpr int kHalf = kKeys / 2;       // keys of a softmax thread
constexpr int kScaleSlots = 4;
constexpr float kFar = 65536.f;        // x - m is taken exactly for an m past this (binary32 steps of 2^-7 and more)

template <int D>
struct Cfg {
  static constexpr int kPieces = D / 64;               // 64-element pieces of a row
  static constexpr int kPieceBytes = 128 * 128;        // 128 rows of one piece
  static constexpr int kImageBytes = kPieces * kPieceBytes;
  static constexpr int kByteTile = kKeys * D;
  static constexpr int kTiles = kImageBytes * 6 + 2 * kByteTile; // Q A, Q B, K x 2, V x 2; int8 K, V
  static constexpr int kOCol = 2 * kKeys;
};

struct Control {
  uint64_t b_full[2], b_empty[2];   // int8 tiles of K, V
  uint64_t k_full[2], v_full[2];
  uint64_t step_done[2];            // S of unit u and the product of unit u - 1, at u % 2
  uint64_t c_full[kScaleSlots];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], pv_done[2], o_done[2], mma_done;
  float4 scale[kScaleSlots][kGroups];
  alignas(8) float top[2][2][kTile];          // per tile and half of the keys: a row's largest score; at an item's end its sum
  long long bounds[2];
  int last_range;                             // of the item that ends after this range
  SharedReq first_req;
  int first_b, first_tile, first_head, first_lo;
  uint32_t tmem_base, abort;
};

template <bool SHARED>
__device__ __forceinline__ ReqOf<SHARED>& first_req(Control& c) { return c.first_req; }
template <bool SHARED>
__device__ __forceinline__ const ReqOf<SHARED>& first_req(const Control& c) { return c.first_req; }

__device__ __forceinline__ bool aborted(const Control& c) { return *reinterpret_cast<const volatile uint32_t*>(&c.abort) != 0u; }

// A wait of a whole warp; false (for every lane) when it ran out: the CTA gives
// up.  (That another role gave up is not looked at here: what waits for it runs
// out in its turn, once per role.)
__device__ __forceinline__ bool warp_wait(Control& c, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xFFFFFFFFu, mbar_wait(bar, parity))) return true;
  atomicOr(&c.abort, 1u);
  return false;
}

__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(kPairBarrier + id), "n"(64) : "memory"); }

// The same, and whether `any` holds for one of the 64 threads.
__device__ __forceinline__ bool pair_any(int id, bool any) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(kPairBarrier + id), "n"(64), "r"(any ? 1u : 0u)
      : "memory");
  return r != 0u;
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
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
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  float v[16];
  tc::tmem_ld16(taddr, v);
#pragma unroll
  for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(v[e]);
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

// One lane of a converged warp, in a form that the compiler knows to be one lane:
// MMAs issued under `lane == 0` took 73 clocks each, not 64 (128 x 128 x 16, idle
// SM; over 100 beside busy warps).
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0u;
}

// A wait that polls without suspending the thread (a suspended one took 200 to 400
// clocks to come back), for the one thread that feeds the tensor pipe.
__device__ __forceinline__ bool poll_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  for (uint32_t it = 0; it < 16u * tc::kSpinLimit; ++it) {   // a second or so
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}

// 16 bytes global -> shared without registers; zeros if not `valid`.
__device__ __forceinline__ void async_copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
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

__device__ __forceinline__ int row_tiles(int rows) { return (rows + kItemRows - 1) / kItemRows; }
// Units of row tile `rt`: up to the last key that its last row sees, at least one.
// `seq` and `late` count from the first of the request's keys.
template <bool SHARED>
__device__ __forceinline__ int tile_units(const AttnParams& p, int n, int late, int seq, int rt) {
  const int last = (min((rt + 1) * kItemRows, n * p.group) - 1) / p.group;
  return max(1, ((SHARED ? min(seq, late + last + 1) : late + last + 1) + kKeys - 1) / kKeys);
}
template <bool SHARED>
__device__ __forceinline__ int tile_units(const AttnParams& p, const ReqOf<SHARED>& r, int rt) {
  return tile_units<SHARED>(p, r.n, late_of(r) - first_key(r), r.seq - first_key(r), rt);
}

// An item of at most kWhole units is not split: leaving and joining partial results
// is not worth it.  A boundary between ranges that falls into such an item moves to its
// nearer end, which leaves ranges unequal: with 8 in place of 5 a prompt of 1500 tokens
// took 54 us in place of 43, 6 x 200 tokens over 900 51 and not 40; with 3 a prompt of
// 500 took 29 and not 25.
constexpr int kWhole = 5;
constexpr int kLeast = 4;   // units that are worth a range of their own
// Ranges are cut in equal parts of units plus kItemCost for each item: beginning and
// ending one (Q, the first scores, the output) takes about as long as that.
constexpr int kItemCost = kPromptItemCost;

// The items of a range: row tiles in order, the heads of a row tile after one
// another.
template <bool SHARED>
struct Walker {
  const AttnParams& p;
  int left;   // units of the range from the current item's first on
  int b, rt, head, lo, hi, units;
  ReqOf<SHARED> r;
  __device__ __forceinline__ Walker(const AttnParams& params, const Control& c, int count)
      : p(params), left(count), b(c.first_b), rt(c.first_tile), head(c.first_head), lo(c.first_lo), r(first_req<SHARED>(c)) {
    units = tile_units<SHARED>(p, r, rt);
    if (lo == units) advance();
    hi = min(units, lo + left);
  }
  __device__ __forceinline__ void advance() {
    lo = 0;
    if (++head == p.kv_heads) {
      head = 0;
      if (++rt == row_tiles(r.rows)) {
        rt = 0;
        do {
          r = load_req<SHARED>(p, ++b);
        } while (r.rows == 0 && b < req_count<SHARED>(p));
      }
      units = tile_units<SHARED>(p, r, rt);
    }
  }
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ void next() {
    left -= hi - lo;
    if (left <= 0) return;
    advance();
    hi = min(units, lo + left);
  }
};

// ---- prelude: units of all items, and where this CTA's range begins -----------------

// Exclusive prefixes of N values over the CTA's threads in place of them, and their
// totals.  `room`: shared memory of its own, N * 24 numbers; one barrier.
template <int N>
__device__ __forceinline__ void block_scan(long long* room, long long (&v)[N], long long (&total)[N]) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 32, "a lane for each warp");
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  long long inc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) inc[i] = v[i];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, inc[i], d);
      if (lane >= d) inc[i] += o;
    }
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < N; ++i) room[i * kWarps + warp] = inc[i];
  }
  __syncthreads();
  long long sums[N];
#pragma unroll
  for (int i = 0; i < N; ++i) sums[i] = lane < kWarps ? room[i * kWarps + lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, sums[i], d);
      if (lane >= d) sums[i] += o;
    }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    total[i] = __shfl_sync(0xFFFFFFFFu, sums[i], 31);
    const long long before = __shfl_sync(0xFFFFFFFFu, sums[i], (warp + 31) & 31);
    v[i] = inc[i] - v[i] + (warp > 0 ? before : 0);
  }
}

// Requests and groups whose lists are copied first in a call with prefixes.
constexpr int kListed = 1024;

// `room`: 12 bytes for each request, 52 up to kListed of them (borrowed from the operand
// images).  False: the CTA has nothing to do.
template <int D, bool SHARED>
__device__ __forceinline__ bool find_range(const AttnParams& p, Control& c, void* room, int& ctas, int& count) {
  const int tid = threadIdx.x;
  const int requests = req_count<SHARED>(p);
  int32_t* first = static_cast<int32_t*>(room);    // row tiles before each request
  int2* req = reinterpret_cast<int2*>(first + ((requests + 1) & ~1));  // its new tokens (0: another launch's) and keys
  const int per = (requests + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, requests), b1 = min(b0 + per, requests);
  long long* sums = reinterpret_cast<long long*>(c.top);   // not in use yet
  Lists lists(p);
  SharedReq* kept = nullptr;   // what is found out about each request
  if constexpr (SHARED) {
    if (requests <= kListed) {
      kept = reinterpret_cast<SharedReq*>(static_cast<unsigned char*>(room) + 12 * kListed + 16);
      lists.copy_to(p, reinterpret_cast<int32_t*>(kept + requests), kThreads);
      __syncthreads();
    }
  }
  long long mine[1] = {0}, tiles[1];
  Costs costs{0.f, 0.f, 0.f};
  for (int b = b0; b < b1; ++b) {
    const ReqOf<SHARED> r = load_from<SHARED>(p, lists, b);
    req[b] = make_int2(r.rows > 0 ? r.n : 0, r.seq - first_key(r));
    mine[0] += row_tiles(r.rows);
    if constexpr (SHARED) {
      if (kept != nullptr) kept[b] = r;
      costs.add(costs_of<D>(p, r));
    }
  }
  if constexpr (SHARED) {   // the warps' sums behind those of the scans
    costs.add_lanes();
    if ((tid & 31) == 0) reinterpret_cast<Costs*>(sums + 6 * 32)[tid >> 5] = costs;
  }
  block_scan(sums, mine, tiles);
  int most = static_cast<int>(gridDim.x);
  if constexpr (SHARED) {
    const int lane = tid & 31;
    costs = lane < kThreads / 32 ? reinterpret_cast<const Costs*>(sums + 6 * 32)[lane] : Costs{0.f, 0.f, 0.f};
    costs.add_lanes();
    most = min(most, many_sms(p, costs));
  }
  long long at = mine[0];
  for (int b = b0; b < b1; ++b) {
    first[b] = static_cast<int32_t>(at);
    at += row_tiles(req[b].x * p.group);
  }
  __syncthreads();
  const int n = static_cast<int>(tiles[0]);
  if (SHARED && kept != nullptr && n <= 32) {
    // As many tiles as lanes, a tile each: every warp finds the range by itself.  (The way
    // below takes 4 us, most of it for code that comes from memory.)
    const int x = tid & 31;
    int b = 0, to = requests;
    while (to - b > 1) {
      const int mid = (b + to) >> 1;
      if (first[mid] <= x) b = mid; else to = mid;
    }
    const int tile = x - first[b];
    const int len = x < n ? tile_units<true>(p, kept[b], tile) : 0;
    const long long cost = x < n ? static_cast<long long>(len + kItemCost) * p.kv_heads : 0;
    long long sum = cost, ranges = x < n ? static_cast<long long>(len <= kWhole ? 1 : (len + kLeast - 1) / kLeast) * p.kv_heads : 0;
    int lens = len;   // of tiles up to this one
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      const int l = __shfl_up_sync(0xFFFFFFFFu, lens, d);
      if (x >= d) {
        sum += o;
        lens += l;
      }
      ranges += __shfl_xor_sync(0xFFFFFFFFu, ranges, d);
    }
    const long long total = __shfl_sync(0xFFFFFFFFu, sum, 31);
    const long long all_units = static_cast<long long>(__shfl_sync(0xFFFFFFFFu, lens, 31)) * p.kv_heads;
    ctas = static_cast<int>(min(static_cast<long long>(most), ranges));
    if (static_cast<int>(blockIdx.x) >= ctas) return false;
    long long bound[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long u = range_begin(total, blockIdx.x + e, ctas);
      const uint32_t ended = __popc(__ballot_sync(0xFFFFFFFFu, sum <= u));   // tiles that end before u: it is in the next
      bound[e] = all_units;
      if (ended >= static_cast<uint32_t>(n)) continue;   // the last range's end
      const int its = __shfl_sync(0xFFFFFFFFu, len, ended), before = __shfl_sync(0xFFFFFFFFu, lens - len, ended);
      const long long off = u - __shfl_sync(0xFFFFFFFFu, sum - cost, ended);
      const int head = off <= 0x7FFFFFFFLL ? static_cast<int>(off) / (its + kItemCost) : static_cast<int>(off / (its + kItemCost));
      const long long start = u - off + static_cast<long long>(head) * (its + kItemCost);
      int lo = static_cast<int>(u - start);
      lo = its <= kWhole ? (2 * lo < its + kItemCost ? 0 : its) : max(0, lo - kItemCost);
      bound[e] = static_cast<long long>(before) * p.kv_heads + static_cast<long long>(head) * its + lo;
      if (tid == static_cast<int>(ended)) {
        if (e == 1) c.last_range = range_of(total, start + kItemCost + its - 1, ctas);
        if (e == 0) {
          c.first_b = b;
          c.first_tile = tile;
          c.first_head = head;
          c.first_lo = lo;
          c.first_req = kept[b];
        }
      }
    }
    __syncthreads();   // c; the room is the operands' again
    count = static_cast<int>(bound[1] - bound[0]);
    return count > 0;
  }
  const int share = (n + kThreads - 1) / kThreads;
  const int x0 = min(tid * share, n), x1 = min(x0 + share, n);
  int from = 0, to = requests;   // the last request that begins at or before x0
  while (to - from > 1) {
    const int mid = (from + to) >> 1;
    if (first[mid] <= x0) from = mid; else to = mid;
  }
  long long part[3] = {0, 0, 0}, all[3];   // cost, units, ranges that this thread's tiles are worth
  for (int x = x0, b = from; x < x1; ++x) {
    while (b + 1 < requests && first[b + 1] <= x) ++b;
    const int len = tile_units<SHARED>(p, req[b].x, SHARED && b < p.groups ? req[b].y : req[b].y - req[b].x, req[b].y, x - first[b]);
    part[0] += static_cast<long long>(len + kItemCost) * p.kv_heads;
    part[1] += static_cast<long long>(len) * p.kv_heads;
    part[2] += static_cast<long long>(len <= kWhole ? 1 : (len + kLeast - 1) / kLeast) * p.kv_heads;
  }
  const long long own_cost = part[0];
  block_scan(sums + 3 * 32, part, all);
  const long long cost = all[0], units = all[1];
  long long before = part[0], before_units = part[1];
  ctas = static_cast<int>(min(static_cast<long long>(most), all[2]));
  const int cta = blockIdx.x;
  if (cta >= ctas) return false;
  const long long u[2] = {range_begin(cost, cta, ctas), range_begin(cost, cta + 1, ctas)};
  if (tid == 0) {
    c.bounds[1] = units;   // the last range's end is in no item
  }
  __syncthreads();
  if (before < cost && u[1] >= before && u[0] < before + own_cost) {
    for (int x = x0, b = from; x < x1; ++x) {
      while (b + 1 < requests && first[b + 1] <= x) ++b;
      const int len = tile_units<SHARED>(p, req[b].x, SHARED && b < p.groups ? req[b].y : req[b].y - req[b].x, req[b].y, x - first[b]);
      const long long of_tile = static_cast<long long>(len + kItemCost) * p.kv_heads;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (u[e] < before || u[e] >= before + of_tile) continue;
        const long long off = u[e] - before;   // (a 64-bit division takes a few hundred clocks)
        const int head = off <= 0x7FFFFFFFLL ? static_cast<int>(off) / (len + kItemCost) : static_cast<int>(off / (len + kItemCost));
        const long long start = before + static_cast<long long>(head) * (len + kItemCost);
        int lo = static_cast<int>(u[e] - start);
        if (len <= kWhole)
          lo = 2 * lo < len + kItemCost ? 0 : len;
        else
          lo = max(0, lo - kItemCost);
        c.bounds[e] = before_units + static_cast<long long>(head) * len + lo;
        if (e == 1) c.last_range = range_of(cost, start + kItemCost + len - 1, ctas);
        if (e == 0) {
          c.first_b = b;
          c.first_tile = x - first[b];
          c.first_head = head;
          c.first_lo = lo;
          first_req<SHARED>(c) = load_from<SHARED>(p, lists, b);
        }
      }
      before += of_tile;
      before_units += static_cast<long long>(len) * p.kv_heads;
    }
  }
  __syncthreads();
  count = static_cast<int>(c.bounds[1] - c.bounds[0]);
  return count > 0;
}

// ---- widening ------------------------------------------------------------------------

// A unit's int8 tile (as the tensor copy swizzles it) into an operand image.  A
// warp takes 8 rows x 64 elements at a time: lane (k, b, c) piece c of row k, or of
// row k ^ 5 for b = 1.  The eight lanes of a shared-memory phase then hold two rows
// whose swizzles differ in bits 0 and 2, and neither the 16-byte loads nor the two
// 16-byte stores touch a bank twice.
template <int D>
__device__ __forceinline__ void widen(const unsigned char* tile, uint32_t image, int tid) {
  constexpr int kPieces = Cfg<D>::kPieces;
  const int lane = tid & 31;
  const int c = lane & 3;
  const int row = (lane >> 3) ^ (lane & 4 ? 5 : 0);      // of 8
  const int at = (tid >> 5) * 8 + row;                   // warp w: row groups w, w + 4, ...
  const unsigned char* src = tile + at * D;
  const uint32_t dst = image + static_cast<uint32_t>(at * 128);
  const uint32_t first = dst + static_cast<uint32_t>((2 * c) ^ row) * 16, second = dst + static_cast<uint32_t>((2 * c + 1) ^ row) * 16;
#pragma unroll
  for (int pc = 0; pc < kPieces; ++pc) {
    const unsigned char* from = src + ((c + 4 * pc) ^ (D == 128 ? row : row >> 1)) * 16;
#pragma unroll 2
    for (int i = 0; i < 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(from + i * 32 * D);
      const uint32_t x = v.x ^ 0x80808080u, y = v.y ^ 0x80808080u, z = v.z ^ 0x80808080u, w = v.w ^ 0x80808080u;
      const uint32_t off = static_cast<uint32_t>(pc * Cfg<D>::kPieceBytes + i * 32 * 128);
      st_shared_v4(first + off, cvt_lo(x), cvt_hi(x), cvt_lo(y), cvt_hi(y));
      st_shared_v4(second + off, cvt_lo(z), cvt_hi(z), cvt_lo(w), cvt_hi(w));
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Largest of 16 scores.
__device__ __forceinline__ float max16(const uint32_t* a) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(__uint_as_float(a[4 * i]), __uint_as_float(a[4 * i + 1]), __uint_as_float(a[4 * i + 2]));
#pragma unroll
  for (int i = 0; i < 2; ++i) m[i] = max3(m[i], m[i + 2], __uint_as_float(a[4 * i + 3]));
  return fmaxf(max3(m[0], m[1], __uint_as_float(a[11])), __uint_as_float(a[15]));
}

// Largest x = c ks s + log2 vs (c ks >= 0) of 16 scores of one scale; `left`: how
// many of them the row sees (MASK).
template <bool MASK>
__device__ __forceinline__ float max_of(const uint32_t* v, const float4& f, int left) {
  if constexpr (MASK) {
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, e < left ? fmaf(__uint_as_float(v[e]), f.x, f.y) : -INFINITY);
    return top;
  } else {
    return fmaf(max16(v), f.x, f.y);
  }
}

// P of 16 scores of one scale to tensor memory, their sum / vs onto l.  EXACT: x as the
// maximum took it, then its distance to m, and only the first `left` scores.  Otherwise c ks
// s + (log2 vs - m), one instruction for two scores less, whose rounding by m's size a large
// m does not allow: P could pass binary16's range or vanish.  (Prompt of 8192: 485 us, 478
// without any regard to large m, 497 with all units EXACT.)
template <bool EXACT>
__device__ __forceinline__ void exp_of(const uint32_t* v, const float4& f, int left, float base, float& l, uint32_t p_at) {
  uint32_t pk[8];
  const float y = EXACT ? f.y : f.y - base;
  const uint64_t ff = pair(f.x, f.x), yy = pair(y, y), mm = pair(-base, -base);
  uint64_t sum = 0;   // two zeros
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    uint64_t x = fma2(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), ff, yy);
    if constexpr (EXACT) x = add2(x, mm);
    float p0, p1;
    unpair(x, p0, p1);
    if constexpr (EXACT) {
      p0 = e < left ? p0 : -INFINITY;
      p1 = e + 1 < left ? p1 : -INFINITY;
    }
    p0 = ex2(p0);
    p1 = ex2(p1);
    sum = add2(sum, pair(p0, p1));
    const __half2 q = __floats2half2_rn(p0, p1);
    pk[e / 2] = *reinterpret_cast<const uint32_t*>(&q);
  }
  float s0, s1;
  unpair(sum, s0, s1);
  l = fmaf(s0 + s1, f.z, l);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(p_at), "r"(pk[0]),
               "r"(pk[1]), "r"(pk[2]), "r"(pk[3]), "r"(pk[4]), "r"(pk[5]), "r"(pk[6]), "r"(pk[7])
               : "memory");
}

// Where P of 16-key group i of a half lies, from the half's first score on: over
// scores that are in registers by then.
__device__ __forceinline__ constexpr uint32_t p_column(int i) { return static_cast<uint32_t>((i >> 1) * 32 + (i & 1) * 8); }

// Whether a row's m is so large that x - m has to be taken exactly.  (m is the same in
// both warps of the rows.)  Not for an infinite one: its row is NaN or sees nothing either
// way, and the rows beside it keep their bits.
__device__ __forceinline__ bool is_far(float m) { return __any_sync(0xFFFFFFFFu, fabsf(m) > kFar && fabsf(m) < INFINITY); }

// 64 of a row's scores (the row's other 64 are another warp's): the running maximum
// m (O and l rescaled when it moves), P in place of the scores, l.  `left`: the
// keys of these 64 that the row sees, looked at only if EXACT, as a unit that needs a
// mask has to be.  True: m has become large, and the unit has to be taken again, EXACT.
// `s_at` the scores, `o_at` this thread's half of O; `mine` the row's place in the
// exchange of the two warps, `other` the other warp's.  A warp whose wait ran out
// takes part in the exchange with NaN, and both give up.  S is read twice, 32 scores
// at a time, in loops that are not unrolled: the code of all roles has to stay in the
// instruction cache (unrolled, the kernel took 1.6 times as long).
template <int D, bool EXACT>
__device__ __forceinline__ bool softmax_unit(uint32_t s_at, uint32_t o_at, const float4* sc, int left, bool first, float& m,
                                             float& l, uint32_t mine, uint32_t other, int pair_id, bool& ok) {
  constexpr int kOnce = EXACT ? 1 : 2;   // groups at a time: few units are EXACT, and their code is to be small
  uint32_t a[16 * kOnce];
  float top = __int_as_float(0x7FC00000);
  if (ok) {
    top = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < 4; i += kOnce) {
      if constexpr (EXACT) {
        tmem_ld16(s_at + 16 * i, a);
        top = fmaxf(top, max_of<true>(a, sc[i], left - 16 * i));
      } else {
        tmem_ld32(s_at + 16 * i, a);
        tmem_ld_wait();
        top = fmaxf(top, fmaxf(max_of<false>(a, sc[i], left), max_of<false>(a + 16, sc[i + 1], left)));
      }
    }
  }
  // In most units no score of the rows passes the maximum by 2^kRoom, and one barrier says so.
  if (pair_any(pair_id, first || !ok || top - m > kRoom)) {
    st_shared_f32(mine, ok ? fmaxf(top, -INFINITY) : top);   // scores that are all NaN count as none
    pair_sync(pair_id);
    const float its = ld_shared_f32(other);
    ok = __all_sync(0xFFFFFFFFu, ok && its == its);
    if (!ok) return false;
    top = fmaxf(top, its);   // not NaN: `its` is not
    if (first) {
      m = top - kBelow;
    } else {
      const bool over = top - m > kRoom;
      const float next = top - kBelow;
      const float keep = over ? ex2(m - next) : 1.f;
      if (over) m = next;
      l *= keep;
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        float o[16];
        tc::tmem_ld16(o_at + 16 * ch, o);
        uint32_t b[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = __float_as_uint(o[e] * keep);
        tc::tmem_st16(o_at + 16 * ch, b);
      }
      tc::tmem_st_wait();
      tc_fence_before();
    }
    pair_sync(pair_id);   // all of O, before either warp lets the next product begin; the exchange is read
    if (!EXACT && is_far(m)) return true;   // both warps have the same rows and the same m
  }
  const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
  for (int i = 0; i < 4; i += kOnce) {
    if constexpr (EXACT) {
      tmem_ld16(s_at + 16 * i, a);
      exp_of<true>(a, sc[i], left - 16 * i, base, l, s_at + p_column(i));
    } else {
      tmem_ld32(s_at + 16 * i, a);
      tmem_ld_wait();
      exp_of<false>(a, sc[i], left, base, l, s_at + p_column(i));
      exp_of<false>(a + 16, sc[i + 1], left, base, l, s_at + p_column(i + 1));
    }
  }
  tc::tmem_st_wait();
  tc_fence_before();
  return false;
}

// Columns of a row of the output.
template <int N>
__device__ __forceinline__ void store_row(__half* dst, const uint32_t (&a)[N], float inv, bool sees) {
#pragma unroll
  for (int e = 0; e < N; e += 8) {
    uint32_t pk[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = sees ? __uint_as_float(a[e + 2 * i]) * inv : 0.f;
      const float v1 = sees ? __uint_as_float(a[e + 2 * i + 1]) * inv : 0.f;
      const __half2 q = __floats2half2_rn(v0, v1);
      pk[i] = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint4*>(dst + e) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  }
}

// Columns of a row's sums.
template <int N>
__device__ __forceinline__ void store_sums(float* dst, const uint32_t (&a)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) *reinterpret_cast<uint4*>(dst + e) = make_uint4(a[e], a[e + 1], a[e + 2], a[e + 3]);
}

// The end of an item: its row sums taken out of tensor memory and finished, or left
// for the range whose arrival completes the item.  Not inlined: its registers are
// not the unit loop's.
template <int D, bool SHARED>
__device__ __noinline__ void finish_item(const AttnParams& p, Control& ctl, ReqOf<SHARED> req, bool own, int head, int base, int lo, bool whole,
                                         bool busy, bool ok, uint32_t o_at, float m, float l) {
  const int r = threadIdx.x & (kTile - 1);
  const int sw = (threadIdx.x >> 5) - kSoftmaxWarp0;
  const int x = sw >> 3, half = (sw >> 2) & 1, pair_id = 4 * x + (sw & 3);
  const uint32_t mine_top = smem_u32(&ctl.top[x][half][r]), other_top = smem_u32(&ctl.top[x][half ^ 1][r]);
  if (!ok) l = unfinished();
  if (busy) {
    st_shared_f32(mine_top, l);
    pair_sync(pair_id);
    l += ld_shared_f32(other_top);
    pair_sync(pair_id);   // before either writes there again
  }
  const bool mine = base + r < req.rows;
  const int rr = base + r;
  const int tok = rr / p.group;
  const bool sees = late_of(req) + tok + 1 > 0;
  const int h = head * p.group + (rr - tok * p.group);
  const size_t part_at = SHARED ? (static_cast<size_t>(own ? p.tokens : 0) + req.t0 + tok) * p.q_heads + h : 0;
  __half* dst = p.out + static_cast<size_t>(req.t0 + tok) * p.out_stride + static_cast<size_t>(h) * D + half * (D / 2);
  constexpr size_t kTileFloats = prompt_slot_floats(D) / 2;
  constexpr size_t kMAt = static_cast<size_t>(D) * kTile, kLAt = static_cast<size_t>(D + 1) * kTile;
  float* slot = p.partial + (static_cast<size_t>(2 * blockIdx.x + (lo == 0 ? 1 : 0)) * 2 + x) * kTileFloats;
  const int quad0 = half * (D / 8);   // this half's first four columns
  if (busy) {
    const float inv = inverse_sum(l, sees);
#pragma unroll 1
    for (int ch = 0; ch < D / 64; ++ch) {
      uint32_t a[32];
      if (ok) {
        tmem_ld32(o_at + 32 * ch, a);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) a[e] = 0u;
      }
      if (whole) {
        if constexpr (SHARED) {
          if (mine) store_sums(p.part + part_at * D + half * (D / 2) + 32 * ch, a);
        } else {
          if (mine) store_row(dst + 32 * ch, a, inv, sees);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          __stcg(reinterpret_cast<float4*>(slot) + static_cast<size_t>(quad0 + 8 * ch + e / 4) * kTile + r,
                 make_float4(__uint_as_float(a[e]), __uint_as_float(a[e + 1]), __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3])));
      }
    }
    tc_fence_before();
  }
  float* lse = p.lse != nullptr && half == 0 ? p.lse + static_cast<size_t>(req.t0 + tok) * p.q_heads + h : nullptr;
  if (whole) {
    if constexpr (SHARED) {
      if (mine && half == 0) {
        p.part_ml[part_at] = make_float2(m, l);
        mark_row(p, req, own, tok, part_at - (own ? static_cast<size_t>(p.tokens) * p.q_heads : 0), 0u);
      }
      return;
    }
    if (mine && lse != nullptr) *lse = sees ? kLn2 * (m == -INFINITY ? 0.f : m) + logf(l) : -INFINITY;
    return;
  }
  if (half == 0) {
    __stcg(slot + kMAt + r, m);
    __stcg(slot + kLAt + r, l);
  }
  // the range in which the item begins tells the join about it
  if constexpr (SHARED) {
    if (lo == 0 && half == 0) {
      if (mine)
        mark_row(p, req, own, tok, part_at - (own ? static_cast<size_t>(p.tokens) * p.q_heads : 0), 1u + kMaxCtas + blockIdx.x);
      if (x == 0 && r == 0)
        p.shared_split[kMaxCtas + blockIdx.x] = SharedSplit{static_cast<long long>(req.t0) * p.group + base, ctl.last_range, 0};
    }
    return;
  }
  if (lo == 0 && x == 0 && half == 0 && r == 0)
    p.split[blockIdx.x] = SplitItem{req.t0, req.n, req.seq, req.rows, base, head, ctl.last_range, 0};
}

// Items that are spread over several ranges, after the other kernel: block (c, y) the
// rows 16 y .. 16 y + 15 of the item that begins in range c.  (Joined by the CTA
// that finished last, an item over 19 ranges, 2.5 MB of partial sums, took 70 us:
// one SM reads 64 bytes a clock.)
constexpr int kJoinRows = 16;
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const SplitItem it = p.split[c];
  const int row = static_cast<int>(blockIdx.y) * kJoinRows + threadIdx.x % kJoinRows;   // of the item
  if (it.last < 0 || it.base + row >= it.rows) return;
  constexpr int kQuads = D / 4 / (kJoinThreads / kJoinRows);   // 4 or 2 groups of four columns a thread
  const int quad0 = static_cast<int>(threadIdx.x) / kJoinRows * kQuads;
  const int x = row / kTile, r = row % kTile;
  constexpr size_t kTileFloats = static_cast<size_t>(kTile) * (D + 2);
  const float* first = p.partial + (static_cast<size_t>(2 * c + 1) * 2 + x) * kTileFloats;
  float top = -INFINITY, sum = 0.f;
  float4 acc[kQuads];
#pragma unroll
  for (int e = 0; e < kQuads; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = c; k <= it.last; ++k) {
    const float* s = k == c ? first : p.partial + (static_cast<size_t>(2 * k) * 2 + x) * kTileFloats;
    const float m = __ldcg(s + static_cast<size_t>(D) * kTile + r);
    const float l = __ldcg(s + static_cast<size_t>(D + 1) * kTile + r);
    float4 v[kQuads];
#pragma unroll
    for (int e = 0; e < kQuads; ++e) v[e] = __ldcg(reinterpret_cast<const float4*>(s) + static_cast<size_t>(quad0 + e) * kTile + r);
    const float up = fmaxf(top, m);
    const float base = up == -INFINITY ? 0.f : up;
    const float fa = ex2(top - base), fb = ex2(m - base);
    top = up;
    sum = sum * fa + l * fb;
#pragma unroll
    for (int e = 0; e < kQuads; ++e) {
      acc[e].x = acc[e].x * fa + v[e].x * fb;
      acc[e].y = acc[e].y * fa + v[e].y * fb;
      acc[e].z = acc[e].z * fa + v[e].z * fb;
      acc[e].w = acc[e].w * fa + v[e].w * fb;
    }
  }
  const int rr = it.base + row;
  const int tok = rr / p.group;
  const int h = it.head * p.group + (rr - tok * p.group);
  const bool sees = it.seq - it.n + tok + 1 > 0;
  const float inv = inverse_sum(sum, sees);
  __half* dst = p.out + static_cast<size_t>(it.t0 + tok) * p.out_stride + static_cast<size_t>(h) * D + 4 * quad0;
#pragma unroll
  for (int e = 0; e < kQuads; ++e) {
    const __half2 q0 = __floats2half2_rn(sees ? acc[e].x * inv : 0.f, sees ? acc[e].y * inv : 0.f);
    const __half2 q1 = __floats2half2_rn(sees ? acc[e].z * inv : 0.f, sees ? acc[e].w * inv : 0.f);
    *reinterpret_cast<uint2*>(dst + 4 * e) = make_uint2(*reinterpret_cast<const uint32_t*>(&q0), *reinterpret_cast<const uint32_t*>(&q1));
  }
  if (p.lse != nullptr && quad0 == 0)
    p.lse[static_cast<size_t>(it.t0 + tok) * p.q_heads + h] = sees ? kLn2 * (top == -INFINITY ? 0.f : top) + logf(sum) : -INFINITY;
}

template <int D, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ CUtensorMap qmap) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];   // the images: swizzle atoms
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  const int warp = tid >> 5;
  const uint32_t images = smem_u32(smem_raw);   // Q A, Q B, K 0, K 1, V 0, V 1
  unsigned char* bytes = smem_raw + 6 * C::kImageBytes;   // int8 K, V
  Control& ctl = *reinterpret_cast<Control*>(bytes + 2 * C::kByteTile);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.b_full[i], 1);
      mbar_init(&ctl.b_empty[i], kConvThreads / 32);
      mbar_init(&ctl.k_full[i], kConvThreads / 32);
      mbar_init(&ctl.v_full[i], kConvThreads / 32);
      mbar_init(&ctl.step_done[i], 1);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i][0], kTile / 32);   // the four warps of 64 keys
      mbar_init(&ctl.p_full[i][1], kTile / 32);
      mbar_init(&ctl.pv_done[i], 1);
      mbar_init(&ctl.o_done[i], 1);
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_empty[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(&ctl.c_full[i], 1);
    mbar_init(&ctl.mma_done, 1);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (SHARED && tid == 32) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
    prefetch_map(&qmap);
  }
  if (!SHARED && tid == 0) p.split[blockIdx.x].last = -1;   // no item begins here and ends later, so far
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int ctas, count;
  if (!find_range<D, SHARED>(p, ctl, smem_raw, ctas, count)) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // not done before the few-rows kernel is
    return;
  }
  if (warp == kMmaWarp) tc::tmem_alloc(&ctl.tmem_base, kTmemCols);
  // The prelude wrote its table where the first Q comes by tensor copies: stores of one
  // proxy before those of the other.
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  Walker<SHARED> w(p, ctl, count);

  if (warp == kMmaWarp) {
    // ---- MMA issue: one lane runs the whole loop -----------------------------------------
    // Before the first unit, and after the product of unit u - 1, the scores of unit
    // u are issued.  The code is kept small (nothing is unrolled but the MMAs of one
    // product) and what can be waited for early is: this thread is on the critical
    // path whenever the tensor pipe runs dry.
    if (elect()) {
      constexpr uint32_t kIdescS = idesc(kKeys, false), kIdescO = idesc(D, true);
      const uint64_t q_desc = swizzled_desc(images, 16, 1024);
      const uint64_t k_desc = swizzled_desc(images + 2 * C::kImageBytes, 16, 1024);
      const uint64_t v_desc = swizzled_desc(images + 4 * C::kImageBytes, C::kPieceBytes, 1024);
      uint32_t used = 0;        // bit x: parity of the products of tile x so far
      uint32_t begun = 0;       // bit x: parity of the items of tile x so far
      int now = 0, next = w.r.rows - w.rt * kItemRows > kTile ? 2 : 1;  // tiles of unit u - 1, of unit u
      int blk = w.lo;           // unit u in its item
      bool first = false, last = true;   // unit u - 1 begins, ends its item
      bool ok = true;
#pragma unroll 1
      for (uint32_t u = 0; u <= static_cast<uint32_t>(count) && ok; ++u) {
        const uint32_t slot = u & 1, prev = slot ^ 1;
        // K of unit u is widened after V of unit u - 1: one wait for both
        ok = next > 0 ? poll_wait(&ctl.k_full[slot], (u >> 1) & 1) : poll_wait(&ctl.v_full[prev], ((u - 1) >> 1) & 1);
#pragma unroll 1
        for (int x = 0; x < 2 && ok; ++x) {
          const uint32_t s_col = tmem + static_cast<uint32_t>(x * kKeys);
          if (x < now) {
            const uint64_t b = v_desc + ((prev * C::kImageBytes) >> 4);
#pragma unroll 1
            for (int h = 0; h < 2 && ok; ++h) {   // half of the keys
              ok = poll_wait(&ctl.p_full[x][h], (used >> x) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < kHalf / 16; ++k)
                tc::mma_f16_ts(tmem + static_cast<uint32_t>(C::kOCol + x * D), s_col + kHalf * h + p_column(k),
                               b + static_cast<uint32_t>((h * kHalf * 128 + k * 2048) >> 4), kIdescO,
                               !first || h > 0 || k > 0 ? 1u : 0u);
            }
            if (!ok) break;
            if (last) mma_commit(&ctl.o_done[x]);
            mma_commit(&ctl.pv_done[x]);
          }
          if (x < next && last) {
            ok = poll_wait(&ctl.q_full[x], (begun >> x) & 1);
            begun ^= 1u << x;
          }
          // the next scores go where P is: its product has to be complete
          if (x < now) {
            ok = ok && poll_wait(&ctl.pv_done[x], (used >> x) & 1);
            used ^= 1u << x;
          }
          if (x < next && ok) {
            tc_fence_after();
            const uint64_t a = q_desc + static_cast<uint32_t>((x * C::kImageBytes) >> 4);
            const uint64_t b = k_desc + ((slot * C::kImageBytes) >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = static_cast<uint32_t>((k >> 2) * C::kPieceBytes + (k & 3) * 32) >> 4;
              mma_ss(s_col, a + off, b + off, kIdescS, k > 0 ? 1u : 0u);
            }
            mma_commit(&ctl.s_full[x]);
            if (blk + 1 == w.hi) mma_commit(&ctl.q_empty[x]);
          }
        }
        if (!ok) break;
        mma_commit(&ctl.step_done[slot]);
        now = next;
        first = blk == w.lo;
        last = ++blk == w.hi;
        if (last) {
          w.next();
          blk = w.lo;
          next = !w.more() ? 0 : w.r.rows - w.rt * kItemRows > kTile ? 2 : 1;
        }
      }
      if (!ok) atomicOr(&ctl.abort, 1u);
      mma_commit(&ctl.mma_done);
      mbar_wait(&ctl.mma_done, 0);
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ---- producer ----------------------------------------------------------------------
    // lanes 0-7: the 16-key groups of the unit two ahead of the one being copied
    const int key16 = (lane & 7) * 16;
    bool live = true;
    int blk = w.lo;
    struct Look {
      int page, head, keys;   // page number as the table has it; the request's keys from this unit's first on
    };
    auto look_up = [&]() -> Look {
      Look k{-1, 0, 0};
      if (live) {
        const int key = first_key(w.r) + blk * kKeys + key16;
        k.head = w.head;
        k.keys = w.r.seq - first_key(w.r) - blk * kKeys;
        if (key < w.r.seq) k.page = __ldg(p.table + static_cast<size_t>(table_row(w.r, w.b)) * p.table_stride + (key >> p.page_shift));
        if (++blk == w.hi) {
          w.next();
          live = w.more();
          blk = w.lo;
        }
      }
      return k;
    };
    struct Scales {
      float k, v;
    };
    auto scales_of = [&](const Look& k) -> Scales {
      Scales s{0.f, 1.f};   // a page number outside the pool reads as zeros
      if (k.page >= 0 && k.page < p.pages) {
        const size_t at = static_cast<size_t>(k.page) * p.kv_heads + k.head;
        s.k = __ldg(p.k_scale + at);
        s.v = __ldg(p.v_scale + at);
      }
      return s;
    };
    const int per_page = 1 << p.page_shift;
    const int step = per_page >> 4;              // groups per copy
    const int copies = kKeys >> p.page_shift;    // pages of a unit
    const uint32_t copy_bytes = static_cast<uint32_t>(per_page * D);
    Look l0 = look_up(), l1 = look_up();
    Scales s0 = scales_of(l0);
    const uint32_t posts = p.stall != 0 ? 1u : static_cast<uint32_t>(count);
    uint32_t n = 0;
    for (; n < posts; ++n) {
      const Look l2 = look_up();
      const Scales s1 = scales_of(l1);
      // one copy per page that holds keys of the request; what is not copied is
      // whatever was there (finite, and its P are 0)
      const int pg = __shfl_sync(0xFFFFFFFFu, l0.page, (lane * step) & 7);   // lane i < copies issues copy i
      const bool mine = lane < copies && lane * per_page < l0.keys;
      const int block = pg >= 0 && pg < p.pages ? pg * p.kv_heads + l0.head : p.pages * p.kv_heads;
      const uint32_t total = static_cast<uint32_t>(__popc(__ballot_sync(0xFFFFFFFFu, mine))) * copy_bytes;
      if (n > 0 && !warp_wait(ctl, &ctl.b_empty[0], (n - 1) & 1)) break;
      if (lane == 0) mbar_arrive_expect_tx(&ctl.b_full[0], total);
      __syncwarp();
      if (mine) tensor_g2s(bytes + lane * copy_bytes, &kmap, 0, block, &ctl.b_full[0]);
      // the unit four before is done (its K image has been written over): the slot is free
      if (lane < kGroups) {
        const PageScale ps = page_scale(p, s0.k, s0.v);
        ctl.scale[n % kScaleSlots][lane] = make_float4(ps.c, ps.lv, ps.iv, 0.f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.c_full[n % kScaleSlots]);
      if (n > 0 && !warp_wait(ctl, &ctl.b_empty[1], (n - 1) & 1)) {
        mbar_wait(&ctl.b_full[0], n & 1);
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&ctl.b_full[1], total);
      __syncwarp();
      if (mine) tensor_g2s(bytes + C::kByteTile + lane * copy_bytes, &vmap, 0, block, &ctl.b_full[1]);
      l0 = l1;
      l1 = l2;
      s0 = s1;
    }
    // Wait (bounded) for the copies in flight.
    if (n > 0) {
      mbar_wait(&ctl.b_full[0], (n - 1) & 1);
      mbar_wait(&ctl.b_full[1], (n - 1) & 1);
    }
  } else if (warp < kSoftmaxWarp0) {
    // ---- Q ---------------------------------------------------------------------------
    const int x = warp - kQWarp0;
    uint32_t items = 0;
    for (; w.more(); w.next()) {
      const int row0 = w.rt * kItemRows + x * kTile;
      const int rows = w.r.rows - row0;
      if (rows <= 0) continue;
      if (items > 0 && !warp_wait(ctl, &ctl.q_empty[x], (items - 1) & 1)) break;
      ++items;
      if (p.q_box != 0) {
        // whole tokens: the tile's rows as one box of (128 / group) tokens x group heads per 64-element piece
        if (lane == 0) {
          mbar_arrive_expect_tx(&ctl.q_full[x], C::kImageBytes);
#pragma unroll
          for (int pc = 0; pc < C::kPieces; ++pc)
            tensor_g2s_at(smem_raw + x * C::kImageBytes + pc * C::kPieceBytes, &qmap, 64 * pc, w.head * p.group,
                          w.r.t0 + row0 / p.group, &ctl.q_full[x]);
        }
        __syncwarp();
        continue;
      }
      constexpr int kChunks = D / 8;            // 16-byte pieces of a row
      constexpr int kRowsAtOnce = 32 / kChunks; // 2 or 4
      const int c = lane % kChunks;
      const uint32_t image = images + static_cast<uint32_t>(x) * C::kImageBytes + static_cast<uint32_t>((c >> 3) * C::kPieceBytes);
      int tok = (row0 + lane / kChunks) / p.group;
      int hd = row0 + lane / kChunks - tok * p.group;
      const __half* base = p.q + static_cast<size_t>(w.r.t0) * p.q_stride + static_cast<size_t>(w.head) * p.group * D + c * 8;
#pragma unroll 4
      for (int r = lane / kChunks; r < kTile; r += kRowsAtOnce) {
        const bool in = r < rows;
        const __half* src = base + static_cast<size_t>(tok) * p.q_stride + static_cast<size_t>(hd) * D;
        async_copy16(image + static_cast<uint32_t>(r * 128 + (((c & 7) ^ (r & 7)) * 16)), in ? src : p.q, in);
        hd += kRowsAtOnce;
        while (hd >= p.group) {
          hd -= p.group;
          ++tok;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (p.negate)
        for (int r = lane / kChunks; r < kTile; r += kRowsAtOnce) {
          uint4* at = reinterpret_cast<uint4*>(smem_raw + (image - images) + r * 128 + (((c & 7) ^ (r & 7)) * 16));
          const uint4 v = *at;
          *at = make_uint4(v.x ^ 0x80008000u, v.y ^ 0x80008000u, v.z ^ 0x80008000u, v.w ^ 0x80008000u);
        }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.q_full[x]);
    }
    if (p.q_box != 0 && items > 0) mbar_wait(&ctl.q_full[x], (items - 1) & 1);  // its last copy
  } else if (warp >= kConvWarp0) {
    // ---- widening ----------------------------------------------------------------------
    const int ct = tid - 32 * kConvWarp0;
    for (uint32_t n = 0; n < static_cast<uint32_t>(count); ++n) {
      const uint32_t slot = n & 1;
      if (!warp_wait(ctl, &ctl.b_full[0], n & 1) || (n >= 2 && !warp_wait(ctl, &ctl.step_done[slot], ((n - 2) >> 1) & 1))) break;
      widen<D>(bytes, images + (2 + slot) * C::kImageBytes, ct);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.k_full[slot]);
        mbar_arrive(&ctl.b_empty[0]);
      }
      if (!warp_wait(ctl, &ctl.b_full[1], n & 1) || (n >= 2 && !warp_wait(ctl, &ctl.step_done[slot ^ 1], ((n - 1) >> 1) & 1))) break;
      widen<D>(bytes + C::kByteTile, images + (4 + slot) * C::kImageBytes, ct);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.v_full[slot]);
        mbar_arrive(&ctl.b_empty[1]);
      }
    }
  } else {
    // ---- softmax -----------------------------------------------------------------------
    const int x = (warp - kSoftmaxWarp0) >> 3;
    const int half = ((warp - kSoftmaxWarp0) >> 2) & 1;       // of the keys; of O's columns
    const int r = tid & (kTile - 1);        // row of the tile = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + static_cast<uint32_t>(x * kKeys + half * kHalf);
    const uint32_t o_at = tmem + lanes + static_cast<uint32_t>(C::kOCol + x * D + half * (D / 2));
    const uint32_t mine_top = smem_u32(&ctl.top[x][half][r]), other_top = smem_u32(&ctl.top[x][half ^ 1][r]);
    const int pair_id = 4 * x + (warp & 3);
    uint32_t n = 0, used = 0, items = 0;
    bool ok = true;
    for (; w.more(); w.next()) {
      const int rows = w.r.rows - w.rt * kItemRows - x * kTile;  // of this tile
      const int steps = w.hi - w.lo;
      if (rows <= 0) {
        n += static_cast<uint32_t>(steps);
        continue;
      }
      const int lim = sees_before<SHARED>(w.r, (w.rt * kItemRows + x * kTile + r) / p.group);   // keys that this row sees
      const int lim_min = __shfl_sync(0xFFFFFFFFu, lim, 0);
      const bool busy = (warp & 3) * 32 < rows;             // the warp has rows at all
      float m = -INFINITY, l = 0.f;
      bool exact = false;
      for (int j = 0; j < steps; ++j, ++n, ++used) {
        // The scales first: they are there long before the scores.  Not at an item's first
        // unit: after units that this tile skipped, the scales' barrier may be any number of
        // phases behind, and a parity wait would pass for an old one.  Behind unit n's scores
        // it is in phase n / kScaleSlots or past it: K of unit n is copied after the scales of
        // unit n - 1 are announced.
        if (j == 0) ok = ok && mbar_wait(&ctl.s_full[x], used & 1);
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(&ctl.c_full[n % kScaleSlots], (n / kScaleSlots) & 1) &&
                                         mbar_wait(&ctl.s_full[x], used & 1));
        if (!ok && lane == 0) atomicOr(&ctl.abort, 1u);
        if (busy) {
          if (ok) tc_fence_after();
          const float4* sc = &ctl.scale[n % kScaleSlots][half * (kGroups / 2)];
          const int key0 = first_key(w.r) + (w.lo + j) * kKeys;
          const int left = lim - key0 - half * kHalf;     // of this half of the unit
          // from its first masked unit on an item is masked
          exact = exact || key0 + kKeys > lim_min;
          bool first = j == 0;
          if (__builtin_expect(!exact, 1)) {
            exact = softmax_unit<D, false>(s_at, o_at, sc, left, first, m, l, mine_top, other_top, pair_id, ok);
            first = false;
          }
          if (__builtin_expect(exact, 0)) softmax_unit<D, true>(s_at, o_at, sc, left, first, m, l, mine_top, other_top, pair_id, ok);
        } else if (j == 0) {
          // Warps without rows meet as well (the others do in softmax_unit): the first
          // product, which writes over all of O, waits for this half's warps only, and the
          // other half's may still be reading the last item's O.
          pair_sync(pair_id);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[x][half]);
      }
      // ---- the item's sums: finished, or to be joined ---------------------------------
      ok = ok && warp_wait(ctl, &ctl.o_done[x], items & 1);
      ++items;
      if (ok) tc_fence_after();
      const int base = w.rt * kItemRows + x * kTile;
      finish_item<D, SHARED>(p, ctl, w.r, SHARED && w.b >= p.groups, w.head, base, w.lo, w.lo == 0 && w.hi == w.units, busy, ok, o_at, m, l);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");   // not done before the few-rows kernel is
}

template <int D, bool SHARED>
exl3_status launch(const AttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                   bool after_step, cudaStream_t stream) {
  constexpr int kSmem = Cfg<D>::kTiles + static_cast<int>(sizeof(Control));
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(Cfg<D>::kTiles >= 12 * EXL3_MAX_REQUESTS + 8, "room for the requests before the tiles");
  static_assert(Cfg<D>::kTiles >= 12 * kListed + 16 + (sizeof(SharedReq) + 8) * kListed + 8, "room for what is kept of them");
  static std::atomic<unsigned long long> allowed{0};
  if (!allow_smem(prompt_kernel<D, SHARED>, kSmem, allowed)) return EXL3_ERR_CUDA;
  const int ctas = prompt_ctas();
  // After the few-rows kernel a CTA begins as soon as an SM is free: the two write
  // nothing in common (one of 100 tokens beside 8 single ones over 300 keys: 38 us, so 31;
  // 2 of 500 beside 11 over up to 8 K: 135, so 132).
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t own = {};
  own.gridDim = dim3(static_cast<unsigned>(ctas));
  own.blockDim = dim3(kThreads);
  own.dynamicSmemBytes = kSmem;
  own.stream = stream;
  own.attrs = attr;
  own.numAttrs = after_step ? 1 : 0;
  if (cudaLaunchKernelEx(&own, prompt_kernel<D, SHARED>, p, kmap, vmap, qmap) != cudaSuccess) return EXL3_ERR_CUDA;
  exl3_status st = launch_status();
  if (st != EXL3_OK) return st;
  if constexpr (SHARED) return EXL3_OK;   // what puts prefixes and own keys together joins too
  // a table whose rows hold no item that is ever split leaves nothing to join
  if (p.most <= static_cast<long long>(kWhole) * kKeys) return EXL3_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), kItemRows / kJoinRows);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join_kernel<D>, p) != cudaSuccess) return EXL3_ERR_CUDA;
  return launch_status();
}

}  // namespace

exl3_status launch_prompt(const AttnParams& p, const exl3_kv_cache& c, bool after_step, cudaStream_t stream) {
  CUtensorMap km, vm;
  exl3_status st;
  if ((st = cache_map(&km, c.k, c, c.page_size)) != EXL3_OK || (st = cache_map(&vm, c.v, c, c.page_size)) != EXL3_OK) return st;
  AttnParams q = p;
  q.negate = p.c < 0.f;
  q.c = fabsf(p.c);
  // a tile of whole tokens can be copied as one box; the other groups (and a
  // negative scale) take the rows one by one (8 K clocks, the box 2 K)
  q.q_box = kTile % p.group == 0 && !q.negate ? 1 : 0;
  CUtensorMap qm = km;
  if (q.q_box != 0 && (st = query_map(&qm, p, c.head_dim, kTile / p.group)) != EXL3_OK) return st;
  if (p.group_start != nullptr)
    return c.head_dim == 64 ? launch<64, true>(q, km, vm, qm, after_step, stream) : launch<128, true>(q, km, vm, qm, after_step, stream);
  return c.head_dim == 64 ? launch<64, false>(q, km, vm, qm, after_step, stream) : launch<128, false>(q, km, vm, qm, after_step, stream);
}

}  // namespace attn
}  // namespace exl3
