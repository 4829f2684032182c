// Shared by the attention kernels: parameters, the numbering of the work, the
// PTX that both use, and the join of partial results.
//
// Mathematics.  With k_j = ks_j * K_j and v_j = vs_j * V_j (K, V int8, one scale
// per page and head) and c = scale * log2(e), a row's result is
//   x_j = c ks_j (q . K_j) + log2 vs_j,   max_j x_j - 15.9 <= m <= max_j x_j - 7,   P_j = 2^(x_j - m),
//   out = (sum_j P_j V_j) / l,   l = sum_j P_j / vs_j,   lse = ln 2 * m + ln l.
// The value's scale rides in the exponent, so V enters the product as it is
// stored and P (rounded to binary16 for the tensor cores) keeps its 11 bits
// whatever the pages' scales are, as it would not if it were multiplied by a
// small scale first; the sum l takes it out again, in binary32.  m follows the running
// maximum from 2^7 below it and is only moved when a score passes it by more than
// 2^15.9, so the accumulators are rescaled rarely.  The row's largest P is then between
// 2^7 and 2^15.9: a P keeps its 11 bits down to 2^-21 of it and is cut at 2^-32 of it, where one
// key outweighs the others by that much (with a largest P of 1 many keys next to one of
// 2^25 times their weight added nothing to the numerator and all of theirs to l).  More
// moves than from a largest P of 1: a prompt of 8192 tokens 478 us in place of 470 (481
// with moves at 2^15), steps the same.
//
// Work.  An item is one (request, key/value head, tile of query rows); it has
// as many units (tiles of keys) as its rows see.  The units of all items, in
// order, are cut into equal ranges, one for each CTA, whatever the requests'
// lengths are.  An item inside one range is finished there; one that crosses
// ranges leaves partial results (m, l and the sums, binary32), which the CTA whose
// arrival completes the item (few rows) or a second kernel (many rows) joins in the
// order of the keys, so the result does not depend on the order of the CTAs.
// Everything is computed from the lengths in device memory.
#pragma once

#include "exl3_kv.cuh"
#include "exl3_tc.cuh"

namespace exl3 {
namespace attn {

using tc::bulk_g2s;
using tc::mbar_arrive;
using tc::mbar_arrive_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::smem_u32;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRoom = 15.9f;    // log2 of the largest P: binary16 ends at 2^16
constexpr float kBelow = 7.f;     // m's distance to the maximum when it is set; kRoom - kBelow powers of two to the next move
// log2 that stands for a value scale of 0 and all below 2^-90: V of less than 2^-83 add
// nothing to a binary16 output, but their P have to count in l, within binary32's range
// (the logarithm of 2^-130, say, left 1 / scale infinite).
constexpr float kTinyScale = -90.f;
constexpr int kMaxCtas = 160 * 4; // ranges that the workspace has counters for

// An item of the many-rows kernel that begins in a range and ends in a later one.
struct SplitItem {
  int t0, n, seq, rows;   // its request
  int base, head;         // its first row, its key/value head
  int last;               // the range in which it ends, -1: no such item
  int unused;
};

// The same for the parts of a row in calls with prefixes, in either kernel.
struct SharedSplit {
  long long first;        // number of the item's first row: token * group + head of the group
  int last, unused;
};

struct AttnParams {
  const __half* q;
  const int32_t* q_start;
  const int32_t* seq_len;
  const int32_t* table;
  const float* k_scale;
  const float* v_scale;
  __half* out;
  float* lse;
  long long q_stride, out_stride;
  float c;                 // scale * log2(e)
  int q_box;               // prompt kernel: Q comes by tensor copies of whole tokens
  int negate;              // prompt kernel: c is the absolute value, Q changes its sign
  int stall;               // test hook: the producers post the first unit of a range only
  int followed;            // few rows: the other kernel may begin where this one's blocks end
  int q_heads, kv_heads, group, requests, tokens;
  int table_stride, pages, page_shift;
  long long most;          // keys that a table row holds
  int rows_lo, rows_hi;    // requests with rows in [rows_lo, rows_hi] are this launch's
  uint32_t* status;
  // few rows, zero between calls: [kMaxCtas] arrivals at the item that begins in CTA c and ends later, then
  // [2 * kMaxCtas] at the part of an item that begins with slot 2c, 2c + 1 of `partial`
  uint32_t* arrived;
  SplitItem* split;        // [kMaxPromptCtas]: many rows, that item
  float* partial;          // [2 * kMaxCtas] slots: 2c the item that began before CTA c's range, 2c + 1 the one that ends after it
  // calls with prefixes only
  const int32_t* group_start;
  const int32_t* prefix_len;
  int groups, align;       // prefixes count up to a multiple of `align` keys, whole units of the kernel that goes on
  int prefix_hi;           // the few-rows kernel takes requests of up to rows_hi rows and prefixes of up to prefix_hi
  int many;                // this launch is the other kernel
  int both, sms;           // both kernels run, side by side on the SMs
  int step_tile, step_shift;  // rows of the few-rows kernel's tiles, their logarithm
  SharedSplit* shared_split;  // [kMaxCtas] ranges of the few-rows kernel, then [kMaxPromptCtas] of the other
  uint32_t* flag;          // [tokens][q_heads] what mark_row says of a row's own keys
  uint32_t* where;         // [tokens][q_heads] and of its prefix
  float* part;             // sums of every row over the prefix, then over its own keys: [2][tokens][q_heads][head_dim]
  float2* part_ml;         // their m and l: [2][tokens][q_heads]
};

// A request as the kernels see it; lengths are cut to what the table and the
// arrays hold.  In a call with prefixes (SHARED) `groups` of these come before the
// requests: the prefix of group g with the rows of all its requests.
struct Req {
  int t0, n, rows;  // first token, new tokens, rows (new * group), 0 if another launch's
  int seq;          // cached tokens, the new ones included; a prefix's length
};
struct SharedReq : Req {
  int late;         // token i of it sees the keys before min(seq, late + i + 1)
  int k0;           // its first key: those before are its group's prefix
  int row;          // of the block table
  int other;        // rows, if the other launch's
};
template <bool SHARED>
struct ReqType {
  using type = Req;
};
template <>
struct ReqType<true> {
  using type = SharedReq;
};
template <bool SHARED>
using ReqOf = typename ReqType<SHARED>::type;

__device__ __forceinline__ int late_of(const Req& r) { return r.seq - r.n; }
__device__ __forceinline__ int late_of(const SharedReq& r) { return r.late; }
__device__ __forceinline__ int first_key(const Req&) { return 0; }
__device__ __forceinline__ int first_key(const SharedReq& r) { return r.k0; }
__device__ __forceinline__ int table_row(const Req&, int b) { return b; }
__device__ __forceinline__ int table_row(const SharedReq& r, int) { return r.row; }

template <bool SHARED>
__device__ __forceinline__ int req_count(const AttnParams& p) { return SHARED ? p.groups + p.requests : p.requests; }

// The lists that a call's work is found from: the caller's, or a copy in shared memory.  (What
// is shared takes a chain of a dozen reads; from memory it took 4.5 us of either kernel.)
struct Lists {
  const int32_t *q_start, *seq_len, *group_start, *prefix_len;
  __device__ __forceinline__ explicit Lists(const AttnParams& p)
      : q_start(p.q_start), seq_len(p.seq_len), group_start(p.group_start), prefix_len(p.prefix_len) {}
  // Room for 2 * req_count + 2 numbers; the block's threads meet before it is read.
  __device__ __forceinline__ void copy_to(const AttnParams& p, int32_t* room, int threads) {
    const int n = p.requests, g = p.groups;
    int32_t *q = room, *s = q + n + 1, *a = s + n, *l = a + g + 1;
    for (int i = threadIdx.x; i <= n; i += threads) {
      q[i] = q_start[i];
      if (i < n) s[i] = seq_len[i];
    }
    for (int i = threadIdx.x; i <= g; i += threads) {
      a[i] = group_start[i];
      if (i < g) l[i] = prefix_len[i];
    }
    q_start = q;
    seq_len = s;
    group_start = a;
    prefix_len = l;
  }
};

__device__ __forceinline__ int first_token(const AttnParams& p, const Lists& l, int b) { return min(max(l.q_start[b], 0), p.tokens); }
__device__ __forceinline__ int cached_tokens(const AttnParams& p, const Lists& l, int b) {
  return static_cast<int>(min(static_cast<long long>(max(l.seq_len[b], 0)), p.most));
}
// A request's rows, which are this launch's or the other's.
template <bool SHARED>
__device__ __forceinline__ void set_rows(const AttnParams& p, ReqOf<SHARED>& r, int most_few) {
  const long long all = static_cast<long long>(r.n) * p.group;
  if constexpr (SHARED) {
    const int rows = static_cast<int>(min(all, 0x7FFFFFFFLL));
    const bool mine = (rows > most_few) == (p.many != 0);
    r.rows = mine ? rows : 0;
    r.other = mine ? 0 : rows;
  } else {
    r.rows = all >= p.rows_lo && all <= p.rows_hi ? static_cast<int>(all) : 0;
  }
}

struct Group {
  int a, e, prefix;  // requests a .. e - 1; the shared keys, 0 where one request alone would share them
};
__device__ __forceinline__ Group load_group(const AttnParams& p, const Lists& l, int g) {
  Group x;
  x.a = min(max(l.group_start[g], 0), p.requests);
  x.e = min(max(l.group_start[g + 1], x.a), p.requests);
  const long long len = min(static_cast<long long>(max(l.prefix_len[g], 0)), p.most);
  x.prefix = x.e - x.a > 1 ? static_cast<int>(len) & ~(p.align - 1) : 0;
  return x;
}

// A prefix: its pages are those of the first request that holds all of it.
__device__ __forceinline__ SharedReq load_prefix(const AttnParams& p, const Lists& l, int g) {
  SharedReq r{};
  const Group x = load_group(p, l, g);
  if (x.prefix == 0) return r;
  for (int b = x.a; b < x.e; ++b) {
    const int n = max(first_token(p, l, b + 1) - first_token(p, l, b), 0);
    if (cached_tokens(p, l, b) - n < x.prefix) continue;
    r.t0 = first_token(p, l, x.a);
    r.n = max(first_token(p, l, x.e) - r.t0, 0);
    r.seq = r.late = x.prefix;
    r.row = b;
    set_rows<true>(p, r, p.prefix_hi);
    break;
  }
  return r;
}

template <bool SHARED>
__device__ __forceinline__ ReqOf<SHARED> make_req(const AttnParams& p, const Lists& l, int b) {
  ReqOf<SHARED> r{};
  if constexpr (SHARED) {
    if (b < p.groups) return load_prefix(p, l, b);
    b -= p.groups;
  }
  if (b < p.requests) {
    const int a = first_token(p, l, b);
    const int e = first_token(p, l, b + 1);
    r.t0 = a;
    r.n = max(e - a, 0);
    set_rows<SHARED>(p, r, p.rows_hi);
    r.seq = cached_tokens(p, l, b);
    if constexpr (SHARED) {
      r.late = r.seq - r.n;
      r.row = b;
      int g = -1, hi = p.groups;   // the last group that begins at b or before
      while (hi - g > 1) {
        const int mid = (g + hi) >> 1;
        if (l.group_start[mid] <= b) g = mid; else hi = mid;
      }
      if (g >= 0) {
        const Group x = load_group(p, l, g);
        if (b < x.e && r.late >= x.prefix) r.k0 = x.prefix;
      }
    }
  }
  return r;
}

static __device__ __noinline__ SharedReq load_shared(const AttnParams& p, int b) { return make_req<true>(p, Lists(p), b); }

// From a copy of the lists where there may be one.  (Their pointers want registers that a
// call without prefixes does not have to spare.)
template <bool SHARED>
__device__ __forceinline__ ReqOf<SHARED> load_from(const AttnParams& p, const Lists& l, int b) {
  if constexpr (SHARED)
    return make_req<true>(p, l, b);
  else
    return make_req<false>(p, Lists(p), b);
}
// Where it is seldom needed.
template <bool SHARED>
__device__ __forceinline__ ReqOf<SHARED> load_req(const AttnParams& p, int b) {
  if constexpr (SHARED)
    return load_shared(p, b);
  else
    return make_req<false>(p, Lists(p), b);
}

// Up to 32 groups and requests: lane b's, from one round of reads and exchanges.
__device__ __forceinline__ SharedReq load_lanes(const AttnParams& p) {
  const int lane = threadIdx.x & 31;
  const int b = lane - p.groups;   // its request
  const bool group = b < 0, own = b >= 0 && b < p.requests;
  const int32_t* two = group ? p.group_start + lane : p.q_start + (own ? b : 0);
  const int first = two[0], second = two[1];
  const int len = group ? p.prefix_len[lane] : own ? p.seq_len[b] : 0;
  const int a = min(max(first, 0), group ? p.requests : p.tokens);
  const int e = min(max(second, 0), group ? p.requests : p.tokens);
  const int cut = static_cast<int>(min(static_cast<long long>(max(len, 0)), p.most));
  SharedReq r{};
  const int prefix = group && e - a > 1 ? cut & ~(p.align - 1) : 0;
  if (own) {
    r.t0 = a;
    r.n = max(e - a, 0);
    r.seq = cut;
    r.late = r.seq - r.n;
    r.row = b;
  }
  for (int g = 0; g < p.groups; ++g) {
    const int shared = __shfl_sync(0xFFFFFFFFu, prefix, g);
    if (shared == 0) continue;
    const int from = __shfl_sync(0xFFFFFFFFu, a, g), to = __shfl_sync(0xFFFFFFFFu, e, g);
    const bool holds = own && b >= from && b < to && r.late >= shared;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, holds);
    if (holds) r.k0 = shared;
    const int t0 = __shfl_sync(0xFFFFFFFFu, a, p.groups + from), t1 = __shfl_sync(0xFFFFFFFFu, e, p.groups + to - 1);
    if (lane == g && who != 0u) {
      r.t0 = t0;
      r.n = max(t1 - t0, 0);
      r.seq = r.late = shared;
      r.row = __ffs(static_cast<int>(who)) - 1 - p.groups;
    }
  }
  set_rows<true>(p, r, group ? p.prefix_hi : p.rows_hi);
  return r;
}

// Where a row's sums lie, for the kernel that puts them together: 0, in p.part as a whole;
// 1 + c, in parts that begin with the slots of range c of this launch (the many-rows kernel's
// ranges are numbered behind the other's).  For its own keys besides: whether
// it has a prefix, whether it sees a key at all.
constexpr uint32_t kHasPrefix = 1, kSees = 2;
__device__ __forceinline__ void mark_row(const AttnParams& p, const SharedReq& r, bool own, int tok, size_t at, uint32_t code) {
  if (own)
    p.flag[at] = code << 2 | (r.k0 > 0 ? kHasPrefix : 0u) | (r.late + tok + 1 > 0 ? kSees : 0u);
  else
    p.where[at] = code;
}

// The first key that token `tok` of a request does not see.
template <bool SHARED>
__device__ __forceinline__ int sees_before(const ReqOf<SHARED>& r, int tok) {
  return SHARED ? min(r.seq, late_of(r) + tok + 1) : late_of(r) + tok + 1;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// In place of a row's sum l where a wait ran out before all of its keys were read: it
// stays through the joins and makes the row's output NaN.
__device__ __forceinline__ float unfinished() { return __int_as_float(0x7FC00000); }

// The row's result from its sums: `sees` whether it sees a key at all.
__device__ __forceinline__ float inverse_sum(float l, bool sees) { return sees ? __fdividef(1.f, l) : 0.f; }

// What a score x has to pass before m moves.  Rounded down, so that x - m (exact for an x of
// m's size) is at most kRoom for an x that does not pass, however large both are: rounded to
// nearest, P left binary16's range at scores from 2^24 or so on.
__device__ __forceinline__ float room_above(float m) { return __fadd_rd(m, kRoom); }

struct PageScale {
  float c;  // c ks
  float lv; // log2 vs
  float iv; // 1 / 2^lv
};

__device__ __forceinline__ PageScale page_scale(const AttnParams& p, float ks, float vs) {
  PageScale s;
  s.c = ks * p.c;
  s.lv = vs >= 0.f && vs <= 0x1p-90f ? kTinyScale : log2f(vs);   // NaN stays NaN
  // of the rounded logarithm, so that l and the sums agree; finite, so that it spoils no row whose P is 0
  s.iv = vs != vs ? 1.f : exp2f(-s.lv);
  return s;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tensor_g2s_at(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Tensor copy of a box of tokens of one page and head: coordinates (0, token,
// page * kv_heads + head).
__device__ __forceinline__ void tensor_g2s(void* dst, const CUtensorMap* map, int token, int block, uint64_t* bar) {
  tensor_g2s_at(dst, map, 0, token, block, bar);
}

// Exact binary16 of the int8 in bytes 0, 1 (resp. 2, 3) of x, whose top bits are
// flipped: 0x64uu is the binary16 1024 + u, and u - 128 is the value.
__device__ __forceinline__ uint32_t half2_sub1152(uint32_t v) {
  const uint32_t k = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t cvt_lo(uint32_t flipped) { return half2_sub1152(__byte_perm(flipped, 0x64646464u, 0x4140)); }
__device__ __forceinline__ uint32_t cvt_hi(uint32_t flipped) { return half2_sub1152(__byte_perm(flipped, 0x64646464u, 0x4342)); }

// CTA `c` of `ctas` takes the units [c * units / ctas, (c + 1) * units / ctas).  (Of
// 64-bit divisions, each a few hundred clocks, a short call notices four.)
constexpr long long kFewUnits = 1LL << 22;   // times kMaxCtas: 32 bits
__device__ __forceinline__ long long range_begin(long long units, int c, int ctas) {
  if (units < kFewUnits) return static_cast<uint32_t>(units) * static_cast<uint32_t>(c) / static_cast<uint32_t>(ctas);
  return static_cast<long long>(static_cast<unsigned long long>(units) * c / ctas);
}
__device__ __forceinline__ int range_of(long long units, long long u, int ctas) {
  if (units < kFewUnits)
    return static_cast<int>((static_cast<uint32_t>(u + 1) * static_cast<uint32_t>(ctas) - 1u) / static_cast<uint32_t>(units));
  return static_cast<int>((static_cast<unsigned long long>(u + 1) * ctas - 1) / units);
}

// The keys or values as [pages * kv_heads][page_size][head_dim] bytes, boxes of
// `rows` tokens, 16-byte pieces swizzled.
exl3_status cache_map(CUtensorMap* map, const int8_t* base, const exl3_kv_cache& c, int rows);

// Q as [tokens][q_heads][head_dim], boxes of `tokens` tokens x a group's heads x 64
// elements in the 128-byte swizzle.
exl3_status query_map(CUtensorMap* map, const AttnParams& p, int head_dim, int tokens);

// The status word, the arrival counters and the split items come first in the workspace.
constexpr int kMaxPromptCtas = 160;
constexpr int kCounters = 3 * kMaxCtas;
constexpr size_t head_bytes() { return 256 + sizeof(uint32_t) * kCounters + sizeof(SplitItem) * kMaxPromptCtas; }

// Up to kStepRows query rows per key/value head, in tiles of at most kStepTile that
// each read the cache (the later ones from L2).  Against the other kernel, whose
// tiles of 128 rows are mostly empty then: 32 rows 34 us to 52 (16 requests of up to
// 4000 keys) and 35 to 44 (one of 32000), 48 rows 46 to 47, 45 to 44 and 16 to 25 (4 of
// 1000), 64 rows 57 to 48, 54 to 44 and 16 to 25.
constexpr int kStepRows = 48;
constexpr int kStepTile = 16;
constexpr size_t step_slot_floats(int head_dim) { return static_cast<size_t>(kStepTile) * (head_dim + 2); }

// More: tiles of 256 rows.
// A slot of partial results: for either MMA tile four columns of all 128 rows after one
// another, then the rows' m, then their l.
constexpr size_t prompt_slot_floats(int head_dim) { return static_cast<size_t>(256) * (head_dim + 2); }
inline int prompt_ctas() {
  const int sms = device_sm_count();
  return sms < kMaxPromptCtas ? sms : kMaxPromptCtas;
}
// Keys of a unit of the few-rows kernel (`step`) and of the other; what an item costs there
// besides its units, in units.
constexpr int step_unit(int head_dim) { return 4096 / head_dim; }
constexpr int kPromptUnit = 128;
constexpr int kStepItemCost = 4;
constexpr int kPromptItemCost = 3;

// A call with prefixes that takes both kernels lets them run side by side: the many-rows
// kernel is bound by its tensor cores and the chain around them, the other by memory and
// its own latencies, and both begin and end with some microseconds of latency.  The SMs
// are divided by the time that each kernel's work takes of an SM: a unit of the many-rows
// kernel 1.97 us, one of the other 0.16 us with three blocks an SM and 0.21 us with two. (Of
// ratios from 8 to 20 13 and 10 were best over nine calls: 64 requests behind 32000 tokens 71, 68, 67
// and 77 us with 10, 12, 14 and 18; 40 with drafted tokens 68, 66 and 72 with 8, 10 and 12.)
// What a request adds to either (x: many-rows units, y: the other's, and the many-rows kernel's
// row tiles), for a key/value head; roughly, for the sums only divide the SMs.
struct Costs {
  float x, y, tiles;
  __device__ __forceinline__ void add(const Costs& c) {
    x += c.x;
    y += c.y;
    tiles += c.tiles;
  }
  __device__ __forceinline__ void add_lanes() {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      add(Costs{__shfl_xor_sync(0xFFFFFFFFu, x, d), __shfl_xor_sync(0xFFFFFFFFu, y, d), __shfl_xor_sync(0xFFFFFFFFu, tiles, d)});
  }
};
template <int D>
__device__ __forceinline__ Costs costs_of(const AttnParams& p, const SharedReq& r) {
  const int keys = r.seq - r.k0;
  const int few = p.many ? r.other : r.rows, many = p.many ? r.rows : r.other;
  Costs c;
  c.tiles = static_cast<float>((static_cast<uint32_t>(many) + 255u) >> 8);
  c.x = c.tiles * static_cast<float>((keys >> 7) + 1 + kPromptItemCost);
  c.y = static_cast<float>((static_cast<uint32_t>(few) + p.step_tile - 1u) >> p.step_shift) * static_cast<float>(keys / step_unit(D) + 1 + (p.step_shift > 3 ? 2 : 1) * kStepItemCost);
  return c;
}
// SMs of the many-rows kernel.  A few items, which are split anyway, are split evenly, so that no
// range ends one item and begins another.
__device__ __forceinline__ int many_sms(const AttnParams& p, const Costs& c) {
  const float x = c.x * (p.step_shift > 3 ? 10.f : 13.f), items = c.tiles * static_cast<float>(p.kv_heads);
  if (x == 0.f) return 0;
  float n = static_cast<float>(p.sms) * __fdividef(x, x + c.y);
  if (4.f * items <= n) {
    n = rintf(__fdividef(n, items)) * items;
    if (n > static_cast<float>(p.sms)) n -= items;
  }
  return c.y == 0.f ? min(__float2int_rn(n), p.sms) : min(max(__float2int_rn(n), 1), p.sms - 1);
}

exl3_status launch_prompt(const AttnParams& p, const exl3_kv_cache& c, bool after_step, cudaStream_t stream);
exl3_status launch_step(const AttnParams& p, const exl3_kv_cache& c, bool wide, cudaStream_t stream);

}  // namespace attn
}  // namespace exl3
