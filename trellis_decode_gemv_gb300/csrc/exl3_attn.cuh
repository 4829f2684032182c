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
};

// A request as the kernels see it; lengths are cut to what the table and the
// arrays hold.
struct Req {
  int t0, n, rows;  // first token, new tokens, rows (new * group), 0 if another launch's
  int seq;          // cached tokens, the new ones included
};

__device__ __forceinline__ Req load_req(const AttnParams& p, int b) {
  Req r{0, 0, 0, 0};
  if (b < p.requests) {
    const int a = min(max(p.q_start[b], 0), p.tokens);
    const int e = min(max(p.q_start[b + 1], 0), p.tokens);
    r.t0 = a;
    r.n = max(e - a, 0);
    const long long rows = static_cast<long long>(r.n) * p.group;
    r.rows = rows >= p.rows_lo && rows <= p.rows_hi ? static_cast<int>(rows) : 0;
    r.seq = static_cast<int>(min(static_cast<long long>(max(p.seq_len[b], 0)), p.most));
  }
  return r;
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
constexpr size_t prompt_slot_floats(int head_dim) { return static_cast<size_t>(256) * (head_dim + 2); }
exl3_status launch_prompt(const AttnParams& p, const exl3_kv_cache& c, bool after_step, cudaStream_t stream);
exl3_status launch_step(const AttnParams& p, const exl3_kv_cache& c, bool wide, cudaStream_t stream);

}  // namespace attn
}  // namespace exl3
