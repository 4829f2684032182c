// exl3_rotary: rotary positions on the queries and keys of a step.
//
// Pair i of a head's first r elements turns by position * f_i.  f_i comes as a
// 64-bit fraction of a turn, so the product modulo 2^64 is the angle without its
// whole turns whatever the position is, in one integer multiplication; what is left,
// in [-1/2, 1/2) of a turn, keeps its 24 bits as binary32.
//
// A block takes some tokens.  Their cosines and sines are computed once, into
// shared memory, and used by all heads; a thread then takes 16 elements of a head at a
// time, 8 pairs (or elements to copy), as two 16-byte vectors.
// Bytes bound the large calls and the launch the small ones.
#include "exl3_kv.cuh"

namespace exl3 {
namespace rotary {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTable = 2048;   // cosines and sines of a block

struct RotaryParams {
  const __half* in[2];    // queries, keys
  __half* out[2];
  long long in_stride[2], out_stride[2];
  const int32_t* position;
  const uint64_t* freqs;
  float factor;
  int heads, q_heads, dim, part, tokens, each;   // each: tokens of a block
};

__device__ __forceinline__ float2 turn(float a, float b, const float2& cs) {
  return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(b, cs.x, a * cs.y));
}

// Two vectors of 8 elements: pair i the elements i of both, or two neighbours of one.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn16(uint4& x, uint4& y, const float2* cs) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
  uint32_t* b = reinterpret_cast<uint32_t*>(&y);
  const float4* c4 = reinterpret_cast<const float4*>(cs);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = c4[i];
    const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
    if constexpr (INTERLEAVED) {
      uint32_t* w = i < 2 ? a + 2 * i : b + 2 * (i - 2);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(w));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(w + 1));
      const float2 u = turn(p.x, p.y, c0), v = turn(q.x, q.y, c1);
      const __half2 r = __floats2half2_rn(u.x, u.y), s = __floats2half2_rn(v.x, v.y);
      w[0] = *reinterpret_cast<const uint32_t*>(&r);
      w[1] = *reinterpret_cast<const uint32_t*>(&s);
    } else {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(a + i));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(b + i));
      const float2 u = turn(p.x, q.x, c0), v = turn(p.y, q.y, c1);
      const __half2 r = __floats2half2_rn(u.x, v.x), s = __floats2half2_rn(u.y, v.y);
      a[i] = *reinterpret_cast<const uint32_t*>(&r);
      b[i] = *reinterpret_cast<const uint32_t*>(&s);
    }
  }
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ __align__(16) float2 table[kMostTable];
  chained_begin();
  const int tid = threadIdx.x;
  const int t0 = static_cast<int>(blockIdx.x) * p.each;
  const int here = min(p.each, p.tokens - t0);
  const int half = p.part >> 1;
  for (int i = tid; i < here * half; i += kThreads) {
    const int t = i / half;
    const uint64_t angle = static_cast<uint64_t>(static_cast<int64_t>(p.position[t0 + t])) * p.freqs[i - t * half];
    float s, c;
    sincospif(__ll2float_rn(static_cast<long long>(angle)) * 0x1p-63f, &s, &c);
    table[i] = make_float2(c * p.factor, s * p.factor);
  }
  __syncthreads();
  const int units = p.dim >> 4;       // of a head, 16 elements each
  const int turned = p.part >> 4;
  const int rows = here * p.heads;    // heads of all tokens
  for (int i = tid; i < rows * units; i += kThreads) {
    const int row = i / units, u = i - row * units;
    const int t = row / p.heads, head = row - t * p.heads;
    const int side = head >= p.q_heads ? 1 : 0;
    const int h = head - (side ? p.q_heads : 0);
    int e0, e1;
    if (u < turned) {
      e0 = INTERLEAVED ? 16 * u : 8 * u;
      e1 = INTERLEAVED ? 16 * u + 8 : 8 * u + half;
    } else {
      e0 = 16 * u;
      e1 = 16 * u + 8;
    }
    const __half* src = p.in[side] + static_cast<size_t>(t0 + t) * p.in_stride[side] + static_cast<size_t>(h) * p.dim;
    __half* dst = p.out[side] + static_cast<size_t>(t0 + t) * p.out_stride[side] + static_cast<size_t>(h) * p.dim;
    uint4 x = *reinterpret_cast<const uint4*>(src + e0), y = *reinterpret_cast<const uint4*>(src + e1);
    if (u < turned && p.position[t0 + t] >= 0) turn16<INTERLEAVED>(x, y, table + t * half + 8 * u);
    *reinterpret_cast<uint4*>(dst + e0) = x;
    *reinterpret_cast<uint4*>(dst + e1) = y;
  }
}

}  // namespace
}  // namespace rotary
}  // namespace exl3

using namespace exl3;

extern "C" exl3_status exl3_rotary(const exl3_half* q, long long q_stride, exl3_half* q_out, long long q_out_stride,
                                   int q_heads, const exl3_half* k, long long k_stride, exl3_half* k_out,
                                   long long k_out_stride, int k_heads, int head_dim, int rotary_dim, int interleaved,
                                   const int32_t* position, const uint64_t* freqs, float factor, int tokens,
                                   exl3_stream_t stream) {
  if (tokens < 0) return EXL3_ERR_BATCH;
  if (head_dim < 16 || head_dim > 512 || head_dim % 16 != 0 || rotary_dim < 16 || rotary_dim > head_dim ||
      rotary_dim % 16 != 0 || q_heads < 1 || q_heads > 65535 || k_heads < 0 || k_heads > 65535 || !(factor - factor == 0.f))
    return EXL3_ERR_SHAPE;
  exl3_status st;
  if ((st = kv::check_stride(q_stride, q_heads, head_dim)) != EXL3_OK ||
      (st = kv::check_stride(q_out_stride, q_heads, head_dim)) != EXL3_OK)
    return st;
  if (k_heads > 0 && ((st = kv::check_stride(k_stride, k_heads, head_dim)) != EXL3_OK ||
                      (st = kv::check_stride(k_out_stride, k_heads, head_dim)) != EXL3_OK))
    return st;
  if (tokens == 0) return EXL3_OK;
  if (q == nullptr || q_out == nullptr || (k_heads > 0 && (k == nullptr || k_out == nullptr)) || position == nullptr ||
      freqs == nullptr)
    return EXL3_ERR_NULL;
  if (!aligned16(q) || !aligned16(q_out) || (k_heads > 0 && (!aligned16(k) || !aligned16(k_out))) ||
      !kv::aligned_to(position, 4) || !kv::aligned_to(freqs, 8))
    return EXL3_ERR_ALIGN;
  // the outputs lie apart, and over an input only as q and k themselves: every element is read before it is written
  kv::Span in[2] = {kv::halves(q, tokens, 1ll * q_heads * head_dim, q_stride), {}};
  kv::Span out[2] = {kv::halves(q_out, tokens, 1ll * q_heads * head_dim, q_out_stride), {}};
  if (k_heads > 0) {
    in[1] = kv::halves(k, tokens, 1ll * k_heads * head_dim, k_stride);
    out[1] = kv::halves(k_out, tokens, 1ll * k_heads * head_dim, k_out_stride);
  }
  if (kv::meet(out[0], out[1])) return EXL3_ERR_SHAPE;
  for (int o = 0; o < 2; ++o)
    for (int i = 0; i < 2; ++i)
      if (!(o == i && in[i].at == out[o].at && (in[i].stride == out[o].stride || tokens == 1)) && kv::meet(out[o], in[i])) return EXL3_ERR_SHAPE;
  rotary::RotaryParams p{};
  p.in[0] = reinterpret_cast<const __half*>(q);
  p.in[1] = reinterpret_cast<const __half*>(k);
  p.out[0] = reinterpret_cast<__half*>(q_out);
  p.out[1] = reinterpret_cast<__half*>(k_out);
  p.in_stride[0] = q_stride;
  p.in_stride[1] = k_stride;
  p.out_stride[0] = q_out_stride;
  p.out_stride[1] = k_out_stride;
  p.position = position;
  p.freqs = freqs;
  p.factor = factor;
  p.heads = q_heads + k_heads;
  p.q_heads = q_heads;
  p.dim = head_dim;
  p.part = rotary_dim;
  p.tokens = tokens;
  // a few units for each thread of a block, if the tokens then still fill the SMs
  const long long units = static_cast<long long>(p.heads) * (head_dim / 16);
  p.each = 1;
  while (p.each * units < 4 * rotary::kThreads && 2 * p.each * (rotary_dim / 2) <= rotary::kMostTable &&
         tokens / (2 * p.each) >= 4 * device_sm_count())
    p.each *= 2;
  const unsigned blocks = static_cast<unsigned>((tokens + (p.each - 1ll)) / p.each);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return interleaved != 0 ? launch_chained(rotary::rotary_kernel<true>, dim3(blocks), rotary::kThreads, 0, cs, p)
                          : launch_chained(rotary::rotary_kernel<false>, dim3(blocks), rotary::kThreads, 0, cs, p);
}
