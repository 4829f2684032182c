// exl3_rms_norm and exl3_rms_norm_i8: the residual's addition and the
// root-mean-square norm before the projections.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * w
//
// in binary32 from the binary16 inputs; y from the sum before it is rounded to
// binary16, so that the residual's rounding enters the next layer only once.
// For the int8 projections y does not leave the registers: for each of them the
// signs, the 128-point transform and the quantizer of exl3_quantize_act follow
// on the binary32 values.
//
// Every input is read once and every output written once, so bytes bound the
// large calls and the launch the small ones.  A row's values stay in the
// registers of its threads between the sum and the outputs, eight to a vector
// and up to eight vectors a thread; a row of up to 1024 values is a warp's, a
// longer one a block's.
#include "exl3_kv.cuh"

namespace exl3 {
namespace norm {
namespace {

constexpr int kMostOuts = EXL3_MAX_NORM_OUTS;
// Threads of a block: a thread's vectors and their sums want registers.
template <int VECS, bool WARP>
constexpr int most_threads() { return WARP ? 128 : VECS <= 2 ? 1024 : 512; }
static_assert(EXL3_MAX_NORM <= 8 * 8 * most_threads<8, false>(), "a row fits its block's registers");

struct NormParams {
  const __half* x;
  const __half* residual;
  const __half* weight;
  __half* y;
  __half* h;
  const __half* signs[kMostOuts];
  int8_t* q;
  float* qscale;
  long long x_stride, residual_stride;
  float eps;
  int rows, n, outs;
};

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 128-point transform of the values of 16 lanes, 8 each in order.
__device__ __forceinline__ void hadamard128(float (&f)[8], int lane) {
#pragma unroll
  for (int d = 1; d < 8; d <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const float a = f[i], b = f[i + d];
        f[i] = a + b;
        f[i + d] = a - b;
      }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const bool up = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, f[i], d);
      f[i] = up ? o - f[i] : f[i] + o;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] *= 0.08838834764831845f;   // 1 / sqrt(128)
}

// GROUP threads a row, ROWS rows a block, VECS vectors of eight values a thread.
template <int VECS, bool I8, bool WARP>
__global__ void __launch_bounds__(most_threads<VECS, WARP>()) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[32];
  const int lane = threadIdx.x & 31;
  const int group = WARP ? 32 : static_cast<int>(blockDim.x);
  const int at = WARP ? lane : static_cast<int>(threadIdx.x);
  const long long row = WARP ? static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.rows) return;   // a whole warp
  const int vecs = p.n >> 3;
  const __half* x = p.x + row * p.x_stride;
  const __half* r = p.residual != nullptr ? p.residual + row * p.residual_stride : nullptr;
  uint4 raw[VECS], add[VECS], wt[VECS];
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int v = at + k * group;
    raw[k] = v < vecs ? *reinterpret_cast<const uint4*>(x + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
    add[k] = r != nullptr && v < vecs ? *reinterpret_cast<const uint4*>(r + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int v = at + k * group;
    wt[k] = v < vecs ? __ldg(reinterpret_cast<const uint4*>(p.weight + 8 * v)) : make_uint4(0u, 0u, 0u, 0u);
  }
  float f[VECS][8];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    widen8(raw[k], f[k]);
    if (r != nullptr) {
      float g[8];
      widen8(add[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[k][i] += g[i];
      const int v = at + k * group;
      if (v < vecs && p.h != nullptr) *reinterpret_cast<uint4*>(p.h + row * p.n + 8 * v) = narrow8(f[k]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(f[k][i], f[k][i], sum);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if constexpr (!WARP) {
    if (lane == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = lane < static_cast<int>(blockDim.x >> 5) ? sums[lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  }
  const float inv = __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(p.n)) + p.eps);
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    float g[8];
    widen8(wt[k], g);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[k][i] = f[k][i] * inv * g[i];
    const int v = at + k * group;
    if constexpr (!I8) {
      if (v < vecs) *reinterpret_cast<uint4*>(p.y + row * p.n + 8 * v) = narrow8(f[k]);
    }
  }
  if constexpr (I8) {
#pragma unroll 1
    for (int o = 0; o < p.outs; ++o) {
      const __half* s = p.signs[o];
      const size_t to = static_cast<size_t>(o) * p.rows + row;
#pragma unroll
      for (int k = 0; k < VECS; ++k) {
        const int v = at + k * group;   // 16 lanes of a block of 128 are all in the row or all past it
        float z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = f[k][i];
        if (s != nullptr) {
          float g[8];
          widen8(v < vecs ? __ldg(reinterpret_cast<const uint4*>(s + 8 * v)) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] *= g[i];
          hadamard128(z, lane);
        }
        // |z| as bits orders as numbers do, infinity and NaN above them
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(z[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const bool bad = top >= 0x7F800000u;
        const float scale = bad ? __int_as_float(0x7FC00000) : __fdiv_rn(__uint_as_float(top), 127.f);
        uint32_t b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          b[i] = bad || !(scale > 0.f) ? 0u : static_cast<uint32_t>(__float2int_rn(__fdiv_rn(z[i], scale)));
        if (v < vecs) {
          const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
          const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
          *reinterpret_cast<uint2*>(p.q + to * p.n + 8 * v) = make_uint2(lo, hi);
          if ((lane & 15) == 0) p.qscale[to * (p.n >> 7) + (v >> 4)] = scale;
        }
      }
    }
  }
}

template <int VECS, bool I8>
exl3_status launch_block(const NormParams& p, int threads, cudaStream_t cs) {
  norm_kernel<VECS, I8, false><<<static_cast<unsigned>(p.rows), threads, 0, cs>>>(p);
  return launch_status();
}

template <bool I8>
exl3_status launch(const NormParams& p, cudaStream_t cs) {
  const int vecs = p.n / 8;
  if (vecs <= 128) {
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(p.rows) + 3) / 4);
    if (vecs <= 32)
      norm_kernel<1, I8, true><<<blocks, 128, 0, cs>>>(p);
    else if (vecs <= 64)
      norm_kernel<2, I8, true><<<blocks, 128, 0, cs>>>(p);
    else
      norm_kernel<4, I8, true><<<blocks, 128, 0, cs>>>(p);
    return launch_status();
  }
  // One vector a thread while the rows leave SMs idle, else as many as a thread takes.
  const bool few = p.rows <= device_sm_count();
  const int take = vecs > 2048 ? 8 : !few ? 4 : vecs > 1024 ? 2 : 1;
  const int threads = ((vecs + take - 1) / take + 31) & ~31;
  switch (take) {
    case 1: return launch_block<1, I8>(p, threads, cs);
    case 2: return launch_block<2, I8>(p, threads, cs);
    case 4: return launch_block<4, I8>(p, threads, cs);
    default: return launch_block<8, I8>(p, threads, cs);
  }
}

exl3_status check(const exl3_half* x, long long x_stride, const exl3_half* residual, long long residual_stride,
                  const exl3_half* weight, float eps, int rows, int n, int multiple) {
  if (rows < 0) return EXL3_ERR_BATCH;
  if (n < multiple || n % multiple != 0 || n > EXL3_MAX_NORM || !(eps >= 0.f) || eps > 3.4e38f) return EXL3_ERR_SHAPE;
  if (x_stride < n || (x_stride & 7) != 0 || (residual != nullptr && (residual_stride < n || (residual_stride & 7) != 0)))
    return EXL3_ERR_SHAPE;
  if (rows == 0) return EXL3_OK;
  if (x == nullptr || weight == nullptr) return EXL3_ERR_NULL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight)) return EXL3_ERR_ALIGN;
  return EXL3_OK;
}

}  // namespace
}  // namespace norm
}  // namespace exl3

using namespace exl3;

extern "C" exl3_status exl3_rms_norm(const exl3_half* x, long long x_stride, const exl3_half* residual,
                                     long long residual_stride, const exl3_half* weight, float eps, int rows, int n,
                                     exl3_half* y, exl3_half* h, exl3_stream_t stream) {
  const exl3_status st = norm::check(x, x_stride, residual, residual_stride, weight, eps, rows, n, 8);
  if (st != EXL3_OK || rows == 0) return st;
  if (y == nullptr) return EXL3_ERR_NULL;
  if (!aligned16(y) || !aligned16(h)) return EXL3_ERR_ALIGN;
  norm::NormParams p{};
  p.x = reinterpret_cast<const __half*>(x);
  p.residual = reinterpret_cast<const __half*>(residual);
  p.weight = reinterpret_cast<const __half*>(weight);
  p.y = reinterpret_cast<__half*>(y);
  p.h = reinterpret_cast<__half*>(h);
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.eps = eps;
  p.rows = rows;
  p.n = n;
  return norm::launch<false>(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" exl3_status exl3_rms_norm_i8(const exl3_half* x, long long x_stride, const exl3_half* residual,
                                        long long residual_stride, const exl3_half* weight, float eps, int rows, int n,
                                        const exl3_half* const* signs, int outs, int8_t* q, float* qscale,
                                        exl3_half* h, exl3_stream_t stream) {
  if (outs < 1 || outs > EXL3_MAX_NORM_OUTS) return EXL3_ERR_BATCH;
  const exl3_status st = norm::check(x, x_stride, residual, residual_stride, weight, eps, rows, n, 128);
  if (st != EXL3_OK || rows == 0) return st;
  if (signs == nullptr || q == nullptr || qscale == nullptr) return EXL3_ERR_NULL;
  if (!aligned16(q) || !aligned16(h) || !kv::aligned_to(qscale, 4)) return EXL3_ERR_ALIGN;
  norm::NormParams p{};
  for (int o = 0; o < outs; ++o) {
    if (!aligned16(signs[o])) return EXL3_ERR_ALIGN;
    p.signs[o] = reinterpret_cast<const __half*>(signs[o]);
  }
  p.x = reinterpret_cast<const __half*>(x);
  p.residual = reinterpret_cast<const __half*>(residual);
  p.weight = reinterpret_cast<const __half*>(weight);
  p.h = reinterpret_cast<__half*>(h);
  p.q = q;
  p.qscale = qscale;
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.eps = eps;
  p.rows = rows;
  p.n = n;
  p.outs = outs;
  return norm::launch<true>(p, reinterpret_cast<cudaStream_t>(stream));
}
