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

// sqrt(128) times the 128-point transform of the values of 16 lanes, 8 each in order, two to a
// register pair.  Instructions bound a large call with rotations, so: two values to an
// addition, and shuffles whose sums are one fused operation.  With the quantizer's one quotient
// for a block's values, 2000 rows of 4096 for three projections take 27 us; single additions and a
// division for each value took 43, and no less with half of the registers exchanged in place of
// all shuffled, whose selections cost what it saves.
__device__ __forceinline__ void hadamard128(uint64_t (&f)[4], int lane) {
  const uint64_t minus = pair(-1.f, -1.f);
#pragma unroll
  for (int d = 1; d < 4; d <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((i & d) == 0) {
        const uint64_t a = f[i], b = f[i + d];
        f[i] = add2(a, b);
        f[i + d] = fma2(b, minus, a);
      }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpair(f[i], a, b);
    f[i] = pair(a + b, a - b);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const float sign = (lane & d) != 0 ? -1.f : 1.f;
    const uint64_t signs = pair(sign, sign);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpair(f[i], a, b);
      a = __shfl_xor_sync(0xFFFFFFFFu, a, d);
      b = __shfl_xor_sync(0xFFFFFFFFu, b, d);
      f[i] = fma2(f[i], signs, pair(a, b));
    }
  }
}

// The largest |value| of three, NaN if there is one.
__device__ __forceinline__ float most3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// GROUP threads a row, ROWS rows a block, VECS vectors of eight values a thread.
template <int VECS, bool I8, bool WARP>
__global__ void __launch_bounds__(most_threads<VECS, WARP>()) norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[32];
  chained_begin();
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
      if (v < vecs && p.h != nullptr && blockIdx.y == 0) *reinterpret_cast<uint4*>(p.h + row * p.n + 8 * v) = narrow8(f[k]);
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
    for (int o = blockIdx.y; o < p.outs; o += gridDim.y) {
      const __half* s = p.signs[o];
      const size_t to = static_cast<size_t>(o) * p.rows + row;
#pragma unroll
      for (int k = 0; k < VECS; ++k) {
        const int v = at + k * group;   // 16 lanes of a block of 128 are all in the row or all past it
        uint64_t z[4];
        float unit = 1.f / 127.f;   // of the scale, for a largest value of 1
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = pair(f[k][2 * i], f[k][2 * i + 1]);
        if (s != nullptr) {
          float g[8];
          widen8(v < vecs ? __ldg(reinterpret_cast<const uint4*>(s + 8 * v)) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = mul2(z[i], pair(g[2 * i], g[2 * i + 1]));
          hadamard128(z, lane);
          unit = 0.08838834764831845f / 127.f;   // 1 / sqrt(128)
        }
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpair(z[i], x[2 * i], x[2 * i + 1]);
        // |z| as bits orders as numbers do, infinity and NaN above them
        uint32_t top = __float_as_uint(most3(most3(x[0], x[1], x[2]), most3(x[3], x[4], x[5]), most3(x[6], x[7], 0.f)));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const bool bad = top >= 0x7F800000u;
        const float most = __uint_as_float(top);
        // (anything but 0 is far above 2^-120: the product of two binary16 numbers and a root)
        const float inv = bad || !(most > 0x1p-120f) ? 0.f : __fdiv_rn(127.f, most);
        const uint64_t by = pair(inv, inv), magic = pair(12582912.f, 12582912.f);   // 1.5 * 2^23: a sum's last bits are the integer
        uint32_t q[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t n = fma2(z[i], by, magic);
          q[2 * i] = static_cast<uint32_t>(n);
          q[2 * i + 1] = static_cast<uint32_t>(n >> 32);
        }
        if (v < vecs) {
          *reinterpret_cast<uint2*>(p.q + to * p.n + 8 * v) =
              bad ? make_uint2(0u, 0u) : make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
          if ((lane & 15) == 0) p.qscale[to * (p.n >> 7) + (v >> 4)] = bad ? __int_as_float(0x7FC00000) : most * unit;
        }
      }
    }
  }
}

template <int VECS, bool I8>
exl3_status launch_block(const NormParams& p, int threads, cudaStream_t cs) {
  // few rows: the outputs side by side, the norm computed for each of them (not where one of
  // them writes h over what the others read)
  const bool apart = p.h == nullptr || (p.h != p.x && p.h != p.residual);
  const unsigned outs = I8 && apart && static_cast<long long>(p.rows) * p.outs <= 2 * device_sm_count() ? p.outs : 1;
  return launch_chained(norm_kernel<VECS, I8, false>, dim3(static_cast<unsigned>(p.rows), outs), threads, 0, cs, p);
}

template <bool I8>
exl3_status launch(const NormParams& p, cudaStream_t cs) {
  const int vecs = p.n / 8;
  if (vecs <= 128) {
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(p.rows) + 3) / 4);
    if (vecs <= 32) return launch_chained(norm_kernel<1, I8, true>, dim3(blocks), 128, 0, cs, p);
    if (vecs <= 64) return launch_chained(norm_kernel<2, I8, true>, dim3(blocks), 128, 0, cs, p);
    return launch_chained(norm_kernel<4, I8, true>, dim3(blocks), 128, 0, cs, p);
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

// Whether what is written of `to` (rows of n) meets an input other than as that input itself.
bool over_inputs(const kv::Span& to, const NormParams& p) {
  const struct {
    const __half* at;
    long long stride;
  } in[2] = {{p.x, p.x_stride}, {p.residual, p.residual_stride}};
  for (const auto& i : in)
    if (!(i.at == to.at && (i.stride == p.n || p.rows == 1)) && kv::meet(to, kv::halves(i.at, p.rows, p.n, i.stride))) return true;
  return kv::meet(to, kv::halves(p.weight, 1, p.n, p.n));
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
  // y and h lie apart, and over an input only as that input itself: every row is read before it is written
  const kv::Span of_y = kv::bytes(y, 2ll * rows * n), of_h = kv::bytes(residual != nullptr ? h : nullptr, 2ll * rows * n);
  if (kv::meet(of_y, of_h) || norm::over_inputs(of_y, p) || norm::over_inputs(of_h, p)) return EXL3_ERR_SHAPE;
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
  const long long values = 1ll * rows * n;
  const kv::Span of_h = kv::bytes(residual != nullptr ? h : nullptr, 2 * values), of_q = kv::bytes(q, outs * values),
                 of_scale = kv::bytes(qscale, outs * (values / 32));
  if (kv::meet(of_q, of_scale) || norm::over_inputs(of_h, p)) return EXL3_ERR_SHAPE;
  for (const kv::Span& to : {of_q, of_scale}) {
    if (kv::meet(to, of_h) || kv::meet(to, kv::halves(x, rows, n, x_stride)) || kv::meet(to, kv::halves(residual, rows, n, residual_stride)) ||
        kv::meet(to, kv::halves(weight, 1, n, n)))
      return EXL3_ERR_SHAPE;
  }
  return norm::launch<true>(p, reinterpret_cast<cudaStream_t>(stream));
}
