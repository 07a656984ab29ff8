// Quantisation to 8-bit integers with one scale per row (engram_quantize_i8): s = amax /
// 127 rounded to fp32, or the smallest power of two with amax <= 127 s, and codes x
// (127 / amax) or x / s, to the nearest whole number, ties to the even one.
#include "common.h"

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kSmallest = 8u << 23;      // 2^-119

struct RowScale {
  float scale, inv;
  bool bad;
};

template <bool POW2>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale r;
  r.bad = top >= 0x7F800000u;
  r.scale = r.inv = 0.f;
  if (r.bad) {
    r.scale = __uint_as_float(0x7FC00000u);
  } else if (top >= kSmallest) {
    if (POW2) {
      // amax = m 2^E, 1 <= m < 2: 2^(E - 6) reaches 127 / 64 of 2^E
      const uint32_t field = (top >> 23) - 6 + ((top & 0x7FFFFFu) > 0x7E0000u);
      r.scale = __uint_as_float(field << 23);
      r.inv = __uint_as_float((254u - field) << 23);
    } else {
      const float amax = __uint_as_float(top);
      r.scale = amax / 127.f;
      // only the largest fp32 rounds to a scale whose 127 steps overflow
      if (isinf(127.f * r.scale)) r.scale = __uint_as_float(__float_as_uint(r.scale) - 1);
      r.inv = 127.f / amax;
    }
  }
  return r;
}

// The whole number nearest to the product x inv, which fp32 may have rounded onto or
// off a half: there the product's exact residue decides.
__device__ __forceinline__ float code_of(float x, float inv) {
#pragma clang fp contract(off)      // p - n is of the rounded product
  const float p = x * inv;
  float n = rintf(p);
  const float off = p - n;
  if (fabsf(off) == 0.5f) {
    const float rest = fmaf(x, inv, -p);
    if (rest != 0.f) n = p + copysignf(0.5f, rest);
  }
  return n;
}

template <bool F32>
__device__ __forceinline__ float load1(const void *src, int64_t i) {
  return F32 ? reinterpret_cast<const float *>(src)[i]
             : engram::bf16_to_f32(reinterpret_cast<const uint16_t *>(src)[i]);
}

template <bool F32, bool POW2>
__global__ __launch_bounds__(kThreads) void quantize_i8_kernel(const void *src, int64_t cols,
                                                               int64_t ld, int64_t out_cols,
                                                               int8_t *__restrict__ codes,
                                                               float *__restrict__ scales,
                                                               void *values) {
  __shared__ uint32_t red[kThreads / 64];
  const int64_t row = blockIdx.x;
  uint32_t top = 0;
  for (int64_t c = threadIdx.x; c < cols; c += kThreads)
    top = max(top, __float_as_uint(load1<F32>(src, row * ld + c)) & 0x7FFFFFFFu);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = max(top, red[w]);
  const RowScale r = row_scale<POW2>(top);
  if (threadIdx.x == 0) scales[row] = r.scale;
  for (int64_t c = threadIdx.x; c < out_cols; c += kThreads) {
    float n = 0.f;
    if (c < cols && !r.bad) n = code_of(load1<F32>(src, row * ld + c), r.inv);
    codes[row * out_cols + c] = (int8_t)(int)n;
    if (values != nullptr && c < cols) {
      const float v = n * r.scale;
      if (F32)
        reinterpret_cast<float *>(values)[row * ld + c] = v;
      else
        reinterpret_cast<uint16_t *>(values)[row * ld + c] = (uint16_t)engram::pack_bf16x2(v, v);
    }
  }
}

}  // namespace

hipError_t engram_launch_quantize_i8(bool f32, bool pow2, const void *src, int64_t rows,
                                     int64_t cols, int64_t ld, int64_t out_cols, int8_t *codes,
                                     float *scales, void *values, hipStream_t stream) {
  if (rows <= 0) return hipSuccess;
  const dim3 grid((unsigned)rows);
#define ENGRAM_QUANTIZE(F, P)                                                                   \
  hipLaunchKernelGGL((quantize_i8_kernel<F, P>), grid, dim3(kThreads), 0, stream, src, cols, ld, \
                     out_cols, codes, scales, values)
  if (f32 && pow2) ENGRAM_QUANTIZE(true, true);
  else if (f32) ENGRAM_QUANTIZE(true, false);
  else if (pow2) ENGRAM_QUANTIZE(false, true);
  else ENGRAM_QUANTIZE(false, false);
#undef ENGRAM_QUANTIZE
  return hipGetLastError();
}
