// Quantisation to 4-bit block floating point: per 32 consecutive values one E8M0
// scale 2^(floor(log2 max|x|) - 2) and 32 E2M1 codes {0, .5, 1, 1.5, 2, 3, 4, 6}
// with a sign, rounded to nearest (ties to even) and saturating at 6.
//
// floor(log2 max|x|) is the exponent field of the largest magnitude, so the
// maximum is taken on the values' bits (as integers, where infinities and NaN
// lie above every finite value), and the scale's code is that field minus 2, at
// least 0 (2^-127: zeros and subnormals). v_cvt_scalef32_pk_fp4 divides by the
// scale and rounds; it matched the formula bit for bit on 1e6 values, ties
// included, over the scales 2^-127 .. 2^126. A block that holds an infinity or a
// NaN has no scale: it is marked with the E8M0 NaN (0xFF) and zero codes.
//
// One pass, bound by HBM: a thread owns 8 values (16 or 32 bytes in, 4 bytes of
// codes out), four neighbouring threads a block, which exchange their maxima
// within the quad; 64 threads read 1 or 2 KB in a row. One group a thread: two in
// flight took 254 us for 237 at 25600 x 6144 fp32 with values (1.34 GB, 5.7 TB/s), and
// 8.4 for 5.9 at 4093 x 1001 bf16. Codes and scales alone take 122 us (0.71 GB, 5.9
// TB/s), from bf16 70. A stride that is not a multiple of 8 moves value by value: 25600 x
// 6143 fp32 takes 266 us, 605 with values.
#include "common.h"
#include "fast_div.h"

namespace {

constexpr int kThreads = 256;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void *src, int64_t row_off, int64_t col, int64_t cols,
                                      uint32_t (&bits)[8]) {
  if (VEC && col + 8 <= cols) {
    if (F32) {
      const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(src) + row_off + col);
      const uint4 a = p[0], b = p[1];
      bits[0] = a.x; bits[1] = a.y; bits[2] = a.z; bits[3] = a.w;
      bits[4] = b.x; bits[5] = b.y; bits[6] = b.z; bits[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(src) + row_off + col);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bits[2 * e] = w[e] << 16;
        bits[2 * e + 1] = w[e] & 0xFFFF0000u;
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bits[e] = 0u;
    if (col + e < cols)
      bits[e] = F32 ? reinterpret_cast<const uint32_t *>(src)[row_off + col + e]
                    : (uint32_t)reinterpret_cast<const uint16_t *>(src)[row_off + col + e] << 16;
  }
}

// The larger of this lane's value and another lane's of the quad.
template <int PERM>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, PERM, 0xF, 0xF, true));
}
constexpr int kSwapPairs = 0xB1;      // lanes 1, 0, 3, 2
constexpr int kSwapHalves = 0x4E;     // lanes 2, 3, 0, 1

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void *dst, int64_t row_off, int64_t col, int64_t cols,
                                       const float (&f)[8]) {
  if (VEC && col + 8 <= cols) {
    engram::Chunk8<F32>::store(dst, (row_off + col) / 8, f);
    // keeps the compiler from merging these with the single stores below (267 us
    // for 237 at 25600 x 6144)
    asm volatile("" ::: "memory");
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (col + e < cols) {
      if (F32)
        reinterpret_cast<float *>(dst)[row_off + col + e] = f[e];
      else
        reinterpret_cast<uint16_t *>(dst)[row_off + col + e] =
            (uint16_t)engram::pack_bf16x2(f[e], f[e]);
    }
  }
}

// src and values may be the same buffer (each value is read and written by one
// thread), so neither is marked restrict.
template <bool F32, bool VEC>
__global__ __launch_bounds__(kThreads) void quantize_mx4_kernel(
    const void *src, int64_t cols, int64_t ld, uint32_t *__restrict__ codes,
    uint8_t *__restrict__ scales, void *values, EngramFastDiv groups, int64_t total) {
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < total;
       g += (int64_t)gridDim.x * kThreads) {
    // A quad of threads is one block of 32: total is a multiple of 4, so the four are
    // in or out of range together.
    const int64_t row = groups.div(g);
    const int64_t col = (g - row * groups.d) * 8;
    uint32_t bits[8], top = 0;
    load8<F32, VEC>(src, row * ld, col, cols, bits);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, bits[e] & 0x7FFFFFFFu);
    top = quad_max<kSwapHalves>(quad_max<kSwapPairs>(top));
    const uint32_t field = top >> 23;
    const bool finite = field < 255u;
    const uint32_t s = finite ? (field > 2u ? field - 2u : 0u) : 255u;
    // 2^(s - 127); 2^-127 is a subnormal fp32
    const float scale = __uint_as_float(s > 0u ? s << 23 : 0x00400000u);
    uint32_t word = 0;
    if (finite) {
#define ENGRAM_CVT_FP4(i)                                                                       \
  word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, __uint_as_float(bits[2 * (i)]),         \
                                                  __uint_as_float(bits[2 * (i) + 1]), scale, i);
      ENGRAM_CVT_FP4(0)
      ENGRAM_CVT_FP4(1)
      ENGRAM_CVT_FP4(2)
      ENGRAM_CVT_FP4(3)
#undef ENGRAM_CVT_FP4
    }
    codes[g] = word;
    if ((g & 3) == 0) scales[g >> 2] = (uint8_t)s;
    if (values != nullptr) {
      // the codes times the scale, exact; NaN in a marked block
      const float by = finite ? scale : __uint_as_float(0x7FC00000u);
      float f[8];
#define ENGRAM_FP4_VALUES(i)                                                                    \
  {                                                                                             \
    const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.f, i);                      \
    f[2 * (i)] = v[0] * by;                                                                     \
    f[2 * (i) + 1] = v[1] * by;                                                                 \
  }
      ENGRAM_FP4_VALUES(0)
      ENGRAM_FP4_VALUES(1)
      ENGRAM_FP4_VALUES(2)
      ENGRAM_FP4_VALUES(3)
#undef ENGRAM_FP4_VALUES
      store8<F32, VEC>(values, row * ld, col, cols, f);
    }
  }
}

}  // namespace

hipError_t engram_launch_quantize_mx4(bool f32, const void *src, int64_t rows, int64_t cols,
                                      int64_t ld, int64_t out_cols, uint8_t *codes,
                                      uint8_t *scales, void *values, hipStream_t stream) {
  if (rows <= 0 || out_cols <= 0) return hipSuccess;
  const EngramFastDiv groups(out_cols / 8);
  const int64_t total = rows * groups.d;
  const int64_t tiles = (total + kThreads - 1) / kThreads;
  const int64_t limit = (int64_t)1 << 22;
  const dim3 grid((unsigned)(tiles < limit ? tiles : limit));
  uint32_t *words = reinterpret_cast<uint32_t *>(codes);
  const bool vec = ld % 8 == 0;
#define ENGRAM_QUANTIZE(F, V)                                                                   \
  hipLaunchKernelGGL((quantize_mx4_kernel<F, V>), grid, dim3(kThreads), 0, stream, src, cols, ld, \
                     words, scales, values, groups, total)
  if (f32 && vec) ENGRAM_QUANTIZE(true, true);
  else if (f32) ENGRAM_QUANTIZE(true, false);
  else if (vec) ENGRAM_QUANTIZE(false, true);
  else ENGRAM_QUANTIZE(false, false);
#undef ENGRAM_QUANTIZE
  return hipGetLastError();
}
