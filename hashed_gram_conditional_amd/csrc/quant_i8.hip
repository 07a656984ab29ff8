// Quantisation to 8-bit integers with one scale per row (engram_quantize_i8): s = amax /
// 127 rounded to fp32, or the smallest power of two with amax <= 127 s, and codes x
// (127 / amax) or x / s, to the nearest whole number, ties to the even one.
//
// A code is that of the exact product with the fp32 factor: the fp32 product decides it
// unless it falls on a half, where its rounding error says on which side the exact one lies.
// The row's maximum is taken on the values' bits (as integers, where infinities and NaN lie
// above every finite value). A bf16 value q s is rounded to fp32 first, which gives the
// bf16 number that one rounding would: amax is a bf16 number then, A 2^e with A < 2^8, and q A /
// 127 is the middle of two bf16 numbers or at least 2^-16 of itself away from one, because
// 2^j q A and 127 times an odd number, both below 2^16, differ by 1 or more; and in the middle
// q or A is a multiple of 127, and q s is exact or amax.
//
// One pass, bound by HBM: a row waits for its maximum in the registers of a wave (up to 1024
// columns) or a block (up to 8192). 25600 x 6144 fp32 with values take 280 us (1.42 GB, 5.1
// TB/s), 40960 x 5120 bf16 with values 180 us (1.05 GB, 5.8 TB/s), 256 x 6144 bf16 5.8 us.
// Rows read value by value, twice, took 453, 516 and 9.5 us.
#include "common.h"

namespace {

constexpr int kThreads = 256;
constexpr int kLongThreads = 1024;
constexpr uint32_t kSmallest = 8u << 23;      // 2^-119

struct RowScale {
  float scale, inv;
  float most;               // of a code's magnitude
  bool bad;
};

template <bool POW2>
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale r;
  r.bad = top >= 0x7F800000u;
  r.scale = r.inv = 0.f;
  r.most = 127.f;
  if (r.bad) {
    r.scale = __uint_as_float(0x7FC00000u);
  } else if (top >= kSmallest) {
    if (POW2) {
      // amax = m 2^E, 1 <= m < 2: 2^(E - 6) reaches 127 / 64 of 2^E
      const uint32_t field = (top >> 23) - 6 + ((top & 0x7FFFFFu) > 0x7E0000u);
      r.scale = __uint_as_float(field << 23);
      r.inv = __uint_as_float((254u - field) << 23);
      if (field == 249u) r.most = 63.f;      // 64 steps of 2^122 would not be finite
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

// 16 bytes at any address of a number
template <bool F32>
struct __attribute__((packed, aligned(F32 ? 4 : 2))) Anywhere {
  uint32_t w[4];
};

// Eight consecutive values from `col` on, zeros behind the row. VEC: rows start at multiples
// of 8 values; others move in the same 16-byte accesses, which the hardware takes at any
// address (25600 x 6143 fp32 592 -> 275 us against value by value, bf16 395 -> 185).
template <bool F32, bool VEC>
struct Eight {
  float f[8];
  __device__ __forceinline__ void load(const void *src, int64_t row_off, int64_t col, int64_t cols) {
    if (VEC && col + 8 <= cols) {
      engram::Chunk8<F32> c;
      c.load_nt(src, (row_off + col) / 8);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = c[e];
      return;
    }
    if (col + 8 <= cols) {
      const auto *p = reinterpret_cast<const Anywhere<F32> *>(reinterpret_cast<const char *>(src) +
                                                              (row_off + col) * (F32 ? 4 : 2));
      const Anywhere<F32> a = p[0];
      if (F32) {
        const Anywhere<F32> b = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = __uint_as_float(a.w[e]);
          f[4 + e] = __uint_as_float(b.w[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = engram::bf16_to_f32(a.w[e / 2] >> (16 * (e % 2)) & 0xFFFFu);
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = 0.f;
      if (col + e < cols)
        f[e] = F32 ? reinterpret_cast<const float *>(src)[row_off + col + e]
                   : engram::bf16_to_f32(reinterpret_cast<const uint16_t *>(src)[row_off + col + e]);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = max(t, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    return t;
  }
  // the codes, as numbers, in place of the values, and packed
  template <bool POW2>
  __device__ __forceinline__ uint2 encode(const RowScale &r) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // x / s is exact where s is a power of two
      f[e] = r.bad ? 0.f
             : POW2 ? fminf(fmaxf(rintf(f[e] * r.inv), -r.most), r.most)
                    : code_of(f[e], r.inv);
      w[e / 4] |= ((uint32_t)(int)f[e] & 0xFFu) << (8 * (e % 4));
    }
    return make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void store(void *dst, int64_t row_off, int64_t col, int64_t cols, float scale) const {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e] * scale;
    if (VEC && col + 8 <= cols) {
      engram::Chunk8<F32>::store_nt(dst, (row_off + col) / 8, v);
      // keeps the compiler from merging these with the single stores below
      asm volatile("" ::: "memory");
      return;
    }
    if (col + 8 <= cols) {
      auto *p = reinterpret_cast<Anywhere<F32> *>(reinterpret_cast<char *>(dst) + (row_off + col) * (F32 ? 4 : 2));
      Anywhere<F32> a;
      if (F32) {
        Anywhere<F32> b;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a.w[e] = __float_as_uint(v[e]);
          b.w[e] = __float_as_uint(v[4 + e]);
        }
        p[1] = b;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) a.w[e] = engram::pack_bf16x2(v[2 * e], v[2 * e + 1]);
      }
      p[0] = a;
      asm volatile("" ::: "memory");
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (col + e < cols) {
        if (F32)
          reinterpret_cast<float *>(dst)[row_off + col + e] = v[e];
        else
          reinterpret_cast<uint16_t *>(dst)[row_off + col + e] = (uint16_t)engram::pack_bf16x2(v[e], v[e]);
      }
    }
  }
};

// The largest of LANES neighbouring lanes'.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, engram::kWave));
  return v;
}

// A row in the registers of TEAM threads (8 to 64 lanes of a wave, or the block), CPT groups of
// 8 a thread.
// src and values may be the same buffer (each value is read and written by one thread), so
// neither is marked restrict. The grid walks the rows.
template <bool F32, bool VEC, bool POW2, int TEAM, int CPT>
__global__ __launch_bounds__(kThreads) void quantize_i8_kernel(const void *src, int64_t rows, int64_t cols,
                                                               int64_t ld, int64_t out_cols,
                                                               uint2 *__restrict__ codes,
                                                               float *__restrict__ scales, void *values) {
  constexpr int kTeams = kThreads / TEAM;
  __shared__ uint32_t red[2][kThreads / 64];
  const int at = threadIdx.x % TEAM;
  const int64_t groups = out_cols / 8;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / TEAM; row < rows;
       row += (int64_t)gridDim.x * kTeams) {
    Eight<F32, VEC> x[CPT];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CPT; ++i) x[i].load(src, row * ld, (int64_t)(at + i * TEAM) * 8, cols);
#pragma unroll
    for (int i = 0; i < CPT; ++i) top = max(top, x[i].top());
    top = lanes_max<(TEAM < 64 ? TEAM : 64)>(top);
    if (TEAM > 64) {
      // the next row's barrier stands between these reads and the writes after it
      if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) top = max(top, red[slot][w]);
      slot ^= 1;
    }
    const RowScale r = row_scale<POW2>(top);
    if (at == 0) scales[row] = r.scale;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int64_t g = at + i * TEAM;
      if (g >= groups) break;
      const uint2 w = x[i].template encode<POW2>(r);
      codes[row * groups + g] = w;
      if (values != nullptr) x[i].store(values, row * ld, g * 8, cols, r.scale);
    }
  }
}

// A longer row: read twice, the second time from L2.
template <bool F32, bool VEC, bool POW2>
__global__ __launch_bounds__(kLongThreads) void quantize_i8_long_kernel(const void *src, int64_t rows,
                                                                        int64_t cols, int64_t ld,
                                                                        int64_t out_cols,
                                                                        uint2 *__restrict__ codes,
                                                                        float *__restrict__ scales,
                                                                        void *values) {
  __shared__ uint32_t red[2][kLongThreads / 64];
  const int64_t groups = out_cols / 8;
  int slot = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    Eight<F32, VEC> x;
    uint32_t top = 0;
#pragma unroll 4
    for (int64_t g = threadIdx.x; g < groups; g += kLongThreads) {
      x.load(src, row * ld, g * 8, cols);
      top = max(top, x.top());
    }
    top = lanes_max<64>(top);
    if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLongThreads / 64; ++w) top = max(top, red[slot][w]);
    slot ^= 1;
    const RowScale r = row_scale<POW2>(top);
    if (threadIdx.x == 0) scales[row] = r.scale;
    for (int64_t g = threadIdx.x; g < groups; g += kLongThreads) {
      x.load(src, row * ld, g * 8, cols);
      const uint2 w = x.template encode<POW2>(r);
      codes[row * groups + g] = w;
      if (values != nullptr) x.store(values, row * ld, g * 8, cols, r.scale);
    }
  }
}

// Rows of up to 1024 columns take 8 to 64 lanes each, of up to 8192 a block, in the registers
// of which they fit; longer ones are read twice.
template <bool F32, bool VEC, bool POW2>
void launch(const void *src, int64_t rows, int64_t cols, int64_t ld, int64_t out_cols, uint2 *codes,
            float *scales, void *values, hipStream_t stream) {
  // at most 2^32 threads to a launch
  const int64_t most = (int64_t)1 << 21;
  const int64_t teams = out_cols <= 64 ? 32 : out_cols <= 128 ? 16 : out_cols <= 256 ? 8 : out_cols <= 1024 ? 4 : 1;
  const int64_t blocks = (rows + teams - 1) / teams;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
#define ENGRAM_QUANTIZE(T, C)                                                                   \
  hipLaunchKernelGGL((quantize_i8_kernel<F32, VEC, POW2, T, C>), grid, dim3(kThreads), 0, stream, src, \
                     rows, cols, ld, out_cols, codes, scales, values)
  if (out_cols <= 64) ENGRAM_QUANTIZE(8, 1);
  else if (out_cols <= 128) ENGRAM_QUANTIZE(16, 1);
  else if (out_cols <= 256) ENGRAM_QUANTIZE(32, 1);
  else if (out_cols <= 512) ENGRAM_QUANTIZE(64, 1);
  else if (out_cols <= 1024) ENGRAM_QUANTIZE(64, 2);
  else if (out_cols <= 2048) ENGRAM_QUANTIZE(kThreads, 1);
  else if (out_cols <= 4096) ENGRAM_QUANTIZE(kThreads, 2);
  else if (out_cols <= 6144) ENGRAM_QUANTIZE(kThreads, 3);
  else if (out_cols <= 8192) ENGRAM_QUANTIZE(kThreads, 4);
  else
    hipLaunchKernelGGL((quantize_i8_long_kernel<F32, VEC, POW2>), grid, dim3(kLongThreads), 0, stream, src, rows,
                       cols, ld, out_cols, codes, scales, values);
#undef ENGRAM_QUANTIZE
}

}  // namespace

hipError_t engram_launch_quantize_i8(bool f32, bool pow2, const void *src, int64_t rows,
                                     int64_t cols, int64_t ld, int64_t out_cols, int8_t *codes,
                                     float *scales, void *values, hipStream_t stream) {
  if (rows <= 0) return hipSuccess;
  uint2 *words = reinterpret_cast<uint2 *>(codes);
  const bool vec = ld % 8 == 0;
#define ENGRAM_QUANTIZE(F, V, P) launch<F, V, P>(src, rows, cols, ld, out_cols, words, scales, values, stream)
#define ENGRAM_QUANTIZE_KIND(F, V) \
  if (pow2) ENGRAM_QUANTIZE(F, V, true); else ENGRAM_QUANTIZE(F, V, false)
  if (f32 && vec) {
    ENGRAM_QUANTIZE_KIND(true, true);
  } else if (f32) {
    ENGRAM_QUANTIZE_KIND(true, false);
  } else if (vec) {
    ENGRAM_QUANTIZE_KIND(false, true);
  } else {
    ENGRAM_QUANTIZE_KIND(false, false);
  }
#undef ENGRAM_QUANTIZE_KIND
#undef ENGRAM_QUANTIZE
  return hipGetLastError();
}
