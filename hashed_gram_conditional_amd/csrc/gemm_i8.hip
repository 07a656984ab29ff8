// Step 4 with 8-bit integer operands: kv[t, c] = s_t s_c sum_k e[t, k] W[c, k]. The sum is
// exact in 32 bits (in_dim < 2^17 codes of at most 128); it is converted to fp32, scaled
// by the channel, then by the token, and rounded to kv's type.
#include "gemm_tiles.h"

using namespace engram_gemm;

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct I8Operands {
  const int8_t *w_codes;     // [N, K]
  const float *w_scales;     // [N]
  const int8_t *e_codes;     // [M, K]
  const float *e_scales;     // [M]
  int M, N, K;
};

constexpr int kTile = 128, kStep = 64, kLd = kStep + 16;

template <bool F32>
__global__ __launch_bounds__(256) void i8_kernel(I8Operands op, void *__restrict__ kv, int tiles_n) {
  __shared__ __align__(16) uint8_t w[kTile * kLd], e[kTile * kLd];
  const int n0 = (int)(blockIdx.x % tiles_n) * kTile, m0 = (int)(blockIdx.x / tiles_n) * kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave >> 1, wm = wave & 1;
  i32x16 acc[2][2];
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  for (int k0 = 0; k0 < op.K; k0 += kStep) {
    __syncthreads();
    for (int q = tid; q < kTile * (kStep / 16); q += 256) {
      const int row = q / (kStep / 16), c = q % (kStep / 16) * 16;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (k0 + c < op.K) {
        if (n0 + row < op.N) a = *reinterpret_cast<const uint4 *>(op.w_codes + (int64_t)(n0 + row) * op.K + k0 + c);
        if (m0 + row < op.M) b = *reinterpret_cast<const uint4 *>(op.e_codes + (int64_t)(m0 + row) * op.K + k0 + c);
      }
      *reinterpret_cast<uint4 *>(w + row * kLd + c) = a;
      *reinterpret_cast<uint4 *>(e + row * kLd + c) = b;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStep / 32; ++s) {
      i32x4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const i32x4 *>(w + (wn * 64 + i * 32 + (lane & 31)) * kLd + s * 32 + (lane >> 5) * 16);
        b[i] = *reinterpret_cast<const i32x4 *>(e + (wm * 64 + i * 32 + (lane & 31)) * kLd + s * 32 + (lane >> 5) * 16);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int m = m0 + wm * 64 + j * 32 + (lane & 31);
    if (m >= op.M) continue;
    const float es = op.e_scales[m];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + wn * 64 + i * 32 + g * 8 + (lane >> 5) * 4;
        if (n >= op.N) continue;
        const float4 s = *reinterpret_cast<const float4 *>(op.w_scales + n);
        const float f[4] = {(float)acc[i][j][g * 4] * s.x * es, (float)acc[i][j][g * 4 + 1] * s.y * es,
                            (float)acc[i][j][g * 4 + 2] * s.z * es, (float)acc[i][j][g * 4 + 3] * s.w * es};
        if (F32)
          *reinterpret_cast<float4 *>(reinterpret_cast<float *>(kv) + (int64_t)m * op.N + n) =
              make_float4(f[0], f[1], f[2], f[3]);
        else
          *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(kv) + (int64_t)m * op.N + n) =
              make_uint2(engram::pack_bf16x2(f[0], f[1]), engram::pack_bf16x2(f[2], f[3]));
      }
  }
}

}  // namespace

hipError_t engram_launch_gemm_i8(const int8_t *w_codes, const float *w_scales, const int8_t *e_codes,
                                 const float *e_scales, bool f32, void *kv, int64_t m, int64_t n,
                                 int64_t k, hipStream_t stream) {
  if (m <= 0 || n <= 0) return hipSuccess;
  const I8Operands op{w_codes, w_scales, e_codes, e_scales, (int)m, (int)n, (int)k};
  const int tiles_n = (int)((n + kTile - 1) / kTile), tiles_m = (int)((m + kTile - 1) / kTile);
  const dim3 grid((unsigned)(tiles_n * tiles_m));
  if (f32)
    hipLaunchKernelGGL((i8_kernel<true>), grid, dim3(256), 0, stream, op, kv, tiles_n);
  else
    hipLaunchKernelGGL((i8_kernel<false>), grid, dim3(256), 0, stream, op, kv, tiles_n);
  return hipGetLastError();
}
