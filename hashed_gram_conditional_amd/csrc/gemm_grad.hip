// Gradient of the projection's weight from 8-bit codes of its inputs: dW[n, k] = sum_t
// d_kv[t, n] s_t q[t, k]. Both operands have the summed index outermost; LDS reads that
// transpose 4 x 16 blocks (ds_read_b64_tr_b16) bring it innermost for the MFMA.
#include "gemm_tiles.h"

using namespace engram_gemm;

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

struct GradOperands {
  const uint16_t *d_kv;      // [T, N] bf16
  const int8_t *e_codes;     // [T, K]
  const float *e_scales;     // [T]
  int T, N, K;
};

constexpr int kTile = 128, kStep = 32, kLd = kTile + 8;

__device__ __forceinline__ s16x4 read_tr(const uint16_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}

__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <bool F32>
__global__ __launch_bounds__(256) void grad_kernel(GradOperands op, void *__restrict__ grad,
                                                   int accumulate, int tiles_k) {
  __shared__ __align__(16) uint16_t dk[kStep * kLd], ek[kStep * kLd];
  const int k0 = (int)(blockIdx.x % tiles_k) * kTile, n0 = (int)(blockIdx.x / tiles_k) * kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wk = wave >> 1, wn = wave & 1;
  const int group = lane >> 4, in = lane & 15;
  // this lane's address in a 16 (t) x 32 block: row, column
  const int tr_row = (group >> 1) * 8 + in / 4, tr_col = (group & 1) * 16 + in % 4 * 4;
  f32x16 acc[2][2];
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  for (int t0 = 0; t0 < op.T; t0 += kStep) {
    __syncthreads();
    for (int q = tid; q < kStep * (kTile / 8); q += 256) {
      const int row = q / (kTile / 8), c = q % (kTile / 8) * 8;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (t0 + row < op.T) {
        if (n0 + c < op.N) a = *reinterpret_cast<const uint4 *>(op.d_kv + (int64_t)(t0 + row) * op.N + n0 + c);
        if (k0 + c < op.K) {
          const float s = op.e_scales[t0 + row];
          const uint2 codes = *reinterpret_cast<const uint2 *>(op.e_codes + (int64_t)(t0 + row) * op.K + k0 + c);
          float f[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            f[x] = s * (float)(int8_t)(codes.x >> (8 * x));
            f[4 + x] = s * (float)(int8_t)(codes.y >> (8 * x));
          }
          b.x = engram::pack_bf16x2(f[0], f[1]);
          b.y = engram::pack_bf16x2(f[2], f[3]);
          b.z = engram::pack_bf16x2(f[4], f[5]);
          b.w = engram::pack_bf16x2(f[6], f[7]);
        }
      }
      *reinterpret_cast<uint4 *>(dk + row * kLd + c) = a;
      *reinterpret_cast<uint4 *>(ek + row * kLd + c) = b;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStep / 16; ++s) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint16_t *pe = ek + (s * 16 + tr_row) * kLd + wk * 64 + i * 32 + tr_col;
        const uint16_t *pd = dk + (s * 16 + tr_row) * kLd + wn * 64 + i * 32 + tr_col;
        a[i] = join(read_tr(pe), read_tr(pe + 4 * kLd));
        b[i] = join(read_tr(pd), read_tr(pd + 4 * kLd));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = n0 + wn * 64 + j * 32 + (lane & 31);
    if (n >= op.N) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int k = k0 + wk * 64 + i * 32 + g * 8 + (lane >> 5) * 4;
        if (k >= op.K) continue;
        float f[4] = {acc[i][j][g * 4], acc[i][j][g * 4 + 1], acc[i][j][g * 4 + 2], acc[i][j][g * 4 + 3]};
        const int64_t at = (int64_t)n * op.K + k;
        if (F32) {
          float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(grad) + at);
          float4 v = make_float4(f[0], f[1], f[2], f[3]);
          if (accumulate) {
            const float4 o = *p;
            v = make_float4(o.x + f[0], o.y + f[1], o.z + f[2], o.w + f[3]);
          }
          *p = v;
        } else {
          uint2 *p = reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(grad) + at);
          if (accumulate) {
            const uint2 o = *p;
            f[0] += engram::bf16_to_f32(o.x & 0xFFFFu);
            f[1] += engram::bf16_to_f32(o.x >> 16);
            f[2] += engram::bf16_to_f32(o.y & 0xFFFFu);
            f[3] += engram::bf16_to_f32(o.y >> 16);
          }
          *p = make_uint2(engram::pack_bf16x2(f[0], f[1]), engram::pack_bf16x2(f[2], f[3]));
        }
      }
  }
}

}  // namespace

hipError_t engram_launch_gemm_grad(const uint16_t *d_kv, const int8_t *e_codes, const float *e_scales,
                                   bool f32, void *grad, int accumulate, int64_t t, int64_t n,
                                   int64_t k, hipStream_t stream) {
  const GradOperands op{d_kv, e_codes, e_scales, (int)t, (int)n, (int)k};
  const int tiles_n = (int)((n + kTile - 1) / kTile), tiles_k = (int)((k + kTile - 1) / kTile);
  const dim3 grid((unsigned)(tiles_n * tiles_k));
  if (f32)
    hipLaunchKernelGGL((grad_kernel<true>), grid, dim3(256), 0, stream, op, grad, accumulate, tiles_k);
  else
    hipLaunchKernelGGL((grad_kernel<false>), grid, dim3(256), 0, stream, op, grad, accumulate, tiles_k);
  return hipGetLastError();
}
