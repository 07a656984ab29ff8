// Step 4 with the projection weight in 4-bit block floating point: kv = e W^T, W as
// E2M1 codes (two to a byte) and e as E2M1 or E4M3 codes, both with one E8M0
// scale per 32 consecutive inputs. v_mfma_scale_f32_32x32x64_f8f6f4 takes the two
// formats as they are, multiplies the codes exactly, applies both block scales and
// accumulates in fp32; kv is rounded once to bf16.
//
// Lane layout of that MFMA (measured on gfx950): lane l of half h = l / 32 holds
// row l % 32. Its 16 bytes of E2M1 are inputs [32 h, 32 h + 32) of the 64 in order;
// its 32 bytes of E4M3 are inputs [16 h, 16 h + 16) and [32 + 16 h, 48 + 16 h). The
// scale of inputs [32 h, 32 h + 32) comes from the lanes of half h, from one byte of
// a register that the instruction selects. That register must be a vector one.
//
// A product over the inputs may take them in any order that both operands share.
// Here half h of a wave takes blocks 4 h .. 4 h + 3 of each 8 blocks (256 inputs),
// one per MFMA: a lane's four E2M1 blocks are then 64 contiguous bytes and their
// scales one aligned dword, whose byte i serves MFMA i with no shift. in_dim is a
// multiple of 128, so the four blocks of a half exist together or not at all.
#include "gemm_tiles.h"

using namespace engram_gemm;

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Mx4Operands {
  const uint8_t *w_codes;    // [N, K / 2]
  const uint8_t *w_scales;   // [N, K / 32]
  const uint8_t *e_codes;    // [M, K / 2] (E2M1) or [M, K] (E4M3)
  const uint8_t *e_scales;   // [M, K / 32]
  int M, N, K;
};

constexpr int kFp4 = 4, kFp8 = 0;      // operand formats of the MFMA

__device__ __forceinline__ i32x8 fp4_operand(uint4 v) {
  i32x8 r = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
  return r;
}

__device__ __forceinline__ i32x8 fp8_operand(uint4 lo, uint4 hi) {
  i32x8 r = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  return r;
}

// MFMA i (0..3) of a 256-input unit: W block against e block, scale byte i of each.
template <int EF, int I>
__device__ __forceinline__ f32x16 mfma_unit(i32x8 w, i32x8 e, f32x16 acc, uint32_t ws, uint32_t es) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, e, acc, kFp4, EF, I, (int)ws, I, (int)es);
}

// ---- a few tokens: the weight straight from memory to registers -------------------
// A block takes 32 weight rows against 32 MT tokens; its waves split the inputs
// (unit u belongs to wave u % waves) and their sums meet in LDS in wave order. Each
// weight byte is loaded once, by the lane that multiplies it.
constexpr int kThinWaves = 4;

template <int EF, int MT>
struct ThinUnit {
  uint4 w[4];
  uint4 e[MT][EF == kFp4 ? 4 : 8];
  uint32_t ws, es[MT];
};

template <int EF, int MT>
__device__ __forceinline__ void thin_load(ThinUnit<EF, MT> &t, const Mx4Operands &op, int unit,
                                          int n, const int (&m)[MT], int h) {
  const int KB = op.K / 32;
  const int b = unit * 8 + 4 * h;
  const bool in = b < KB;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  const uint8_t *w = op.w_codes + (int64_t)n * (op.K / 2) + b * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) t.w[i] = in ? reinterpret_cast<const uint4 *>(w)[i] : none;
  t.ws = in ? *reinterpret_cast<const uint32_t *>(op.w_scales + (int64_t)n * KB + b) : 0x7F7F7F7Fu;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    if (EF == kFp4) {
      const uint8_t *e = op.e_codes + (int64_t)m[j] * (op.K / 2) + b * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) t.e[j][i] = in ? reinterpret_cast<const uint4 *>(e)[i] : none;
    } else {
      // halves of blocks 8 unit + i and 8 unit + 4 + i
      const uint8_t *e = op.e_codes + (int64_t)m[j] * op.K + unit * 256 + 16 * h;
      const bool second = unit * 8 + 4 < KB;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.e[j][2 * i % 8] = *reinterpret_cast<const uint4 *>(e + i * 32);
        t.e[j][(2 * i + 1) % 8] = second ? *reinterpret_cast<const uint4 *>(e + 128 + i * 32) : none;
      }
    }
    t.es[j] = in ? *reinterpret_cast<const uint32_t *>(op.e_scales + (int64_t)m[j] * KB + b)
                 : 0x7F7F7F7Fu;
  }
}

template <int EF, int MT, int I>
__device__ __forceinline__ void thin_mfma(f32x16 (&acc)[MT], const ThinUnit<EF, MT> &t) {
  const i32x8 w = fp4_operand(t.w[I]);
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const i32x8 e = EF == kFp4 ? fp4_operand(t.e[j][I]) : fp8_operand(t.e[j][2 * I % 8], t.e[j][(2 * I + 1) % 8]);
    acc[j] = mfma_unit<EF, I>(w, e, acc[j], t.ws, t.es[j]);
  }
}

template <int EF, int MT>
__global__ __launch_bounds__(kThinWaves * 64) void mx4_thin_kernel(Mx4Operands op,
                                                                   uint16_t *__restrict__ kv) {
  __shared__ float part[kThinWaves - 1][MT * 16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = lane & 31, h = lane >> 5;
  const int n0 = blockIdx.x * 32, m0 = blockIdx.y * 32 * MT;
  // rows past the end repeat the last one; their outputs are not stored
  const int n = min(n0 + row, op.N - 1);
  int m[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) m[j] = min(m0 + j * 32 + row, op.M - 1);
  f32x16 acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
  const int units = (op.K + 255) / 256;
  for (int u = wave; u < units; u += kThinWaves) {
    ThinUnit<EF, MT> t;
    thin_load<EF, MT>(t, op, u, n, m, h);
    thin_mfma<EF, MT, 0>(acc, t);
    thin_mfma<EF, MT, 1>(acc, t);
    thin_mfma<EF, MT, 2>(acc, t);
    thin_mfma<EF, MT, 3>(acc, t);
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) part[wave - 1][j * 16 + r][lane] = acc[j][r];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
#pragma unroll
    for (int w = 0; w < kThinWaves - 1; ++w)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] += part[w][j * 16 + r][lane];
    // accumulator r: column n0 + 8 (r / 4) + 4 h + r % 4 of token m0 + 32 j + row
    const int t = m0 + j * 32 + row;
    if (t >= op.M) continue;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = n0 + g * 8 + h * 4;
      if (c < op.N) {
        uint2 v;
        v.x = engram::pack_bf16x2(acc[j][g * 4 + 0], acc[j][g * 4 + 1]);
        v.y = engram::pack_bf16x2(acc[j][g * 4 + 2], acc[j][g * 4 + 3]);
        *reinterpret_cast<uint2 *>(kv + (int64_t)t * op.N + c) = v;
      }
    }
  }
}

}  // namespace

hipError_t engram_gemm_mx4_workspace(int64_t m, int64_t n, int64_t k, bool e_fp4, size_t *bytes) {
  (void)m; (void)n; (void)k; (void)e_fp4;
  *bytes = 0;
  return hipSuccess;
}

hipError_t engram_launch_gemm_mx4(const uint8_t *w_codes, const uint8_t *w_scales,
                                  const uint8_t *e_codes, const uint8_t *e_scales, bool e_fp4,
                                  uint16_t *kv, int64_t m, int64_t n, int64_t k, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
  (void)workspace; (void)workspace_bytes;
  if (m <= 0 || n <= 0) return hipSuccess;
  const Mx4Operands op{w_codes, w_scales, e_codes, e_scales, (int)m, (int)n, (int)k};
  const dim3 block(kThinWaves * 64);
  const dim3 grid((unsigned)((n + 31) / 32), (unsigned)((m + 63) / 64));
  if (e_fp4)
    hipLaunchKernelGGL((mx4_thin_kernel<kFp4, 2>), grid, block, 0, stream, op, kv);
  else
    hipLaunchKernelGGL((mx4_thin_kernel<kFp8, 2>), grid, block, 0, stream, op, kv);
  return hipGetLastError();
}
