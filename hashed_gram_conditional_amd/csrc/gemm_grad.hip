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

constexpr int kStep = 64;                 // tokens per step
constexpr int kTile = 256;                // columns of either operand
constexpr int kRow = kTile * 2;           // bytes of a row in LDS
constexpr int kPatch = 4096;              // LDS of a wave for storing part of its tile

__device__ __forceinline__ s16x4 read_tr(const uint8_t *p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
}

__device__ __forceinline__ bf16x8 join(s16x4 a, s16x4 b) {
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Two codes (bytes 2 i and 2 i + 1 of w's low or high half) times s, as bf16.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, int i, float s) {
  return engram::pack_bf16x2((float)(int8_t)(w >> (16 * i)) * s, (float)(int8_t)(w >> (16 * i + 8)) * s);
}

// Stores 32 rows (n) x COLS columns (k, one or two accumulators) of a wave in whole cache
// lines, through LDS: a lane's accumulators are 4 columns of one row at a time. ADD: added
// to what is there, in fp32, and rounded once.
template <bool F32, bool ADD, int COLS>
__device__ __forceinline__ void store_patch(const f32x16 &a0, const f32x16 &a1, uint8_t *patch,
                                            void *__restrict__ grad, int N, int K, int n, int k, int lane) {
  constexpr bool kWide = F32 || ADD;                     // fp32 in the patch
  constexpr int kBytes = COLS * (kWide ? 4 : 2), kChunks = kBytes / 16;
  const int frow = lane & 31, fk = lane >> 5;
#pragma unroll
  for (int i = 0; i < COLS / 32; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x16 &a = i ? a1 : a0;
      if (kWide)
        *reinterpret_cast<float4 *>(patch + frow * kBytes + (((i * 8 + g * 2 + fk) ^ (frow & (kChunks - 1))) << 4)) =
            make_float4(a[g * 4], a[g * 4 + 1], a[g * 4 + 2], a[g * 4 + 3]);
      else
        *reinterpret_cast<uint2 *>(patch + frow * kBytes + (((i * 4 + g) ^ (frow & (kChunks - 1))) << 4) + fk * 8) =
            make_uint2(engram::pack_bf16x2(a[g * 4], a[g * 4 + 1]), engram::pack_bf16x2(a[g * 4 + 2], a[g * 4 + 3]));
    }
  const int c = lane % kChunks, col = k + c * (kWide ? 4 : 8);
#pragma unroll
  for (int q = 0; q < 32 * kChunks / 64; ++q) {
    const int t = (q * 64 + lane) / kChunks;
    engram::u32x4 v = *reinterpret_cast<const engram::u32x4 *>(patch + t * kBytes + ((c ^ (t & (kChunks - 1))) << 4));
    if (n + t >= N || col >= K) continue;
    const int64_t at = (int64_t)(n + t) * K + col;
    if (F32) {
      engram::u32x4 *p = reinterpret_cast<engram::u32x4 *>(reinterpret_cast<float *>(grad) + at);
      if (ADD) {
        const engram::u32x4 o = *p;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = __float_as_uint(__uint_as_float(o[x]) + __uint_as_float(v[x]));
      }
      __builtin_nontemporal_store(v, p);
    } else if (ADD) {
      uint2 *p = reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(grad) + at);
      const uint2 o = *p;
      *p = make_uint2(engram::pack_bf16x2(__uint_as_float(v[0]) + engram::bf16_to_f32(o.x & 0xFFFFu),
                                          __uint_as_float(v[1]) + engram::bf16_to_f32(o.x >> 16)),
                      engram::pack_bf16x2(__uint_as_float(v[2]) + engram::bf16_to_f32(o.y & 0xFFFFu),
                                          __uint_as_float(v[3]) + engram::bf16_to_f32(o.y >> 16)));
    } else {
      __builtin_nontemporal_store(v, reinterpret_cast<engram::u32x4 *>(reinterpret_cast<uint16_t *>(grad) + at));
    }
  }
}

// A block sums the tokens [split * per, (split + 1) * per) of one 256 x 256 tile (four waves
// of 128 x 128) in steps of 64, two stages. d_kv goes global -> LDS by direct loads; codes go
// through registers, where they are scaled and rounded to bf16: those of step kt + 2 are
// requested at the end of step kt and written to LDS during step kt + 1, whose stage is the
// other one. In a row of LDS the 64-byte group of column c sits at group ^ (t % 4), so that
// the four rows of a transposing read fall into different banks.
template <bool F32, bool ADD>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grad_kernel(GradOperands op, void *__restrict__ grad, int tiles_n, int tiles_k,
                 int tiles, int per) {
  __shared__ __align__(1024) uint8_t d0[kStep * kRow], d1[kStep * kRow];
  __shared__ __align__(1024) uint8_t e0[kStep * kRow], e1[kStep * kRow];
  __shared__ __align__(1024) uint8_t out[4 * kPatch];
  const int split = (int)blockIdx.x / tiles;
  int n0, k0;
  tile_origin_of((int)blockIdx.x - split * tiles, tiles_n, tiles_k, kTile, n0, k0);
  const int t_first = split * per, t_last = min(op.T, t_first + per);
  const int steps = ((t_last - t_first + kStep - 1) / kStep + 1) & ~1;      // a step of zeros if odd
  if (gridDim.x > (unsigned)tiles) grad = reinterpret_cast<float *>(grad) + (int64_t)split * op.N * op.K;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave >> 1, wn = wave & 1;
  // direct load i of a wave fills 1 KB: rows 16 wave + 2 i and the next (lane p: row p / 32,
  // slot p % 32)
  const int d_row = (wave * 16 + (lane >> 5)) * op.N * 2;
  const int d_v0 = d_row + (((lane & 31) ^ (lane >> 5 << 2)) << 4);
  const int d_v1 = d_row + (((lane & 31) ^ ((2 + (lane >> 5)) << 2)) << 4);
  // codes: 16 threads a row of 256, four rows a thread, 16 apart
  const int c_row = tid >> 4, c_col = tid & 15;
  const int e_v = c_row * op.K + c_col * 16;
  const int e_w = c_row * kRow + (((c_col * 2) ^ ((c_row & 3) << 2)) << 4);
  // a lane's address in a 16 (t) x 32 block: row, and the bytes of its column
  const int group = lane >> 4, in = lane & 15;
  const int tr_row = (group >> 1) * 8 + in / 4;
  const int tr_x = (tr_row & 3) << 6, tr_c = (group & 1) * 32 + in % 4 * 8;
  const int a_base = tr_row * kRow + tr_c, b_base = a_base;
#define GR_D(st) ((st) ? d1 : d0)
#define GR_E(st) ((st) ? e1 : e0)
  uint4 codes[4];
  float scale[4];
// requests step kt_: codes and scales into registers, d_kv into stage st; rows behind the
// last token are zeros
#define GR_LOAD(kt_, st)                                                                       \
  {                                                                                            \
    const int t_ = t_first + (kt_) * kStep;                                                    \
    const int rows_ = t_ >= t_last ? 0 : t_last - t_ < kStep ? t_last - t_ : kStep;            \
    const int64_t at_ = rows_ > 0 ? t_ : 0;                                                    \
    const __amdgpu_buffer_rsrc_t rsD = __builtin_amdgcn_make_buffer_rsrc(                      \
        const_cast<uint16_t *>(op.d_kv + at_ * op.N + n0), 0,                                  \
        rows_ > 0 ? (rows_ * op.N - n0) * 2 : 0, kBufferFlags);                                \
    const __amdgpu_buffer_rsrc_t rsE = __builtin_amdgcn_make_buffer_rsrc(                      \
        const_cast<int8_t *>(op.e_codes + at_ * op.K + k0), 0, rows_ > 0 ? rows_ * op.K - k0 : 0, \
        kBufferFlags);                                                                         \
    const __amdgpu_buffer_rsrc_t rsS = __builtin_amdgcn_make_buffer_rsrc(                      \
        const_cast<float *>(op.e_scales + at_), 0, rows_ * 4, kBufferFlags);                   \
    _Pragma("unroll") for (int i = 0; i < 4; ++i) {                                            \
      codes[i] = load16(rsE, e_v, i * 16 * op.K);                                              \
      scale[i] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsS, c_row * 4, i * 64, 0)); \
    }                                                                                          \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds(    \
        rsD, ENGRAM_LDS(&GR_D(st)[(wave * 8 + i) * 1024]), 16, (i & 1) ? d_v1 : d_v0,          \
        i * 4 * op.N, 0, 0);                                                                   \
  }
#define GR_WRITE(st, i)                                                                        \
  {                                                                                            \
    uint4 lo_, hi_;                                                                            \
    lo_.x = scaled_pair(codes[i].x, 0, scale[i]);                                              \
    lo_.y = scaled_pair(codes[i].x, 1, scale[i]);                                              \
    lo_.z = scaled_pair(codes[i].y, 0, scale[i]);                                              \
    lo_.w = scaled_pair(codes[i].y, 1, scale[i]);                                              \
    hi_.x = scaled_pair(codes[i].z, 0, scale[i]);                                              \
    hi_.y = scaled_pair(codes[i].z, 1, scale[i]);                                              \
    hi_.z = scaled_pair(codes[i].w, 0, scale[i]);                                              \
    hi_.w = scaled_pair(codes[i].w, 1, scale[i]);                                              \
    *reinterpret_cast<uint4 *>(&GR_E(st)[e_w + (i) * 16 * kRow]) = lo_;                        \
    *reinterpret_cast<uint4 *>(&GR_E(st)[(e_w ^ 16) + (i) * 16 * kRow]) = hi_;                 \
  }
// fragments of tokens 16 s .. 16 s + 15: columns wk * 128 + 32 i of e, wn * 128 + 32 j of d_kv
#define GR_FRAG(buf, base, w, i, s)                                                            \
  join(read_tr(&(buf)[(base) + (s) * 16 * kRow + (((w) * 256 + (i) * 64) ^ tr_x)]),            \
       read_tr(&(buf)[(base) + ((s) * 16 + 4) * kRow + (((w) * 256 + (i) * 64) ^ tr_x)]))
#define GR_FRAGS(st, s, fa, fb)                                                                \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) fa[i] = GR_FRAG(GR_E(st), a_base, wk, i, s);   \
  _Pragma("unroll") for (int j = 0; j < 4; ++j) fb[j] = GR_FRAG(GR_D(st), b_base, wn, j, s);
#define GR_MFMA(fa, fb)                                                                        \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) _Pragma("unroll") for (int j = 0; j < 4; ++j)  \
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
#define GR_FENCE() __builtin_amdgcn_sched_barrier(0)
#define GR_GROUP(mask, n) __builtin_amdgcn_sched_group_barrier(mask, n, 0)
// 16 MFMAs, a fragment's read behind each, and between them the conversion of two rows
#define GR_MIX()                                                                               \
  _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) {                                          \
    GR_GROUP(0x008, 1); GR_GROUP(0x100, 1); GR_GROUP(0x002, 6);                                \
    if (g_ % 4 == 3) GR_GROUP(0x200, 1);                                                       \
  }                                                                                            \
  GR_FENCE();
#define GR_STEP(kt_, P, Q)                                                                     \
  {                                                                                            \
    GR_FRAGS(P, 1, fa1, fb1)                                                                   \
    GR_MFMA(fa0, fb0)                                                                          \
    _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) { GR_GROUP(0x008, 1); GR_GROUP(0x100, 1); } \
    GR_FENCE();                                                                                \
    GR_FRAGS(P, 2, fa0, fb0)                                                                   \
    GR_WRITE(Q, 0)                                                                             \
    GR_WRITE(Q, 1)                                                                             \
    GR_MFMA(fa1, fb1)                                                                          \
    GR_MIX()                                                                                   \
    GR_FRAGS(P, 3, fa1, fb1)                                                                   \
    GR_WRITE(Q, 2)                                                                             \
    GR_WRITE(Q, 3)                                                                             \
    GR_MFMA(fa0, fb0)                                                                          \
    GR_MIX()                                                                                   \
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");                   \
    GR_FENCE();                                                                                \
    GR_FRAGS(Q, 0, fa0, fb0)                                                                   \
    GR_LOAD((kt_) + 2, P)                                                                      \
    GR_MFMA(fa1, fb1)                                                                          \
    _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) {                                        \
      GR_GROUP(0x008, 1); GR_GROUP(0x100, 2); GR_GROUP(0x020, 2);                              \
    }                                                                                          \
    GR_FENCE();                                                                                \
  }
  f32x16 acc[4][4];
  bf16x8 fa0[4], fb0[4], fa1[4], fb1[4];
  zero_acc(acc);
  if (steps > 0) {
    GR_LOAD(0, 0)
    GR_WRITE(0, 0)
    GR_WRITE(0, 1)
    GR_WRITE(0, 2)
    GR_WRITE(0, 3)
    GR_LOAD(1, 1)
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    GR_FENCE();
    GR_FRAGS(0, 0, fa0, fb0)
    for (int kt = 0; kt < steps; kt += 2) {
      GR_STEP(kt, 0, 1)
      GR_STEP(kt + 1, 1, 0)
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  uint8_t *patch = out + wave * kPatch;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; i += F32 || ADD ? 1 : 2)
      store_patch<F32, ADD, F32 || ADD ? 32 : 64>(acc[i][j], acc[i + (F32 || ADD ? 0 : 1)][j], patch, grad, op.N,
                                                  op.K, n0 + wn * 128 + j * 32, k0 + wk * 128 + i * 32, lane);
#undef GR_STEP
#undef GR_MIX
#undef GR_GROUP
#undef GR_FENCE
#undef GR_MFMA
#undef GR_FRAGS
#undef GR_FRAG
#undef GR_WRITE
#undef GR_LOAD
#undef GR_E
#undef GR_D
}

// The splits' parts, summed in order.
template <bool F32>
__global__ __launch_bounds__(256) void grad_join_kernel(const float *__restrict__ part, int splits,
                                                        void *__restrict__ grad, int accumulate, int64_t quads) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (q >= quads) return;
  float4 v = reinterpret_cast<const float4 *>(part)[q];
  for (int s = 1; s < splits; ++s) {
    const float4 o = reinterpret_cast<const float4 *>(part)[s * quads + q];
    v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
  }
  if (F32) {
    float4 *p = reinterpret_cast<float4 *>(grad) + q;
    if (accumulate) {
      const float4 o = *p;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *p = v;
  } else {
    uint2 *p = reinterpret_cast<uint2 *>(grad) + q;
    if (accumulate) {
      const uint2 o = *p;
      v = make_float4(v.x + engram::bf16_to_f32(o.x & 0xFFFFu), v.y + engram::bf16_to_f32(o.x >> 16),
                      v.z + engram::bf16_to_f32(o.y & 0xFFFFu), v.w + engram::bf16_to_f32(o.y >> 16));
    }
    *p = make_uint2(engram::pack_bf16x2(v.x, v.y), engram::pack_bf16x2(v.z, v.w));
  }
}

// How many parts the tokens are split into: as many as fit the CUs beside each other, each
// of at least 256 tokens.
int grad_splits(int64_t t, int64_t n, int64_t k, int cus) {
  const int64_t tiles = ((n + kTile - 1) / kTile) * ((k + kTile - 1) / kTile);
  const int64_t most = (t + 255) / 256, fit = cus / tiles;
  const int64_t s = most < fit ? most : fit;
  return (int)(s > 1 ? s : 1);
}

}  // namespace

size_t engram_gemm_grad_workspace(int64_t t, int64_t n, int64_t k) {
  int cus = 0;
  if (cu_count(cus) != hipSuccess) {
    (void)hipGetLastError();
    return 0;
  }
  const int s = grad_splits(t, n, k, cus);
  return s > 1 ? (size_t)s * n * k * sizeof(float) : 0;
}

hipError_t engram_launch_gemm_grad(const uint16_t *d_kv, const int8_t *e_codes, const float *e_scales,
                                   bool f32, void *grad, int accumulate, int64_t t, int64_t n,
                                   int64_t k, float *workspace, hipStream_t stream) {
  const GradOperands op{d_kv, e_codes, e_scales, (int)t, (int)n, (int)k};
  const int tiles_n = (int)((n + kTile - 1) / kTile), tiles_k = (int)((k + kTile - 1) / kTile);
  const int tiles = tiles_n * tiles_k;
  int cus = 0;
  const hipError_t err = cu_count(cus);
  if (err != hipSuccess) return err;
  const int splits = workspace != nullptr ? grad_splits(t, n, k, cus) : 1;
  // whole steps a split
  const int per = (int)(((t + splits - 1) / splits + kStep - 1) / kStep * kStep);
  if (splits > 1) {
    hipLaunchKernelGGL((grad_kernel<true, false>), dim3((unsigned)(tiles * splits)), dim3(256), 0, stream, op,
                       workspace, tiles_n, tiles_k, tiles, per);
    const int64_t quads = n * k / 4;
    const dim3 grid((unsigned)((quads + 255) / 256));
    if (f32)
      hipLaunchKernelGGL((grad_join_kernel<true>), grid, dim3(256), 0, stream, workspace, splits, grad,
                         accumulate, quads);
    else
      hipLaunchKernelGGL((grad_join_kernel<false>), grid, dim3(256), 0, stream, workspace, splits, grad,
                         accumulate, quads);
  } else {
#define ENGRAM_GRAD(F, A)                                                                       \
  hipLaunchKernelGGL((grad_kernel<F, A>), dim3((unsigned)tiles), dim3(256), 0, stream, op, grad, \
                     tiles_n, tiles_k, tiles, per)
    if (f32 && accumulate) ENGRAM_GRAD(true, true);
    else if (f32) ENGRAM_GRAD(true, false);
    else if (accumulate) ENGRAM_GRAD(false, true);
    else ENGRAM_GRAD(false, false);
#undef ENGRAM_GRAD
  }
  return hipGetLastError();
}
