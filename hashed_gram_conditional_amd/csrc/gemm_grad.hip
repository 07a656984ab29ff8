// Gradient of the projection's weight from 8-bit codes of its inputs: dW[n, k] = sum_t
// d_kv[t, n] s_t q[t, k], in the bf16 MFMA with fp32 sums. s_t q[t, k] is rounded to bf16, as
// d_kv is: s_t belongs to the summed index, so it cannot wait for the sum. For codes near 127 the
// rounding reaches 0.49 of a code step, the quantiser's own half step; in the mean square of normal
// values whose largest is four standard deviations it is 0.05 of a step beside the quantiser's
// 0.29, and a gradient is 1.66e-3 of its norm away from that of the unrounded values (4096 and
// 32768 tokens; powers of two, whose products are bf16 numbers, 1e-7). FINE (ENGRAM_F32_FINE)
// takes two bf16 terms and twice the MFMAs: 2.5e-6 (sums in fp32 throughout 1.1e-6 and 3.2e-6), in
// 19.3 ms where one term takes 9.25 (32768 x 25600 x 6144) and 378 us where it takes 229 (509 tokens).
//
// Both operands have the summed index outermost, the MFMA reads it innermost. The kernel turns
// them on the way through registers, where the codes have to pass anyway. Other ways measured
// at 32768 x 25600 x 6144: LDS reads that transpose (ds_read_b64_tr_b16; half the rate of
// 16-byte reads, 2650 cycles of LDS a step beside 2048 of the MFMAs) 10.0 ms; the codes scaled
// and turned by a launch before, direct loads of them here, 10.0 ms; this 9.1-9.5 ms, 1.09-1.13
// PFLOP/s. Power and stalls bound it together: the clock falls to 1.7-1.8 GHz, and the matrix units
// are busy 59 % of that; with codes and gradients of zero the same kernel takes 7.5 ms, and MFMAs
// with LDS reads alone 6.3 ms. 509 tokens take 223-230 us into fp32 (629 MB of gradients; 240 to 280
// in the first hundred passes after idling), of which each of the ten rounds of tiles spends 13 us
// in its eight steps and 10 us in its first loads and its stores; one block
// per CU that walks the tiles with the next one's loads ahead saved 2 % there and lost 9 %
// in the long sum, whose addresses it had to form anew in every step.
#include <type_traits>

#include "gemm_tiles.h"

using namespace engram_gemm;

namespace {

struct GradOperands {
  const uint16_t *d_kv;      // [T, N] bf16
  const int8_t *e_codes;     // [T, K]
  const float *e_scales;     // [T]
  int T, N, K;
};

// Tokens per step, whose values of a column fill a row of LDS. FINE: half as many, each of e's
// values as two bf16 numbers.
template <bool FINE>
constexpr int kStep = FINE ? 32 : 64;
constexpr int kTile = 256;                // columns of either operand
constexpr int kRow = 128;                 // bytes of a column in LDS
constexpr int kPatch = 4096;              // LDS of a wave for storing part of its tile

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

// Two scaled values, as pairs of bf16 numbers: their roundings, and the roundings of what those
// drop, in all within 2^-17 of the value. A rounding that is not finite has nothing beside it.
__device__ __forceinline__ void two_terms(float a, float b, uint32_t &high, uint32_t &low) {
#pragma clang fp contract(off)      // a and b are the rounded products
  high = engram::pack_bf16x2(a, b);
  const float x = a - __uint_as_float(high << 16), y = b - __uint_as_float(high & 0xFFFF0000u);
  low = engram::pack_bf16x2(fabsf(x) < INFINITY ? x : 0.f, fabsf(y) < INFINITY ? y : 0.f);
}

// Word `at` of a register set, which is a constant where it is unrolled.
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int at) {
  return at == 0 ? v.x : at == 1 ? v.y : at == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t word_of(const uint2 &v, int at) { return at == 0 ? v.x : v.y; }
__device__ __forceinline__ uint32_t word_of(uint32_t v, int) { return v; }

__device__ __forceinline__ uint2 load8(__amdgpu_buffer_rsrc_t rs, int voff, int soff) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, voff, soff, 0);
  return make_uint2((uint32_t)v[0], (uint32_t)v[1]);
}

// Tile `bid`: each XCD takes a contiguous range of tiles, in groups of 2 tiles of d_kv's
// columns by all of e's, so that its 32 blocks share 2 panels of d_kv and 16 of codes. By the
// bytes alone 4 by 8 would be less to read (512 bytes of d_kv a token and 256 of codes), but
// measured 2 is ahead or within 1 % (tokens x d_kv's columns x e's, us in groups of 1, 2, 4 and 8):
// 32768 x 25600 x 6144 9190, 9130, 9290, 9580; 32768 x 5120 x 6144 1771, 1755, 1760, 1796; 8192 x
// 8192 x 8192 926, 912, 915, 922; 16384 x 25600 x 1024 815, 825, 832, 841; 16384 x 1536 x 6144 386,
// 384, 388, 390; 16384 x 1024 x 25600 830, 822, 827, 827.
constexpr int kGroupN = 2;

__device__ __forceinline__ void grad_tile(int bid, int tiles_n, int tiles_k, int &n0, int &k0) {
  const int full = tiles_n * tiles_k / kXcds * kXcds;
  if (bid < full) bid = (bid % kXcds) * (full / kXcds) + bid / kXcds;
  const int group = bid / (kGroupN * tiles_k);
  const int size = min(tiles_n - group * kGroupN, kGroupN);
  const int local = bid - group * kGroupN * tiles_k;
  n0 = (group * kGroupN + local % size) * kTile;
  k0 = local / size * kTile;
}

// A block sums the tokens [split * per, (split + 1) * per) of one 256 x 256 tile (four waves
// of 128 x 128) in steps of 64, two stages. LDS holds a step as the MFMA reads it, the tokens
// innermost: column c is a row of 128 bytes, tokens 8 g .. 8 g + 7 its chunk g, in slot g ^ f(c).
// Both operands are turned on the way through registers: a thread loads 8 columns of 8 tokens
// of each, and pairs of neighbouring tokens meet in one byte permutation (d_kv) or in the
// rounding of two scaled codes to bf16 (e). A register set is requested again, for the step
// after next, as soon as it is written to LDS, so that its loads have a whole step.
//
// FINE: a step is 32 tokens, chunks 0 to 3 of d_kv's columns, and of e's the four chunks of the
// first terms and the four of the second. A thread loads 4 columns of 8 tokens.
template <bool F32, bool ADD, bool FINE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grad_kernel(GradOperands op, void *__restrict__ grad, int tiles_n, int tiles_k,
                 int tiles, int per) {
  __shared__ __align__(1024) uint8_t d0[kTile * kRow], d1[kTile * kRow];
  __shared__ __align__(1024) uint8_t e0[kTile * kRow], e1[kTile * kRow];
  __shared__ __align__(1024) uint8_t out[4 * kPatch];
  const int split = (int)blockIdx.x / tiles;
  int n0, k0;
  grad_tile((int)blockIdx.x - split * tiles, tiles_n, tiles_k, n0, k0);
  const int t_first = split * per, t_last = min(op.T, t_first + per);
  constexpr int kTokens = kStep<FINE>;
  const int steps = ((t_last - t_first + kTokens - 1) / kTokens + 1) & ~1;  // a step of zeros if odd
  if (gridDim.x > (unsigned)tiles) grad = reinterpret_cast<float *>(grad) + (int64_t)split * op.N * op.K;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave >> 1, wn = wave & 1;
  // a thread's 8 tokens (group) and 8 (FINE: 4) columns
  constexpr int kCols = FINE ? 4 : 8;
  const int tg = tid / (kTile / kCols), tc = tid % (kTile / kCols);
  const int d_v = tg * 8 * op.N * 2 + tc * kCols * 2, e_v = tg * 8 * op.K + tc * kCols;
  // f(c) = (c ^ c / 8) % 8: a thread's columns, and eight threads' columns of the same number,
  // lie in different slots
  const int w_base = tc * kCols * kRow, w_x = FINE ? tg ^ (tc & 1) * 4 ^ (tc >> 1 & 7) : tg ^ (tc & 7);
  const int frow = lane & 31, h = lane >> 5;
  const int a_base = (wk * 128 + frow) * kRow, b_base = (wn * 128 + frow) * kRow;
  const int f_x = (frow ^ frow >> 3) & 7;
#define GR_D(st) ((st) ? d1 : d0)
#define GR_E(st) ((st) ? e1 : e0)
  std::conditional_t<FINE, uint2, uint4> dv[8];
  std::conditional_t<FINE, uint32_t, uint2> ev[8];
  float4 sv[2];
// Rows behind the last token are zeros.
#define GR_ROWS(kt_)                                                                           \
    const int t_ = t_first + (kt_) * kTokens;                                                  \
    const int rows_ = t_ >= t_last ? 0 : t_last - t_ < kTokens ? t_last - t_ : kTokens;        \
    const int64_t at_ = rows_ > 0 ? t_ : 0;
// requests d_kv of step kt_, or its codes and scales
#define GR_LOADD(kt_)                                                                          \
  {                                                                                            \
    GR_ROWS(kt_)                                                                               \
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(                       \
        const_cast<uint16_t *>(op.d_kv + at_ * op.N + n0), 0,                                  \
        rows_ > 0 ? (rows_ * op.N - n0) * 2 : 0, kBufferFlags);                                \
    _Pragma("unroll") for (int r = 0; r < 8; ++r) {                                            \
      if constexpr (FINE) dv[r] = load8(rs, d_v, r * op.N * 2);                                \
      else dv[r] = load16(rs, d_v, r * op.N * 2);                                              \
    }                                                                                          \
  }
#define GR_LOADE(kt_)                                                                          \
  {                                                                                            \
    GR_ROWS(kt_)                                                                               \
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(                       \
        const_cast<int8_t *>(op.e_codes + at_ * op.K + k0), 0, rows_ > 0 ? rows_ * op.K - k0 : 0, \
        kBufferFlags);                                                                         \
    const __amdgpu_buffer_rsrc_t rsS = __builtin_amdgcn_make_buffer_rsrc(                      \
        const_cast<float *>(op.e_scales + at_), 0, rows_ * 4, kBufferFlags);                   \
    _Pragma("unroll") for (int r = 0; r < 8; ++r) {                                            \
      if constexpr (FINE) ev[r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, e_v, r * op.K, 0); \
      else ev[r] = load8(rs, e_v, r * op.K);                                                   \
    }                                                                                          \
    _Pragma("unroll") for (int r = 0; r < 2; ++r)                                              \
      sv[r] = __builtin_bit_cast(float4, load16(rsS, tg * 32, r * 16));                        \
  }
#define GR_AT(buf, j, x) (*reinterpret_cast<uint4 *>(&(buf)[w_base + (j) * kRow + ((w_x ^ (j) ^ (x)) << 4)]))
// column j of d_kv: the low or high halves of word j / 2 of the 8 tokens, in pairs
#define GR_PAIR(r, j)                                                                          \
  __builtin_amdgcn_perm(word_of(dv[(r) + 1], (j) / 2), word_of(dv[r], (j) / 2), (j) & 1 ? 0x07060302u : 0x05040100u)
#define GR_WRITED(st)                                                                          \
  _Pragma("unroll") for (int j = 0; j < kCols; ++j)                                            \
    GR_AT(GR_D(st), j, 0) = make_uint4(GR_PAIR(0, j), GR_PAIR(2, j), GR_PAIR(4, j), GR_PAIR(6, j));
// columns 4 q .. 4 q + 3 of e; FINE: both terms of columns 2 q and 2 q + 1
#define GR_CODE(r, c) ((float)(int8_t)(word_of(ev[r], (c) / 4) >> (8 * ((c) & 3))))
#define GR_VALUE(r, j) (GR_CODE(r, j) * ((r) % 4 == 0 ? sv[(r) / 4].x : (r) % 4 == 1 ? sv[(r) / 4].y : \
                                         (r) % 4 == 2 ? sv[(r) / 4].z : sv[(r) / 4].w))
#define GR_WRITEE(st, q)                                                                       \
  if constexpr (FINE) {                                                                        \
    _Pragma("unroll") for (int j = 2 * (q); j < 2 * (q) + 2; ++j) {                            \
      uint4 high_, low_;                                                                       \
      two_terms(GR_VALUE(0, j), GR_VALUE(1, j), high_.x, low_.x);                              \
      two_terms(GR_VALUE(2, j), GR_VALUE(3, j), high_.y, low_.y);                              \
      two_terms(GR_VALUE(4, j), GR_VALUE(5, j), high_.z, low_.z);                              \
      two_terms(GR_VALUE(6, j), GR_VALUE(7, j), high_.w, low_.w);                              \
      GR_AT(GR_E(st), j, 0) = high_;                                                           \
      GR_AT(GR_E(st), j, 4) = low_;                                                            \
    }                                                                                          \
  } else {                                                                                     \
    _Pragma("unroll") for (int j = 4 * (q); j < 4 * (q) + 4; ++j)                              \
      GR_AT(GR_E(st), j, 0) = make_uint4(engram::pack_bf16x2(GR_VALUE(0, j), GR_VALUE(1, j)),  \
                                         engram::pack_bf16x2(GR_VALUE(2, j), GR_VALUE(3, j)),  \
                                         engram::pack_bf16x2(GR_VALUE(4, j), GR_VALUE(5, j)),  \
                                         engram::pack_bf16x2(GR_VALUE(6, j), GR_VALUE(7, j))); \
  }
// fragments s of a step: half h of a wave takes tokens 8 (4 h + s) .. + 7; FINE: tokens 8 (2 (s / 2)
// + h) .. + 7, of e the first terms where s is even, the second where it is odd
#define GR_FRAG(buf, base, i, c)                                                               \
  (*reinterpret_cast<const bf16x8 *>(&(buf)[(base) + (i) * 32 * kRow + (((c) ^ f_x ^ ((i) * 4 & 7)) << 4)]))
#define GR_FRAGS(st, s, fa, fb)                                                                \
  _Pragma("unroll") for (int i = 0; i < 4; ++i)                                                \
    fa[i] = GR_FRAG(GR_E(st), a_base, i, FINE ? (s) % 2 * 4 + (s) / 2 * 2 + h : 4 * h + (s));  \
  _Pragma("unroll") for (int j = 0; j < 4; ++j)                                                \
    fb[j] = GR_FRAG(GR_D(st), b_base, j, FINE ? (s) / 2 * 2 + h : 4 * h + (s));
#define GR_MFMA(fa, fb)                                                                        \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) _Pragma("unroll") for (int j = 0; j < 4; ++j)  \
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
#define GR_FENCE() __builtin_amdgcn_sched_barrier(0)
#define GR_GROUP(mask, n) __builtin_amdgcn_sched_group_barrier(mask, n, 0)
// 16 MFMAs, between the first of them the next fragments' reads, and V vector instructions
// and the LDS writes that they lead to, one per W MFMAs
#define GR_MIX(V, W)                                                                           \
  _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) {                                          \
    GR_GROUP(0x008, 1);                                                                        \
    if (g_ < 8) GR_GROUP(0x100, 1);                                                            \
    GR_GROUP(0x002, V);                                                                        \
    if (g_ % (W) == (W) - 1) GR_GROUP(0x200, 1);                                               \
  }                                                                                            \
  GR_FENCE();
#define GR_STEP(kt_, P, Q)                                                                     \
  {                                                                                            \
    GR_FRAGS(P, 1, fa1, fb1)                                                                   \
    GR_WRITED(Q)                                                                               \
    GR_MFMA(fa0, fb0)                                                                          \
    GR_MIX(2, 2)                                                                               \
    GR_LOADD((kt_) + 2)                                                                        \
    GR_FRAGS(P, 2, fa0, fb0)                                                                   \
    GR_WRITEE(Q, 0)                                                                            \
    GR_MFMA(fa1, fb1)                                                                          \
    GR_MIX(6, 4)                                                                               \
    GR_FRAGS(P, 3, fa1, fb1)                                                                   \
    GR_WRITEE(Q, 1)                                                                            \
    GR_MFMA(fa0, fb0)                                                                          \
    GR_MIX(6, 4)                                                                               \
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");                            \
    GR_FENCE();                                                                                \
    GR_LOADE((kt_) + 2)                                                                        \
    GR_FRAGS(Q, 0, fa0, fb0)                                                                   \
    GR_MFMA(fa1, fb1)                                                                          \
    _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) {                                        \
      GR_GROUP(0x008, 1); GR_GROUP(0x100, 1); GR_GROUP(0x020, 1);                              \
    }                                                                                          \
    GR_FENCE();                                                                                \
  }
  f32x16 acc[4][4];
  bf16x8 fa0[4], fb0[4], fa1[4], fb1[4];
  zero_acc(acc);
  if (steps > 0) {
    GR_LOADD(0)
    GR_LOADE(0)
    GR_WRITED(0)
    GR_LOADD(1)
    GR_WRITEE(0, 0)
    GR_WRITEE(0, 1)
    GR_LOADE(1)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    GR_FENCE();
    GR_FRAGS(0, 0, fa0, fb0)
    for (int kt = 0; kt < steps; kt += 2) {
      GR_STEP(kt, 0, 1)
      GR_STEP(kt + 1, 1, 0)
    }
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
#undef GR_VALUE
#undef GR_CODE
#undef GR_PAIR
#undef GR_AT
#undef GR_WRITEE
#undef GR_WRITED
#undef GR_LOADE
#undef GR_LOADD
#undef GR_ROWS
#undef GR_FENCE
#undef GR_MFMA
#undef GR_FRAGS
#undef GR_FRAG
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
// of at least 256 tokens, so that only up to half as many tiles as CUs are split. Split and
// whole (us, fp32, tokens x e's columns x d_kv's, parts): 512 x 1024 x 1024, 2: 20, 20; 600 x 512 x
// 512, 3: 18, 22; 1024 x 1024 x 1024, 4: 22, 30; 4096 x 1024 x 1024, 16: 37, 91; 4096 x 2048 x 4096,
// 2: 91, 100; 8192 x 6144 x 1024, 2: 123, 175; 32768 x 1536 x 2560, 4: 266, 748. Above half, tiles
// of 129 to 255, whole: 4096 x 6144 x 1536 (144 tiles) 95, 32768 x 6144 x 1536 750, 32768 x 4096 x
// 2560 (160) 756, with the other CUs idle.
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
                                   bool f32, bool fine, void *grad, int accumulate, int64_t t, int64_t n,
                                   int64_t k, float *workspace, hipStream_t stream) {
  const GradOperands op{d_kv, e_codes, e_scales, (int)t, (int)n, (int)k};
  const int tiles_n = (int)((n + kTile - 1) / kTile), tiles_k = (int)((k + kTile - 1) / kTile);
  const int tiles = tiles_n * tiles_k;
  int cus = 0;
  const hipError_t err = cu_count(cus);
  if (err != hipSuccess) return err;
  const int splits = workspace != nullptr ? grad_splits(t, n, k, cus) : 1;
  // whole steps a split
  const int per = (int)(((t + splits - 1) / splits + 63) / 64 * 64);
  if (splits > 1) {
    const dim3 blocks((unsigned)(tiles * splits));
    if (fine)
      hipLaunchKernelGGL((grad_kernel<true, false, true>), blocks, dim3(256), 0, stream, op, workspace, tiles_n,
                         tiles_k, tiles, per);
    else
      hipLaunchKernelGGL((grad_kernel<true, false, false>), blocks, dim3(256), 0, stream, op, workspace, tiles_n,
                         tiles_k, tiles, per);
    const int64_t quads = n * k / 4;
    const dim3 grid((unsigned)((quads + 255) / 256));
    if (f32)
      hipLaunchKernelGGL((grad_join_kernel<true>), grid, dim3(256), 0, stream, workspace, splits, grad,
                         accumulate, quads);
    else
      hipLaunchKernelGGL((grad_join_kernel<false>), grid, dim3(256), 0, stream, workspace, splits, grad,
                         accumulate, quads);
  } else {
#define ENGRAM_GRAD(F, A, X)                                                                       \
  hipLaunchKernelGGL((grad_kernel<F, A, X>), dim3((unsigned)tiles), dim3(256), 0, stream, op, grad, \
                     tiles_n, tiles_k, tiles, per)
    if (fine && accumulate) ENGRAM_GRAD(true, true, true);
    else if (fine) ENGRAM_GRAD(true, false, true);
    else if (f32 && accumulate) ENGRAM_GRAD(true, true, false);
    else if (f32) ENGRAM_GRAD(true, false, false);
    else if (accumulate) ENGRAM_GRAD(false, true, false);
    else ENGRAM_GRAD(false, false, false);
#undef ENGRAM_GRAD
  }
  return hipGetLastError();
}
