// Step 4 with 8-bit integer operands: kv[t, c] = s_t s_c sum_k e[t, k] W[c, k]. The sum is
// exact in 32 bits (in_dim < 2^17 codes of at most 128); it is converted to fp32, scaled
// by the channel, then by the token, and rounded to kv's type.
//
// Few tokens are bound by W's stream: 1 token against 25600 rows of 6144 takes 27 us (5.8
// TB/s), 256 tokens 52 us, of which the loads alone take about 40. Many tokens are bound by
// power: 32768 tokens take 4.5 ms, 2.3 POPS at 1.8-2.0 GHz with the matrix units 53-59 % busy.
// The same kernel without its loads reaches 3.1 POPS, MFMAs alone 3.3 (4.3 where every code
// is zero), and with all loads served by L2 2.5; a ring of four half steps, a deeper prefetch,
// was no faster.
//
// v_mfma_i32_32x32x32_i8 takes 16 bytes a lane: lane l holds row l % 32, inputs [16 h, 16 h +
// 16) of the 32 for its half h = l / 32. A sum over the inputs may take them in any order
// that both operands share: of the 128 inputs of a K-step, half h of a wave takes 16-byte
// chunk 4 h + s in MFMA s.
//
// Both operands go global -> LDS by direct loads, 128 bytes (a cache line) of a row at a
// time; chunk c of a row sits in slot c ^ f(row), so that the 8 rows a quarter-wave reads
// fall into 8 different slots of 128 bytes. Inputs behind the last one are zeros of W (loads
// from an offset behind the buffer), whatever e's chunk holds there.
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

constexpr int kStep = 128;                 // inputs, and bytes of a row, per K-step
constexpr int kPatch = 4096;               // LDS of a wave for storing part of its tile
constexpr int kBehind = (int)0x80000000u;  // an offset behind every operand panel

__device__ __forceinline__ i32x16 mfma_i8(i32x4 w, i32x4 e, i32x16 acc) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(w, e, acc, 0, 0, 0);
}

// Stores 32 tokens x COLS columns (one or two accumulators) of a wave in whole cache lines:
// a lane's accumulators are 4 columns of one token at a time, so they pass through LDS
// (16-byte chunk c of token t in slot c ^ t % chunks). ws points at the columns' scales,
// es is this lane's token's.
template <bool F32, int COLS>
__device__ __forceinline__ void store_patch(const i32x16 &a0, const i32x16 &a1, const float *ws, float es,
                                            uint8_t *patch, void *__restrict__ kv, int M, int N, int m,
                                            int n, int lane) {
  constexpr int kRow = COLS * (F32 ? 4 : 2), kChunks = kRow / 16;
  const int frow = lane & 31, fk = lane >> 5;
#pragma unroll
  for (int i = 0; i < COLS / 32; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const i32x16 &a = i ? a1 : a0;
      const float4 s = *reinterpret_cast<const float4 *>(ws + i * 32 + g * 8 + fk * 4);
      const float f[4] = {(float)a[g * 4] * s.x * es, (float)a[g * 4 + 1] * s.y * es,
                          (float)a[g * 4 + 2] * s.z * es, (float)a[g * 4 + 3] * s.w * es};
      if (F32) {
        *reinterpret_cast<float4 *>(patch + frow * kRow + (((i * 8 + g * 2 + fk) ^ (frow & (kChunks - 1))) << 4)) =
            make_float4(f[0], f[1], f[2], f[3]);
      } else {
        *reinterpret_cast<uint2 *>(patch + frow * kRow + (((i * 4 + g) ^ (frow & (kChunks - 1))) << 4) + fk * 8) =
            make_uint2(engram::pack_bf16x2(f[0], f[1]), engram::pack_bf16x2(f[2], f[3]));
      }
    }
  const int c = lane % kChunks, col = n + c * (F32 ? 4 : 8);
#pragma unroll
  for (int q = 0; q < 32 * kChunks / 64; ++q) {
    const int t = (q * 64 + lane) / kChunks;
    const engram::u32x4 v =
        *reinterpret_cast<const engram::u32x4 *>(patch + t * kRow + ((c ^ (t & (kChunks - 1))) << 4));
    if (m + t < M && col < N) {
      if (F32)
        __builtin_nontemporal_store(v, reinterpret_cast<engram::u32x4 *>(
                                           reinterpret_cast<float *>(kv) + (int64_t)(m + t) * N + col));
      else
        __builtin_nontemporal_store(v, reinterpret_cast<engram::u32x4 *>(
                                           reinterpret_cast<uint16_t *>(kv) + (int64_t)(m + t) * N + col));
    }
  }
}

#define I8_LDS(p) ((__attribute__((address_space(3))) void *)(p))
#define I8_CHUNK(buf, off, c, sw) (*reinterpret_cast<const i32x4 *>(&(buf)[(off) + (((c) ^ (sw)) << 4)]))
#define I8_FENCE() __builtin_amdgcn_sched_barrier(0)
#define I8_GROUP(mask, n) __builtin_amdgcn_sched_group_barrier(mask, n, 0)

// ---- many tokens: 256 x 256 tiles through LDS ---------------------------------------
// Four waves of 128 x 128 outputs, K-steps in two stages. One block per CU walks the tiles:
// the loads of the two steps behind a tile's last are the next tile's first two, so they
// are in flight while the finished tile is stored, and the stores while the next begins.
// An odd number of steps is rounded up with a step of zeros, so that a tile begins in
// stage 0.
template <bool F32>
__global__ __launch_bounds__(kWideThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void i8_wide_kernel(I8Operands op, void *__restrict__ kv, int tiles_m, int tiles_n) {
  // The stages are separate LDS variables: the compiler then knows that direct loads
  // into one and reads of another do not meet, and waits for nothing in between.
  __shared__ __align__(1024) uint8_t w0[BN * kStep], w1[BN * kStep];
  __shared__ __align__(1024) uint8_t e0[BM * kStep], e1[BM * kStep];
  __shared__ __align__(1024) uint8_t out[4 * kPatch];
  __shared__ __align__(16) float sc[2][BN + BM];          // the tile's scales, by its parity
  const int tiles = tiles_m * tiles_n;
  const int ke = ((op.K + kStep - 1) / kStep + 1) & ~1;
  const int ld = op.K;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wm = wave & 1;
  // direct load i of a wave fills 1 KB: 8 rows of 128 bytes (lane p: row p / 8, slot p % 8)
  const int dl_c = (lane & 7) ^ (lane >> 3);
  const int dl_row = (wave * 64 + (lane >> 3)) * ld;
  const int v0 = dl_row + dl_c * 16, v1 = dl_row + (dl_c ^ 1) * 16;
  const int frow = lane & 31, h = lane >> 5;
  const int fsw = (frow & 7) ^ ((frow >> 3) & 1);
  const int a_base = (wn * 128 + frow) * kStep, b_base = (wm * 128 + frow) * kStep;
  __amdgpu_buffer_rsrc_t rsW, rsE, rsS;
// The operands of tile t_, from which the loads come; behind the last tile nothing does.
// Waves 0 and 1 load W's scales, 2 and 3 e's.
#define I8_AIM(t_)                                                                             \
  {                                                                                            \
    const int at_ = (t_);                                                                      \
    int am_ = 0, an_ = 0;                                                                      \
    if (at_ < tiles) tile_origin_of(at_, tiles_m, tiles_n, BN, am_, an_);                      \
    const int rw_ = at_ < tiles ? min(BN, op.N - an_) : 0;                                     \
    const int re_ = at_ < tiles ? min(BM, op.M - am_) : 0;                                     \
    rsW = __builtin_amdgcn_make_buffer_rsrc(                                                   \
        const_cast<int8_t *>(op.w_codes + (int64_t)an_ * ld), 0, rw_ * ld, kBufferFlags);      \
    rsE = __builtin_amdgcn_make_buffer_rsrc(                                                   \
        const_cast<int8_t *>(op.e_codes + (int64_t)am_ * ld), 0, re_ * ld, kBufferFlags);      \
    rsS = wave < 2 ? __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(op.w_scales + an_), 0, \
                                                       rw_ * 4, kBufferFlags)                  \
                   : __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(op.e_scales + am_), 0, \
                                                       re_ * 4, kBufferFlags);                 \
  }
#define I8_W(st) ((st) ? w1 : w0)
#define I8_E(st) ((st) ? e1 : e0)
#define I8_LOADSTEP(kt_, st)                                                                   \
  {                                                                                            \
    const int left_ = op.K / 16 - (kt_) * 8;                                                   \
    const int wv0_ = dl_c < left_ ? v0 : kBehind, wv1_ = (dl_c ^ 1) < left_ ? v1 : kBehind;    \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds(    \
        rsW, I8_LDS(&I8_W(st)[(wave * 8 + i) * 1024]), 16, (i & 1) ? wv1_ : wv0_,              \
        i * 8 * ld + (kt_) * kStep, 0, 0);                                                     \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds(    \
        rsE, I8_LDS(&I8_E(st)[(wave * 8 + i) * 1024]), 16, (i & 1) ? v1 : v0,                  \
        i * 8 * ld + (kt_) * kStep, 0, 0);                                                     \
  }
#define I8_LOADS(par_)                                                                         \
  _Pragma("unroll") for (int i = 0; i < 2; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds(      \
      rsS, I8_LDS(&sc[par_][wave * 128 + i * 64]), 4, ((wave & 1) * 128 + lane) * 4, i * 256, 0, 0);
#define I8_FRAGS(st, s, fa, fb)                                                                \
  _Pragma("unroll") for (int i = 0; i < 4; ++i)                                                \
    fa[i] = I8_CHUNK(I8_W(st), a_base + i * 32 * kStep, 4 * h + (s), fsw);                     \
  _Pragma("unroll") for (int j = 0; j < 4; ++j)                                                \
    fb[j] = I8_CHUNK(I8_E(st), b_base + j * 32 * kStep, 4 * h + (s), fsw);
#define I8_MFMA(fa, fb)                                                                        \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) _Pragma("unroll") for (int j = 0; j < 4; ++j)  \
    acc[i][j] = mfma_i8(fa[i], fb[j], acc[i][j]);
#define I8_BARRIER() asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
// the first step of a tile: the stores of the one before may be outstanding, all of them
// (as many as the counter holds), as they were issued behind the loads
#define I8_BARRIER0()                                                                          \
  if (stores)                                                                                  \
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(F32 ? 63 : 32) : "memory"); \
  else                                                                                         \
    I8_BARRIER()
// 16 MFMAs with the next fragments' reads between the first of them
#define I8_PART(P, s, ra, rb, fa, fb)                                                          \
  I8_FRAGS(P, (s) + 1, ra, rb)                                                                 \
  I8_MFMA(fa, fb)                                                                              \
  _Pragma("unroll") for (int g_ = 0; g_ < 8; ++g_) { I8_GROUP(0x100, 1); I8_GROUP(0x008, 1); } \
  I8_FENCE();
// One step from stage P: its last fragments are read before the barrier, the next
// step's first ones (stage Q) behind it, while stage P takes step `ahead`. The LDS
// reads come before the new direct loads: the compiler, which cannot see the wait
// inside the barrier, puts a full vmcnt wait before them.
#define I8_STEP(ahead, P, Q, BARRIER, LOAD)                                                    \
  {                                                                                            \
    I8_PART(P, 0, fa1, fb1, fa0, fb0)                                                          \
    I8_PART(P, 1, fa0, fb0, fa1, fb1)                                                          \
    I8_PART(P, 2, fa1, fb1, fa0, fb0)                                                          \
    BARRIER                                                                                    \
    I8_FENCE();                                                                                \
    I8_FRAGS(Q, 0, fa0, fb0)                                                                   \
    I8_LOADSTEP(ahead, P)                                                                      \
    LOAD                                                                                       \
    I8_MFMA(fa1, fb1)                                                                          \
    _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) {                                        \
      I8_GROUP(0x008, 1); I8_GROUP(0x100, 2); I8_GROUP(0x020, 2);                              \
    }                                                                                          \
    I8_FENCE();                                                                                \
  }
  i32x16 acc[4][4];
  i32x4 fa0[4], fb0[4], fa1[4], fb1[4];
#define I8_ZERO()                                                                              \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) _Pragma("unroll") for (int j = 0; j < 4; ++j)  \
    _Pragma("unroll") for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  I8_ZERO()
  I8_AIM((int)blockIdx.x)
  I8_LOADS(0)
  I8_LOADSTEP(0, 0)
  I8_LOADSTEP(1, 1)
  I8_BARRIER()
  bool stores = false;                // a whole tile's stores were issued behind the loads
  int par = 0;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    // read again behind the stores, whose registers they would otherwise take
    I8_FRAGS(0, 0, fa0, fb0)
    for (int kt = 0; kt < ke; kt += 2) {
      int ahead = kt + 2, to = par;
      if (ahead >= ke) {              // the next tile's first steps
        I8_AIM(t + (int)gridDim.x)
        ahead = 0;
        to ^= 1;
      }
      I8_STEP(ahead, 0, 1, I8_BARRIER0(), I8_LOADS(to))
      stores = false;
      I8_STEP(ahead + 1, 1, 0, I8_BARRIER(), )
    }
    int m0, n0;
    tile_origin_of(t, tiles_m, tiles_n, BN, m0, n0);
    uint8_t *patch = out + wave * kPatch;
    // the lane through a swap with itself, which stays in the loop: addresses formed
    // from it are formed anew for each tile; kept over the K loop they spill
    const int l = __builtin_amdgcn_mov_dpp(lane, 0xE4, 0xF, 0xF, true);
    const float *ws = sc[par] + wn * 128, *es = sc[par] + BN + wm * 128 + (l & 31);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = es[j * 32];
      if (F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store_patch<true, 32>(acc[i][j], acc[i][j], ws + i * 32, s, patch, kv, op.M, op.N,
                                m0 + wm * 128 + j * 32, n0 + wn * 128 + i * 32, l);
      } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2)
          store_patch<false, 64>(acc[i][j], acc[i + 1][j], ws + i * 32, s, patch, kv, op.M, op.N,
                                 m0 + wm * 128 + j * 32, n0 + wn * 128 + i * 32, l);
      }
    }
    I8_ZERO()
    stores = m0 + BM <= op.M && n0 + BN <= op.N;
    par ^= 1;
  }
  // direct loads issued behind the last tile land before the block's LDS is freed
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#undef I8_ZERO
#undef I8_STEP
#undef I8_PART
#undef I8_BARRIER0
#undef I8_BARRIER
#undef I8_MFMA
#undef I8_FRAGS
#undef I8_LOADS
#undef I8_LOADSTEP
#undef I8_E
#undef I8_W
#undef I8_AIM
}

// ---- few blocks: small tiles, the operands streamed far ahead ------------------------
// A block of WV waves takes 64 MT tokens against 64 NB weight rows over the whole of K, two
// waves along the tokens and WV / 2 along the rows, so that a wave holds 32 MT x 32 NI
// outputs. Both operands go into a ring of R K-steps. The one barrier of a step stands before its last MFMAs: by then the step's
// slot has been read and takes the loads of step kt + R, and step kt + 1 has landed: of
// the loads issued, those of the R - 2 steps behind it may be outstanding. Every step
// issues the same number of loads, and steps are rounded up to a multiple of R with steps
// of zeros, so the count holds throughout.
//
// ONCE: one block holds all tokens, so that W's rows are read by one block alone and are
// marked nontemporal, which leaves L2 to e (1 token 30.4 -> 27.1 us, 256 tokens 55.5 -> 53.1;
// where two blocks share them 55.7 -> 57.7).
constexpr int kNontemporal = 2;            // of a buffer load's cache policy

template <int NB, int MT>
constexpr int ring_of() {
  return NB + MT <= 3 ? 6 : NB + MT <= 4 ? 4 : 3;
}

template <bool F32, int NB, int MT, int WV, bool ONCE>
__global__ __launch_bounds__(64 * WV) __attribute__((amdgpu_waves_per_eu(WV / 4, WV / 4)))
void i8_skinny_kernel(I8Operands op, void *__restrict__ kv, int tiles_n) {
  constexpr int NI = NB * 4 / WV;
  constexpr int R = ring_of<NB, MT>();
  constexpr int kRows = 64 * NB, kToks = 64 * MT;
  constexpr int kSlot = (kRows + kToks) * kStep;        // the W rows, then the e rows
  constexpr int kLW = kRows / 8 / WV, kLE = kToks / 8 / WV;
  constexpr int kLoads = kLW + kLE;                     // direct loads of a wave and step
  // one LDS variable per slot: the compiler tells direct loads into up to eight apart
  __shared__ __align__(1024) uint8_t s0[kSlot], s1[kSlot], s2[kSlot];
  __shared__ __align__(1024) uint8_t s3[R > 3 ? kSlot : 16], s4[R > 4 ? kSlot : 16], s5[R > 5 ? kSlot : 16];
  static_assert(R * kSlot <= 160 * 1024 && WV * kPatch <= kSlot, "LDS");
  // The token tiles of the same rows go to one XCD, eight row tiles at a time.
  const int tiles_m = (int)gridDim.x / tiles_n;
  const int ahead = (int)blockIdx.x / (8 * tiles_m) * 8, left = (int)blockIdx.x - ahead * tiles_m;
  const int wide = min(8, tiles_n - ahead);
  const int n0 = (ahead + left % wide) * kRows, m0 = left / wide * kToks;
  const int ld = op.K, steps = (op.K + kStep - 1) / kStep;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wm = wave & 1;
  const int frow = lane & 31, h = lane >> 5;
  const __amdgpu_buffer_rsrc_t rsW = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t *>(op.w_codes + (int64_t)n0 * ld), 0, min(kRows, op.N - n0) * ld, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsE = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t *>(op.e_codes + (int64_t)m0 * ld), 0, min(kToks, op.M - m0) * ld, kBufferFlags);
  const int dl_c = (lane & 7) ^ (lane >> 3);
  const int w_v0 = (wave * (kRows / WV) + (lane >> 3)) * ld + dl_c * 16;
  const int w_v1 = (wave * (kRows / WV) + (lane >> 3)) * ld + (dl_c ^ 1) * 16;
  const int e_v0 = (wave * (kToks / WV) + (lane >> 3)) * ld + dl_c * 16;
  const int e_v1 = (wave * (kToks / WV) + (lane >> 3)) * ld + (dl_c ^ 1) * 16;
  const int fsw = (frow & 7) ^ ((frow >> 3) & 1);
  const int a_base = (wn * 32 * NI + frow) * kStep, b_base = (kRows + wm * 32 * MT + frow) * kStep;
#define IK_SLOT(u) ((u) % R == 0 ? s0 : (u) % R == 1 ? s1 : (u) % R == 2 ? s2 : (u) % R == 3 ? s3 : (u) % R == 4 ? s4 : s5)
#define IK_LOAD(kt_, u)                                                                        \
  {                                                                                            \
    const int left_ = op.K / 16 - (kt_) * 8;                                                   \
    const int wv0_ = dl_c < left_ ? w_v0 : kBehind, wv1_ = (dl_c ^ 1) < left_ ? w_v1 : kBehind; \
    _Pragma("unroll") for (int i = 0; i < kLE; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds( \
        rsE, I8_LDS(&IK_SLOT(u)[kRows * kStep + (wave * kLE + i) * 1024]), 16,              \
        (i & 1) ? e_v1 : e_v0, i * 8 * ld + (kt_) * kStep, 0, 0);                              \
    _Pragma("unroll") for (int i = 0; i < kLW; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds( \
        rsW, I8_LDS(&IK_SLOT(u)[(wave * kLW + i) * 1024]), 16, (i & 1) ? wv1_ : wv0_,       \
        i * 8 * ld + (kt_) * kStep, 0, ONCE ? kNontemporal : 0);                               \
  }
#define IK_FRAGS(u, s, fa, fb)                                                                 \
  _Pragma("unroll") for (int i = 0; i < NI; ++i)                                               \
    fa[i] = I8_CHUNK(IK_SLOT(u), a_base + i * 32 * kStep, 4 * h + (s), fsw);                   \
  _Pragma("unroll") for (int j = 0; j < MT; ++j)                                               \
    fb[j] = I8_CHUNK(IK_SLOT(u), b_base + j * 32 * kStep, 4 * h + (s), fsw);
#define IK_MFMA(fa, fb)                                                                        \
  _Pragma("unroll") for (int i = 0; i < NI; ++i) _Pragma("unroll") for (int j = 0; j < MT; ++j) \
    acc[i][j] = mfma_i8(fa[i], fb[j], acc[i][j]);
#define IK_BARRIER()                                                                           \
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((R - 2) * kLoads) : "memory");
#define IK_MIX()                                                                               \
  _Pragma("unroll") for (int g_ = 0; g_ < NI + MT; ++g_) { I8_GROUP(0x100, 1); I8_GROUP(0x008, 1); } \
  I8_FENCE();
#define IK_STEP(u)                                                                             \
  {                                                                                            \
    IK_FRAGS(u, 1, fa1, fb1)                                                                   \
    IK_MFMA(fa0, fb0)                                                                          \
    IK_MIX()                                                                                   \
    IK_FRAGS(u, 2, fa0, fb0)                                                                   \
    IK_MFMA(fa1, fb1)                                                                          \
    IK_MIX()                                                                                   \
    IK_FRAGS(u, 3, fa1, fb1)                                                                   \
    IK_MFMA(fa0, fb0)                                                                          \
    IK_MIX()                                                                                   \
    IK_BARRIER()                                                                               \
    I8_FENCE();                                                                                \
    IK_FRAGS((u) + 1, 0, fa0, fb0)                                                             \
    I8_FENCE();                                                                                \
    IK_LOAD(kt + (u) + R, u)                                                                   \
    IK_MFMA(fa1, fb1)                                                                          \
    _Pragma("unroll") for (int g_ = 0; g_ < NI * MT; ++g_) { I8_GROUP(0x008, 1); I8_GROUP(0x020, 2); } \
    I8_FENCE();                                                                                \
  }
  i32x16 acc[NI][MT];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  i32x4 fa0[NI], fb0[MT], fa1[NI], fb1[MT];
  IK_LOAD(0, 0)
  I8_FENCE();
  IK_LOAD(1, 1)
  I8_FENCE();
  IK_LOAD(2, 2)
  I8_FENCE();
  if constexpr (R > 3) IK_LOAD(3, 3)
  I8_FENCE();
  if constexpr (R > 4) IK_LOAD(4, 4)
  I8_FENCE();
  if constexpr (R > 5) IK_LOAD(5, 5)
  I8_FENCE();
  // step 0 has landed when the R - 1 behind it are outstanding
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((R - 1) * kLoads) : "memory");
  I8_FENCE();
  IK_FRAGS(0, 0, fa0, fb0)
  for (int kt = 0; kt < steps; kt += R) {
    IK_STEP(0)
    IK_STEP(1)
    IK_STEP(2)
    if constexpr (R > 3) IK_STEP(3)
    if constexpr (R > 4) IK_STEP(4)
    if constexpr (R > 5) IK_STEP(5)
  }
  // every direct load has landed before a slot holds the outputs
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#undef IK_STEP
#undef IK_MIX
#undef IK_BARRIER
#undef IK_MFMA
#undef IK_FRAGS
#undef IK_LOAD
  __shared__ __align__(16) float sc[kRows + kToks];
  for (int x = tid; x < kRows + kToks; x += 64 * WV) {
    const int at = x < kRows ? n0 + x : m0 + x - kRows;
    sc[x] = at < (x < kRows ? op.N : op.M) ? (x < kRows ? op.w_scales : op.e_scales)[at] : 0.f;
  }
  __syncthreads();
  uint8_t *patch = s0 + wave * kPatch;
  constexpr int kCols = F32 || NI == 1 ? 32 : 64;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const float es = sc[kRows + wm * 32 * MT + j * 32 + frow];
#pragma unroll
    for (int i = 0; i < NI; i += kCols / 32)
      store_patch<F32, kCols>(acc[i][j], acc[i + kCols / 32 - 1][j], sc + wn * 32 * NI + i * 32, es, patch, kv,
                              op.M, op.N, m0 + wm * 32 * MT + j * 32, n0 + wn * 32 * NI + i * 32, lane);
  }
#undef IK_SLOT
}

template <bool F32, int NB, int MT, int WV>
hipError_t launch_skinny(const I8Operands &op, void *kv, hipStream_t stream) {
  const int tiles_n = (op.N + 64 * NB - 1) / (64 * NB), tiles_m = (op.M + 64 * MT - 1) / (64 * MT);
  const dim3 grid((unsigned)(tiles_n * tiles_m)), block(64 * WV);
  if (tiles_m == 1)
    hipLaunchKernelGGL((i8_skinny_kernel<F32, NB, MT, WV, true>), grid, block, 0, stream, op, kv, tiles_n);
  else
    hipLaunchKernelGGL((i8_skinny_kernel<F32, NB, MT, WV, false>), grid, block, 0, stream, op, kv, tiles_n);
  return hipGetLastError();
}

// The smallest tile whose blocks fit the CUs at once: a larger one leaves CUs idle and, at few
// tokens, multiplies padding. Where none fits, the blocks come in rounds, a round of whole 256 x
// 256 tiles as long as 1.3 to 1.9 of 128 x 256: those are taken where their rounds number up
// to 5 / 3 of the whole tiles' (us, 6144 inputs, 128 x 256 against 256 x 256; 1 round to 1:
// 300 x 20480 48, 73; 2 to 2: 128 x 66048 116, 172 and 600 x 25600 95, 146; 3 to 2: 768 x 25600
// 128, 153 and 4096 x 5120 158, 172; 2 to 1: 256 x 33024 96, 77 and 300 x 25600 76, 77; 4 to 2:
// 1003 x 25600 170, 156; 7 to 4: 2048 x 25600 362, 359). From 129 to 256 tokens they are 256
// tokens by 128 rows, as many blocks, so that W is read once.
template <bool F32>
hipError_t launch_i8(const I8Operands &op, void *kv, hipStream_t stream) {
  int cus = 0;
  const hipError_t err = cu_count(cus);
  if (err != hipSuccess) return err;
  const auto rounds = [&](int toks, int rows) {
    const int64_t blocks = ((int64_t)op.M + toks - 1) / toks * (((int64_t)op.N + rows - 1) / rows);
    return (blocks + cus - 1) / cus;
  };
  if (rounds(64, 64) == 1) return launch_skinny<F32, 1, 1, 4>(op, kv, stream);
  if (rounds(64, 128) == 1) return launch_skinny<F32, 2, 1, 4>(op, kv, stream);
  if (rounds(128, 128) == 1) return launch_skinny<F32, 2, 2, 8>(op, kv, stream);
  if (3 * rounds(128, 256) <= 5 * rounds(BM, BN))
    return op.M <= 256 && op.M > 128 ? launch_skinny<F32, 2, 4, 8>(op, kv, stream)
                                     : launch_skinny<F32, 4, 2, 8>(op, kv, stream);
  const int tiles_m = (op.M + BM - 1) / BM, tiles_n = (op.N + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  hipLaunchKernelGGL((i8_wide_kernel<F32>), dim3((unsigned)(tiles > cus ? cus : tiles)), dim3(kWideThreads),
                     0, stream, op, kv, tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t engram_launch_gemm_i8(const int8_t *w_codes, const float *w_scales, const int8_t *e_codes,
                                 const float *e_scales, bool f32, void *kv, int64_t m, int64_t n,
                                 int64_t k, hipStream_t stream) {
  if (m <= 0 || n <= 0) return hipSuccess;
  const I8Operands op{w_codes, w_scales, e_codes, e_scales, (int)m, (int)n, (int)k};
  return f32 ? launch_i8<true>(op, kv, stream) : launch_i8<false>(op, kv, stream);
}
