// Step 4 with the projection weight in 4-bit block floating point: kv = e W^T, W as
// E2M1 codes (two to a byte) and e as E2M1 or E4M3 codes, both with one E8M0
// scale per 32 consecutive inputs. v_mfma_scale_f32_32x32x64_f8f6f4 takes the two
// formats as they are, multiplies the codes exactly, applies both block scales and
// accumulates in fp32; kv is rounded once to bf16.
//
// With two E2M1 operands nothing is lost before fp32. With an E4M3 operand the instruction
// first adds the products of eight consecutive inputs in fixed point, the last place 2^-13
// of the largest product's power of two. That is taken as it is: 256 tokens x 25600 from
// 6144 normal inputs lie as far from the 64-bit product as fp32 sums rounded to bf16 do
// (1.6552e-3 of its norm, both), with 0.4 % of the values on the neighbour of the nearest
// bf16 (0.001 %). Sums without it need the bf16 instruction, at half the 8-bit rate and on
// four times W's bytes of LDS.
//
// Lane layout of that MFMA (measured on gfx950): lane l of half h = l / 32 holds
// row l % 32. Its 16 bytes of E2M1 are inputs [32 h, 32 h + 32) of the 64 in order;
// its 32 bytes of E4M3 are inputs [16 h, 16 h + 16) and [32 + 16 h, 48 + 16 h). The
// scale of inputs [32 h, 32 h + 32) comes from the lanes of half h, from one byte of
// a register that the instruction selects. That register must be a vector one: with a
// constant operand the upper half's blocks lost their scale.
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

// ---- many tokens: 256 x 256 tiles through LDS ---------------------------------------
// gemm_mx_kernel's tiles and two-stage schedule on the narrower operands. A K-step
// is 128 bytes of an e row: 256 inputs of E2M1 or 128 of E4M3, and 128 or 64 bytes of
// a W row. Both operands go global -> LDS by direct loads; 16-byte chunk c of a row
// sits in slot c ^ f(row), so the 8 rows a quarter-wave reads fall into 8 different
// slots of 128 bytes. Scales come for two K-steps at once (16 or 8 bytes of a row, half
// as many cache lines as one step at a time) and are kept in registers.
//
// One block per CU walks the tiles: the loads of the two steps behind a tile's last
// are the next tile's first two, so they are in flight while the finished tile is
// stored, and the stores while the next one begins (32768 x 1024 x 25600: 655 -> 560 us,
// with 6144 inputs 2.57 -> 2.55 ms: there power sets the clock, 1.76 GHz with the matrix
// units 54 % busy; an MFMA loop of nothing else reaches 6.4 PFLOP/s, with the LDS reads
// 6.0, this kernel 4.0). An odd number of K-steps costs that overlap (32768 x 25600 in us:
// E4M3 with 8, 9 and 10 steps 764, 911 and 895; E2M1 with 4, 5 and 6 steps 589, 757 and
// 754). The E4M3 instance keeps 17 registers in scratch memory and reads one of them, an
// LDS address, in every K-step, with a wait in front of 11 of its 12 direct loads.
template <int EF>
struct WideCfg {
  static constexpr int kStep = EF == kFp4 ? 256 : 128;      // inputs of a K-step
  static constexpr int kSub = kStep / 64;                   // MFMAs along K
  static constexpr int kWRow = kStep / 2;                   // bytes of a W row
  static constexpr int kERow = 128;                         // bytes of an e row
  static constexpr int kSc = kStep / 32;                    // scale bytes of a row
};

constexpr int kPatch = 4096;          // LDS of a wave for storing 32 tokens x 64 columns

// Stores 32 tokens (j) x 64 columns (accumulators i, i + 1) of a wave in whole cache
// lines. A lane's accumulators are 4 columns of one token at a time, 16 bytes of a
// line with its partner's: stored from the registers, a tile's 128 KB took 4 times as
// many write transactions as lines. So they pass through LDS (chunk c of token t in
// slot c ^ t % 8), and 8 lanes store 128 bytes of a token. The stores are marked
// nontemporal, so that kv does not push the operands' panels out of L2 (2.83 -> 2.57
// ms at 32768 x 6144 x 25600). GUARD: the tile passes the end of kv.
template <bool GUARD>
__device__ __forceinline__ void store_patch(const f32x16 &a0, const f32x16 &a1, uint8_t *patch,
                                            uint16_t *__restrict__ kv, int M, int N, int m, int n,
                                            int lane) {
  const int frow = lane & 31, fk = lane >> 5;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x16 &a = i ? a1 : a0;
      uint2 v;
      v.x = engram::pack_bf16x2(a[g * 4 + 0], a[g * 4 + 1]);
      v.y = engram::pack_bf16x2(a[g * 4 + 2], a[g * 4 + 3]);
      *reinterpret_cast<uint2 *>(patch + frow * 128 + (((i * 4 + g) ^ (frow & 7)) << 4) + fk * 8) = v;
    }
  const int col = n + (lane & 7) * 8;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int t = q * 8 + (lane >> 3);
    const engram::u32x4 v =
        *reinterpret_cast<const engram::u32x4 *>(patch + t * 128 + (((lane & 7) ^ (t & 7)) << 4));
    if (!GUARD || (m + t < M && col < N))
      __builtin_nontemporal_store(v, reinterpret_cast<engram::u32x4 *>(kv + (int64_t)(m + t) * N + col));
  }
}
constexpr int kTileStores = 32;       // store instructions of a wave and tile

// The tiles blockIdx.x, blockIdx.x + gridDim.x, ... of tiles_m x tiles_n. With an odd
// number of K-steps each block has one tile (the stages would change places).
template <int EF>
__device__ __forceinline__ void wide_walk(const Mx4Operands &op, uint16_t *__restrict__ kv, int tiles_m,
                                          int tiles_n) {
  using Cfg = WideCfg<EF>;
  constexpr int kSub = Cfg::kSub, kWRow = Cfg::kWRow, kSc = Cfg::kSc;
  constexpr int kWLoads = BN * kWRow / 1024 / 4;            // direct loads of a wave and step
  constexpr int kSLoads = (BN + BM) * 2 * kSc / 256 / 4;    // of a wave and two steps
  constexpr int kReads = EF == kFp4 ? 8 : 12;               // LDS reads of one set of fragments
  constexpr int kScBytes = (BN + BM) * 2 * kSc;
  // The stages are separate LDS variables: the compiler then knows that direct loads
  // into one and reads of another do not meet, and waits for nothing in between. (The
  // patches share the scales' variable: reads of one that no load meets would wait for
  // all of them.)
  __shared__ __align__(1024) uint8_t w0[BN * kWRow], w1[BN * kWRow];
  __shared__ __align__(1024) uint8_t e0[BM * Cfg::kERow], e1[BM * Cfg::kERow];
  __shared__ __align__(1024) uint8_t sc[kScBytes + 4 * kPatch];   // W rows, e rows; patches
  const int tiles = tiles_m * tiles_n;
  const int ke = (op.K + Cfg::kStep - 1) / Cfg::kStep;
  const int KB = op.K / 32;
  const int w_ld = op.K / 2, e_ld = EF == kFp4 ? op.K / 2 : op.K;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wm = wave & 1;
  // Direct load i of a wave fills 1 KB: 8 rows of 128 bytes (lane p: row p / 8, slot
  // p % 8) or 16 rows of 64 (row p / 4, slot p % 4).
  const int dl_c = (lane & 7) ^ (lane >> 3);
  const int dl_row = wave * 64 + (lane >> 3);
  const int e_v0 = dl_row * e_ld + dl_c * 16, e_v1 = dl_row * e_ld + (dl_c ^ 1) * 16;
  const int w_v0 = EF == kFp4 ? dl_row * w_ld + dl_c * 16
                              : (wave * 64 + (lane >> 2)) * w_ld + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
  const int w_v1 = EF == kFp4 ? dl_row * w_ld + (dl_c ^ 1) * 16 : w_v0;
  constexpr int kWInstRows = EF == kFp4 ? 8 : 16;
  // scale dword q of a row: 2 kSc / 4 dwords a row, 256 / (2 kSc) rows an instruction
  constexpr int kSRows = 256 / (2 * kSc);
  const int s_v = ((wave & 1) * 128 + lane / (64 / kSRows)) * KB + (lane % (64 / kSRows)) * 4;

  const int frow = lane & 31, h = lane >> 5;
  const int fsw = (frow & 7) ^ ((frow >> 3) & 1);
  const int a_base = (wn * 128 + frow) * kWRow, b_base = (wm * 128 + frow) * Cfg::kERow;
  const int a_sw = EF == kFp4 ? fsw : (frow >> 1) & 3;
  const int as_base = (wn * 128 + frow) * 2 * kSc + h * (kSc / 2);
  const int bs_base = (BN + wm * 128 + frow) * 2 * kSc + h * (kSc / 2);

  // The operands of tile t_, from which the loads come; behind the last tile nothing
  // does. Waves 0 and 1 load W's scales, 2 and 3 e's.
  __amdgpu_buffer_rsrc_t rsW, rsE, rsS;
#define M4_AIM(t_)                                                                             \
  {                                                                                            \
    const int at_ = (t_);                                                                      \
    int am_ = 0, an_ = 0;                                                                      \
    if (at_ < tiles) tile_origin_of(at_, tiles_m, tiles_n, BN, am_, an_);                      \
    const int rw_ = at_ < tiles ? min(BN, op.N - an_) : 0;                                     \
    const int re_ = at_ < tiles ? min(BM, op.M - am_) : 0;                                     \
    rsW = __builtin_amdgcn_make_buffer_rsrc(                                                   \
        const_cast<uint8_t *>(op.w_codes + (int64_t)an_ * w_ld), 0, rw_ * w_ld, kBufferFlags); \
    rsE = __builtin_amdgcn_make_buffer_rsrc(                                                   \
        const_cast<uint8_t *>(op.e_codes + (int64_t)am_ * e_ld), 0, re_ * e_ld, kBufferFlags); \
    rsS = wave < 2 ? __builtin_amdgcn_make_buffer_rsrc(                                        \
                         const_cast<uint8_t *>(op.w_scales + (int64_t)an_ * KB), 0, rw_ * KB,  \
                         kBufferFlags)                                                         \
                   : __builtin_amdgcn_make_buffer_rsrc(                                        \
                         const_cast<uint8_t *>(op.e_scales + (int64_t)am_ * KB), 0, re_ * KB,  \
                         kBufferFlags);                                                        \
  }

#define M4_W(st) ((st) ? w1 : w0)
#define M4_E(st) ((st) ? e1 : e0)
#define M4_LDS(p) ((__attribute__((address_space(3))) void *)(p))
#define M4_LOADW(kt_, st, i)                                                                   \
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsW, M4_LDS(&M4_W(st)[(wave * kWLoads + (i)) * 1024]), 16, \
                                           ((i) & 1) ? w_v1 : w_v0,                            \
                                           (i) * kWInstRows * w_ld + (kt_) * kWRow, 0, 0);
#define M4_LOADE(kt_, st, i)                                                                   \
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsE, M4_LDS(&M4_E(st)[(wave * 8 + (i)) * 1024]), 16, \
                                           ((i) & 1) ? e_v1 : e_v0,                            \
                                           (i) * 8 * e_ld + (kt_) * Cfg::kERow, 0, 0);
// the scales of steps kt_ and kt_ + 1 (kt_ even)
#define M4_LOADS(kt_)                                                                          \
  _Pragma("unroll") for (int i = 0; i < kSLoads; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds( \
      rsS, M4_LDS(&sc[(wave * kSLoads + i) * 256]), 4, s_v, i * kSRows * KB + (kt_) * kSc, 0, 0);
#define M4_LOADSTEP(kt_, st)                                                                   \
  _Pragma("unroll") for (int i = 0; i < kWLoads; ++i) { M4_LOADW(kt_, st, i) }                 \
  _Pragma("unroll") for (int i = 0; i < 8; ++i) { M4_LOADE(kt_, st, i) }
#define M4_CHUNK(buf, base, c, sw) \
  (*reinterpret_cast<const uint4 *>(&(buf)[(base) + (((c) ^ (sw)) << 4)]))
#define M4_FRAGS(st, s, fa, fb)                                                                \
  _Pragma("unroll") for (int i = 0; i < 4; ++i)                                                \
    fa[i] = fp4_operand(M4_CHUNK(M4_W(st), a_base + i * 32 * kWRow, kSub * h + (s), a_sw));    \
  _Pragma("unroll") for (int j = 0; j < 4; ++j)                                                \
    fb[j] = EF == kFp4                                                                         \
                ? fp4_operand(M4_CHUNK(M4_E(st), b_base + j * 32 * 128, kSub * h + (s), fsw))  \
                : fp8_operand(M4_CHUNK(M4_E(st), b_base + j * 32 * 128, 2 * (s) + h, fsw),     \
                              M4_CHUNK(M4_E(st), b_base + j * 32 * 128, 2 * (kSub + (s)) + h, fsw));
// this lane's scales of step q (0 or 1) of a pair, as the low bytes of a word
#define M4_SCALE(base, q)                                                                      \
  (EF == kFp4 ? *reinterpret_cast<const uint32_t *>(&sc[(base) + (q) * kSc])                   \
              : (uint32_t)*reinterpret_cast<const uint16_t *>(&sc[(base) + (q) * kSc]))
#define M4_SCALES(q, sA, sB)                                                                   \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) sA[i] = M4_SCALE(as_base + i * 32 * 2 * kSc, q); \
  _Pragma("unroll") for (int j = 0; j < 4; ++j) sB[j] = M4_SCALE(bs_base + j * 32 * 2 * kSc, q);
#define M4_MFMA(s, fa, fb, sA, sB)                                                             \
  _Pragma("unroll") for (int i = 0; i < 4; ++i) _Pragma("unroll") for (int j = 0; j < 4; ++j)  \
    acc[i][j] = mfma_unit<EF, s>(fa[i], fb[j], acc[i][j], sA[i], sB[j]);
#define M4_BARRIER() asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
// the first step of a tile: the stores of the one before may be outstanding, all of
// them, as they were issued behind the loads
#define M4_BARRIER0()                                                                          \
  if (stores)                                                                                  \
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kTileStores) : "memory"); \
  else                                                                                         \
    M4_BARRIER()
// E2M1, in_dim an odd multiple of 128: the last step's upper four blocks lie in the
// next row. Scales of 2^-127 on both sides take their products below the smallest
// fp32, to zero.
#define M4_TAIL(kt_, sA, sB)                                                                   \
  if constexpr (EF == kFp4) {                                                                  \
    const uint32_t keep = ((kt_) + 1) * 8 > KB && h ? 0u : ~0u;                                \
    _Pragma("unroll") for (int i = 0; i < 4; ++i) { sA[i] &= keep; sB[i] &= keep; }            \
  }

  f32x16 acc[4][4];
  i32x8 fa0[4], fb0[4], fa1[4], fb1[4];
  uint32_t sA0[4], sB0[4], sA1[4], sB1[4];
  zero_acc(acc);
  M4_AIM((int)blockIdx.x)
  M4_LOADS(0)
  M4_LOADSTEP(0, 0)
  M4_LOADSTEP(1, 1)
  M4_BARRIER()
// One step from stage P: its last fragments are read before the barrier, the next
// step's first ones (stage Q) behind it, while stage P takes step `ahead`. The LDS
// reads come before the new direct loads: the compiler, which cannot see the wait
// inside the barrier, puts a full vmcnt wait before them.
#define M4_FENCE() __builtin_amdgcn_sched_barrier(0)
#define M4_GROUP(mask, n) __builtin_amdgcn_sched_group_barrier(mask, n, 0)
// 16 MFMAs with the next fragments' reads between the first of them
#define M4_PART(P, s, ra, rb, fa, fb, sA, sB)                                                  \
  M4_FRAGS(P, (s) + 1, ra, rb)                                                                 \
  M4_MFMA(s, fa, fb, sA, sB)                                                                   \
  _Pragma("unroll") for (int g_ = 0; g_ < kReads; ++g_) { M4_GROUP(0x100, 1); M4_GROUP(0x008, 1); } \
  M4_FENCE();
#define M4_STEP(kt_, ahead, P, Q, sA, sB, BARRIER, READ, LOAD)                                 \
  {                                                                                            \
    M4_TAIL(kt_, sA, sB)                                                                       \
    if constexpr (kSub == 4) {                                                                 \
      M4_PART(P, 0, fa1, fb1, fa0, fb0, sA, sB)                                                \
      M4_PART(P, 1, fa0, fb0, fa1, fb1, sA, sB)                                                \
      M4_PART(P, 2, fa1, fb1, fa0, fb0, sA, sB)                                                \
    } else {                                                                                   \
      M4_PART(P, 0, fa1, fb1, fa0, fb0, sA, sB)                                                \
    }                                                                                          \
    BARRIER                                                                                    \
    M4_FENCE();                                                                                \
    M4_FRAGS(Q, 0, fa0, fb0)                                                                   \
    READ                                                                                       \
    M4_LOADSTEP(ahead, P)                                                                      \
    LOAD                                                                                       \
    M4_MFMA((kSub - 1), fa1, fb1, sA, sB)                                                      \
    _Pragma("unroll") for (int g_ = 0; g_ < 16; ++g_) {                                        \
      M4_GROUP(0x008, 1); M4_GROUP(0x100, 2); M4_GROUP(0x020, 2);                              \
    }                                                                                          \
    M4_FENCE();                                                                                \
  }
  bool stores = false;                // a whole tile's stores were issued behind the loads
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    // read again behind the stores, whose registers they would otherwise take
    M4_FRAGS(0, 0, fa0, fb0)
    M4_SCALES(0, sA0, sB0)
    M4_SCALES(1, sA1, sB1)
    int kt = 0;
    for (; kt + 1 < ke; kt += 2) {
      int ahead = kt + 2;
      if (ahead >= ke) {              // the next tile's first steps
        M4_AIM(t + (int)gridDim.x)
        ahead = 0;
      }
      M4_STEP(kt, ahead, 0, 1, sA0, sB0, M4_BARRIER0(), , M4_LOADS(ahead))
      stores = false;
      uint32_t tA[4], tB[4];
      M4_STEP(kt + 1, ahead + 1, 1, 0, sA1, sB1, M4_BARRIER(), M4_SCALES(0, sA0, sB0) M4_SCALES(1, tA, tB), )
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sA1[i] = tA[i];
        sB1[i] = tB[i];
      }
    }
    if (kt < ke) M4_STEP(kt, kt + 2, 0, 1, sA0, sB0, M4_BARRIER(), , )
    int m0, n0;
    tile_origin_of(t, tiles_m, tiles_n, BN, m0, n0);
    uint8_t *patch = sc + kScBytes + wave * kPatch;
    const bool whole = m0 + BM <= op.M && n0 + BN <= op.N;
    // the lane through a swap with itself, which stays in the loop: addresses formed
    // from it are formed anew for each tile; kept over the K loop they spill
    const int l = __builtin_amdgcn_mov_dpp(lane, 0xE4, 0xF, 0xF, true);
    if (whole) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        store_patch<false>(acc[q % 2 * 2][q / 2], acc[q % 2 * 2 + 1][q / 2], patch, kv, op.M, op.N,
                           m0 + wm * 128 + q / 2 * 32, n0 + wn * 128 + q % 2 * 64, l);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        store_patch<true>(acc[q % 2 * 2][q / 2], acc[q % 2 * 2 + 1][q / 2], patch, kv, op.M, op.N,
                          m0 + wm * 128 + q / 2 * 32, n0 + wn * 128 + q % 2 * 64, l);
    }
    zero_acc(acc);
    stores = whole;
  }
  // direct loads issued behind the last tile land before the block's LDS is freed
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#undef M4_STEP
#undef M4_PART
#undef M4_GROUP
#undef M4_FENCE
#undef M4_TAIL
#undef M4_BARRIER0
#undef M4_BARRIER
#undef M4_MFMA
#undef M4_SCALES
#undef M4_SCALE
#undef M4_FRAGS
#undef M4_CHUNK
#undef M4_LOADSTEP
#undef M4_LOADS
#undef M4_LOADE
#undef M4_LOADW
#undef M4_LDS
#undef M4_E
#undef M4_W
#undef M4_AIM
}

template <int EF>
__global__ __launch_bounds__(kWideThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mx4_wide_kernel(Mx4Operands op, uint16_t *__restrict__ kv, int tiles_m, int tiles_n) {
  wide_walk<EF>(op, kv, tiles_m, tiles_n);
}

// ---- few blocks: small tiles, the operands streamed far ahead ------------------------
// A block takes 64 MT tokens against 64 NI weight rows over the whole of K, two waves
// along each, so that a wave holds 32 MT x 32 NI outputs. K-steps of 128 inputs; both
// operands go global -> LDS by direct loads into rings of their own: the weight, which
// comes from HBM, kRw pairs of steps deep (whole cache lines of a row), e, which the
// blocks of a token tile share and L2 holds, kRe steps. The one barrier of a step stands
// before its last MFMAs: by then the step's slots have been read and take the loads of
// step kt + kRe and of the pair kRw ahead, and step kt + 1 has landed. Loads complete in
// order, so the wait for an e batch is one for every weight load issued before it: e is
// requested first, which leaves the weight one step more (100 tokens of E4M3: 24 us for
// 26). Scales go straight to registers, 16 bytes of a row (4 steps) at a time and a
// group ahead.
// 256 tokens of E4M3 against 25600 rows of 6144 take 38-42 us, 34 with every load and
// LDS read left out (launch, ends and MFMAs: the matrix units are busy 45 % of the 200
// CUs' cycles, and barriers and issue take the rest); E2M1 28-31, 22 without loads and
// reads, 28 without the weight's stream alone. 1 token takes 15 us, 5.6 TB/s.
template <int EF, int NI>
struct SkinnyCfg {
  static constexpr int kERow = EF == kFp4 ? 64 : 128;   // bytes of an e row and step
  static constexpr int kRe = 4;
  static constexpr int kRw = EF == kFp4 && NI < 4 ? 4 : 3;
  static constexpr int kUnroll = kRw == 4 ? 8 : 12;     // steps: a multiple of both rings and of 4
};

template <int EF, int NI, int MT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mx4_skinny_kernel(Mx4Operands op, uint16_t *__restrict__ kv, int tiles_n) {
  using Cfg = SkinnyCfg<EF, NI>;
  constexpr int kRe = Cfg::kRe, kRw = Cfg::kRw, kERow = Cfg::kERow;
  constexpr int kRows = 64 * NI, kToks = 64 * MT;
  constexpr int kWLoads = kRows * 128 / 1024 / 4;       // direct loads of a wave and pair
  constexpr int kELoads = kToks * kERow / 1024 / 4;     // of a wave and step
  constexpr int kERows = 1024 / kERow;                  // e rows of a direct load
  constexpr int kSLoads = NI + MT;                      // scale loads of four steps
  // one LDS variable per slot: the compiler tells direct loads into up to eight apart
  __shared__ __align__(1024) uint8_t w0[kRows * 128], w1[kRows * 128], w2[kRows * 128];
  __shared__ __align__(1024) uint8_t w3[kRw == 4 ? kRows * 128 : 16];
  __shared__ __align__(1024) uint8_t e0[kToks * kERow], e1[kToks * kERow];
  __shared__ __align__(1024) uint8_t e2[kToks * kERow], e3[kToks * kERow];
  // The token tiles of the same rows go to one XCD, eight row tiles at a time.
  const int tiles_m = (int)gridDim.x / tiles_n;
  const int ahead = (int)blockIdx.x / (8 * tiles_m) * 8, left = (int)blockIdx.x - ahead * tiles_m;
  const int wide = min(8, tiles_n - ahead);
  const int n0 = (ahead + left % wide) * kRows, m0 = left / wide * kToks;
  const int KB = op.K / 32, KT = op.K / 128;
  const int w_ld = op.K / 2, e_ld = EF == kFp4 ? op.K / 2 : op.K;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave >> 1, wm = wave & 1;
  const int frow = lane & 31, h = lane >> 5;
  const int rows_w = min(kRows, op.N - n0), rows_e = min(kToks, op.M - m0);
  const __amdgpu_buffer_rsrc_t rsW = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(op.w_codes + (int64_t)n0 * w_ld), 0, rows_w * w_ld, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsE = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(op.e_codes + (int64_t)m0 * e_ld), 0, rows_e * e_ld, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsWs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(op.w_scales + (int64_t)n0 * KB), 0, rows_w * KB, kBufferFlags);
  const __amdgpu_buffer_rsrc_t rsEs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(op.e_scales + (int64_t)m0 * KB), 0, rows_e * KB, kBufferFlags);
  // 64-byte rows: chunk c of row r in slot c ^ (r / 2) % 4; 128-byte rows: c ^ f(r)
  const int c64 = (lane & 3) ^ ((lane >> 3) & 3), c128 = (lane & 7) ^ (lane >> 3);
  const int w_v0 = (wave * (kRows / 4) + (lane >> 3)) * w_ld + c128 * 16;
  const int w_v1 = (wave * (kRows / 4) + (lane >> 3)) * w_ld + (c128 ^ 1) * 16;
  const int e_v0 = EF == kFp4 ? (wave * (kToks / 4) + (lane >> 2)) * e_ld + c64 * 16
                              : (wave * (kToks / 4) + (lane >> 3)) * e_ld + c128 * 16;
  const int e_v1 = EF == kFp4 ? e_v0 : (wave * (kToks / 4) + (lane >> 3)) * e_ld + (c128 ^ 1) * 16;
  const int a_sw = (frow & 7) ^ ((frow >> 3) & 1);
  const int b_sw = EF == kFp4 ? (frow >> 1) & 3 : a_sw;
  const int a_base = (wn * 32 * NI + frow) * 128, b_base = (wm * 32 * MT + frow) * kERow;
  const int ws_v = (wn * 32 * NI + frow) * KB, es_v = (wm * 32 * MT + frow) * KB;

#define MK_W(s) ((s) == 0 ? w0 : (s) == 1 ? w1 : (s) == 2 ? w2 : w3)
#define MK_E(s) ((s) == 0 ? e0 : (s) == 1 ? e1 : (s) == 2 ? e2 : e3)
#define MK_LDS(p) ((__attribute__((address_space(3))) void *)(p))
#define MK_LOADW(pair, s)                                                                      \
  _Pragma("unroll") for (int i = 0; i < kWLoads; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds( \
      rsW, MK_LDS(&MK_W(s)[(wave * kWLoads + i) * 1024]), 16, (i & 1) ? w_v1 : w_v0,           \
      i * 8 * w_ld + (pair) * 128, 0, 0);
#define MK_LOADE(kt_, s)                                                                       \
  _Pragma("unroll") for (int i = 0; i < kELoads; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds( \
      rsE, MK_LDS(&MK_E(s)[(wave * kELoads + i) * 1024]), 16, (i & 1) ? e_v1 : e_v0,           \
      i * kERows * e_ld + (kt_) * kERow, 0, 0);
#define MK_SCALES(g)                                                                           \
  _Pragma("unroll") for (int i = 0; i < NI; ++i) wsn[i] = load16(rsWs, ws_v, i * 32 * KB + (g) * 16); \
  _Pragma("unroll") for (int j = 0; j < MT; ++j) esn[j] = load16(rsEs, es_v, j * 32 * KB + (g) * 16);
#define MK_WORD(v, q) ((q) == 0 ? (v).x : (q) == 1 ? (v).y : (q) == 2 ? (v).z : (v).w)
#define MK_CHUNK(buf, off, c, sw) (*reinterpret_cast<const uint4 *>(&(buf)[(off) + (((c) ^ (sw)) << 4)]))
// fragments of sub-step s (0, 1): this half's block 2 h + s of the step's four
#define MK_FRAGS(u, s, fa, fb)                                                                 \
  _Pragma("unroll") for (int i = 0; i < NI; ++i)                                               \
    fa[i] = fp4_operand(MK_CHUNK(MK_W((u) / 2 % kRw), a_base + i * 32 * 128,                   \
                                 (u) % 2 * 4 + 2 * h + (s), a_sw));                            \
  _Pragma("unroll") for (int j = 0; j < MT; ++j)                                               \
    fb[j] = EF == kFp4                                                                         \
                ? fp4_operand(MK_CHUNK(MK_E((u) % kRe), b_base + j * 32 * kERow, 2 * h + (s), b_sw)) \
                : fp8_operand(MK_CHUNK(MK_E((u) % kRe), b_base + j * 32 * kERow, 2 * (s) + h, b_sw), \
                              MK_CHUNK(MK_E((u) % kRe), b_base + j * 32 * kERow, 4 + 2 * (s) + h, b_sw));
#define MK_MFMA(s, fa, fb)                                                                     \
  _Pragma("unroll") for (int i = 0; i < NI; ++i) _Pragma("unroll") for (int j = 0; j < MT; ++j) \
    acc[i][j] = mfma_unit<EF, s>(fa[i], fb[j], acc[i][j], sa[i], sb[j]);
#define MK_FENCE() __builtin_amdgcn_sched_barrier(0)
// what computes may cross, loads may not: the waits count on their order
#define MK_ORDER() __builtin_amdgcn_sched_barrier(0x000F)
#define MK_GROUP(mask, n) __builtin_amdgcn_sched_group_barrier(mask, n, 0)

  f32x16 acc[NI][MT];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  i32x8 fa0[NI], fb0[MT], fa1[NI], fb1[MT];
  uint4 ws[NI], es[MT], wsn[NI], esn[MT];
  uint32_t sa[NI], sb[MT];
  MK_SCALES(0)
#pragma unroll
  for (int i = 0; i < NI; ++i) ws[i] = wsn[i];
#pragma unroll
  for (int j = 0; j < MT; ++j) es[j] = esn[j];
  // in the order in which the steps before the first would have issued them
  MK_LOADW(0, 0)
  if constexpr (kRw == 4) { MK_LOADW(1, 1) }
  MK_LOADE(0, 0)
  MK_FENCE();
  MK_LOADE(1, 1)
  MK_FENCE();
  MK_LOADW(kRw - 2, kRw - 2)
  MK_FENCE();
  MK_LOADE(2, 2)
  MK_FENCE();
  MK_LOADE(3, 3)
  MK_FENCE();
  MK_LOADW(kRw - 1, kRw - 1)
  MK_FENCE();
  // step 0 has landed when only what was issued after it is outstanding
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kRe - 1) * kELoads + 2 * kWLoads)
               : "memory");
  MK_FENCE();
  MK_FRAGS(0, 0, fa0, fb0)
// What may be outstanding at step u's barrier: everything issued behind the e batch of
// step u + 1, which is that of step u + 1 - kRe: kRe - 2 batches, the weight's of the
// odd steps from that one on, the scales (every fourth step) of the steps behind it.
// Only loads that the compiler must issue, and issue there, may be counted: the direct
// loads write LDS and stay where they are, and a scale load of the main loop is read by
// a later turn. A scale load of the last steps is not counted: the compiler may move one to
// where it is read, and deletes one that no step reads.
#define MK_PENDING(u, last)                                        \
  ((kRe - 2) * kELoads + ((u) % 2 == 0 ? 2 : 1) * kWLoads +        \
   (!(last) && (u) % 4 <= kRe - 2 ? kSLoads : 0))
// Step kt + u, of the main loop or of the last steps, which end before the next group of
// scales is due. The LDS reads come before the direct loads of the same step, whose
// slots the compiler believes to be in flight (it cannot see the barrier's wait).
#define MK_STEP(u, last)                                                                       \
  {                                                                                            \
    if ((u) % 4 == 0 && (!(last) || (u) + 4 < Cfg::kUnroll)) { MK_SCALES((kt + (u)) / 4 + 1) } \
    _Pragma("unroll") for (int i = 0; i < NI; ++i) sa[i] = MK_WORD(ws[i], (u) % 4) >> (16 * h); \
    _Pragma("unroll") for (int j = 0; j < MT; ++j) sb[j] = MK_WORD(es[j], (u) % 4) >> (16 * h); \
    MK_FRAGS(u, 1, fa1, fb1)                                                                   \
    MK_MFMA(0, fa0, fb0)                                                                       \
    MK_FENCE();                                                                                \
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(MK_PENDING(u, last))        \
                 : "memory");                                                                  \
    MK_FENCE();                                                                                \
    MK_FRAGS((u) + 1, 0, fa0, fb0)                                                             \
    MK_FENCE();                                                                                \
    MK_LOADE(kt + (u) + kRe, (u) % kRe)                                                        \
    if ((u) % 2 == 1) {                                                                        \
      MK_ORDER();                                                                              \
      MK_LOADW((kt + (u)) / 2 + kRw, (u) / 2 % kRw)                                            \
    }                                                                                          \
    MK_MFMA(1, fa1, fb1)                                                                       \
    _Pragma("unroll") for (int g_ = 0; g_ < 8; ++g_) { MK_GROUP(0x008, 1); MK_GROUP(0x020, 2); } \
    MK_FENCE();                                                                                \
    if ((u) % 4 == 3) {                                                                        \
      _Pragma("unroll") for (int i = 0; i < NI; ++i) ws[i] = wsn[i];                           \
      _Pragma("unroll") for (int j = 0; j < MT; ++j) es[j] = esn[j];                           \
    }                                                                                          \
  }
// The steps behind the last whole unrolling stand apart: branches around steps of the
// main loop made the compiler wait for every load at each of them, as it does here (47
// steps of which 11 stand apart against 48: 256 tokens of E4M3 38.2 us against 37.5, of E2M1
// 30.7 against 28.4, 1 token 14.9 against 15.0).
#define MK_LAST(u)           \
  if (kt + (u) >= KT) break; \
  MK_STEP(u, true)
  int kt = 0;
  for (; kt + Cfg::kUnroll <= KT; kt += Cfg::kUnroll) {
    MK_STEP(0, false) MK_STEP(1, false) MK_STEP(2, false) MK_STEP(3, false)
    MK_STEP(4, false) MK_STEP(5, false) MK_STEP(6, false) MK_STEP(7, false)
    if constexpr (Cfg::kUnroll == 12) {
      MK_STEP(8, false) MK_STEP(9, false) MK_STEP(10, false) MK_STEP(11, false)
    }
  }
  do {
    MK_LAST(0) MK_LAST(1) MK_LAST(2) MK_LAST(3) MK_LAST(4) MK_LAST(5) MK_LAST(6)
    if constexpr (Cfg::kUnroll == 12) { MK_LAST(7) MK_LAST(8) MK_LAST(9) MK_LAST(10) }
  } while (false);
  // every direct load has landed before the slots hold the outputs
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#undef MK_LAST
#undef MK_STEP
#undef MK_PENDING
#undef MK_GROUP
#undef MK_ORDER
#undef MK_FENCE
#undef MK_MFMA
#undef MK_FRAGS
#undef MK_CHUNK
#undef MK_WORD
#undef MK_SCALES
#undef MK_LOADE
#undef MK_LOADW
#undef MK_LDS
#undef MK_E
#undef MK_W
  // 32 tokens x 32 NI columns of a wave at a time through LDS, as store_patch
  constexpr int kChunks = 4 * NI;                       // 16-byte chunks of a token
  constexpr int kPatch = 32 * kChunks * 16;
  static_assert(EF == kFp4 ? kPatch <= kToks * kERow : 2 * kPatch <= kToks * kERow, "patches fit the e slots");
  uint8_t *mine = EF == kFp4 ? (wave == 0 ? e0 : wave == 1 ? e1 : wave == 2 ? e2 : e3)
                             : (wave < 2 ? e0 : e1) + (wave & 1) * kPatch;
  const int col = n0 + wn * 32 * NI + (lane % kChunks) * 8;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint2 v;
        v.x = engram::pack_bf16x2(acc[i][j][g * 4 + 0], acc[i][j][g * 4 + 1]);
        v.y = engram::pack_bf16x2(acc[i][j][g * 4 + 2], acc[i][j][g * 4 + 3]);
        *reinterpret_cast<uint2 *>(mine + (frow * kChunks + ((i * 4 + g) ^ (frow & (kChunks - 1)))) * 16 +
                                   h * 8) = v;
      }
#pragma unroll
    for (int q = 0; q < 32 * kChunks / 64; ++q) {
      const int t = (q * 64 + lane) / kChunks;
      const engram::u32x4 v = *reinterpret_cast<const engram::u32x4 *>(
          mine + (t * kChunks + ((lane % kChunks) ^ (t & (kChunks - 1)))) * 16);
      const int m = m0 + wm * 32 * MT + j * 32 + t;
      if (m < op.M && col < op.N)
        __builtin_nontemporal_store(v, reinterpret_cast<engram::u32x4 *>(kv + (int64_t)m * op.N + col));
    }
  }
}

template <int EF, int NI, int MT>
hipError_t launch_skinny(const Mx4Operands &op, uint16_t *kv, hipStream_t stream) {
  const int tiles_n = (op.N + 64 * NI - 1) / (64 * NI), tiles_m = (op.M + 64 * MT - 1) / (64 * MT);
  hipLaunchKernelGGL((mx4_skinny_kernel<EF, NI, MT>), dim3((unsigned)(tiles_n * tiles_m)), dim3(256), 0,
                     stream, op, kv, tiles_n);
  return hipGetLastError();
}

// The smallest tile whose blocks fit the CUs at once: a larger one leaves CUs idle and, at
// few tokens, multiplies padding (us, E4M3, 6144 inputs: 1 token x 25600 columns 20, 15,
// 20, 34 with tiles of 64 x 64, 64 x 128, 128 x 128, 128 x 256 tokens x rows; 100 x 5120
// 11, 11, 18, 31; 600 x 5120 41, 29, 22, 36). Where no such tile fits, the blocks come in
// rounds, a round of whole 256 x 256 tiles as long as 1.4 to 1.8 of 128 x 256: those are taken
// where their rounds number up to 5 / 3 of the whole tiles' (us, E4M3 and E2M1, 128 x 256
// against 256 x 256; 1 round: 240 blocks of 300 x 20480, E4M3 42, 64; 2 to 2: 600 x 25600
// 83, 126 and 63, 85; 3 to 2: 768 x 25600 115, 135 and 86, 91; 2 to 1: 256 x 33024 76, 67
// and 57, 49; 4 to 2: 1003 x 25600 154, 135 and 114, 94; 7 to 4: 2048 x 25600 281, 285 and
// 207, 191; with 1024 inputs the same sides win). Up to 128 tokens both sides have as
// many blocks: 128 x 66048 83, 125 and 68, 84.
template <int EF>
hipError_t launch_mx4(const Mx4Operands &op, uint16_t *kv, hipStream_t stream) {
  int cus = 0;
  const hipError_t err = cu_count(cus);
  if (err != hipSuccess) return err;
  const auto rounds = [&](int toks, int rows) {
    const int64_t blocks = ((int64_t)op.M + toks - 1) / toks * (((int64_t)op.N + rows - 1) / rows);
    return (blocks + cus - 1) / cus;
  };
  if (rounds(64, 64) == 1) return launch_skinny<EF, 1, 1>(op, kv, stream);
  if (rounds(64, 128) == 1) return launch_skinny<EF, 2, 1>(op, kv, stream);
  if (rounds(128, 128) == 1) return launch_skinny<EF, 2, 2>(op, kv, stream);
  if (3 * rounds(128, 256) <= 5 * rounds(BM, BN)) return launch_skinny<EF, 4, 2>(op, kv, stream);
  const int tiles_m = (op.M + BM - 1) / BM, tiles_n = (op.N + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  const bool even = (op.K + WideCfg<EF>::kStep - 1) / WideCfg<EF>::kStep % 2 == 0;
  hipLaunchKernelGGL((mx4_wide_kernel<EF>), dim3((unsigned)(even && tiles > cus ? cus : tiles)),
                     dim3(kWideThreads), 0, stream, op, kv, tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t engram_launch_gemm_mx4(const uint8_t *w_codes, const uint8_t *w_scales,
                                  const uint8_t *e_codes, const uint8_t *e_scales, bool e_fp4,
                                  uint16_t *kv, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
  if (m <= 0 || n <= 0) return hipSuccess;
  const Mx4Operands op{w_codes, w_scales, e_codes, e_scales, (int)m, (int)n, (int)k};
  return e_fp4 ? launch_mx4<kFp4>(op, kv, stream) : launch_mx4<kFp8>(op, kv, stream);
}
