// Gradient of step 5 (gate.hip) from the streams and the keys and value it was computed
// from, each as they were or as 8-bit codes with one scale per row. Per token t, with d =
// d_out the gradient of the updated streams h' = h + alpha v:
//
//   w = q_w k_w, D = sum h w k, rh = (mean h^2 + eps)^(-1/2), rk of k,
//   s = D rh rk / sqrt(dim), alpha = sigmoid(z), z = sign(s) sqrt(max(|s|, c)) or s
//   c1 = (sum d v) alpha (1 - alpha) z'(s) rh rk / sqrt(dim),
//        z' = 1 / (2 sqrt|s|) where |s| > c, else 0; or 1
//   dh = d + c1 (k w - (D rh^2 / dim) h),  dk = c1 (h w - (D rk^2 / dim) k)
//   dv = sum over the streams of alpha d,  dw = sum over the tokens of c1 h k,
//   dq_w = k_w dw,  dk_w = q_w dw;  at a DEAD position dh = d, dk = dv = 0, no dw
//
// z' has a pole at s = 0, where D's terms cancel: D is summed in 64 bits from exact
// products of h and k, and w = q_w k_w enters it as the product and its rounding error, so
// that s keeps its relative precision there. Everything else is fp32.
//
// Bound by HBM: what the outputs need is read once and they are written once. (Beside that,
// gate_grad_token_kernel requests a DEAD position's saved rows and reads its d_out again where
// d_h is another buffer, and with a team's last token one more, which nothing uses.) A block walks
// the tokens blockIdx.x, blockIdx.x + gridDim.x, ...; a thread owns 8 columns of every stream and
// keeps its part of dw in registers over all of them. The blocks' parts are summed by a second launch in a
// fixed order. 32768 tokens of 4 x 5120 from codes take 1.15 ms (5.88 GB, 5.1 TB/s; stream by
// stream, with a barrier and a wait for loads at each, 2.89 ms; without the sums over the wave
// 1.09 ms), 509 tokens 45 us, of which the stores take 10 and the second launch 5.
#include "common.h"

namespace {

constexpr int kMaxThreads = 1024;

struct GateGradArgs {
  const int32_t *ids;
  EngramDeadRule dead_rule;
  const void *kv, *h;
  const float *kv_scales, *h_scales;   // of codes
  const float *q_w, *k_w;
  const void *d_out;
  void *d_h, *d_kv;
  float *part;                         // [gridDim.x, hc, dim], or NULL
  int tokens, hc, dim;
  float eps, clamp;
  int plain;
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// Eight consecutive saved values: a chunk of floats, or 8 codes.
template <bool I8, bool F32>
struct Saved8 {
  engram::Chunk8<F32> c;
  __device__ __forceinline__ void load(const void *p, int64_t row, int dim, int ci) {
    c.load_nt(p, row * (dim / 8) + ci);
  }
  __device__ __forceinline__ float operator[](int e) const { return c[e]; }
  __device__ __forceinline__ float squares() const {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(c[e], c[e], s);
    return s;
  }
};
template <bool F32>
struct Saved8<true, F32> {
  uint32_t w[2];
  __device__ __forceinline__ void load(const void *p, int64_t row, int dim, int ci) {
    const uint64_t v = __builtin_nontemporal_load(reinterpret_cast<const uint64_t *>(p) +
                                                  row * ((dim + 15) / 16 * 2) + ci);
    w[0] = (uint32_t)v;
    w[1] = (uint32_t)(v >> 32);
  }
  __device__ __forceinline__ float operator[](int e) const {
    return (float)(int8_t)(w[e / 4] >> (8 * (e % 4)));
  }
  __device__ __forceinline__ float squares() const {
    return (float)__builtin_amdgcn_sdot4((int)w[1], (int)w[1],
                                         __builtin_amdgcn_sdot4((int)w[0], (int)w[0], 0, false), false);
  }
};

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, engram::kWave);
  return v;
}

// Sums of HC (2 or 4) numbers over a wave: first halves of the wave change places between two
// streams' numbers, then rows of 16, so that each addition serves two streams; then a row's
// (half's) lanes by shifts. Stream m's sum ends in lane 64 / HC (m + 1) - 1.
template <typename T, int CTRL, int ROWS>
__device__ __forceinline__ T shifted(T v) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, true));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  }
}
// a's sums of lanes l and l + 32 (l and l + 16 of each half) below b's
template <typename T, bool HALVES>
__device__ __forceinline__ T fold(T a, T b) {
  constexpr int kWords = sizeof(T) / 4;
  uint32_t x[kWords], y[kWords];
  __builtin_memcpy(x, &a, sizeof(T));
  __builtin_memcpy(y, &b, sizeof(T));
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const auto r = HALVES ? __builtin_amdgcn_permlane32_swap(x[w], y[w], false, false)
                          : __builtin_amdgcn_permlane16_swap(x[w], y[w], false, false);
    x[w] = r[0];
    y[w] = r[1];
  }
  __builtin_memcpy(&a, x, sizeof(T));
  __builtin_memcpy(&b, y, sizeof(T));
  return a + b;
}
template <typename T, int HC>
__device__ __forceinline__ T sums_of(const T (&v)[HC]) {
  T s;
  if constexpr (HC == 4)
    s = fold<T, false>(fold<T, true>(v[0], v[2]), fold<T, true>(v[1], v[3]));
  else
    s = fold<T, true>(v[0], v[1]);
  s += shifted<T, 0x111, 0xF>(s);
  s += shifted<T, 0x112, 0xF>(s);
  s += shifted<T, 0x114, 0xF>(s);
  s += shifted<T, 0x118, 0xF>(s);
  if constexpr (HC == 2) s += shifted<T, 0x142, 0xA>(s);     // a row's last lane to the next row
  return s;
}

// What the outputs of one stream take from its sums, which are of the saved numbers
// without their scales sh, sk, sv: alpha, and with h and k still without theirs
//   dh = d + ck k w - Bh h,  dk = ch h w - Bk k,  dw = cw h k.
struct StreamGrad {
  float alpha, ch, ck, cw, Bh, Bk;
};
__device__ __forceinline__ StreamGrad stream_grad(const GateGradArgs &a, float shh, float skk, float sdv,
                                                  double dot, float sh, float sk, float sv) {
  const float inv_d = 1.f / (float)a.dim;
  const float rh = 1.f / sqrtf(shh * sh * sh * inv_d + a.eps);
  const float rk = 1.f / sqrtf(skk * sk * sk * inv_d + a.eps);
  const float D = (float)(dot * (double)sh * (double)sk);
  const float norm = rh * rk / sqrtf((float)a.dim);
  const float s = D * norm;
  // a NaN stays one, so that no gradient looks sound that a broken saved row went into
  const float root = sqrtf(fabsf(s) < a.clamp ? a.clamp : fabsf(s));
  const float z = a.plain ? s : copysignf(root, s);
  // alpha (1 - alpha) without the difference of two near ones
  const float small = expf(-fabsf(z));
  float slope = small / ((1.f + small) * (1.f + small));
  if (!a.plain) slope = fabsf(s) <= a.clamp ? 0.f : slope / (2.f * root);
  const float c1 = sdv * sv * slope * norm;
  StreamGrad g;
  g.alpha = (z < 0.f ? small : 1.f) / (1.f + small);
  g.ch = c1 * sh;
  g.ck = c1 * sk;
  g.cw = g.ch * sk;
  g.Bh = D * rh * rh * inv_d * g.ch;
  g.Bk = D * rk * rk * inv_d * g.ck;
  return g;
}

// The outputs of a DEAD position.
template <bool F32>
__device__ __forceinline__ void store_dead(const GateGradArgs &a, int64_t t, int cps, int ci) {
  const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int m = 0; m <= a.hc; ++m)
    engram::Chunk8<F32>::store_nt(a.d_kv, (t * (a.hc + 1) + m) * cps + ci, zero);
  if (a.d_h == a.d_out) return;
  for (int m = 0; m < a.hc; ++m) {
    engram::Chunk8<F32> d;
    d.load_nt(a.d_out, (t * a.hc + m) * cps + ci);
    d.put(a.d_h, (t * a.hc + m) * cps + ci);
  }
}

// Up to HC streams, whose numbers of one token a thread holds together: one barrier a
// token, and the loads of the next token's stream m are issued as soon as this one's are
// used up, so that a token is in flight while another is worked on. The learned scales lie
// in LDS as w = q_w k_w rounded to fp32 and the part of it that this drops, 2^24 times that in
// fp16: 36 bits in all (bf16 left dq_w of 32768 x 4 x 5120 off by 1.3e-6 of its norm where one
// token's s came near 0, against 2e-7). Registers spill inside the loop where they hold most: 13 with
// 4 streams all in bf16, 10 with 4 all in fp32, with 8 streams 1 from codes, 34 and 56 from codes and
// bf16, 84 from bf16; a reload waits for the loads requested before it. From bf16 arrays 8192 x 4 x
// 5120 take 382 us (4.8 TB/s; from codes 311) and 4096 x 8 x 1024 175 us (2.0 TB/s; from codes 95).
// A block has
// `teams` teams of `width` threads, each on a token of its own, which share w; their parts
// of dw meet in LDS at the end. F32: fp32 streams, else bf16. KI8, HI8: keys and value,
// streams as codes.
constexpr int token_threads(bool f32, int hc) { return f32 || hc > 4 ? 512 : 640; }
constexpr int kMaxTokenThreads = 640;
constexpr int kTokenColumns = 25600;          // hc * dim: 150 KB of w

template <bool F32, bool KI8, bool HI8, int HC>
__global__ __launch_bounds__(token_threads(F32, HC)) void gate_grad_token_kernel(GateGradArgs a, int width, int teams) {
  // products of two bf16 numbers or codes are exact in fp32
  constexpr bool kExact = !F32 || (KI8 && HI8);
  constexpr int kFold = HC < 4 ? HC : 4;      // streams whose sums are formed together
  extern __shared__ __align__(16) uint8_t w_lds[];
  __shared__ double red_d[2][kMaxTokenThreads / 64][HC];
  __shared__ float red[2][kMaxTokenThreads / 64][HC][3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int team = __builtin_amdgcn_readfirstlane(tid / width);
  const int first_wave = team * (width >> 6), last_wave = first_wave + (width >> 6);
  const int cps = a.dim / 8, hc = a.hc;
  const bool on = tid - team * width < cps;
  const int ci = on ? tid - team * width : 0;
  float dw[HC][8];
#pragma unroll
  for (int m = 0; m < HC; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[m][e] = 0.f;
  Saved8<HI8, F32> h[HC];
  Saved8<KI8, F32> k[HC], v;
  engram::Chunk8<F32> d[HC];
  const int64_t stride = (int64_t)gridDim.x * teams;
  int64_t t = (int64_t)blockIdx.x * teams + team;
  const int64_t last = a.tokens - 1;
  const int64_t begin = t < last ? t : last;
#pragma unroll
  for (int m = 0; m < HC; ++m) {
    if (m >= hc) break;
    h[m].load(a.h, begin * hc + m, a.dim, ci);
    k[m].load(a.kv, begin * (hc + 1) + m, a.dim, ci);
    d[m].load_nt(a.d_out, (begin * hc + m) * cps + ci);
  }
  v.load(a.kv, begin * (hc + 1) + hc, a.dim, ci);
  float *w_hi = reinterpret_cast<float *>(w_lds);
  f16x8 *w_lo = reinterpret_cast<f16x8 *>(w_lds + (size_t)hc * a.dim * 4);
#pragma unroll 4
  for (int c = tid; c < hc * cps; c += blockDim.x) {
    engram::Chunk8<true> q, k;
    q.load(a.q_w, c);
    k.load(a.k_w, c);
    float hi[8];
    f16x8 lo;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      hi[e] = q[e] * k[e];
      // at most 1 for normal numbers; others have nothing to add
      const float part = fmaf(q[e], k[e], -hi[e]) / hi[e] * 16777216.f;
      lo[e] = (_Float16)(fabsf(part) <= 1.f ? part : 0.f);
    }
    engram::Chunk8<true>::store(w_hi, c, hi);
    w_lo[c] = lo;
  }
  __syncthreads();
  int slot = 0;
  // every team takes as many turns as the block's first: one barrier a turn
  for (int64_t turn = (int64_t)blockIdx.x * teams; turn < a.tokens; turn += stride, t += stride) {
    const bool some = t < a.tokens;
    const int64_t next = t + stride < a.tokens ? t + stride : last;
    const bool live = some && !engram_dead(a.dead_rule, a.ids[t]);
    const int ml = lane < hc ? lane : 0;       // this lane's stream
    float sh = 1.f, sk = 1.f, sv = 1.f;
    if (live) {
      if (HI8) sh = a.h_scales[t * hc + ml];
      if (KI8) sk = a.kv_scales[t * (hc + 1) + ml], sv = a.kv_scales[t * (hc + 1) + hc];
#pragma unroll
      for (int g = 0; g < HC; g += kFold) {
        float shh[kFold], skk[kFold], sdv[kFold];
        double dot[kFold];
#pragma unroll
        for (int x = 0; x < kFold; ++x) {
          const int m = g + x;
          shh[x] = skk[x] = sdv[x] = 0.f;
          dot[x] = 0.0;
          if (m < hc && on) {
            float rest = 0.f, low = 0.f;
            engram::Chunk8<true> w;
            w.load(w_hi, m * cps + ci);
            const f16x8 lo = w_lo[m * cps + ci];
            shh[x] = h[m].squares();
            skk[x] = k[m].squares();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float he = h[m][e], ke = k[m][e];
              sdv[x] = fmaf(d[m][e], v[e], sdv[x]);
              if (kExact) {
                // p q_w k_w in three parts: p w rounded, its error, and what w drops
                const float p = he * ke, r = p * w[e];
                rest += fmaf(p, w[e], -r);
                low = fmaf(r, (float)lo[e], low);
                dot[x] += (double)r;
              } else {
                const double r = (double)he * (double)ke * (double)w[e];
                dot[x] += r;
                low = fmaf((float)r, (float)lo[e], low);
              }
            }
            dot[x] += (double)rest + (double)low * 0x1p-24;
          }
        }
        const float a0 = sums_of(shh), a1 = sums_of(skk), a2 = sums_of(sdv);
        const double a3 = sums_of(dot);
        if (lane % (64 / kFold) == 64 / kFold - 1) {
          const int m = g + lane / (64 / kFold);
          red[slot][wave][m][0] = a0;
          red[slot][wave][m][1] = a1;
          red[slot][wave][m][2] = a2;
          red_d[slot][wave][m] = a3;
        }
      }
    }
    // the next turn's barrier stands between the reads behind this one and the writes after it
    __syncthreads();
    if (live) {
      StreamGrad mine;
      {
        float shh = 0.f, skk = 0.f, sdv = 0.f;
        double dot = 0.0;
        for (int w = first_wave; w < last_wave; ++w) {
          shh += red[slot][w][ml][0];
          skk += red[slot][w][ml][1];
          sdv += red[slot][w][ml][2];
          dot += red_d[slot][w][ml];
        }
        mine = stream_grad(a, shh, skk, sdv, dot, sh, sk, sv);
      }
      float dv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < HC; ++m) {
        if (m >= hc) break;
#define ENGRAM_OF_STREAM(x) __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), m))
        const float alpha = ENGRAM_OF_STREAM(mine.alpha), ch = ENGRAM_OF_STREAM(mine.ch);
        const float ck = ENGRAM_OF_STREAM(mine.ck), cw = ENGRAM_OF_STREAM(mine.cw);
        const float Bh = ENGRAM_OF_STREAM(mine.Bh), Bk = ENGRAM_OF_STREAM(mine.Bk);
#undef ENGRAM_OF_STREAM
        if (on) {
          engram::Chunk8<true> w;
          w.load(w_hi, m * cps + ci);
          float dh[8], dk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float he = h[m][e], ke = k[m][e], de = d[m][e];
            dh[e] = de + (ck * (ke * w[e]) - Bh * he);
            dk[e] = ch * (he * w[e]) - Bk * ke;
            dv[e] = fmaf(alpha, de, dv[e]);
            dw[m][e] = fmaf(cw, he * ke, dw[m][e]);
          }
          engram::Chunk8<F32>::store_nt(a.d_h, (t * hc + m) * cps + ci, dh);
          engram::Chunk8<F32>::store_nt(a.d_kv, (t * (hc + 1) + m) * cps + ci, dk);
        }
        h[m].load(a.h, next * hc + m, a.dim, ci);
        k[m].load(a.kv, next * (hc + 1) + m, a.dim, ci);
        d[m].load_nt(a.d_out, (next * hc + m) * cps + ci);
      }
      if (on) engram::Chunk8<F32>::store_nt(a.d_kv, (t * (hc + 1) + hc) * cps + ci, dv);
    } else {
      if (some && on) store_dead<F32>(a, t, cps, ci);
#pragma unroll
      for (int m = 0; m < HC; ++m) {
        if (m >= hc) break;
        h[m].load(a.h, next * hc + m, a.dim, ci);
        k[m].load(a.kv, next * (hc + 1) + m, a.dim, ci);
        d[m].load_nt(a.d_out, (next * hc + m) * cps + ci);
      }
    }
    v.load(a.kv, next * (hc + 1) + hc, a.dim, ci);
    slot ^= 1;
  }
  if (a.part == nullptr) return;
  // team 0 adds the others' parts, one after another, in w's place
  for (int other = 1; other < teams; ++other) {
    __syncthreads();
    if (team == other && on) {
#pragma unroll
      for (int m = 0; m < HC; ++m) {
        if (m >= hc) break;
        engram::Chunk8<true>::store(w_hi, m * cps + ci, dw[m]);
      }
    }
    __syncthreads();
    if (team == 0 && on) {
#pragma unroll
      for (int m = 0; m < HC; ++m) {
        if (m >= hc) break;
        engram::Chunk8<true> o;
        o.load(w_hi, m * cps + ci);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[m][e] += o[e];
      }
    }
  }
  if (team == 0 && on) {
#pragma unroll
    for (int m = 0; m < HC; ++m) {
      if (m >= hc) break;
      engram::Chunk8<true>::store(a.part, ((int64_t)blockIdx.x * hc + m) * cps + ci, dw[m]);
    }
  }
}

// Any shape, stream by stream, for layers too wide for the other; the block's part of dw is
// added up in the workspace, each value by one thread.
template <bool F32, bool KI8, bool HI8>
__global__ __launch_bounds__(kMaxThreads) void gate_grad_kernel(GateGradArgs a) {
  __shared__ double red_d[2][kMaxThreads / 64];
  __shared__ float red[2][kMaxThreads / 64][3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nwaves = blockDim.x >> 6;
  const int cps = a.dim / 8;
  const bool on = tid < cps;
  const int ci = on ? tid : 0;
  float *part = a.part == nullptr ? nullptr : a.part + (int64_t)blockIdx.x * a.hc * a.dim;
  if (part != nullptr && on) {
    const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int m = 0; m < a.hc; ++m) engram::Chunk8<true>::store(part, m * cps + ci, zero);
  }
  int slot = 0;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    if (engram_dead(a.dead_rule, a.ids[t])) {
      if (on) store_dead<F32>(a, t, cps, ci);
      continue;
    }
    Saved8<KI8, F32> v;
    v.load(a.kv, t * (a.hc + 1) + a.hc, a.dim, ci);
    const float sv = KI8 ? a.kv_scales[t * (a.hc + 1) + a.hc] : 1.f;
    float dv[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int m = 0; m < a.hc; ++m) {
      Saved8<HI8, F32> h;
      Saved8<KI8, F32> k;
      engram::Chunk8<F32> d;
      h.load(a.h, t * a.hc + m, a.dim, ci);
      k.load(a.kv, t * (a.hc + 1) + m, a.dim, ci);
      d.load_nt(a.d_out, (t * a.hc + m) * cps + ci);
      const float sh = HI8 ? a.h_scales[t * a.hc + m] : 1.f;
      const float sk = KI8 ? a.kv_scales[t * (a.hc + 1) + m] : 1.f;
      engram::Chunk8<true> q, kw;
      q.load(a.q_w, (int64_t)m * cps + ci);
      kw.load(a.k_w, (int64_t)m * cps + ci);
      float shh = 0.f, skk = 0.f, sdv = 0.f;
      double dot = 0.0;
      if (on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          shh = fmaf(h[e], h[e], shh);
          skk = fmaf(k[e], k[e], skk);
          sdv = fmaf(d[e], v[e], sdv);
          dot = fma((double)h[e] * (double)k[e], (double)q[e] * (double)kw[e], dot);
        }
      }
      shh = engram::warp_sum(shh);
      skk = engram::warp_sum(skk);
      sdv = engram::warp_sum(sdv);
      dot = warp_sum_d(dot);
      if (lane == 0) {
        red[slot][wave][0] = shh;
        red[slot][wave][1] = skk;
        red[slot][wave][2] = sdv;
        red_d[slot][wave] = dot;
      }
      __syncthreads();
      shh = skk = sdv = 0.f;
      dot = 0.0;
      for (int w = 0; w < nwaves; ++w) {
        shh += red[slot][w][0];
        skk += red[slot][w][1];
        sdv += red[slot][w][2];
        dot += red_d[slot][w];
      }
      slot ^= 1;
      const StreamGrad g = stream_grad(a, shh, skk, sdv, dot, sh, sk, sv);
      if (on) {
        float dh[8], dk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = q[e] * kw[e];
          dh[e] = d[e] + (g.ck * (k[e] * w) - g.Bh * h[e]);
          dk[e] = g.ch * (h[e] * w) - g.Bk * k[e];
          dv[e] = fmaf(g.alpha, d[e], dv[e]);
        }
        if (part != nullptr) {
          engram::Chunk8<true> sum;
          sum.load(part, m * cps + ci);
          float dw[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) dw[e] = fmaf(g.cw, h[e] * k[e], sum[e]);
          engram::Chunk8<true>::store(part, m * cps + ci, dw);
        }
        engram::Chunk8<F32>::store_nt(a.d_h, (t * a.hc + m) * cps + ci, dh);
        engram::Chunk8<F32>::store_nt(a.d_kv, (t * (a.hc + 1) + m) * cps + ci, dk);
      }
    }
    if (on) engram::Chunk8<F32>::store_nt(a.d_kv, (t * (a.hc + 1) + a.hc) * cps + ci, dv);
  }
}

// dq_w and dk_w of 64 columns a block: 16 waves sum every sixteenth block's part, eight
// parts in flight.
constexpr int kSumGroups = 16;

__global__ __launch_bounds__(64 * kSumGroups) void gate_grad_weights_kernel(
    const float *__restrict__ part, int blocks, int n, const float *__restrict__ q_w,
    const float *__restrict__ k_w, float *__restrict__ d_q_w, float *__restrict__ d_k_w,
    int accumulate) {
  __shared__ float red[kSumGroups][64];
  const int lane = threadIdx.x & 63, group = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float sum = 0.f;
  if (col < n) {
    int b = group;
    for (; b + 7 * kSumGroups < blocks; b += 8 * kSumGroups) {
      float v[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = part[(int64_t)(b + x * kSumGroups) * n + col];
      sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; b < blocks; b += kSumGroups) sum += part[(int64_t)b * n + col];
  }
  red[group][lane] = sum;
  __syncthreads();
  if (group != 0 || col >= n) return;
#pragma unroll
  for (int g = 1; g < kSumGroups; ++g) sum += red[g][lane];
  const float q = sum * k_w[col], k = sum * q_w[col];
  d_q_w[col] = accumulate ? d_q_w[col] + q : q;
  d_k_w[col] = accumulate ? d_k_w[col] + k : k;
}

// The launch of a shape: threads a token, teams a block, blocks. The token kernel takes one
// block of wide rows a CU, of the 256, or two of narrow ones, whose teams fill 512 threads;
// the other up to four, as their threads allow.
struct GateGradPlan {
  bool by_token;
  int width, teams, blocks;
};
GateGradPlan plan_of(bool f32, int64_t tokens, int32_t hc, int32_t dim) {
  GateGradPlan p;
  p.width = (dim / 8 + 63) / 64 * 64;
  // eight streams of fp32 numbers do not fit the registers
  p.by_token = p.width <= token_threads(f32, hc) && hc * dim <= kTokenColumns && (!f32 || hc <= 4);
  p.teams = p.by_token && p.width <= 256 ? 512 / p.width : 1;
  const int64_t most = p.by_token ? (p.teams > 1 ? 512 : 256) : p.width <= 128 ? 1024 : p.width <= 320 ? 512 : 256;
  const int64_t turns = (tokens + p.teams - 1) / p.teams;
  p.blocks = (int)(turns < most ? turns : most);
  return p;
}

template <bool F32, bool KI8, bool HI8>
void launch(const GateGradArgs &a, const GateGradPlan &p, hipStream_t stream) {
  const dim3 grid(p.blocks), block(p.width * p.teams);
  const size_t lds = (size_t)a.hc * a.dim * 6;
  if (!p.by_token)
    hipLaunchKernelGGL((gate_grad_kernel<F32, KI8, HI8>), grid, block, 0, stream, a);
  else if (a.hc <= 2)
    hipLaunchKernelGGL((gate_grad_token_kernel<F32, KI8, HI8, 2>), grid, block, lds, stream, a, p.width, p.teams);
  else if (a.hc <= 4)
    hipLaunchKernelGGL((gate_grad_token_kernel<F32, KI8, HI8, 4>), grid, block, lds, stream, a, p.width, p.teams);
  else if constexpr (!F32)
    hipLaunchKernelGGL((gate_grad_token_kernel<F32, KI8, HI8, 8>), grid, block, lds, stream, a, p.width, p.teams);
}

}  // namespace

size_t engram_gate_grad_workspace(bool f32, int64_t tokens, int32_t hc, int32_t dim) {
  return (size_t)plan_of(f32, tokens, hc, dim).blocks * hc * dim * sizeof(float);
}

hipError_t engram_launch_gate_grad(const EngramGateGrad &g, int64_t tokens, int32_t hc, int32_t dim,
                                   float eps, float clamp, int plain, hipStream_t stream) {
  GateGradArgs a;
  a.ids = g.ids;
  a.dead_rule = g.dead_rule;
  a.kv = g.kv;
  a.h = g.h;
  a.kv_scales = g.kv_scales;
  a.h_scales = g.h_scales;
  a.q_w = g.q_w;
  a.k_w = g.k_w;
  a.d_out = g.d_out;
  a.d_h = g.d_h;
  a.d_kv = g.d_kv;
  a.part = g.d_q_w != nullptr ? g.workspace : nullptr;
  a.tokens = (int)tokens;
  a.hc = hc;
  a.dim = dim;
  a.eps = eps;
  a.clamp = clamp;
  a.plain = plain;
  const GateGradPlan p = plan_of(g.f32, tokens, hc, dim);
#define ENGRAM_GATE_GRAD(F)                                                 \
  if (g.kv_i8 && g.h_i8) launch<F, true, true>(a, p, stream); \
  else if (g.kv_i8) launch<F, true, false>(a, p, stream);     \
  else if (g.h_i8) launch<F, false, true>(a, p, stream);      \
  else launch<F, false, false>(a, p, stream)
  if (tokens <= 0) {
    a.part = g.d_q_w;      // no part is read
  } else if (g.f32) {
    ENGRAM_GATE_GRAD(true);
  } else {
    ENGRAM_GATE_GRAD(false);
  }
#undef ENGRAM_GATE_GRAD
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.part == nullptr) return err;
  const int n = hc * dim;
  hipLaunchKernelGGL(gate_grad_weights_kernel, dim3((n + 63) / 64), dim3(64 * kSumGroups), 0, stream,
                     g.workspace, p.blocks, n, g.q_w, g.k_w, g.d_q_w, g.d_k_w, g.accumulate);
  return hipGetLastError();
}
