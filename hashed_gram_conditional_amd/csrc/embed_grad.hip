// Gradient of the table lookup by sorted row ids: dT[r] = scale * sum of d_out[i]
// over the i with row_ids[i] = r, without floating-point atomics, so that the
// same call gives the same bits.
//
//   1. Keys: the row id, or table_rows for an id outside the table (those sort
//      behind every row and are dropped). A stable least-digit radix sort of
//      (key, i) puts each row's occurrences side by side in the order of i.
//      Up to kSmall ids one block sorts in LDS; above, each pass is a
//      histogram per block, a scan per digit and a scatter.
//   2. Runs of equal keys: run u starts at sorted position starts[u]; the number
//      of runs is known only on the device.
//   3. Sums: the sorted positions are cut into chunks of `chunk`; a thread owns
//      one chunk and 8 (bf16) or 4 (fp32) columns, so neighbouring threads read
//      whole rows, and walks the runs that begin in its chunk, adding in fp32 in
//      the order of i. A run longer than kLong is summed piece by piece, a piece
//      per chunk it touches, and
//   4. the pieces are joined: fixed groups of pieces in order, then the groups
//      in order.
//
// Bound by HBM in step 3: d_out is read once, a row's sum written once. The sort
// moves 8 bytes per id and pass.
#include "common.h"
#include "fast_div.h"

namespace {

constexpr int kSmall = 16384;          // ids one block sorts in LDS
constexpr int kSmallThreads = 1024;
constexpr int kSmallItems = kSmall / kSmallThreads;
constexpr int kSmallBits = 8;
constexpr int kLong = 64;              // longest run summed by one thread; >= every chunk

constexpr int kSortThreads = 512;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxBits = 10;           // digit of one pass of the large sort
constexpr int kMaxBlocks = 512;        // blocks of one pass

constexpr int kSumThreads = 256;
constexpr int kJoinThreads = 1024;
constexpr int kJoinChunks = 32;        // chunks one join block looks after

__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t table_rows) {
  return (uint64_t)id < (uint64_t)table_rows ? (uint32_t)id : (uint32_t)table_rows;
}

// Lanes of the wave whose digit equals this lane's (all lanes take part; the
// digit of a lane out of range is one no other lane has).
template <int BITS>
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits) {
  uint64_t mask = ~0ull;
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    if (b < bits) {
      const bool set = (digit >> b) & 1u;
      const uint64_t vote = __ballot(set);
      mask &= set ? vote : ~vote;
    }
  }
  return mask;
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __popcll(mask & ((1ull << (threadIdx.x & 63)) - 1ull));
}

// Inclusive scan over the wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)v, off, engram::kWave);
    if (lane >= off) v += o;
  }
  return v;
}

// Exclusive scan over a block of up to 16 waves; total gets the sum. `part` is
// 17 words of LDS. Every thread must call it.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *part, uint32_t &total) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int waves = blockDim.x >> 6;
  const uint32_t inc = wave_scan(v);
  __syncthreads();
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  if (wave == 0) {
    const uint32_t p = lane < waves ? part[lane] : 0u;
    const uint32_t s = wave_scan(p);
    if (lane < waves) part[lane] = s - p;
    if (lane == waves - 1) part[16] = s;
  }
  __syncthreads();
  total = part[16];
  return part[wave] + inc - v;
}

// What the sums need to know of the sorted ids.
struct Runs {
  const uint32_t *keys;       // [n] sorted
  const uint32_t *order;      // [n] the i of each sorted position
  uint32_t *starts;           // [n + 1] first position of run u; starts[runs] = ids kept
  uint32_t *chunk_run;        // [chunks] the run that holds a chunk's first position
  uint32_t *meta;             // [0] runs, [1] ids kept
  int chunk;
};

// Where the sums go: rows of fp32, at the run's number (compact) or its row id.
struct Sums {
  float *grad;
  int64_t ld;
  int64_t *rows;              // compact: the runs' row ids, then -1 up to n; else NULL
  int64_t *count;             // compact: the number of runs; else NULL
  int dense, accumulate;
};

// Zeroes grad[0 .. rows) x [0 .. dim), groups of 4 or single columns.
__device__ __forceinline__ void zero_grad(const Sums &s, const EngramFastDiv &groups, int vec,
                                          int64_t total, int64_t first, int64_t step) {
  for (int64_t g = first; g < total; g += step) {
    const int64_t row = groups.div(g);
    const int64_t col = g - row * groups.d;
    if (vec)
      *reinterpret_cast<float4 *>(s.grad + row * s.ld + col * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    else
      s.grad[row * s.ld + col] = 0.f;
  }
}

__global__ __launch_bounds__(256) void zero_grad_kernel(Sums s, EngramFastDiv groups, int vec,
                                                        int64_t total) {
  zero_grad(s, groups, vec, total, (int64_t)blockIdx.x * 256 + threadIdx.x,
            (int64_t)gridDim.x * 256);
}

// Block 0: the whole sort and the runs of up to kSmall ids. The other blocks
// (a dense gradient that is not added to) clear the gradient meanwhile.
struct SmallLds {
  uint32_t key[kSmall];
  uint16_t idx[kSmall];
  uint32_t cnt[kSmallThreads / 64][1 << kSmallBits];
  uint32_t part[17];
  uint32_t kept;
};

__global__ __launch_bounds__(kSmallThreads) void small_sort_kernel(
    const int64_t *__restrict__ ids, int n, int64_t table_rows, int bits, Runs r,
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ order_out, Sums s,
    EngramFastDiv zero_groups, int zero_vec, int64_t zero_total) {
  __shared__ SmallLds lds;
  if (blockIdx.x > 0) {
    zero_grad(s, zero_groups, zero_vec, zero_total,
              (int64_t)(blockIdx.x - 1) * kSmallThreads + threadIdx.x,
              (int64_t)(gridDim.x - 1) * kSmallThreads);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int items = (n + kSmallThreads - 1) / kSmallThreads;
  // item i of the thread is position first + 64 i
  const int first = wave * 64 * items + lane;
  for (int p = tid; p < n; p += kSmallThreads) {
    lds.key[p] = key_of(ids[p], table_rows);
    lds.idx[p] = (uint16_t)p;
  }
  if (tid == 0) lds.kept = (uint32_t)n;
  for (int shift = 0; shift < bits; shift += kSmallBits) {
    for (int d = lane; d < (1 << kSmallBits); d += 64) lds.cnt[wave][d] = 0u;
    __syncthreads();
    uint32_t key[kSmallItems], rank[kSmallItems];
    uint16_t idx[kSmallItems];
#pragma unroll
    for (int i = 0; i < kSmallItems; ++i) {
      if (i < items) {
        const int p = first + 64 * i;
        const bool in = p < n;
        key[i] = in ? lds.key[p] : 0u;
        idx[i] = in ? lds.idx[p] : (uint16_t)0;
        const uint32_t d = (key[i] >> shift) & ((1u << kSmallBits) - 1u);
        const uint64_t mask = same_digit<kSmallBits>(d, kSmallBits) & __ballot(in);
        uint32_t before = 0;
        const int leader = mask ? __ffsll((unsigned long long)mask) - 1 : 0;
        if (in && lane == leader) before = atomicAdd(&lds.cnt[wave][d], (uint32_t)__popcll(mask));
        rank[i] = (uint32_t)__shfl((int)before, leader, engram::kWave) + (uint32_t)lanes_below(mask);
      }
    }
    __syncthreads();
    uint32_t sum = 0;
    if (tid < (1 << kSmallBits)) {
#pragma unroll
      for (int w = 0; w < kSmallThreads / 64; ++w) {
        const uint32_t c = lds.cnt[w][tid];
        lds.cnt[w][tid] = sum;
        sum += c;
      }
    }
    uint32_t total;
    const uint32_t base = block_scan(sum, lds.part, total);
    if (tid < (1 << kSmallBits)) {
#pragma unroll
      for (int w = 0; w < kSmallThreads / 64; ++w) lds.cnt[w][tid] += base;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSmallItems; ++i) {
      if (i < items && first + 64 * i < n) {
        const uint32_t d = (key[i] >> shift) & ((1u << kSmallBits) - 1u);
        const uint32_t to = lds.cnt[wave][d] + rank[i];
        lds.key[to] = key[i];
        lds.idx[to] = idx[i];
      }
    }
    __syncthreads();
  }
  __syncthreads();
  uint32_t heads = 0;
  for (int i = 0; i < items; ++i) {
    const int p = first + 64 * i;
    const uint32_t k = p < n ? lds.key[p] : (uint32_t)table_rows;
    const bool head = p < n && k < (uint32_t)table_rows && (p == 0 || lds.key[p - 1] != k);
    heads += (uint32_t)__popcll(__ballot(head));
  }
  uint32_t runs;
  uint32_t at = block_scan(lane == 0 ? heads : 0u, lds.part, runs);
  at = (uint32_t)__shfl((int)at, 0, engram::kWave);
  for (int i = 0; i < items; ++i) {
    const int p = first + 64 * i;
    const uint32_t k = p < n ? lds.key[p] : (uint32_t)table_rows;
    const bool edge = p < n && (p == 0 || lds.key[p - 1] != k);
    const bool head = edge && k < (uint32_t)table_rows;
    const uint64_t vote = __ballot(head);
    const uint32_t upto = at + (uint32_t)lanes_below(vote) + (head ? 1u : 0u);
    at += (uint32_t)__popcll(vote);
    if (p < n) {
      keys_out[p] = k;
      order_out[p] = lds.idx[p];
      if (head) {
        r.starts[upto - 1] = (uint32_t)p;
        if (s.rows != nullptr) s.rows[upto - 1] = (int64_t)k;
      }
      if (k < (uint32_t)table_rows && p % r.chunk == 0) r.chunk_run[p / r.chunk] = upto - 1;
      if (edge && k == (uint32_t)table_rows) lds.kept = (uint32_t)p;
    }
  }
  __syncthreads();
  if (tid == 0) {
    r.starts[runs] = lds.kept;
    r.meta[0] = runs;
    r.meta[1] = lds.kept;
    if (s.count != nullptr) s.count[0] = (int64_t)runs;
  }
}

// ---- the sort of more ids: histogram, scan, scatter per digit ---------------------
// Block b of a pass owns a contiguous range of tiles; counts[d * blocks + b] is
// how many of its keys have digit d, and after the scan how many keys with that
// digit the blocks before it hold.
struct Pass {
  int64_t n;
  int64_t per_block;      // positions of a block, a multiple of kSortTile
  int blocks;
  int shift, bits;
};

template <bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const int64_t *ids, const uint32_t *keys, int64_t p,
                                             int64_t table_rows) {
  return FIRST ? key_of(ids[p], table_rows) : keys[p];
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(
    const int64_t *__restrict__ ids, const uint32_t *__restrict__ keys, int64_t table_rows, Pass a,
    uint32_t *__restrict__ counts) {
  __shared__ uint32_t hist[1 << kMaxBits];
  const int digits = 1 << a.bits;
  for (int d = threadIdx.x; d < digits; d += kSortThreads) hist[d] = 0u;
  __syncthreads();
  const int64_t p0 = blockIdx.x * a.per_block;
  const int64_t p1 = min(a.n, p0 + a.per_block);
  for (int64_t p = p0 + threadIdx.x; p < p1; p += kSortThreads)
    atomicAdd(&hist[(sort_key<FIRST>(ids, keys, p, table_rows) >> a.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kSortThreads)
    counts[(int64_t)d * a.blocks + blockIdx.x] = hist[d];
}

// One block per digit; kMaxBlocks == kSortThreads counts at most.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(uint32_t *__restrict__ counts,
                                                                 uint32_t *__restrict__ totals,
                                                                 int blocks) {
  __shared__ uint32_t part[17];
  uint32_t *c = counts + (int64_t)blockIdx.x * blocks;
  const uint32_t v = (int)threadIdx.x < blocks ? c[threadIdx.x] : 0u;
  uint32_t total;
  const uint32_t before = block_scan(v, part, total);
  if ((int)threadIdx.x < blocks) c[threadIdx.x] = before;
  if (threadIdx.x == 0) totals[blockIdx.x] = total;
}

struct ScatterLds {
  uint32_t base[1 << kMaxBits];
  uint32_t cnt[kSortThreads / 64][1 << kMaxBits];
  uint32_t part[17];
};

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(
    const int64_t *__restrict__ ids, const uint32_t *__restrict__ keys,
    const uint32_t *__restrict__ order, int64_t table_rows, Pass a,
    const uint32_t *__restrict__ counts, const uint32_t *__restrict__ totals,
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ order_out) {
  __shared__ ScatterLds lds;
  constexpr int kWaves = kSortThreads / 64;
  constexpr int kPer = (1 << kMaxBits) / kSortThreads;     // digits of a thread
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int digits = 1 << a.bits;
  {
    uint32_t t[kPer], sum = 0, total;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int d = tid * kPer + k;
      t[k] = d < digits ? totals[d] : 0u;
      sum += t[k];
    }
    uint32_t before = block_scan(sum, lds.part, total);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int d = tid * kPer + k;
      if (d < digits) lds.base[d] = before + counts[(int64_t)d * a.blocks + blockIdx.x];
      before += t[k];
    }
  }
  const int64_t p0 = blockIdx.x * a.per_block;
  const int64_t p1 = min(a.n, p0 + a.per_block);
  for (int64_t tile = p0; tile < p1; tile += kSortTile) {
    for (int d = lane; d < digits; d += 64) lds.cnt[wave][d] = 0u;
    const int64_t first = tile + wave * 64 * kSortItems + lane;
    uint32_t key[kSortItems], idx[kSortItems], rank[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t p = first + 64 * i;
      key[i] = p < p1 ? sort_key<FIRST>(ids, keys, p, table_rows) : 0u;
      idx[i] = FIRST ? (uint32_t)p : p < p1 ? order[p] : 0u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const bool in = first + 64 * i < p1;
      const uint32_t d = (key[i] >> a.shift) & (uint32_t)(digits - 1);
      const uint64_t mask = same_digit<kMaxBits>(d, a.bits) & __ballot(in);
      uint32_t before = 0;
      const int leader = mask ? __ffsll((unsigned long long)mask) - 1 : 0;
      if (in && lane == leader) before = atomicAdd(&lds.cnt[wave][d], (uint32_t)__popcll(mask));
      rank[i] = (uint32_t)__shfl((int)before, leader, engram::kWave) + (uint32_t)lanes_below(mask);
    }
    __syncthreads();
    for (int d = tid; d < digits; d += kSortThreads) {
      uint32_t run = lds.base[d];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const uint32_t c = lds.cnt[w][d];
        lds.cnt[w][d] = run;
        run += c;
      }
      lds.base[d] = run;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      if (first + 64 * i < p1) {
        const uint32_t d = (key[i] >> a.shift) & (uint32_t)(digits - 1);
        const uint32_t to = lds.cnt[wave][d] + rank[i];
        keys_out[to] = key[i];
        order_out[to] = idx[i];
      }
    }
    __syncthreads();
  }
}

// Runs of the sorted keys: the heads of each tile, then their numbers.
__device__ __forceinline__ bool is_edge(const uint32_t *keys, int64_t p, uint32_t k) {
  return p == 0 || keys[p - 1] != k;
}

__global__ __launch_bounds__(kSortThreads) void count_heads_kernel(
    const uint32_t *__restrict__ keys, int64_t n, int64_t table_rows,
    uint32_t *__restrict__ tile_heads) {
  __shared__ uint32_t part[17];
  const int64_t tile = (int64_t)blockIdx.x * kSortTile;
  uint32_t heads = 0, total;
#pragma unroll
  for (int i = 0; i < kSortItems; ++i) {
    const int64_t p = tile + i * kSortThreads + threadIdx.x;
    if (p < n) {
      const uint32_t k = keys[p];
      heads += k < (uint32_t)table_rows && is_edge(keys, p, k) ? 1u : 0u;
    }
  }
  block_scan(heads, part, total);
  if (threadIdx.x == 0) tile_heads[blockIdx.x] = total;
}

__global__ __launch_bounds__(kSortThreads) void write_runs_kernel(
    int64_t n, int64_t table_rows, const uint32_t *__restrict__ tile_heads, Runs r, Sums s) {
  __shared__ uint32_t part[17];
  uint32_t v = 0, at;
  for (int64_t t = threadIdx.x; t < (int64_t)blockIdx.x; t += kSortThreads) v += tile_heads[t];
  block_scan(v, part, at);                      // runs that begin before this tile
  const int64_t tile = (int64_t)blockIdx.x * kSortTile;
  for (int i = 0; i < kSortItems; ++i) {
    const int64_t p = tile + i * kSortThreads + threadIdx.x;
    const uint32_t k = p < n ? r.keys[p] : (uint32_t)table_rows;
    const bool edge = p < n && is_edge(r.keys, p, k);
    const bool head = edge && k < (uint32_t)table_rows;
    uint32_t total;
    const uint32_t upto = at + block_scan(head ? 1u : 0u, part, total) + (head ? 1u : 0u);
    at += total;
    if (p >= n) continue;                       // no barrier follows in this iteration
    if (head) {
      r.starts[upto - 1] = (uint32_t)p;
      if (s.rows != nullptr) s.rows[upto - 1] = (int64_t)k;
    }
    if (k < (uint32_t)table_rows && p % r.chunk == 0) r.chunk_run[p / r.chunk] = upto - 1;
    // the end of the kept ids: the first dropped one, or behind the last position
    const bool dropped = edge && k == (uint32_t)table_rows;
    if (dropped || (p == n - 1 && k < (uint32_t)table_rows)) {
      const uint32_t kept = (uint32_t)(dropped ? p : n);
      r.starts[upto] = kept;
      r.meta[0] = upto;
      r.meta[1] = kept;
      if (s.count != nullptr) s.count[0] = (int64_t)upto;
    }
  }
}

// ---- the sums ----------------------------------------------------------------------
// The last run of the chunk [p0, p1) and whether it begins there and is long.
struct LastRun {
  uint32_t run, start, end;
  bool is_long;
};

__device__ __forceinline__ LastRun last_run(const Runs &r, uint32_t c, uint32_t p0, uint32_t p1,
                                            uint32_t runs, uint32_t kept) {
  LastRun l;
  l.run = runs - 1;
  if (p1 < kept) {
    l.run = r.chunk_run[c + 1];
    if (r.starts[l.run] == p1) --l.run;
  }
  l.start = r.starts[l.run];
  l.end = r.starts[l.run + 1];
  l.is_long = l.start >= p0 && l.end - l.start > (uint32_t)kLong;
  return l;
}

template <bool F32, int VEC>
struct Cols;
template <bool F32>
struct Cols<F32, 8> {
  engram::Chunk8<F32> v;
  __device__ __forceinline__ void load(const void *p, int64_t off) { v.load(p, off / 8); }
  __device__ __forceinline__ float operator[](int e) const { return v[e]; }
};
template <bool F32>
struct Cols<F32, 1> {
  float f;
  __device__ __forceinline__ void load(const void *p, int64_t off) {
    f = F32 ? reinterpret_cast<const float *>(p)[off]
            : engram::bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[off]);
  }
  __device__ __forceinline__ float operator[](int) const { return f; }
};

template <int VEC>
__device__ __forceinline__ void put(float *p, const float (&f)[VEC], bool add) {
  if (VEC == 8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 *q = reinterpret_cast<float4 *>(p) + h;
      float4 o = make_float4(f[4 * h], f[(4 * h + 1) % VEC], f[(4 * h + 2) % VEC], f[(4 * h + 3) % VEC]);
      if (add) {
        const float4 a = *q;
        o = make_float4(a.x + o.x, a.y + o.y, a.z + o.z, a.w + o.w);
      }
      *q = o;
    }
  } else {
    *p = add ? *p + f[0] : f[0];
  }
}

constexpr int kAhead = 8;      // rows of d_out a thread has in flight

template <bool F32, int VEC>
__global__ __launch_bounds__(kSumThreads) void sum_runs_kernel(
    const void *__restrict__ d_out, int64_t out_ld, Runs r, Sums s, float *__restrict__ pieces,
    int64_t piece_ld, int cols, int threads_per_chunk, int64_t chunks, float scale) {
  const int part = threadIdx.x / threads_per_chunk;
  const int per_block = kSumThreads / threads_per_chunk;
  const int64_t chunk = (int64_t)blockIdx.x * per_block + part;
  const int g = blockIdx.y * threads_per_chunk + (threadIdx.x - part * threads_per_chunk);
  if (part >= per_block || chunk >= chunks || g >= cols) return;
  const uint32_t runs = r.meta[0], kept = r.meta[1];
  const uint32_t c = (uint32_t)chunk;
  const uint32_t p0 = c * (uint32_t)r.chunk;
  if (p0 >= kept) return;
  const uint32_t p1 = min(p0 + (uint32_t)r.chunk, kept);
  const int64_t col = (int64_t)g * VEC;

  uint32_t u = r.chunk_run[c];
  uint32_t p = p0;
  const uint32_t s0 = r.starts[u];
  if (s0 < p0) {                      // a run from an earlier chunk leads
    const uint32_t e0 = r.starts[u + 1];
    const uint32_t pe = min(e0, p1);
    if (e0 - s0 > (uint32_t)kLong) {
      float acc[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      for (; p < pe; p += kAhead) {
        Cols<F32, VEC> v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          v[j].load(d_out, (int64_t)r.order[min(p + j, pe - 1)] * out_ld + col);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (p + j < pe) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += v[j][e];
          }
        }
      }
      put<VEC>(pieces + (int64_t)(2 * (uint64_t)c) * piece_ld + col, acc, false);
    }
    p = pe;
    ++u;
  }
  if (p >= p1) return;
  const LastRun l = last_run(r, c, p0, p1, runs, kept);
  const uint32_t end = l.is_long ? p1 : l.end;
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  for (; p < end; p += kAhead) {
    uint32_t k[kAhead + 1];
    Cols<F32, VEC> v[kAhead];
#pragma unroll
    for (int j = 0; j <= kAhead; ++j) k[j] = r.keys[min(p + j, end - 1)];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      v[j].load(d_out, (int64_t)r.order[min(p + j, end - 1)] * out_ld + col);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (p + j >= end) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += v[j][e];
      const bool last = p + j == end - 1;
      if (last || k[j + 1] != k[j]) {
        if (last && l.is_long) {
          put<VEC>(pieces + (int64_t)(2 * (uint64_t)c + 1) * piece_ld + col, acc, false);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] *= scale;
          put<VEC>(s.grad + (int64_t)(s.dense ? k[j] : u) * s.ld + col, acc, s.accumulate);
        }
        ++u;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      }
    }
  }
}

// The long runs: block b joins the pieces of those that begin in its
// kJoinChunks chunks. The threads form groups of one thread per column (4 columns
// where VEC is 4); group g adds a fixed share of the pieces in order, and the
// first group adds the groups in order. Also closes the list of rows with -1.
template <int VEC>
__global__ __launch_bounds__(kJoinThreads) void join_pieces_kernel(
    Runs r, Sums s, const float *__restrict__ pieces, int64_t piece_ld, int cols, int width,
    int64_t chunks, int64_t n, float scale) {
  __shared__ float sums[kJoinThreads * VEC];
  __shared__ uint32_t list[kJoinChunks];
  const int tid = threadIdx.x;
  const uint32_t runs = r.meta[0], kept = r.meta[1];
  const int64_t c0 = (int64_t)blockIdx.x * kJoinChunks;
  if (s.rows != nullptr && blockIdx.y == 0) {
    const int64_t last = min(n, (c0 + kJoinChunks) * r.chunk);
    for (int64_t u = c0 * r.chunk + tid; u < last; u += kJoinThreads)
      if (u >= (int64_t)runs) s.rows[u] = -1;
  }
  if (tid < kJoinChunks) {
    const int64_t c = c0 + tid;
    uint32_t found = 0;
    if (c < chunks && c * r.chunk < (int64_t)kept) {
      const uint32_t p0 = (uint32_t)c * (uint32_t)r.chunk;
      found = last_run(r, (uint32_t)c, p0, min(p0 + (uint32_t)r.chunk, kept), runs, kept).is_long;
    }
    list[tid] = found;
  }
  __syncthreads();
  const int groups = kJoinThreads / width;
  const int group = tid / width;
  const int g = blockIdx.y * width + (tid - group * width);
  const bool active = group < groups && g < cols;
  for (int t = 0; t < kJoinChunks; ++t) {
    if (!list[t]) continue;                     // the same for the whole block
    const uint32_t c = (uint32_t)(c0 + t);
    const uint32_t p0 = c * (uint32_t)r.chunk;
    const LastRun l = last_run(r, c, p0, min(p0 + (uint32_t)r.chunk, kept), runs, kept);
    const int64_t m = (int64_t)((l.end - 1) / (uint32_t)r.chunk) - c + 1;
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    if (active) {
      const int64_t k1 = m * (group + 1) / groups;
      for (int64_t k = m * group / groups; k < k1; k += kAhead) {
        float v[kAhead][VEC];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int64_t kk = k + j < k1 ? k + j : k1 - 1;
          const float *q = pieces + (kk == 0 ? 2 * (int64_t)c + 1 : 2 * ((int64_t)c + kk)) * piece_ld +
                           (int64_t)g * VEC;
          if (VEC == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(q);
            v[j][0] = x.x; v[j][1 % VEC] = x.y; v[j][2 % VEC] = x.z; v[j][3 % VEC] = x.w;
          } else {
            v[j][0] = *q;
          }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (k + j < k1) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[e] += v[j][e];
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sums[e * kJoinThreads + tid] = acc[e];
    __syncthreads();
    if (active && group == 0) {
      for (int q = 1; q < groups; ++q) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += sums[e * kJoinThreads + q * width + tid];
      }
      float *dst = s.grad + (int64_t)(s.dense ? r.keys[l.start] : l.run) * s.ld + (int64_t)g * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        dst[e] = s.accumulate ? dst[e] + acc[e] * scale : acc[e] * scale;
    }
    __syncthreads();
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The workspace of a call, and how it is cut.
struct Plan {
  int64_t n, chunks, tiles;
  int chunk, bits, passes, digit;
  bool vec;
  int64_t piece_ld;
  size_t keys[2], order[2], counts, totals, tile_heads, starts, chunk_run, meta, pieces, bytes;
  Pass pass;
};

// Chunks of 64 positions where those give every CU 2048 threads, else shorter
// ones down to 8, so that small calls use the chip.
Plan make_plan(const EngramEmbedArgs &a) {
  Plan p;
  p.n = a.n_ids;
  p.vec = a.dim % 8 == 0 && a.out_ld % 8 == 0 && a.grad_ld % 4 == 0;
  const int64_t per_chunk = p.vec ? a.dim / 8 : a.dim;
  p.chunk = kLong;
  while (p.chunk > 8 && (p.n / p.chunk) * per_chunk < (int64_t)256 * 2048) p.chunk /= 2;
  p.chunks = (p.n + p.chunk - 1) / p.chunk;
  p.bits = 1;
  while (p.bits < 32 && (a.table_rows >> p.bits) != 0) ++p.bits;
  p.passes = (p.bits + kMaxBits - 1) / kMaxBits;
  p.digit = (p.bits + p.passes - 1) / p.passes;
  p.tiles = (p.n + kSortTile - 1) / kSortTile;
  const int64_t per = p.tiles > 0 ? (p.tiles + kMaxBlocks - 1) / kMaxBlocks : 1;
  p.pass.n = p.n;
  p.pass.per_block = per * kSortTile;
  p.pass.blocks = (int)((p.tiles + per - 1) / per);
  p.piece_ld = ((int64_t)a.dim + 3) / 4 * 4;
  const bool large = p.n > kSmall;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = i == 0 || large ? take((size_t)p.n * 4) : 0;
    p.order[i] = i == 0 || large ? take((size_t)p.n * 4) : 0;
  }
  p.counts = take(large ? ((size_t)p.pass.blocks << p.digit) * 4 : 0);
  p.totals = take(large ? (size_t)4 << p.digit : 0);
  p.tile_heads = take(large ? (size_t)p.tiles * 4 : 0);
  p.starts = take((size_t)(p.n + 1) * 4);
  p.chunk_run = take((size_t)p.chunks * 4);
  p.meta = take(8);
  p.pieces = take((size_t)p.chunks * 2 * (size_t)p.piece_ld * 4);
  p.bytes = at;
  return p;
}

template <bool F32, int VEC>
void launch_sums(const EngramEmbedArgs &a, const Plan &p, const void *d_out, const Runs &r,
                 const Sums &s, float *pieces, hipStream_t stream) {
  const int cols = VEC == 8 ? a.dim / 8 : a.dim;
  const int slices = (cols + kSumThreads - 1) / kSumThreads;
  const int width = (cols + slices - 1) / slices;
  const int per_block = kSumThreads / width;
  const dim3 grid((unsigned)((p.chunks + per_block - 1) / per_block), (unsigned)slices);
  hipLaunchKernelGGL((sum_runs_kernel<F32, VEC>), grid, dim3(kSumThreads), 0, stream, d_out,
                     a.out_ld, r, s, pieces, p.piece_ld, cols, width, p.chunks, a.scale);
}

template <int VEC>
void launch_join(const EngramEmbedArgs &a, const Plan &p, const Runs &r, const Sums &s,
                 const float *pieces, hipStream_t stream) {
  const int cols = VEC == 4 ? a.dim / 4 : a.dim;
  const int slices = (cols + 255) / 256;
  const int width = (cols + slices - 1) / slices;
  const dim3 grid((unsigned)((p.chunks + kJoinChunks - 1) / kJoinChunks), (unsigned)slices);
  hipLaunchKernelGGL((join_pieces_kernel<VEC>), grid, dim3(kJoinThreads), 0, stream, r, s, pieces,
                     p.piece_ld, cols, width, p.chunks, p.n, a.scale);
}

}  // namespace

size_t engram_embed_grad_workspace(const EngramEmbedArgs &a) { return make_plan(a).bytes; }

hipError_t engram_launch_embed_grad(const EngramEmbedArgs &a, const void *d_out,
                                    const int64_t *row_ids, float *grad, int64_t *grad_rows,
                                    int64_t *n_rows, int accumulate, void *workspace,
                                    hipStream_t stream) {
  const Plan p = make_plan(a);
  uint8_t *ws = (uint8_t *)workspace;
  uint32_t *keys[2] = {(uint32_t *)(ws + p.keys[0]), (uint32_t *)(ws + p.keys[1])};
  uint32_t *order[2] = {(uint32_t *)(ws + p.order[0]), (uint32_t *)(ws + p.order[1])};
  uint32_t *counts = (uint32_t *)(ws + p.counts), *totals = (uint32_t *)(ws + p.totals);
  uint32_t *tile_heads = (uint32_t *)(ws + p.tile_heads);
  float *pieces = (float *)(ws + p.pieces);
  const bool dense = n_rows == nullptr;
  const Sums s{grad, a.grad_ld, grad_rows, n_rows, dense ? 1 : 0, accumulate};
  const int zero_vec = a.dim % 4 == 0 && a.grad_ld % 4 == 0 ? 1 : 0;
  const EngramFastDiv zero_groups(zero_vec ? a.dim / 4 : a.dim);
  const int64_t zero_total = dense && !accumulate ? a.table_rows * zero_groups.d : 0;
  Runs r{keys[0], order[0], (uint32_t *)(ws + p.starts), (uint32_t *)(ws + p.chunk_run),
         (uint32_t *)(ws + p.meta), p.chunk};
  if (p.n <= kSmall) {
    const int64_t want = (zero_total + (int64_t)kSmallThreads * 4 - 1) / (kSmallThreads * 4);
    const unsigned blocks = 1u + (unsigned)(want < 1024 ? want : 1024);
    hipLaunchKernelGGL(small_sort_kernel, dim3(blocks), dim3(kSmallThreads), 0, stream, row_ids,
                       (int)p.n, a.table_rows, p.bits, r, keys[0], order[0], s, zero_groups,
                       zero_vec, zero_total);
  } else {
    if (zero_total > 0) {
      const int64_t want = (zero_total + 256 * 4 - 1) / (256 * 4);
      hipLaunchKernelGGL(zero_grad_kernel, dim3((unsigned)(want < 8192 ? want : 8192)), dim3(256), 0,
                         stream, s, zero_groups, zero_vec, zero_total);
    }
    Pass pass = p.pass;
    int at = 1;                       // the buffers the next pass writes are 1 - at
    for (int i = 0; i < p.passes; ++i) {
      pass.shift = i * p.digit;
      pass.bits = p.digit;
      const dim3 grid((unsigned)pass.blocks), block(kSortThreads);
      if (i == 0)
        hipLaunchKernelGGL(sort_count_kernel<true>, grid, block, 0, stream, row_ids,
                           (const uint32_t *)nullptr, a.table_rows, pass, counts);
      else
        hipLaunchKernelGGL(sort_count_kernel<false>, grid, block, 0, stream, row_ids,
                           (const uint32_t *)keys[at], a.table_rows, pass, counts);
      hipLaunchKernelGGL(sort_scan_kernel, dim3(1u << p.digit), block, 0, stream, counts, totals,
                         pass.blocks);
      if (i == 0)
        hipLaunchKernelGGL(sort_scatter_kernel<true>, grid, block, 0, stream, row_ids,
                           (const uint32_t *)nullptr, (const uint32_t *)nullptr, a.table_rows, pass,
                           counts, totals, keys[1 - at], order[1 - at]);
      else
        hipLaunchKernelGGL(sort_scatter_kernel<false>, grid, block, 0, stream, row_ids,
                           (const uint32_t *)keys[at], (const uint32_t *)order[at], a.table_rows,
                           pass, counts, totals, keys[1 - at], order[1 - at]);
      at = 1 - at;
    }
    r.keys = keys[at];
    r.order = order[at];
    hipLaunchKernelGGL(count_heads_kernel, dim3((unsigned)p.tiles), dim3(kSortThreads), 0, stream,
                       r.keys, p.n, a.table_rows, tile_heads);
    hipLaunchKernelGGL(write_runs_kernel, dim3((unsigned)p.tiles), dim3(kSortThreads), 0, stream,
                       p.n, a.table_rows, tile_heads, r, s);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || p.n == 0) return err;
  if (p.vec) {
    if (a.out_f32) launch_sums<true, 8>(a, p, d_out, r, s, pieces, stream);
    else launch_sums<false, 8>(a, p, d_out, r, s, pieces, stream);
    launch_join<4>(a, p, r, s, pieces, stream);
  } else {
    if (a.out_f32) launch_sums<true, 1>(a, p, d_out, r, s, pieces, stream);
    else launch_sums<false, 1>(a, p, d_out, r, s, pieces, stream);
    launch_join<1>(a, p, r, s, pieces, stream);
  }
  return hipGetLastError();
}
