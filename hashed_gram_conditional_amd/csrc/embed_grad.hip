// Gradient of the table lookup by sorted row ids: dT[r] = scale * sum of d_out[i]
// over the i with row_ids[i] = r, without floating-point atomics, so that the
// same call gives the same bits.
//
//   1. Keys: the row id, or table_rows for an id outside the table (those sort
//      behind every row and are dropped). A stable sort of (key, i) puts each
//      row's occurrences side by side in the order of i. Up to kSmall ids, parts
//      of kPart are sorted by counting and merged by rank: an element's place is
//      its place in its own part plus, for every other part, a binary search.
//      Above, a least-digit radix sort: each pass is a histogram per block, a scan
//      per digit and a scatter. (Three launches of 5 to 7 us against eight of 5 to 19
//      us; at 32768 ids of 256 the whole gradient takes 56 us with the merge and 65 to
//      77 with the radix sort.)
//   2. Runs of equal keys: run u starts at sorted position starts[u]; the number
//      of runs is known only on the device.
//   3. Sums: the sorted positions are cut into chunks of `chunk`; a thread owns
//      one chunk and 8 columns (one, where the width or a stride is no whole number
//      of groups), so neighbouring threads read whole rows, and walks the runs that begin in its chunk, adding in fp32 in
//      the order of i. A run longer than `longest` is summed piece by piece, a
//      piece per chunk it touches, and
//   4. the pieces are joined: fixed groups of pieces in order, then the groups
//      in order.
//
// Bound by HBM in step 3: d_out is read once, a row's sum written once. 786432 ids of
// 256 bf16 take 302 us: 69 for the sort and the runs, 223 for the sums (1.02 GB, 4.6
// TB/s), 10 for the join; 255 columns, one value at a time, 405. Small calls are bound by
// the latency of their five launches: 12216 ids take 28 us.
#include "common.h"
#include "fast_div.h"

namespace {

constexpr int kPart = 256;             // ids a block sorts, one per thread
constexpr int kSmall = 32768;          // ids whose keys one block holds in LDS to merge
constexpr int kMergeThreads = 1024;
constexpr int kMergeElems = 64;
constexpr int kMaxChunk = 64;          // positions of a chunk, at most

constexpr int kSortThreads = 512;
constexpr int kSortItems = 8;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxBits = 11;           // digit of one pass of the large sort
constexpr int kMaxBlocks = 1024;       // blocks of one pass
constexpr int kScanThreads = 1024;
constexpr int kScanDigits = 32;

constexpr int kSumThreads = 256;
constexpr int kJoinThreads = 512;
constexpr int kJoinChunks = 8;         // chunks one join block looks after
constexpr int kFewPieces = 16;         // pieces of a run that one group of threads joins
constexpr int kJoinFan = 16;           // groups whose sums one group adds at a time

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

// Ranks of a wave's items among those of equal digit, items in order and lanes in
// order within an item: rank[i] = how many came before. cnt counts the wave's digits
// (zeroed before). A wave's LDS operations run in program order, so the counters'
// additions need no wait between them.
template <int BITS, int ITEMS, class Digit, class In>
__device__ __forceinline__ void wave_ranks(uint32_t *cnt, int bits, Digit digit, In in,
                                           uint32_t (&rank)[ITEMS]) {
  const int lane = threadIdx.x & 63;
  uint32_t before[ITEMS];
  int leader[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const uint32_t d = digit(i);
    const bool mine = in(i);
    const uint64_t mask = same_digit<BITS>(d, bits) & __ballot(mine);
    leader[i] = mask ? __ffsll((unsigned long long)mask) - 1 : 0;
    rank[i] = (uint32_t)lanes_below(mask);
    before[i] = 0;
    if (mine && lane == leader[i]) before[i] = atomicAdd(&cnt[d], (uint32_t)__popcll(mask));
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) rank[i] += (uint32_t)__shfl((int)before[i], leader[i], engram::kWave);
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
  const uint2 *pairs;         // [n] sorted (key, i)
  uint32_t *starts;           // [n + 1] first position of run u; starts[runs] = ids kept
  uint32_t *chunk_run;        // [chunks] the run that holds a chunk's first position
  uint32_t *meta;             // [0] runs, [1] ids kept
  int chunk, chunk_log2;      // positions of a chunk, a power of two
  int longest;                // >= chunk
};

// Where the sums go: rows of fp32, at the run's number (compact) or its row id.
struct Sums {
  float *grad;
  int64_t ld;
  int64_t *rows;              // compact: the runs' row ids, then -1 up to n; else NULL
  int64_t *count;             // compact: the number of runs; else NULL
  int dense, accumulate;
};

// Zeroes grad[0 .. rows) x [0 .. dim): dense rows as one array, else by groups of 4
// or single columns.
struct Zero {
  EngramFastDiv groups;
  int64_t begin, end;         // groups to clear
  int vec, flat;
};

__device__ __forceinline__ void zero_grad(const Sums &s, const Zero &z, int64_t first, int64_t step) {
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  if (z.flat) {
#pragma unroll 4
    for (int64_t g = z.begin + first; g < z.end; g += step)
      reinterpret_cast<float4 *>(s.grad)[g] = none;
    return;
  }
  for (int64_t g = z.begin + first; g < z.end; g += step) {
    const int64_t row = z.groups.div(g);
    const int64_t col = g - row * z.groups.d;
    if (z.vec)
      *reinterpret_cast<float4 *>(s.grad + row * s.ld + col * 4) = none;
    else
      s.grad[row * s.ld + col] = 0.f;
  }
}

// ---- the sort of up to kSmall ids -------------------------------------------------
// The first blocks of a launch do its work; the others (a dense gradient that is not
// added to) clear their share of the gradient meanwhile.
template <int THREADS>
__device__ __forceinline__ bool zero_block(const Sums &s, const Zero &z, int blocks) {
  if ((int)blockIdx.x < blocks) return false;
  zero_grad(s, z, (int64_t)(blockIdx.x - blocks) * THREADS + threadIdx.x,
            (int64_t)(gridDim.x - blocks) * THREADS);
  return true;
}

// Block b: part b in order. A thread counts the part's keys that come before its own:
// in earlier waves the keys not above it, in later waves those below it.
__global__ __launch_bounds__(kPart) void sort_part_kernel(const int64_t *__restrict__ ids, int n,
                                                          int64_t table_rows, uint2 *__restrict__ out,
                                                          int parts, Sums s, Zero z) {
  __shared__ __align__(16) uint32_t keys[kPart];
  if (zero_block<kPart>(s, z, parts)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int p0 = blockIdx.x * kPart;
  const bool in = p0 + tid < n;
  // behind the end: above every key, so that it comes before none
  const uint32_t key = in ? key_of(ids[p0 + tid], table_rows) : UINT32_MAX;
  keys[tid] = key;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int w = 0; w < kPart / 64; ++w) {
    const uint32_t bound = key + (w < wave ? 1u : 0u);
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const uint4 k = reinterpret_cast<const uint4 *>(keys)[w * 16 + q];
      before += (k.x < bound ? 1u : 0u) + (k.y < bound ? 1u : 0u) + (k.z < bound ? 1u : 0u) +
                (k.w < bound ? 1u : 0u);
    }
  }
  // equal keys of the own wave, in the order of the lanes
#pragma unroll
  for (int l = 0; l < 64; ++l) {
    const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)key, l);
    before += k == key && l < lane ? 1u : 0u;
  }
  if (in) out[p0 + before] = make_uint2(key, (uint32_t)(p0 + tid));
}

// Each block places kMergeElems elements of the sorted parts. Thread (q, e) finds how
// many keys of parts q, q + 16, ... come before element e: an equal key of
// an earlier part does, one of a later part does not.
__global__ __launch_bounds__(kMergeThreads) void merge_parts_kernel(const uint2 *__restrict__ in, int n,
                                                                    uint2 *__restrict__ out, int blocks,
                                                                    Sums s, Zero z) {
  __shared__ uint32_t keys[kSmall];
  __shared__ uint32_t place[kMergeElems];
  if (zero_block<kMergeThreads>(s, z, blocks)) return;
  const int tid = threadIdx.x;
  const int e = blockIdx.x * kMergeElems + (tid & (kMergeElems - 1));
  if (tid < kMergeElems) place[tid] = (uint32_t)(e % kPart);
#pragma unroll 8
  for (int p = tid; p < n; p += kMergeThreads) keys[p] = in[p].x;
  __syncthreads();
  if (e < n) {
    const uint32_t key = keys[e];
    const int mine = e / kPart;
    const int parts = (n + kPart - 1) / kPart;
    uint32_t before = 0;
    for (int q = tid / kMergeElems; q < parts; q += kMergeThreads / kMergeElems) {
      if (q == mine) continue;
      const uint32_t *k = keys + q * kPart;
      const int count = min(kPart, n - q * kPart);
      const uint32_t bound = key + (q < mine ? 1u : 0u);
      int at = 0;
#pragma unroll
      for (int step = kPart / 2; step > 0; step >>= 1)
        if (at + step <= count && k[at + step - 1] < bound) at += step;
      if (at < count && k[at] < bound) ++at;
      before += (uint32_t)at;
    }
    atomicAdd(&place[tid & (kMergeElems - 1)], before);
  }
  __syncthreads();
  if (tid < kMergeElems && e < n) out[place[tid]] = in[e];
}
static_assert(kPart % kMergeElems == 0, "a merge block stays within one part");

// ---- the sort of more ids: histogram, scan, scatter per digit ---------------------
// Block b of a pass owns a contiguous range of tiles; counts[b * digits + d] is
// how many of its keys have digit d, and after the scan how many keys with that
// digit the blocks before it hold.
struct Pass {
  int64_t n;
  int64_t per_block;      // positions of a block, a multiple of kSortTile
  int blocks;
  int shift, bits;
};

template <bool FIRST>
__device__ __forceinline__ uint2 sort_pair(const int64_t *ids, const uint2 *pairs, int64_t p,
                                           int64_t table_rows) {
  return FIRST ? make_uint2(key_of(ids[p], table_rows), (uint32_t)p) : pairs[p];
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(
    const int64_t *__restrict__ ids, const uint2 *__restrict__ pairs, int64_t table_rows, Pass a,
    uint32_t *__restrict__ counts, Sums s, Zero z) {
  __shared__ uint32_t hist[1 << kMaxBits];
  if (zero_block<kSortThreads>(s, z, a.blocks)) return;
  const int digits = 1 << a.bits;
  for (int d = threadIdx.x; d < digits; d += kSortThreads) hist[d] = 0u;
  __syncthreads();
  const int64_t p0 = blockIdx.x * a.per_block;
  const int64_t p1 = min(a.n, p0 + a.per_block);
#pragma unroll 4
  for (int64_t p = p0 + threadIdx.x; p < p1; p += kSortThreads)
    atomicAdd(&hist[(sort_pair<FIRST>(ids, pairs, p, table_rows).x >> a.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kSortThreads)
    counts[(int64_t)blockIdx.x * digits + d] = hist[d];
}

// A block scans kScanDigits neighbouring digits: thread (g, d) adds up its share of
// the blocks' counts, the shares are scanned in LDS, then each count is replaced.
__global__ __launch_bounds__(kScanThreads) void sort_scan_kernel(uint32_t *__restrict__ counts,
                                                                 uint32_t *__restrict__ totals,
                                                                 int blocks, int digits) {
  constexpr int kShares = kScanThreads / kScanDigits;
  __shared__ uint32_t sums[kShares][kScanDigits];
  const int d = threadIdx.x % kScanDigits, g = threadIdx.x / kScanDigits;
  const int digit = blockIdx.x * kScanDigits + d;
  const bool in = digit < digits;
  const int b0 = blocks * g / kShares, b1 = blocks * (g + 1) / kShares;
  uint32_t sum = 0;
  if (in) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += counts[(int64_t)b * digits + digit];
  }
  sums[g][d] = sum;
  __syncthreads();
  uint32_t run = 0;
  for (int q = 0; q < g; ++q) run += sums[q][d];
  if (!in) return;
  if (g == kShares - 1) totals[digit] = run + sum;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) {
    const uint32_t c = counts[(int64_t)b * digits + digit];
    counts[(int64_t)b * digits + digit] = run;
    run += c;
  }
}

struct ScatterLds {
  uint32_t base[1 << kMaxBits];
  uint32_t cnt[kSortThreads / 64][1 << kMaxBits];
  uint32_t part[17];
};

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(
    const int64_t *__restrict__ ids, const uint2 *__restrict__ pairs, int64_t table_rows, Pass a,
    const uint32_t *__restrict__ counts, const uint32_t *__restrict__ totals,
    uint2 *__restrict__ out) {
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
      if (d < digits) lds.base[d] = before + counts[(int64_t)blockIdx.x * digits + d];
      before += t[k];
    }
  }
  const int64_t p0 = blockIdx.x * a.per_block;
  const int64_t p1 = min(a.n, p0 + a.per_block);
  for (int64_t tile = p0; tile < p1; tile += kSortTile) {
    for (int d = lane; d < digits; d += 64) lds.cnt[wave][d] = 0u;
    const int64_t first = tile + wave * 64 * kSortItems + lane;
    uint2 pair[kSortItems];
    uint32_t rank[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
      const int64_t p = first + 64 * i;
      pair[i] = p < p1 ? sort_pair<FIRST>(ids, pairs, p, table_rows) : make_uint2(0u, 0u);
    }
    __syncthreads();
    wave_ranks<kMaxBits, kSortItems>(
        lds.cnt[wave], a.bits, [&](int i) { return (pair[i].x >> a.shift) & (uint32_t)(digits - 1); },
        [&](int i) { return first + 64 * i < p1; }, rank);
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
        const uint32_t d = (pair[i].x >> a.shift) & (uint32_t)(digits - 1);
        out[lds.cnt[wave][d] + rank[i]] = pair[i];
      }
    }
    __syncthreads();
  }
}

// ---- the runs ----------------------------------------------------------------------
// Item i of a thread is position first + 64 i, so a wave's positions are contiguous.
template <int ITEMS>
__device__ __forceinline__ void load_heads(const uint2 *pairs, int64_t n, int64_t first, uint32_t none,
                                           uint32_t (&key)[ITEMS], uint32_t (&before)[ITEMS]) {
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t p = first + 64 * i;
    key[i] = p < n ? pairs[p].x : none;
    before[i] = p > 0 && p < n ? pairs[p - 1].x : ~key[i];
  }
}

// The runs that begin in this block's tile, `earlier` runs beginning before it.
template <int ITEMS>
__device__ __forceinline__ void write_runs(int64_t n, int64_t first, uint32_t table_rows, uint32_t earlier,
                                           const uint32_t (&key)[ITEMS], const uint32_t (&before)[ITEMS],
                                           const Runs &r, const Sums &s, uint32_t *part) {
  const int lane = threadIdx.x & 63;
  uint32_t heads = 0, total;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
    heads += (uint32_t)__popcll(__ballot(key[i] < table_rows && before[i] != key[i]));
  uint32_t at = block_scan(lane == 0 ? heads : 0u, part, total);
  at = earlier + (uint32_t)__shfl((int)at, 0, engram::kWave);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int64_t p = first + 64 * i;
    const bool in = p < n;
    const bool edge = in && before[i] != key[i];
    const bool valid = key[i] < table_rows;
    const uint64_t vote = __ballot(edge && valid);
    const uint32_t upto = at + (uint32_t)lanes_below(vote) + (edge && valid ? 1u : 0u);
    at += (uint32_t)__popcll(vote);
    if (edge && valid) {
      r.starts[upto - 1] = (uint32_t)p;
      if (s.rows != nullptr) s.rows[upto - 1] = (int64_t)key[i];
    }
    if (in && valid && (p & (r.chunk - 1)) == 0) r.chunk_run[p >> r.chunk_log2] = upto - 1;
    // the end of the kept ids: the first dropped one, or behind the last position
    const bool dropped = edge && !valid;
    if (dropped || (p == n - 1 && valid)) {
      const uint32_t kept = (uint32_t)(dropped ? p : n);
      r.starts[upto] = kept;
      r.meta[0] = upto;
      r.meta[1] = kept;
      if (s.count != nullptr) s.count[0] = (int64_t)upto;
    }
  }
}

// Up to kSmall sorted ids: each block counts the heads before its tile itself.
constexpr int kSmallTile = 1024;
__global__ __launch_bounds__(kSmallTile) void small_runs_kernel(int n, int64_t table_rows, Runs r,
                                                                int blocks, Sums s, Zero z) {
  __shared__ uint32_t part[17];
  if (zero_block<kSmallTile>(s, z, blocks)) return;
  const int tid = threadIdx.x;
  const uint32_t none = (uint32_t)table_rows;
  if (n == 0) {
    if (tid == 0) {
      r.meta[0] = r.meta[1] = 0u;
      if (s.count != nullptr) s.count[0] = 0;
    }
    return;
  }
  const int64_t tile = (int64_t)blockIdx.x * kSmallTile;
  uint32_t key[1], before[1], heads = 0, earlier;
  load_heads<1>(r.pairs, n, tile + tid, none, key, before);
#pragma unroll 8
  for (int64_t p = tid; p < tile; p += kSmallTile) {
    const uint32_t k = r.pairs[p].x, b = p > 0 ? r.pairs[p - 1].x : ~k;
    heads += k < none && b != k ? 1u : 0u;
  }
  block_scan(heads, part, earlier);
  write_runs<1>(n, tile + tid, none, earlier, key, before, r, s, part);
}

// More: the heads of each tile, then their numbers.
constexpr int kHeadThreads = 512;
constexpr int kHeadItems = 8;
constexpr int kHeadTile = kHeadThreads * kHeadItems;

__global__ __launch_bounds__(kHeadThreads) void count_heads_kernel(
    const uint2 *__restrict__ pairs, int64_t n, int64_t table_rows, uint32_t *__restrict__ tile_heads) {
  __shared__ uint32_t part[17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t key[kHeadItems], before[kHeadItems], heads = 0, total;
  load_heads<kHeadItems>(pairs, n, (int64_t)blockIdx.x * kHeadTile + wave * 64 * kHeadItems + lane,
                         (uint32_t)table_rows, key, before);
#pragma unroll
  for (int i = 0; i < kHeadItems; ++i)
    heads += key[i] < (uint32_t)table_rows && before[i] != key[i] ? 1u : 0u;
  block_scan(heads, part, total);
  if (threadIdx.x == 0) tile_heads[blockIdx.x] = total;
}

__global__ __launch_bounds__(kHeadThreads) void write_runs_kernel(
    int64_t n, int64_t table_rows, const uint32_t *__restrict__ tile_heads, Runs r, Sums s) {
  __shared__ uint32_t part[17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t first = (int64_t)blockIdx.x * kHeadTile + wave * 64 * kHeadItems + lane;
  uint32_t key[kHeadItems], before[kHeadItems];
  load_heads<kHeadItems>(r.pairs, n, first, (uint32_t)table_rows, key, before);
  uint32_t v = 0, earlier;
  for (int64_t t = threadIdx.x; t < (int64_t)blockIdx.x; t += kHeadThreads) v += tile_heads[t];
  block_scan(v, part, earlier);
  write_runs<kHeadItems>(n, first, (uint32_t)table_rows, earlier, key, before, r, s, part);
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
  l.is_long = l.start >= p0 && l.end - l.start > (uint32_t)r.longest;
  return l;
}

template <bool F32, int VEC>
struct Cols;
template <bool F32>
struct Cols<F32, 8> {
  engram::Chunk8<F32> v;
  __device__ __forceinline__ void load(const void *p, int64_t off) { v.load_nt(p, off / 8); }
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
    if (e0 - s0 > (uint32_t)r.longest) {
      float acc[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      for (; p < pe; p += kAhead) {
        Cols<F32, VEC> v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          v[j].load(d_out, (int64_t)r.pairs[min(p + j, pe - 1)].y * out_ld + col);
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
    uint2 k[kAhead + 1];
    Cols<F32, VEC> v[kAhead];
#pragma unroll
    for (int j = 0; j <= kAhead; ++j) k[j] = r.pairs[min(p + j, end - 1)];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) v[j].load(d_out, (int64_t)k[j].y * out_ld + col);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (p + j >= end) continue;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] += v[j][e];
      const bool last = p + j == end - 1;
      if (last || k[j + 1].x != k[j].x) {
        if (last && l.is_long) {
          put<VEC>(pieces + (int64_t)(2 * (uint64_t)c + 1) * piece_ld + col, acc, false);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] *= scale;
          put<VEC>(s.grad + (int64_t)(s.dense ? k[j].x : u) * s.ld + col, acc, s.accumulate);
        }
        ++u;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      }
    }
  }
}

// The pieces [k0, k1) of the long run that begins in chunk c, added in order.
template <int VEC>
__device__ __forceinline__ void add_pieces(const float *__restrict__ pieces, int64_t piece_ld, int64_t col,
                                           int64_t c, int64_t k0, int64_t k1, float (&acc)[VEC]) {
  for (int64_t k = k0; k < k1; k += kAhead) {
    float v[kAhead][VEC];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t kk = k + j < k1 ? k + j : k1 - 1;
      const float *q = pieces + (kk == 0 ? 2 * c + 1 : 2 * (c + kk)) * piece_ld + col;
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

// The long runs: block b joins the pieces of those that begin in its kJoinChunks
// chunks. The threads form groups of one thread per column (4 columns where VEC is
// 4). A run of few pieces is one group's, added in order; of a longer one each group
// adds a fixed share of the pieces in order, every kJoinFan-th one the groups up to the
// next such, and the first group those. With 8 to 512 groups a term of a run of m so
// passes through fewer than 200 + m / 64 additions: 64 of its chunk, m / (8 * 8) + 2 of its
// group, 16 and 32 of the groups. (The first group adding all of them, 512 for narrow
// rows, took 4096 ids of one row through 520, and 29 us for 25 at one column.)
// Also closes the list of rows with -1.
template <int VEC>
__global__ __launch_bounds__(kJoinThreads) void join_pieces_kernel(
    Runs r, Sums s, const float *__restrict__ pieces, int64_t piece_ld, int cols, int width,
    int64_t chunks, int64_t n, float scale) {
  __shared__ float sums[kJoinThreads * VEC];
  __shared__ LastRun list[kJoinChunks];
  const int tid = threadIdx.x;
  const uint32_t runs = r.meta[0], kept = r.meta[1];
  const int64_t c0 = (int64_t)blockIdx.x * kJoinChunks;
  if (s.rows != nullptr && blockIdx.y == 0) {
    const int64_t last = min(n, (c0 + kJoinChunks) * r.chunk);
    for (int64_t u = c0 * r.chunk + tid; u < last; u += kJoinThreads)
      if (u >= (int64_t)runs) s.rows[u] = -1;
  }
  bool any = false;
  if (tid < kJoinChunks) {
    const int64_t c = c0 + tid;
    LastRun l;
    l.is_long = false;
    if (c < chunks && c * r.chunk < (int64_t)kept) {
      const uint32_t p0 = (uint32_t)c * (uint32_t)r.chunk;
      l = last_run(r, (uint32_t)c, p0, min(p0 + (uint32_t)r.chunk, kept), runs, kept);
    }
    list[tid] = l;
    any = l.is_long;
  }
  if (!__syncthreads_or(any)) return;
  const int groups = kJoinThreads / width;
  const int group = tid / width;
  const int g = blockIdx.y * width + (tid - group * width);
  const bool active = group < groups && g < cols;
  const int64_t col = (int64_t)g * VEC;
  const auto count = [&](int t) {
    return (int64_t)((list[t].end - 1) >> r.chunk_log2) - (c0 + t) + 1;
  };
  const auto store = [&](const LastRun &l, const float (&acc)[VEC]) {
    float *dst = s.grad + (int64_t)(s.dense ? r.pairs[l.start].x : l.run) * s.ld + col;
#pragma unroll
    for (int e = 0; e < VEC; ++e) dst[e] = s.accumulate ? dst[e] + acc[e] * scale : acc[e] * scale;
  };
  if (active) {
    for (int t = group; t < kJoinChunks; t += groups) {
      if (!list[t].is_long || count(t) > kFewPieces) continue;
      float acc[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
      add_pieces<VEC>(pieces, piece_ld, col, c0 + t, 0, count(t), acc);
      store(list[t], acc);
    }
  }
  for (int t = 0; t < kJoinChunks; ++t) {
    if (!list[t].is_long || count(t) <= kFewPieces) continue;      // the same for the whole block
    const int64_t m = count(t);
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
    if (active)
      add_pieces<VEC>(pieces, piece_ld, col, c0 + t, m * group / groups, m * (group + 1) / groups, acc);
#pragma unroll
    for (int e = 0; e < VEC; ++e) sums[e * kJoinThreads + tid] = acc[e];
    __syncthreads();
    if (active && group % kJoinFan == 0) {
      for (int q = group + 1; q < min(group + kJoinFan, groups); ++q) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += sums[e * kJoinThreads + q * width + tid - group * width];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) sums[e * kJoinThreads + tid] = acc[e];
    }
    __syncthreads();
    if (active && group == 0) {
      for (int q = kJoinFan; q < groups; q += kJoinFan) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += sums[e * kJoinThreads + q * width + tid];
      }
      store(list[t], acc);
    }
    __syncthreads();
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The workspace of a call, and how it is cut.
struct Plan {
  int64_t n, chunks, head_tiles;
  int chunk, longest, bits, passes, digit;
  bool vec;
  int64_t piece_ld;
  size_t pairs[2], counts, totals, tile_heads, starts, chunk_run, meta, pieces, bytes;
  Pass pass;
};

// Chunks of 64 positions where those give every CU 2048 threads, else shorter ones
// down to 8, so that small calls use the chip; a thread follows a run behind its
// chunk for as long as a chunk, up to 64 positions in all.
Plan make_plan(const EngramEmbedArgs &a) {
  Plan p;
  p.n = a.n_ids;
  p.vec = a.dim % 8 == 0 && a.out_ld % 8 == 0 && a.grad_ld % 4 == 0;
  const int64_t per_chunk = p.vec ? a.dim / 8 : a.dim;
  p.chunk = kMaxChunk;
  while (p.chunk > 8 && (p.n / p.chunk) * per_chunk < (int64_t)256 * 2048) p.chunk /= 2;
  p.longest = 2 * p.chunk < kMaxChunk ? 2 * p.chunk : kMaxChunk;
  p.chunks = (p.n + p.chunk - 1) / p.chunk;
  p.bits = 1;
  while (p.bits < 32 && (a.table_rows >> p.bits) != 0) ++p.bits;
  p.passes = (p.bits + kMaxBits - 1) / kMaxBits;
  p.digit = (p.bits + p.passes - 1) / p.passes;
  p.head_tiles = (p.n + kHeadTile - 1) / kHeadTile;
  const int64_t tiles = (p.n + kSortTile - 1) / kSortTile;
  const int64_t per = tiles > 0 ? (tiles + kMaxBlocks - 1) / kMaxBlocks : 1;
  p.pass.n = p.n;
  p.pass.per_block = per * kSortTile;
  p.pass.blocks = (int)((tiles + per - 1) / per);
  p.piece_ld = ((int64_t)a.dim + 3) / 4 * 4;
  const bool large = p.n > kSmall;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  for (int i = 0; i < 2; ++i) p.pairs[i] = take((size_t)p.n * 8);
  p.counts = take(large ? ((size_t)p.pass.blocks << p.digit) * 4 : 0);
  p.totals = take(large ? (size_t)4 << p.digit : 0);
  p.tile_heads = take(large ? (size_t)p.head_tiles * 4 : 0);
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
  const int slices = (cols + 63) / 64;
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
  uint2 *pairs[2] = {(uint2 *)(ws + p.pairs[0]), (uint2 *)(ws + p.pairs[1])};
  uint32_t *counts = (uint32_t *)(ws + p.counts), *totals = (uint32_t *)(ws + p.totals);
  uint32_t *tile_heads = (uint32_t *)(ws + p.tile_heads);
  float *pieces = (float *)(ws + p.pieces);
  const bool dense = n_rows == nullptr;
  const Sums s{grad, a.grad_ld, grad_rows, n_rows, dense ? 1 : 0, accumulate};
  const bool zero_vec = a.dim % 4 == 0 && a.grad_ld % 4 == 0;
  Zero z{EngramFastDiv(zero_vec ? a.dim / 4 : a.dim), 0, 0, zero_vec, zero_vec && a.grad_ld == a.dim};
  const int64_t zero_total = dense && !accumulate ? a.table_rows * z.groups.d : 0;
  // blocks that clear the groups [z.begin, z.end), 4 groups a thread
  const auto zero_blocks = [&](int threads) {
    const int64_t want = (z.end - z.begin + threads * 4 - 1) / (threads * 4);
    const int64_t most = ((int64_t)1 << 30) / threads;
    return (unsigned)(want < most ? want : most);
  };
  Runs r{pairs[1], (uint32_t *)(ws + p.starts), (uint32_t *)(ws + p.chunk_run),
         (uint32_t *)(ws + p.meta), p.chunk, __builtin_ctz(p.chunk), p.longest};
  if (p.n <= kSmall) {
    const int parts = (int)((p.n + kPart - 1) / kPart);
    const int merges = parts > 1 ? (int)((p.n + kMergeElems - 1) / kMergeElems) : 0;
    const int tiles = p.n > 0 ? (int)((p.n + kSmallTile - 1) / kSmallTile) : 1;
    uint2 *sorted = pairs[parts > 1 ? 0 : 1];
    // Clearing is shared out over the three launches. The shares matter little: with
    // these, with thirds and with half of it in the first, 8191 ids and 99092 x 1024
    // values took 98, 101 and 97 us, 509 ids of the same 87, 88 and 84, and 32000 ids of
    // 99092 x 256 77, 76 and 76.
    z.end = zero_total / 8;
    if (parts + zero_blocks(kPart) > 0)
      hipLaunchKernelGGL(sort_part_kernel, dim3((unsigned)parts + zero_blocks(kPart)), dim3(kPart), 0,
                         stream, row_ids, (int)p.n, a.table_rows, sorted, parts, s, z);
    z.begin = z.end;
    if (merges > 0) {
      z.end = zero_total / 2;
      hipLaunchKernelGGL(merge_parts_kernel, dim3((unsigned)merges + zero_blocks(kMergeThreads)),
                         dim3(kMergeThreads), 0, stream, (const uint2 *)sorted, (int)p.n, pairs[1], merges,
                         s, z);
      z.begin = z.end;
    }
    z.end = zero_total;
    hipLaunchKernelGGL(small_runs_kernel, dim3((unsigned)tiles + zero_blocks(kSmallTile)),
                       dim3(kSmallTile), 0, stream, (int)p.n, a.table_rows, r, tiles, s, z);
  } else {
    z.end = zero_total;               // cleared beside the first count
    Pass pass = p.pass;
    int at = 1;                       // the next pass writes pairs[1 - at]
    for (int i = 0; i < p.passes; ++i) {
      pass.shift = i * p.digit;
      pass.bits = p.digit;
      const dim3 grid((unsigned)pass.blocks), block(kSortThreads);
      const uint2 *from = pairs[at];
      if (i == 0)
        hipLaunchKernelGGL(sort_count_kernel<true>, dim3((unsigned)pass.blocks + zero_blocks(kSortThreads)),
                           block, 0, stream, row_ids, from, a.table_rows, pass, counts, s, z);
      else
        hipLaunchKernelGGL(sort_count_kernel<false>, grid, block, 0, stream, row_ids, from, a.table_rows,
                           pass, counts, s, z);
      hipLaunchKernelGGL(sort_scan_kernel, dim3(((1u << p.digit) + kScanDigits - 1) / kScanDigits),
                         dim3(kScanThreads), 0, stream, counts, totals, pass.blocks, 1 << p.digit);
      if (i == 0)
        hipLaunchKernelGGL(sort_scatter_kernel<true>, grid, block, 0, stream, row_ids, from, a.table_rows,
                           pass, counts, totals, pairs[1 - at]);
      else
        hipLaunchKernelGGL(sort_scatter_kernel<false>, grid, block, 0, stream, row_ids, from, a.table_rows,
                           pass, counts, totals, pairs[1 - at]);
      at = 1 - at;
    }
    r.pairs = pairs[at];
    hipLaunchKernelGGL(count_heads_kernel, dim3((unsigned)p.head_tiles), dim3(kHeadThreads), 0, stream,
                       r.pairs, p.n, a.table_rows, tile_heads);
    hipLaunchKernelGGL(write_runs_kernel, dim3((unsigned)p.head_tiles), dim3(kHeadThreads), 0, stream,
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
