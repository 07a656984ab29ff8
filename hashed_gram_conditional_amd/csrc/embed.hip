// Table lookup with scaling: out[i] = scale * table[row_ids[i]], zero rows for ids
// outside the table, bf16 or fp32 rows in, bf16 or fp32 rows out.
//
// One pass over the output: each thread owns groups of 8 consecutive values of
// an output row (16 bytes of bf16, 32 of fp32), so a row of 256 is 32
// neighbouring threads and both sides move in whole cache lines whatever the
// rows' order. kUnroll groups are requested before any is stored, to cover the
// latency of random rows. The product is formed in fp32 and rounded once to the
// output type (nearest, ties to even). Bound by HBM: 786432 rows of 256 from fp32 to
// bf16 take 189 us (1.02 GB, 5.4 TB/s) with nontemporal stores, which leave the cache
// to repeated rows, and 211 us with plain ones; four groups a thread 194 us. Widths and
// strides that are not multiples of 8 move value by value: 255 columns take 471 us (2.2
// TB/s), from bf16 to bf16 453 against 114.
#include "common.h"
#include "fast_div.h"

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;
// Lookups in a host-resident table leave the other CUs to concurrent work.
constexpr int kHostBlocks = 32;

template <bool F32>
__device__ __forceinline__ float load_one(const void *p, int64_t i) {
  return F32 ? reinterpret_cast<const float *>(p)[i]
             : engram::bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]);
}

template <bool F32>
__device__ __forceinline__ void store_one(void *p, int64_t i, float v) {
  if (F32)
    reinterpret_cast<float *>(p)[i] = v;
  else
    reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)engram::pack_bf16x2(v, v);
}

// VEC = 8: rows made of whole, aligned groups of 8. VEC = 1: any width and stride.
template <bool TF32, bool OF32, int VEC, int U>
__global__ __launch_bounds__(kThreads) void embed_kernel(
    const void *__restrict__ table, int64_t table_rows, int64_t table_ld,
    const int64_t *__restrict__ row_ids, void *__restrict__ out, int64_t out_ld, float scale,
    EngramFastDiv groups, int64_t total) {
  constexpr int64_t kTile = (int64_t)kThreads * U;
  for (int64_t g0 = (int64_t)blockIdx.x * kTile + threadIdx.x; g0 < total;
       g0 += (int64_t)gridDim.x * kTile) {
    int64_t row[U], id[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t g = g0 + u * kThreads;
      row[u] = groups.div(g);
      col[u] = (int)(g - row[u] * groups.d);
      id[u] = g < total ? row_ids[row[u]] : -1;
    }
    if (VEC == 8) {
      engram::Chunk8<TF32> v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u].zero();
        if ((uint64_t)id[u] < (uint64_t)table_rows) v[u].load(table, id[u] * (table_ld / 8) + col[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g0 + u * kThreads < total) {
          // an id outside the table gives +0 whatever the scale's sign
          const bool in = (uint64_t)id[u] < (uint64_t)table_rows;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = in ? v[u][e] * scale : 0.f;
          engram::Chunk8<OF32>::store_nt(out, row[u] * (out_ld / 8) + col[u], f);
        }
      }
    } else {
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = (uint64_t)id[u] < (uint64_t)table_rows
                   ? load_one<TF32>(table, id[u] * table_ld + col[u]) * scale
                   : 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (g0 + u * kThreads < total) store_one<OF32>(out, row[u] * out_ld + col[u], v[u]);
    }
  }
}

template <bool TF32, bool OF32>
hipError_t launch_typed(const EngramEmbedArgs &a, const void *table, const int64_t *row_ids,
                        void *out, bool host_table, hipStream_t stream) {
  const bool vec = a.dim % 8 == 0 && a.table_ld % 8 == 0 && a.out_ld % 8 == 0;
  const EngramFastDiv groups(vec ? a.dim / 8 : a.dim);
  const int64_t total = a.n_ids * groups.d;
  const int64_t tiles = (total + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  const int64_t limit = host_table ? kHostBlocks : (int64_t)1 << 22;
  const dim3 grid((unsigned)(tiles < limit ? tiles : limit));
  if (vec)
    hipLaunchKernelGGL((embed_kernel<TF32, OF32, 8, kUnroll>), grid, dim3(kThreads), 0, stream,
                       table, a.table_rows, a.table_ld, row_ids, out, a.out_ld, a.scale, groups,
                       total);
  else
    hipLaunchKernelGGL((embed_kernel<TF32, OF32, 1, kUnroll>), grid, dim3(kThreads), 0, stream,
                       table, a.table_rows, a.table_ld, row_ids, out, a.out_ld, a.scale, groups,
                       total);
  return hipGetLastError();
}

}  // namespace

hipError_t engram_launch_embed(const EngramEmbedArgs &a, const void *table,
                               const int64_t *row_ids, void *out, bool host_table,
                               hipStream_t stream) {
  if (a.n_ids <= 0) return hipSuccess;
  if (a.table_f32)
    return a.out_f32 ? launch_typed<true, true>(a, table, row_ids, out, host_table, stream)
                     : launch_typed<true, false>(a, table, row_ids, out, host_table, stream);
  return a.out_f32 ? launch_typed<false, true>(a, table, row_ids, out, host_table, stream)
                   : launch_typed<false, false>(a, table, row_ids, out, host_table, stream);
}
