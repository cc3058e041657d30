// Compaction of a paged cache (sm_100a): row j of request b becomes row kept[b][j], in place, for
// j = 0 .. kept_lengths[b] - 1, with the same for its scales and its accumulated weights.  kept is
// strictly ascending, so kept[j] >= j and the order of the tokens is preserved (causal masks and
// "the last num_recent keys" keep their meaning).
//
// In place, without waits between CTAs.  Row j may be the source of an earlier row j' <= j only
// (kept[j'] = j), so a worker that walks the rows upwards, and for each chunk of rows first reads all
// its sources and then writes all its destinations, never reads a row it has overwritten: the sources
// of later chunks lie at or above their own rows.  That order is only needed within one column of the
// rows, so the row is cut into slices of 64 (or 32) bytes and each CTA moves one slice of all of a
// request's rows: CTAs share no bytes, a barrier of the CTA separates a chunk's reads from its
// writes, and nothing waits for another CTA.  The scales and the accumulated weights are further such
// columns, moved as 4-byte words.
//
// What bounds it: HBM, one read and one write of every moved row.  The slices of a request are
// neighbouring CTAs, which walk the rows at the same pace, so the 128-byte lines they share are
// fetched once.  A request has 9 slices of 576 bytes, four CTAs of 256 threads to an SM (128 requests of 8k
// cut to 4k: 119 us, 0.79 of the copy rate; two of 512: 128).  With few requests the slices are 32 bytes wide
// (a DRAM sector) and the CTAs larger, and what is in flight per SM bounds it (4 requests of 128k cut to
// 64k: 146 us, 0.32; a cluster per slice, whose barrier waits for the writes, gave 141 and cost the full
// batches 13 %).
#pragma once
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

struct CompactParams {
  const int32_t* kept;             // row stride kept_stride
  const int32_t* kept_lengths;     // [B]
  const uint32_t* lut;             // [B, max_pages]
  const uint32_t* slut;            // [B, max_pages]: the scales' pages (lut itself when they share ids)
  uint8_t* blocks;                 // [NB, KVD, NL, P, row_bytes]
  float* scales;                   // [NSB, KVD, NL, P, row_words] or null
  float* scores;                   // row stride scores_stride, or null
  unsigned int* status;
  long long kept_stride, scores_stride;
  int max_kept, scores_cols;
  int P, KVD, NL, layer, NB, NSB, max_pages;
  int row_bytes, row_words;        // of a token in one kv plane
  int slices;                      // CTAs per (request, kv plane) that move cache rows
  FastDiv divP, divW;              // by the page size and by row_words
};


// Plain loads through L2, kept on their side of the chunk's barrier.
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_row(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// A column of the rows of one request: element x of row t lies at base + row(t) * pitch + x, in units
// of V, with row(t) found through a page table (table != null) or t itself (rows < limit).
template <typename V>
struct CompactColumn {
  V* base;
  long long pitch;
  const uint32_t* table;
  uint32_t pool, plane, limit;
};

// Moves the column for rows 0 .. m - 1, `per_row` elements each, U elements per thread and chunk.
template <typename V, int THREADS, int U, typename RowOf>
__device__ __forceinline__ void compact_walk(const CompactParams& p, const int32_t* kept, uint32_t m, uint32_t per_row,
                                             RowOf row_of, const CompactColumn<V>& col) {
  const uint32_t total = m * per_row;
  for (uint32_t e0 = 0; e0 < total; e0 += U * THREADS) {
    // three rounds of independent loads: the kept indices, the page ids, the rows
    uint32_t to[U], x[U], from[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t e = e0 + u * THREADS + threadIdx.x;
      to[u] = row_of(min(e, total - 1));
      x[u] = min(e, total - 1) - to[u] * per_row;
      from[u] = e < total ? static_cast<uint32_t>(kept[to[u]]) : to[u];
    }
    const V* src[U];
    V* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      src[u] = nullptr;
      dst[u] = nullptr;
      if (from[u] == to[u]) continue;                    // already in its place
      uint32_t fr = from[u], tr = to[u];
      bool ok = from[u] > to[u] && from[u] < col.limit;
      long long frow = fr, trow = tr;
      if (col.table) {
        const uint32_t fp = p.divP.div(fr), tp = p.divP.div(tr);
        ok = ok && fp < static_cast<uint32_t>(p.max_pages);
        const uint32_t fb = ok ? col.table[fp] : ~0u, tb = ok ? col.table[tp] : ~0u;
        ok = fb < col.pool && tb < col.pool;
        frow = ((static_cast<long long>(fb) * p.KVD + col.plane) * p.NL + p.layer) * p.P + (fr - fp * p.P);
        trow = ((static_cast<long long>(tb) * p.KVD + col.plane) * p.NL + p.layer) * p.P + (tr - tp * p.P);
      }
      if (!ok) {
        raise_status(p.status, STATUS_BOUNDS);           // left as it is
        continue;
      }
      src[u] = col.base + frow * col.pitch + x[u];
      dst[u] = col.base + trow * col.pitch + x[u];
    }
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u]) v[u] = ld_row(src[u]);
    __syncthreads();                                     // the chunk has been read
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u]) *dst[u] = v[u];
  }
}

// The cache rows: a CTA moves one slice of SLICE bytes of every row, SLICE / 16 lanes per row, U rows per
// lane and chunk.  The three dependent rounds of a chunk overlap with the chunks before it: while chunk n
// waits for its barrier and is written, chunk n + 1's rows are on their way and chunk n + 2's pages are
// looked up.  (Its rows may be read before chunk n is written: they lie at or above chunk n + 1.)
template <int SLICE, int THREADS, int U>
__device__ __forceinline__ void compact_rows(const CompactParams& p, const int32_t* kept, uint32_t m, const uint32_t* lut,
                                             int plane, int slice) {
  constexpr int LPR = SLICE / 16;                        // lanes per row
  constexpr uint32_t ROWS = THREADS / LPR;           // rows of a chunk per step u
  constexpr uint32_t CHUNK = ROWS * U;
  constexpr uint32_t NONE = ~0u;
  uint8_t* base = p.blocks + slice * SLICE + (threadIdx.x & (LPR - 1)) * 16;
  const uint32_t j0 = threadIdx.x / LPR;
  const uint32_t kv = static_cast<uint32_t>(plane) * p.NL + p.layer, pages = static_cast<uint32_t>(p.KVD) * p.NL;
  // rows of a chunk: kept index and own index of each step; then pool rows (NONE: nothing to move)
  auto indices = [&](uint32_t c0, uint32_t (&from)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = c0 + u * ROWS + j0;
      from[u] = j < m ? static_cast<uint32_t>(kept[j]) : j;
    }
  };
  auto rows = [&](uint32_t c0, const uint32_t (&from)[U], uint32_t (&src)[U], uint32_t (&dst)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = c0 + u * ROWS + j0, f = from[u];
      src[u] = NONE;
      dst[u] = NONE;
      if (f == j) continue;                              // already in its place
      const uint32_t fp = p.divP.div(f), tp = p.divP.div(j);
      const bool in = f > j && fp < static_cast<uint32_t>(p.max_pages);
      const uint32_t fb = in ? lut[fp] : NONE, tb = in ? lut[tp] : NONE;
      if (fb < static_cast<uint32_t>(p.NB) && tb < static_cast<uint32_t>(p.NB)) {
        src[u] = (fb * pages + kv) * p.P + (f - fp * p.P);   // below 2^31: the pool's rows are
        dst[u] = (tb * pages + kv) * p.P + (j - tp * p.P);
      } else {
        raise_status(p.status, STATUS_BOUNDS);           // left as it is
      }
    }
  };
  uint32_t from[U], src[U], dst[U], next_dst[U];
  uint4 v[U], next[U];
  auto load = [&](uint4 (&to)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] != NONE) to[u] = ld_row(reinterpret_cast<const uint4*>(base + static_cast<size_t>(src[u]) * p.row_bytes));
  };
  indices(0, from);
  rows(0, from, src, dst);
  load(v);
  indices(CHUNK, from);
  rows(CHUNK, from, src, next_dst);
  indices(2 * CHUNK, from);
  for (uint32_t c0 = 0; c0 < m; c0 += CHUNK) {
    load(next);                                          // chunk n + 1
    __syncthreads();                                     // chunk n has been read by every thread
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] != NONE) *reinterpret_cast<uint4*>(base + static_cast<size_t>(dst[u]) * p.row_bytes) = v[u];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = next[u];
      dst[u] = next_dst[u];
    }
    rows(c0 + 2 * CHUNK, from, src, next_dst);
    indices(c0 + 3 * CHUNK, from);
  }
}

// grid (kv planes * slices + kv planes (scales) + 1 (accumulated weights), requests)
template <int SLICE, int THREADS, int U>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) mla_compact_kernel(const __grid_constant__ CompactParams p) {
  const int b = blockIdx.y;
  const int32_t given = p.kept_lengths[b];
  const uint32_t m = min(max(given, 0), p.max_kept);
  if (given != static_cast<int32_t>(m) && blockIdx.x == 0 && threadIdx.x == 0) raise_status(p.status, STATUS_BOUNDS);
  if (m == 0) return;
  const int32_t* kept = p.kept + b * p.kept_stride;
  const uint32_t* lut = p.lut + static_cast<size_t>(b) * p.max_pages;
  const uint32_t* slut = p.slut + static_cast<size_t>(b) * p.max_pages;
  int i = blockIdx.x;
  if (i < p.KVD * p.slices) {
    const int plane = i / p.slices, slice = i - plane * p.slices;
    compact_rows<SLICE, THREADS, U>(p, kept, m, lut, plane, slice);
    return;
  }
  i -= p.KVD * p.slices;
  if (i < p.KVD) {
    if (!p.scales) return;
    const CompactColumn<uint32_t> col{reinterpret_cast<uint32_t*>(p.scales), p.row_words, slut,
                                      static_cast<uint32_t>(p.NSB), static_cast<uint32_t>(i), ~0u};
    compact_walk<uint32_t, THREADS, 8>(p, kept, m, p.row_words, [&](uint32_t e) { return p.divW.div(e); }, col);
    return;
  }
  if (!p.scores) return;
  const CompactColumn<uint32_t> col{reinterpret_cast<uint32_t*>(p.scores + b * p.scores_stride), 1, nullptr, 0u, 0u,
                                    static_cast<uint32_t>(p.scores_cols)};
  compact_walk<uint32_t, THREADS, 8>(p, kept, m, 1, [](uint32_t e) { return e; }, col);
}

}  // namespace mla
