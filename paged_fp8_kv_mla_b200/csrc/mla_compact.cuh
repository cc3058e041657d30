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
// fetched once.  A request has 9 slices of 576 bytes; 128 requests of 8k cut to 4k take 120 us, 0.78 of the
// copy rate.  With few requests the slices are 32 bytes wide (a DRAM sector) and the CTAs larger (64 registers a thread, 20 bytes spilt), and what
// bounds it is the rate at which an SM's load unit takes scattered 32-byte pieces, on as many SMs as there are
// slices: 4 requests of 128k cut to 64k 113 us, 0.4 of the copy rate on 72 SMs, and one such request 110 (floor
// 12) on 18.  (Copies held in registers instead of shared memory: 119 and 146; a cluster per slice, whose barrier
// waits for the writes: 134 and 141.)  The words of a column (scales, sums) are walked by one CTA, a chunk at a time:
// for one scale a token that ends with the rows, but the scales of an e4m3 cache with 8 kv heads of 128 are what a
// long request waits for: 4 of 128k to 64k 854 us (floor 169; bf16, without scales, 457 of 328), 32 of 8k to 4k 133
// (85; bf16 192 of 164).
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

// A plain load through L2, kept on its side of the chunk's barrier.
__device__ __forceinline__ uint32_t ld_word(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// A column of 4-byte words of the rows of one request (the scales, the accumulated weights): word x of row t lies
// at base + row(t) * pitch + x, with row(t) found through a page table (table != null) or t itself (rows < limit).
struct CompactColumn {
  uint32_t* base;
  long long pitch;
  const uint32_t* table;
  uint32_t pool, plane, limit;
};

// Moves the column for rows 0 .. m - 1, `per_row` words each, U words per thread and chunk.
template <int THREADS, int U, typename RowOf>
__device__ __forceinline__ void compact_walk(const CompactParams& p, const int32_t* kept, uint32_t m, uint32_t per_row,
                                             RowOf row_of, const CompactColumn& col) {
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
    const uint32_t* src[U];
    uint32_t* dst[U];
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
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u]) v[u] = ld_word(src[u]);
    __syncthreads();                                     // the chunk has been read
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u]) *dst[u] = v[u];
  }
}

// The cache rows: a CTA moves one slice of SLICE bytes of every row, SLICE / 16 lanes per row, U rows per
// lane and chunk.  A chunk passes four stations, one per turn of the loop: its kept indices are loaded, its
// pages looked up, its rows copied into shared memory (cp.async, S chunks deep, each lane into slots of its
// own), and, once all of the CTA's copies of the chunk are in, written.  Rows may be read before earlier
// chunks are written: they lie at or above their own chunk.
constexpr uint32_t CMP_SLOT = 20;                        // bytes per lane, row and chunk: 16 and the row it goes to
template <int SLICE, int THREADS, int U, int S>
__device__ __forceinline__ void compact_rows(const CompactParams& p, const int32_t* kept, uint32_t m, const uint32_t* lut,
                                             int plane, int slice) {
  constexpr int LPR = SLICE / 16;                        // lanes per row
  constexpr uint32_t ROWS = THREADS / LPR;               // rows of a chunk per step u
  constexpr uint32_t CHUNK = ROWS * U;
  constexpr uint32_t NONE = ~0u;
  extern __shared__ __align__(16) uint8_t cmp_smem[];
  const uint32_t data = ptx::smem_u32(cmp_smem) + threadIdx.x * 16;                                   // [S][U][THREADS]
  uint32_t* dest = reinterpret_cast<uint32_t*>(cmp_smem + S * U * THREADS * 16) + threadIdx.x;        // [S][U][THREADS]
  uint8_t* base = p.blocks + slice * SLICE + (threadIdx.x & (LPR - 1)) * 16;
  const uint32_t j0 = threadIdx.x / LPR;
  const uint32_t kv = static_cast<uint32_t>(plane) * p.NL + p.layer, pages = static_cast<uint32_t>(p.KVD) * p.NL;
  const uint32_t chunks = (m + CHUNK - 1) / CHUNK;
  uint32_t from[U];                                      // station 1: sources of chunk c
  auto indices = [&](uint32_t c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = c * CHUNK + u * ROWS + j0;
      from[u] = j < m ? static_cast<uint32_t>(kept[j]) : j;
    }
  };
  uint32_t fb[U], tb[U], fs[U], ts[U];                   // station 2: blocks (NONE: no such page) and slots
  auto lookup = [&](uint32_t c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = c * CHUNK + u * ROWS + j0, f = from[u];
      const uint32_t fp = p.divP.div(f), tp = p.divP.div(j);
      fs[u] = f - fp * p.P;
      ts[u] = f == j ? NONE : j - tp * p.P;              // NONE: already in its place
      const bool in = f > j && fp < static_cast<uint32_t>(p.max_pages);
      fb[u] = in ? lut[fp] : NONE;
      tb[u] = in ? lut[tp] : NONE;
    }
  };
  auto copy = [&](uint32_t s) {                          // station 3, into slots s
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t d = NONE;
      if (ts[u] != NONE) {
        if (fb[u] < static_cast<uint32_t>(p.NB) && tb[u] < static_cast<uint32_t>(p.NB)) {
          const uint32_t src = (fb[u] * pages + kv) * p.P + fs[u];   // below 2^31: the pool's rows are
          d = (tb[u] * pages + kv) * p.P + ts[u];
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                       :: "r"(data + (s * U + u) * THREADS * 16), "l"(base + static_cast<size_t>(src) * p.row_bytes) : "memory");
        } else {
          raise_status(p.status, STATUS_BOUNDS);         // left as it is
        }
      }
      dest[(s * U + u) * THREADS] = d;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  indices(0);
  for (uint32_t c = 0; c < S; ++c) {                     // chunks 0 .. S - 2 on their way, S - 1 looked up
    lookup(c);
    indices(c + 1);
    if (c < S - 1) copy(c);
  }
  uint32_t s = 0;
  for (uint32_t c = 0; c < chunks; ++c) {
    copy(s == 0 ? S - 1 : s - 1);                        // chunk c + S - 1, where chunk c - 1 was
    lookup(c + S);
    indices(c + S + 1);
    asm volatile("cp.async.wait_group %0;" :: "n"(S - 1) : "memory");
    __syncthreads();                                     // chunk c has been read by every thread
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t d = dest[(s * U + u) * THREADS];
      if (d != NONE)
        *reinterpret_cast<uint4*>(base + static_cast<size_t>(d) * p.row_bytes) = ptx::ld_shared_v4(data + (s * U + u) * THREADS * 16);
    }
    s = s + 1 == S ? 0 : s + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// grid (kv planes * slices + kv planes (scales) + 1 (accumulated weights), requests)
template <int SLICE, int THREADS, int U, int S, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) mla_compact_kernel(const __grid_constant__ CompactParams p) {
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
    compact_rows<SLICE, THREADS, U, S>(p, kept, m, lut, plane, slice);
    return;
  }
  i -= p.KVD * p.slices;
  if (i < p.KVD) {
    if (!p.scales) return;
    const CompactColumn col{reinterpret_cast<uint32_t*>(p.scales), p.row_words, slut,
                            static_cast<uint32_t>(p.NSB), static_cast<uint32_t>(i), ~0u};
    compact_walk<THREADS, 8>(p, kept, m, p.row_words, [&](uint32_t e) { return p.divW.div(e); }, col);
    return;
  }
  if (!p.scores) return;
  const CompactColumn col{reinterpret_cast<uint32_t*>(p.scores + b * p.scores_stride), 1, nullptr, 0u, 0u,
                          static_cast<uint32_t>(p.scores_cols)};
  compact_walk<THREADS, 8>(p, kept, m, 1, [](uint32_t e) { return e; }, col);
}

}  // namespace mla
