// Decode attention over a paged cache with separate keys and values per kv head (sm_100a): kv plane 0
// holds K, plane 1 holds V, in bf16 or in e4m3 with one fp32 scale per token and head.  With G = H / HKV
// query heads per kv head, for request b, query token i and query head h (kv head h / G):
//   x[t] = softmax_scale <q[b,i,h,:], K[t]>  for t <= L_b + i,
//   lse  = ln sum_t exp(x[t]),   out[b,i,h,:] = sum_t exp(x[t] - lse) V[t].
//
// What bounds it.  A kv head's key and value are 4 D bytes (bf16) for 4 D flop per query row, so up to
// some hundred rows per kv head the cache's bytes set the time: every K and V byte is to cross HBM once,
// at full rate, and the arithmetic has to stay out of the way.  The rows that share a kv head
// (R = T * G of them) are few, so the products run on the warp-level 16 x 8 x 16 MMA with the query rows
// as its 8 columns: a tcgen05 tile has 128 rows, most of them empty here, and its accumulator would have
// to come back from tensor memory for every rescale.
//
// Who does what.  Eight consumer warps per CTA (one CTA per SM).  A warp owns 8 rows of one kv head (16
// where the head has more than 8; its scores, weights and O stay in its registers, no exchange within a
// tile) and, where fewer than eight (head, row tile) pairs exist, every kw-th group of keys; those kw warps
// merge once, at the end of a piece.  All warps read the same tile, so K and V are loaded once for all of
// up to 128 rows, and a tile's rows are read as whole contiguous runs of the page over the CTA's heads.  A
// ninth warp keeps a ring of tiles full by TMA: one box per page run and plane, [column of 128 (64)
// bytes][key], in the matching shared-memory swizzle, so that ldmatrix reads rows without bank conflicts.
//
// The weights enter the value product as two bf16 terms for a bf16 cache: one alone would add as much error as
// the rounding of the output, and the second costs nothing that shows (165 us with and without it, below).
//
// e4m3.  The values are converted to f16, exactly, as they leave shared memory (two per instruction),
// and never to anything wider: each row of q is brought to f16 with a power of two of its own (exact down to
// 2^-30 of the row's largest value, whatever the rows beside it hold), K's scale multiplies the score, and V's scale goes into the weight, relative to a
// running power-of-two bound of V's scales so that f16 holds it with 11 bits (down to 2^-23 of the bound).
// The instructions of this are what keeps an e4m3 cache from the copy rate: the loads alone run at it.  (One power
// of two for a warp's rows together cost nothing elsewhere, but took 130 instead of 140 us for 64 requests of 8k, 16
// rows a head of 64; a row's infinity, NaN or much larger values then spoilt its neighbours'.)
//
// Work split.  The tiles of all (request, head group, row group) items, with each item's fixed cost, laid
// end to end are cut into equal contiguous ranges, one per CTA.  An item cut by a range's end leaves
// normalised fp32 partials and their log-sum-exp in the workspace and a second kernel joins them; each CTA
// names the item whose head it holds and the last CTA of it, so the join needs no plan and nothing has to
// start at zero.
// Where all requests are short (up to four tiles), each CTA takes one item and the second launch is
// left out.
//
// Measured (floor, the cache's bytes at the copy rate): 64 requests of 1 to 32k, 2 tokens, 32/8 heads of 128,
// bf16 165 us (155), e4m3 97 (80); 128 of 8k, 64/8 heads of 128, e4m3 337 to 376 by machine (338); heads of 64,
// e4m3 200 (174); 2 short requests 5.6.  Above 8 rows a head (64 of 8k, 128/8 heads: 226, floor 170) and with one kv
// head (128 of 8k: 69, floor 42) the latency of a warp's own chain shows, with two warps to a scheduler.  All
// eight variants with heads of 128 and five of the ten with heads of 64 spill 24 to 88 bytes at the launch's 168
// registers a thread.  Prompts are right but far from what a prefill takes: every row group
// walks to its request's end, past the last key its rows see, and reads K and V again (2048 tokens, nothing cached, 32/8
// heads of 128, bf16: 328 us, floor 21).
#pragma once
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

constexpr int MHA_WARPS = 8;                      // consumer warps
constexpr int MHA_THREADS = 32 * (MHA_WARPS + 4);   // consumers, and a warpgroup for the producer warp
constexpr int MHA_ROWS = 16 * MHA_WARPS;          // rows of a CTA at most
constexpr int MHA_MAX_STAGES = 8;
constexpr uint32_t MHA_SMEM_LIMIT = 232448;

struct MhaParams {
  CUtensorMap tmap;                // blocks as {column bytes, rows, columns}; box {.., box_rows, ncols}
  const uint16_t* q;               // bf16 bits [B, T, H, D]
  const float* scales;             // [NSB, KVD, NL, P, HKV, 1] (e4m3 only)
  const uint32_t* cache_lengths;   // [B]
  const uint32_t* lut;             // [B, max_pages]
  const uint32_t* slut;            // [B, max_pages]: lut itself where the scales share the ids
  uint16_t* out;                   // bf16 bits [B, T, H, D]
  float* lse;                      // [B, T, H] or null
  float* part_o;                   // [2 NC][MHA_ROWS][D]
  float* part_lse;                 // [2 NC][MHA_ROWS], base 2
  int4* desc;                      // [NC]: request (-1: none), item of the request, last CTA
  unsigned int* status;
  unsigned long long wait_limit_ns;
  int B, T, H, HKV, R, P, KVD, NL, layer, NB, NSB, max_pages;
  unsigned int max_cache_length;
  int hg, mt, kw;                  // kv heads per CTA, row tiles per CTA, warps over the keys of a tile
  int row_tile;                    // rows of a warp: 8 or 16
  int head_groups, row_groups;     // of a request: its items
  int tile, box_rows, box_shift, stages;   // keys per tile, keys per box (a power of two) and its log2, ring depth
  uint32_t plane_bytes, stage_bytes;   // of a tile's K (or V); of a ring stage
  int one_item;                    // 1: CTA c computes item c alone
  FastDiv divP, divG;              // by the page size and by G = H / HKV
  float scale_log2;                // softmax_scale * log2(e)
};

// D (16 x 8) += A (16 x 16) B (16 x 8), both operands f16 or both bf16.
template <bool F16>
__device__ __forceinline__ void mma_16816(float2& c0, float2& c1, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c0.x), "+f"(c0.y), "+f"(c1.x), "+f"(c1.y)
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c0.x), "+f"(c0.y), "+f"(c1.x), "+f"(c1.y)
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Named barrier that also tells whether `v` holds for any thread.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r) : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(v)) : "memory");
  return r != 0;
}
// Over the eight lanes that share lane % 4 (the keys of a column of scores).
__device__ __forceinline__ float keys_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float keys_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
__device__ __forceinline__ float warp_max(float v) {   // v >= 0
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t mha_length(const MhaParams& p, int b) {
  return min(p.cache_lengths[b], p.max_cache_length);
}
__device__ __forceinline__ int mha_tiles(const MhaParams& p, int b) {   // of one item of request b
  return static_cast<int>((mha_length(p, b) + p.T + p.tile - 1) / p.tile);
}

// What an item costs beside its tiles (q, the epilogue), in tiles.  The ranges are cut by this cost: batches
// of long and very short requests otherwise leave many short ones to a few CTAs (64 ragged requests, e4m3:
// the last CTA ended at 102 us where the median ended at 79; 116 us a call with 0, 102 with 2, 97 with 4).
constexpr int MHA_ITEM_COST = 4;

// A CTA's piece of an item: tiles [ta, tb) of nt.
struct MhaPiece {
  int b, item, ta, tb, nt;
};
// Walks the pieces of a CTA's range of the items' costs laid end to end; the first MHA_ITEM_COST units of an
// item hold no tile.  t0: the range's first unit within its first item, left: units left.
struct MhaWalker {
  int b, item, t0;
  long long left;
  __device__ __forceinline__ bool next(const MhaParams& p, MhaPiece& u) {
    do {
      if (left <= 0 || b >= p.B) return false;
      u.b = b;
      u.item = item;
      u.nt = mha_tiles(p, b);
      const int end = static_cast<int>(min(static_cast<long long>(u.nt + MHA_ITEM_COST), t0 + left));
      u.ta = max(t0 - MHA_ITEM_COST, 0);
      u.tb = max(end - MHA_ITEM_COST, 0);
      left -= end - t0;
      t0 = 0;
      if (++item == p.head_groups * p.row_groups) {
        item = 0;
        ++b;
      }
    } while (u.ta == u.tb);
    return true;
  }
};

// Shared memory after the ring: the warps' merge buffers (kw > 1), then the barriers.
template <int D>
__host__ __device__ constexpr uint32_t mha_merge_bytes() { return (MHA_WARPS / 2) * 16 * (D + 2) * 4; }
constexpr uint32_t MHA_MISC_BYTES = 8 * 4 * MHA_MAX_STAGES + 4 * MHA_MAX_STAGES + 64 + 8 * (MHA_WARPS + 4) + 64;

// One warp's state: 8 NR query rows of one kv head.  Both products are formed transposed, keys and dims as
// the MMA's 16 rows, query rows as its 8 columns: S^T = K Q^T and O^T = V^T P^T, so that up to eight rows
// (the usual group) waste nothing, where rows on the 16-side would be half padding in every score, weight
// and register of O.  Thread (g, t) = (lane / 4, lane % 4) holds, of a group of 8 rows, rows 2t and 2t + 1.
template <int D, bool FP8, int NR>
struct MhaRows {
  static constexpr int CW = D * (FP8 ? 1 : 2) < 128 ? D * (FP8 ? 1 : 2) : 128;   // bytes of a column
  uint32_t qb[NR][D / 16][2];      // q as B fragments (bf16, or f16 times a power of two)
  float2 o[D / 16][NR][2];         // O^T: dims A and B of a 16-dim block (dim_a, dim_b), rows 2t and 2t + 1
  float m[NR][2];                  // reference maxima (base 2) of rows 2t, 2t + 1
  float2 l[NR];                    // this thread's part of their sums
  uint32_t last[NR][2];            // their last visible keys
  float2 xs[FP8 ? NR : 1];         // score factors: of rows 2t and 2t + 1, or the one of all rows
  float vref;                      // e4m3: power-of-two bound of V's scales so far (0: none yet)
  uint32_t koff, voff;             // this lane's place in a 16-key block of K and V

  static __device__ __forceinline__ uint32_t swizzle(uint32_t r) { return CW == 128 ? (r & 7u) << 4 : ((r >> 1) & 3u) << 4; }
  static __device__ __forceinline__ int dim_a(int k, int g) { return 16 * k + (FP8 ? 2 * g : g); }
  static __device__ __forceinline__ int dim_b(int k, int g) { return 16 * k + (FP8 ? 2 * g + 1 : g + 8); }

  // Query rows row0 .. row0 + 8 NR - 1 of kv head kvh (rows past the last one are zero).  For e4m3 caches each
  // row is brought to f16 by a power of two (its largest value into [2^12, 2^13)).
  __device__ __forceinline__ void load_q(const MhaParams& p, int b, int kvh, int row0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    if (!FP8) xs[0] = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      uint32_t m2 = 0;
      const int r = row0 + 8 * u + g;
      const bool have = r < p.R;
      const int i = have ? static_cast<int>(p.divG.div(r)) : 0;
      const int h = kvh * p.divG.d + (r - i * p.divG.d);
      const uint16_t* src = p.q + ((static_cast<size_t>(b) * p.T + i) * p.H + h) * D;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if (!FP8) {
          qb[u][k][0] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * t) : 0u;
          qb[u][k][1] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * t) : 0u;
        } else {
          const uint2 v = have ? *reinterpret_cast<const uint2*>(src + 16 * k + 4 * t) : make_uint2(0, 0);
          qb[u][k][0] = v.x;
          qb[u][k][1] = v.y;
          m2 = __vmaxu2(__vmaxu2(m2, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int re = row0 + 8 * u + 2 * t + e;
        last[u][e] = mha_length(p, b) + (re < p.R ? p.divG.div(re) : 0u);
        m[u][e] = -INFINITY;
      }
      l[u] = make_float2(0.f, 0.f);
      if (FP8) {                                         // row g lies in the four lanes of g, its scores in those of t = g / 2
        uint32_t big = max(m2 & 0xFFFFu, m2 >> 16);
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int e = big == 0 ? 0 : min(max(12 - (static_cast<int>(big >> 7) - 127), -115), 126);
        const float f = pow2(e), own = big >= 0x7F80u ? __uint_as_float(0x7FC00000u) : p.scale_log2 * pow2(-e);
        xs[u] = make_float2(__shfl_sync(0xffffffffu, own, 8 * t), __shfl_sync(0xffffffffu, own, 8 * t + 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qb[u][k][x] = ptx::pack_f16x2(__uint_as_float(qb[u][k][x] << 16) * f, __uint_as_float(qb[u][k][x] & 0xFFFF0000u) * f);
      }
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int u = 0; u < NR; ++u) o[k][u][0] = o[k][u][1] = make_float2(0.f, 0.f);
    vref = 0.f;
    // ldmatrix addresses of this lane: K as A fragments by key (lane & 15) and 16-byte half (lane / 16); V^T
    // as A fragments, through transposing loads, by key (lane & 7) + 8 (lane / 16) and half (lane / 8) & 1.
    // A row's swizzle depends on the key's low bits only, which a step's multiple of 16 does not change.
    const uint32_t kr = lane & 15, vr = (lane & 7) + ((lane >> 4) << 3);
    koff = kr * CW + (((lane >> 4) * 16) ^ swizzle(kr));
    voff = vr * CW + ((((lane >> 3) & 1) * 16) ^ swizzle(vr));
  }

  // A step takes 16 KS keys, at consecutive rows of a page run.
  // Products: s[16-key block][row group][0: key g, 1: key g + 8] of rows 2t (x) and 2t + 1 (y).
  // kcol: the head's first column at the step's first row; pitch: bytes from column to column.
  template <int KS>
  __device__ __forceinline__ void scores(uint32_t kcol, uint32_t pitch, float2 (&s)[KS][NR][2]) const {
#pragma unroll
    for (int y = 0; y < KS; ++y)
#pragma unroll
      for (int u = 0; u < NR; ++u) s[y][u][0] = s[y][u][1] = make_float2(0.f, 0.f);
    const uint32_t a0 = kcol + koff, a1 = a0 + pitch;
    if (!FP8) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t a[4];
          ldsm4(((k * 32 < CW ? a0 : a1) ^ ((k * 32) % CW)) + y * 16 * CW, a);
#pragma unroll
          for (int u = 0; u < NR; ++u) mma_16816<false>(s[y][u][0], s[y][u][1], a, qb[u][k][0], qb[u][k][1]);
        }
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2)
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t kb[4];
          ldsm4((a0 ^ (k * 16)) + y * 16 * CW, kb);
#pragma unroll
          for (int x = 0; x < 2; ++x) {   // a lane's four consecutive dims are its two k pairs (q is permuted alike)
            const uint32_t a[4] = {ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[2 * x])),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[2 * x + 1])),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[2 * x] >> 16)),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[2 * x + 1] >> 16))};
#pragma unroll
            for (int u = 0; u < NR; ++u) mma_16816<true>(s[y][u][0], s[y][u][1], a, qb[u][k + x][0], qb[u][k + x][1]);
          }
        }
    }
  }

  // Scores to weights (pb: B fragments of the value product; for a bf16 cache, whose 8 bits would be the
  // largest error before the output's rounding, pl: what that rounding left, multiplied as well) against a reference maximum that trails the
  // running one by at most LAZY (log2): weights stay below 2^LAZY and O is rescaled rarely.  ks, vs: the
  // scales of the step's first key, sstep bytes from key to key; key0: the first key, n: stored keys.
  static constexpr float LAZY = 6.f;
  // e4m3: a weight times its V scale is stored in f16 as a multiple of vref 2^-VSHIFT, so that at most 2^(LAZY +
  // VSHIFT), half of f16's range, is stored, and it has all 11 bits while the product is above 2^-23 vref: an
  // all-zero row, whose scale is 1, costs rows of small values nothing.
  static constexpr int VSHIFT = 9;
  template <int KS>
  __device__ __forceinline__ void weights(const MhaParams& p, float2 (&s)[KS][NR][2], uint32_t ks, uint32_t vs, uint32_t sstep,
                                          uint32_t key0, uint32_t n, int lane, uint32_t (&pb)[KS][NR][2], uint32_t (&pl)[KS][NR][2]) {
    const int g = lane >> 2;
    float sv[KS][2];
    if (FP8) {
      ks += g * sstep;
      vs += g * sstep;
    }
#pragma unroll
    for (int y = 0; y < KS; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x) {     // key 16 y + 8 x + g
        float kf = 1.f;
        if (FP8) {
          kf = ptx::ld_shared_f32(ks);
          sv[y][x] = ptx::ld_shared_f32(vs);
          ks += 8 * sstep;
          vs += 8 * sstep;
        }
#pragma unroll
        for (int u = 0; u < NR; ++u)
          s[y][u][x] = __fmul2_rn(s[y][u][x], FP8 ? make_float2(xs[FP8 ? u : 0].x * kf, xs[FP8 ? u : 0].y * kf) : xs[0]);
      }
    if (key0 + 16 * KS - 1 > n - p.T) {   // some row may not see some of the keys
#pragma unroll
      for (int y = 0; y < KS; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t key = key0 + 16 * y + 8 * x + g;
#pragma unroll
          for (int u = 0; u < NR; ++u) {
            if (key > last[u][0]) s[y][u][x].x = -INFINITY;
            if (key > last[u][1]) s[y][u][x].y = -INFINITY;
          }
          if (FP8 && key >= n) sv[y][x] = 0.f;
        }
    }
    float top = 0.f, mx[NR][2];
    bool due = false;
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      mx[u][0] = s[0][u][0].x;
      mx[u][1] = s[0][u][0].y;
#pragma unroll
      for (int y = 0; y < KS; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          mx[u][0] = fmaxf(mx[u][0], s[y][u][x].x);
          mx[u][1] = fmaxf(mx[u][1], s[y][u][x].y);
          if (FP8 && u == 0) top = fmaxf(top, fabsf(sv[y][x]));
        }
      due = due || mx[u][0] > m[u][0] + LAZY || mx[u][1] > m[u][1] + LAZY;
    }
    if (__any_sync(0xffffffffu, due || (FP8 && top > vref))) {
      float ref = vref;
      if (FP8) {
        top = warp_max(top);
        if (top > vref) ref = pow2(min(max(static_cast<int>(__float_as_uint(top) >> 23) - 126, VSHIFT - 126), 126));
      }
      const float vc = FP8 && ref != vref ? vref / ref : 1.f;
      vref = ref;
#pragma unroll
      for (int u = 0; u < NR; ++u) {
        const float m0 = fmaxf(m[u][0], keys_max(mx[u][0])), m1 = fmaxf(m[u][1], keys_max(mx[u][1]));
        // ex2(-inf) = 0; a row that has seen no key yet keeps -inf
        const float2 c = make_float2(m0 == -INFINITY ? 0.f : ptx::ex2_approx(m[u][0] - m0),
                                     m1 == -INFINITY ? 0.f : ptx::ex2_approx(m[u][1] - m1));
        l[u] = __fmul2_rn(l[u], c);
        const float2 cv = __fmul2_rn(c, make_float2(vc, vc));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          o[k][u][0] = __fmul2_rn(o[k][u][0], cv);
          o[k][u][1] = __fmul2_rn(o[k][u][1], cv);
        }
        m[u][0] = m0;
        m[u][1] = m1;
      }
    }
    // 2^VSHIFT / vref: a power of two's reciprocal has the mirrored exponent
    const float inv = FP8 && vref > 0.f ? __uint_as_float(0x7F000000u + (VSHIFT << 23) - __float_as_uint(vref)) : 0.f;
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const float2 r = make_float2(m[u][0] == -INFINITY ? 0.f : -m[u][0], m[u][1] == -INFINITY ? 0.f : -m[u][1]);
#pragma unroll
      for (int y = 0; y < KS; ++y)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 e = __fadd2_rn(s[y][u][x], r);
          float2 w = make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
          l[u] = __fadd2_rn(l[u], w);
          if (FP8) {
            const float f = sv[y][x] * inv;
            w = __fmul2_rn(w, make_float2(f, f));
            pb[y][u][x] = transpose8(ptx::pack_f16x2(w.x, w.y));
          } else {
            const uint32_t h = ptx::pack_bf16x2(w.x, w.y);
            pb[y][u][x] = transpose8(h);
            pl[y][u][x] = transpose8(ptx::pack_bf16x2(w.x - __uint_as_float(h << 16), w.y - __uint_as_float(h & 0xFFFF0000u)));
          }
        }
    }
  }

  // O^T += V^T P^T; vcol, pitch as for scores.
  template <int KS>
  __device__ __forceinline__ void values(uint32_t vcol, uint32_t pitch, const uint32_t (&pb)[KS][NR][2],
                                         const uint32_t (&pl)[KS][NR][2]) {
    const uint32_t a0 = vcol + voff, a1 = a0 + pitch;
    if (!FP8) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t a[4];
          ldsm4_t(((k * 32 < CW ? a0 : a1) ^ ((k * 32) % CW)) + y * 16 * CW, a);
#pragma unroll
          for (int u = 0; u < NR; ++u) {
            mma_16816<false>(o[k][u][0], o[k][u][1], a, pb[y][u][0], pb[y][u][1]);
            mma_16816<false>(o[k][u][0], o[k][u][1], a, pl[y][u][0], pl[y][u][1]);
          }
        }
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2)       // 32 dims: two blocks of 16, whose even dims are A, odd dims B
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t vb[4];
          ldsm4_t((a0 ^ (k * 16)) + y * 16 * CW, vb);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a[4] = {ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(vb[x], 0, 0x4420))),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(vb[x], 0, 0x4431))),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(vb[x + 2], 0, 0x4420))),
                                   ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(vb[x + 2], 0, 0x4431)))};
#pragma unroll
            for (int u = 0; u < NR; ++u) mma_16816<true>(o[k + x][u][0], o[k + x][u][1], a, pb[y][u][0], pb[y][u][1]);
          }
        }
    }
  }

  // The last step of a request: rows of V past its end hold anything, and a weight of 0 does not silence an
  // infinity.  Zeroes this head's part of rows `from` .. 16 KS - 1 (each warp for itself, before it reads).
  template <int KS>
  __device__ __forceinline__ void clear_tail(uint32_t vcol, uint32_t pitch, uint32_t from, int lane) const {
    constexpr uint32_t UNITS = CW / 16, COLS = D * (FP8 ? 1 : 2) / CW;
    for (uint32_t x = from * UNITS + lane; x < 16 * KS * UNITS; x += 32)
#pragma unroll
      for (uint32_t c = 0; c < COLS; ++c) ptx::st_shared_v4(vcol + c * pitch + x * 16, 0, 0, 0, 0);
    __syncwarp();
  }

  // The whole sums of the rows, and O in its own units.
  __device__ __forceinline__ void finish_sums() {
    const float unit = vref * pow2(-VSHIFT);
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      l[u] = make_float2(keys_sum(l[u].x), keys_sum(l[u].y));
      if (FP8)
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) o[k][u][x] = __fmul2_rn(o[k][u][x], make_float2(unit, unit));
    }
  }
  // Hands the state to, or takes it from, a warp with other keys of the same rows.
  __device__ __forceinline__ void put(float* buf, int lane) const {
    float2* mine = reinterpret_cast<float2*>(buf) + lane;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int u = 0; u < NR; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) mine[((k * NR + u) * 2 + x) * 32] = o[k][u][x];
    if (lane < 4)
#pragma unroll
      for (int u = 0; u < NR; ++u)
        reinterpret_cast<float4*>(buf + 16 * D)[u * 4 + lane] = make_float4(m[u][0], l[u].x, m[u][1], l[u].y);
  }
  __device__ __forceinline__ void add(const float* buf, int lane) {
    const float2* theirs = reinterpret_cast<const float2*>(buf) + lane;
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const float4 ml = reinterpret_cast<const float4*>(buf + 16 * D)[u * 4 + (lane & 3)];
      const float m0 = fmaxf(m[u][0], ml.x), m1 = fmaxf(m[u][1], ml.z);
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
      const float2 a = make_float2(ptx::ex2_approx(m[u][0] - r0), ptx::ex2_approx(m[u][1] - r1));
      const float2 c = make_float2(ptx::ex2_approx(ml.x - r0), ptx::ex2_approx(ml.z - r1));
      l[u] = make_float2(l[u].x * a.x + ml.y * c.x, l[u].y * a.y + ml.w * c.y);
      m[u][0] = m0;
      m[u][1] = m1;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          o[k][u][x] = __ffma2_rn(theirs[((k * NR + u) * 2 + x) * 32], c, __fmul2_rn(o[k][u][x], a));
    }
  }
};

template <int D, bool FP8, int KS, int NR>
__global__ void __launch_bounds__(MHA_THREADS, 1) mla_mha_decode_kernel(const __grid_constant__ MhaParams p) {
  using Rows = MhaRows<D, FP8, NR>;
  constexpr int RT = 8 * NR;                             // rows of a warp
  constexpr int CPH = D * (FP8 ? 1 : 2) / Rows::CW;      // columns per head
  extern __shared__ uint8_t mha_smem_raw[];
  const uint32_t raw = ptx::smem_u32(mha_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = mha_smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t merge = p.stages * p.stage_bytes;
  const uint32_t sbar = merge + (p.kw > 1 ? mha_merge_bytes<D>() : 0);
  const uint32_t sbad = sbar + 8 * 4 * MHA_MAX_STAGES;             // per stage: runs without a page
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + sbad + 4 * MHA_MAX_STAGES);
  int* start = reinterpret_cast<int*>(smem + sbad + 4 * MHA_MAX_STAGES + 16);   // request, item, tile
  long long* tot = reinterpret_cast<long long*>(smem + sbad + 4 * MHA_MAX_STAGES + 64);
  // K and V of a tile are handed over separately: K is free once its scores are formed, while its V waits
  auto full_k = [&](uint32_t s) { return base + sbar + 8 * s; };
  auto full_v = [&](uint32_t s) { return base + sbar + 8 * (MHA_MAX_STAGES + s); };
  auto empty_k = [&](uint32_t s) { return base + sbar + 8 * (2 * MHA_MAX_STAGES + s); };
  auto empty_v = [&](uint32_t s) { return base + sbar + 8 * (3 * MHA_MAX_STAGES + s); };
  const int active = p.hg * p.mt * p.kw;
  const int items = p.head_groups * p.row_groups;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(full_k(s), 1);
      ptx::mbar_init(full_v(s), 1);
      ptx::mbar_init(empty_k(s), active);
      ptx::mbar_init(empty_v(s), active);
    }
    *abort = 0u;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap);
  }
  // this CTA's range of the items' tiles, and where it starts
  long long all = 0, nc = 1, r0 = 0, r1 = 0;
  if (p.one_item) {
    if (threadIdx.x == 0) {
      start[0] = blockIdx.x / items;
      start[1] = blockIdx.x - start[0] * items;
      start[2] = 0;
    }
    r1 = mha_tiles(p, blockIdx.x / items) + MHA_ITEM_COST;
    __syncthreads();
  } else {
    long long mine = 0;
    for (int b = threadIdx.x; b < p.B; b += MHA_THREADS) mine += static_cast<long long>(mha_tiles(p, b) + MHA_ITEM_COST) * items;
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) tot[warp] = mine;
    __syncthreads();
    for (int w = 0; w < MHA_THREADS / 32; ++w) all += tot[w];
    nc = min(static_cast<long long>(gridDim.x), all);    // no empty range among the first nc
    r0 = blockIdx.x < nc ? all * blockIdx.x / nc : all;
    r1 = blockIdx.x < nc ? all * (blockIdx.x + 1ll) / nc : all;
    __syncthreads();
    long long before = 0;
    for (int b0 = 0; b0 < p.B && before <= r0; b0 += MHA_THREADS) {
      const int b = b0 + threadIdx.x;
      const int cost = b < p.B ? mha_tiles(p, b) + MHA_ITEM_COST : 0;
      const long long n = static_cast<long long>(cost) * items;
      long long inc = n;
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (lane == 31) tot[warp] = inc;
      __syncthreads();
      long long off = before;
      for (int w = 0; w < warp; ++w) off += tot[w];
      if (off + inc - n <= r0 && r0 < off + inc) {
        const long long in = r0 - (off + inc - n);
        start[0] = b;
        start[1] = static_cast<int>(in / cost);
        start[2] = static_cast<int>(in % cost);
      }
      for (int w = 0; w < MHA_THREADS / 32; ++w) before += tot[w];
      __syncthreads();
    }
  }
  MhaWalker walk{start[0], start[1], start[2], r1 - r0};
  const uint64_t lim = p.wait_limit_ns;
  auto wait = [&](uint32_t b, uint32_t parity) {         // whole warp, all or none
    return __all_sync(0xffffffffu, wait_bar(b, parity, abort, p.status, 0, lim)) != 0;
  };

  // 384 threads of 168 registers: the producer's warpgroup hands 112 a thread on to the
  // consumers (8 warps x 224 + 4 x 56 = 12 x 168).
  if (warp >= MHA_WARPS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ------------------------------------------------------------------ producer (the group's first warp)
    uint32_t n = 0;                                      // tiles issued
    const int runs = p.tile / p.box_rows;
    const uint32_t sc_bytes = FP8 ? p.box_rows * p.HKV * 4u : 0u;
    const uint32_t box_bytes = p.hg * CPH * p.box_rows * Rows::CW;
    MhaPiece u;
    bool live = warp == MHA_WARPS;
    while (live && walk.next(p, u)) {
      const uint32_t stored = mha_length(p, u.b) + p.T;
      if (lane == 0 && u.ta == 0 && u.item == 0 && p.cache_lengths[u.b] > p.max_cache_length)
        raise_status(p.status, STATUS_BOUNDS);
      const int head0 = (u.item / p.row_groups) * p.hg;
      for (int j = u.ta; j < u.tb; ++j, ++n) {
        const uint32_t s = n % p.stages, use = n / p.stages;
        const uint32_t t = static_cast<uint32_t>(j) * p.tile + lane * p.box_rows;
        const bool in = lane < runs && t < stored;
        bool have = in;
        int row = 0;
        size_t srow = 0;
        if (in) {
          const uint32_t page = p.divP.div(t), slot = t - page * p.P;
          const size_t e = static_cast<size_t>(u.b) * p.max_pages + page;
          const uint32_t blk = p.lut[e], sblk = FP8 ? p.slut[e] : 0u;
          have = blk < static_cast<uint32_t>(p.NB) && (!FP8 || sblk < static_cast<uint32_t>(p.NSB));
          if (!have) raise_status(p.status, STATUS_BOUNDS);
          row = static_cast<int>((static_cast<uint64_t>(blk) * p.KVD * p.NL + p.layer) * p.P + slot);
          if (FP8) srow = (static_cast<size_t>(sblk) * p.KVD * p.NL + p.layer) * p.P + slot;
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, in && !have);
        const uint32_t got = __popc(__ballot_sync(0xffffffffu, have));
        const uint32_t dst = base + s * p.stage_bytes + lane * box_bytes, bytes = got * (box_bytes + sc_bytes);
        const uint32_t sd = base + s * p.stage_bytes + 2 * p.plane_bytes + lane * sc_bytes;
        const int plane_rows = p.NL * p.P;
        // the weights need V's scales before V itself: they come, and go, with K
        if (!wait(empty_k(s), (use & 1) ^ 1)) { live = false; break; }
        if (lane == 0) {
          ptx::st_shared_u32(base + sbad + 4 * s, bad);
          ptx::mbar_arrive_expect_tx(full_k(s), bytes + got * sc_bytes);
        }
        __syncwarp();
        if (have) {
          ptx::tma_load_3d(dst, &p.tmap, 0, row, head0 * CPH, full_k(s));
          if (FP8) {
            ptx::bulk_load(sd, p.scales + srow * p.HKV, sc_bytes, full_k(s));
            ptx::bulk_load(sd + p.tile * p.HKV * 4, p.scales + (srow + plane_rows) * p.HKV, sc_bytes, full_k(s));
          }
        }
        if (!wait(empty_v(s), (use & 1) ^ 1)) { ++n; live = false; break; }
        if (lane == 0) ptx::mbar_arrive_expect_tx(full_v(s), got * box_bytes);
        __syncwarp();
        if (have) ptx::tma_load_3d(dst + p.plane_bytes, &p.tmap, 0, row + plane_rows, head0 * CPH, full_v(s));
      }
    }
    for (uint32_t s = 0; s < static_cast<uint32_t>(p.stages) && s < n; ++s)   // no copy may land after the CTA is gone
    {
      drain_bar(full_k(s), ((n - 1 - s) / p.stages) & 1, 10000000ull);
      drain_bar(full_v(s), ((n - 1 - s) / p.stages) & 1, 10000000ull);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // ------------------------------------------------------------------ consumers
    const int kp = warp / (p.hg * p.mt), pair = warp - kp * p.hg * p.mt;
    const int hl = pair / p.mt, rt = pair - hl * p.mt;   // kv head and row tile within the CTA
    Rows w;
    MhaPiece u;
    uint32_t stk = 0, stv = 0, kpar = 0, vpar = 0;       // next K and V stage, and their phases
    bool live = warp < active;
    int4 mine = make_int4(-1, 0, 0, 0);                  // the item this CTA holds the head of, if it is cut
    while (live && walk.next(p, u)) {
      const int hgi = u.item / p.row_groups, rgi = u.item - hgi * p.row_groups;
      const int kvh = hgi * p.hg + hl, row0 = (rgi * p.mt + rt) * RT;
      const bool work = kvh < p.HKV && row0 < p.R;
      const uint32_t stored = mha_length(p, u.b) + p.T;
      w.load_q(p, u.b, work ? kvh : 0, work ? row0 : p.R, lane);
      // Steps of this warp: keys (kp + x kw) 16 KS of each tile.  The scores of the next step are formed
      // beside the value product of this one: two independent streams of loads, conversions and MMAs.
      const uint32_t pitch = p.box_rows * Rows::CW, box_bytes = p.hg * CPH * pitch, sstep = p.HKV * 4;
      const uint32_t my_k = base + hl * CPH * pitch, my_s = base + 2 * p.plane_bytes + kvh * 4, vscales = p.tile * sstep;
      struct Step {
        uint32_t k, sc, key0;                            // addresses of its K and scales; first key
        bool ok;                                         // has keys, and a page
      };
      auto locate = [&](uint32_t stage, int j, uint32_t g, uint32_t bad) {
        Step t;
        const uint32_t run = g >> p.box_shift, at = stage * p.stage_bytes;
        t.key0 = static_cast<uint32_t>(j) * p.tile + g;
        t.k = my_k + at + run * box_bytes + (g - (run << p.box_shift)) * Rows::CW;
        t.sc = my_s + at + g * sstep;
        t.ok = work && t.key0 < stored && !((bad >> run) & 1u);
        return t;
      };
      auto enter = [&](uint32_t stage, uint32_t& bad) {  // K of the next tile (and V's scales) are in
        if (!wait(full_k(stage), kpar)) return false;
        bad = ptx::ld_shared_u32(base + sbad + 4 * stage);
        return true;
      };
      const uint32_t g0 = kp * 16 * KS, gstep = p.kw * 16 * KS;
      uint32_t bad = 0;
      float2 s[KS][NR][2];
      Step cur{};
      if (u.ta < u.tb) {
        if (!enter(stk, bad)) live = false;
        cur = locate(stk, u.ta, g0, bad);
        if (live && cur.ok) w.template scores<KS>(cur.k, pitch, s);
      }
      for (int j = u.ta; j < u.tb && live; ++j) {
        bool have_v = false;
        for (uint32_t g = g0; g < static_cast<uint32_t>(p.tile) && live; g += gstep) {
          const bool end = g + gstep >= static_cast<uint32_t>(p.tile);   // this warp's last step of the tile
          const bool more = !end || j + 1 < u.tb;
          uint32_t pb[KS][NR][2], pl[KS][NR][2];
          if (cur.ok) w.template weights<KS>(p, s, cur.sc, cur.sc + vscales, sstep, cur.key0, stored, lane, pb, pl);
          if (end) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(empty_k(stk));   // the tile's K and scales are read
            if (++stk == static_cast<uint32_t>(p.stages)) {
              stk = 0;
              kpar ^= 1;
            }
            if (more && !enter(stk, bad)) { live = false; break; }
          }
          if (!have_v) {
            if (!wait(full_v(stv), vpar)) { live = false; break; }
            have_v = true;
          }
          Step nxt = cur;
          if (more) nxt = locate(stk, end ? j + 1 : j, end ? g0 : g + gstep, bad);
          if (cur.ok) {
            const uint32_t v = cur.k + p.plane_bytes;
            if (cur.key0 + 16 * KS > stored) {
              w.template clear_tail<KS>(v, pitch, stored - cur.key0, lane);
              ptx::fence_proxy_async_smem();             // before the stage's next copy
            }
            // (the last step of a piece forms its own scores again: nothing reads them)
            w.template scores<KS>(nxt.k, pitch, s);
            w.template values<KS>(v, pitch, pb, pl);
          } else if (nxt.ok) {
            w.template scores<KS>(nxt.k, pitch, s);
          }
          cur = nxt;
          if (!more) cur.ok = false;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty_v(stv));
        if (++stv == static_cast<uint32_t>(p.stages)) {
          stv = 0;
          vpar ^= 1;
        }
      }
      w.finish_sums();
      if (p.kw > 1) {
        // (on an aborted call too: the last barrier tells every warp that one of them gave up)
        // the upper half of the warps over the keys hands its state to the lower half, and so on
        for (int half = p.kw >> 1; half > 0; half >>= 1) {
          float* buf = reinterpret_cast<float*>(smem + merge) + (pair * half + (kp & (half - 1))) * 16 * (D + 2);
          if (kp >= half && kp < 2 * half) w.put(buf, lane);
          ptx::named_bar_sync(1, 32 * active);
          if (kp < half) w.add(buf, lane);
          live = !bar_any(1, 32 * active, !live);
        }
      }
      if (!live) break;
      const bool head = u.ta == 0, whole = head && u.tb == u.nt;
      if (!whole && head) {
        // the CTA of the item's last tile: the largest c whose range starts at or before it
        const long long end = r1 + (u.nt - u.tb) - 1;
        long long c = end * nc / all;
        while (c + 1 < nc && all * (c + 1) / nc <= end) ++c;
        mine = make_int4(u.b, u.item, static_cast<int>(c), 0);
      }
      if (work && kp == 0) {
        const int gg = lane >> 2, t = lane & 3;
#pragma unroll
        for (int v = 0; v < 2 * NR; ++v) {
          const int x = v >> 1, e = v & 1, r = row0 + 8 * x + 2 * t + e;   // row group, row of the thread's two
          if (r >= p.R) continue;
          const float sum = e ? w.l[x].y : w.l[x].x;
          const bool some = sum > 0.f || sum != sum;     // (a NaN is passed on)
          const float inv = some ? 1.f / sum : 0.f, lse2 = some ? w.m[x][e] + log2f(sum) : -INFINITY;
          if (whole) {
            const int i = static_cast<int>(p.divG.div(r));
            const size_t row = (static_cast<size_t>(u.b) * p.T + i) * p.H + kvh * p.divG.d + (r - i * p.divG.d);
            uint16_t* out = p.out + row * D;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t ab = ptx::pack_bf16x2((e ? w.o[k][x][0].y : w.o[k][x][0].x) * inv, (e ? w.o[k][x][1].y : w.o[k][x][1].x) * inv);
              if (FP8) {
                *reinterpret_cast<uint32_t*>(out + Rows::dim_a(k, gg)) = ab;   // dims 2g, 2g + 1
              } else {
                out[Rows::dim_a(k, gg)] = static_cast<uint16_t>(ab);
                out[Rows::dim_b(k, gg)] = static_cast<uint16_t>(ab >> 16);
              }
            }
            if (p.lse && gg == 0) p.lse[row] = lse2 * 0.6931471805599453f;
          } else {
            const size_t row = (static_cast<size_t>(2 * blockIdx.x + (head ? 1 : 0)) * MHA_ROWS) + pair * RT + 8 * x + 2 * t + e;
            float* out = p.part_o + row * D;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              out[Rows::dim_a(k, gg)] = (e ? w.o[k][x][0].y : w.o[k][x][0].x) * inv;
              out[Rows::dim_b(k, gg)] = (e ? w.o[k][x][1].y : w.o[k][x][1].x) * inv;
            }
            if (gg == 0) p.part_lse[row] = lse2;
          }
        }
      }
    }
    if (!p.one_item && warp == 0 && lane == 0) p.desc[blockIdx.x] = !*abort ? mine : make_int4(-1, 0, 0, 0);
  }
  ptx::griddep_launch_dependents();
}

// Joins the pieces of the item whose head CTA blockIdx.x holds: slot 1 of that CTA, slot 0 of the CTAs
// after it.  One warp per row; lane x holds values x * D / 32 ...
template <int D>
__global__ void __launch_bounds__(256) mla_mha_join_kernel(const __grid_constant__ MhaParams p) {
  ptx::griddep_wait();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 0) return;
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int pair = row / p.row_tile, hl = pair / p.mt, rt = pair - hl * p.mt;
  const int hgi = d.y / p.row_groups, rgi = d.y - hgi * p.row_groups;
  const int kvh = hgi * p.hg + hl, r = (rgi * p.mt + rt) * p.row_tile + row % p.row_tile;
  if (pair >= p.hg * p.mt || kvh >= p.HKV || r >= p.R) return;
  const int c0 = blockIdx.x, parts = d.z - c0 + 1;
  auto slot = [&](int k) { return (static_cast<size_t>(2 * (c0 + k) + (k == 0)) * MHA_ROWS) + row; };
  float mx = -INFINITY;
  for (int k = lane; k < parts; k += 32) mx = fmaxf(mx, p.part_lse[slot(k)]);
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  constexpr int V = D / 32;
  float sum = 0.f, acc[V];
#pragma unroll
  for (int x = 0; x < V; ++x) acc[x] = 0.f;
  const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const size_t at = slot(k);
    const float w = ptx::ex2_approx(p.part_lse[at] - ref);
    sum += w;
    const float* src = p.part_o + at * D + lane * V;
#pragma unroll
    for (int x = 0; x < V; x += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + x);
      acc[x] += w * v.x;
      acc[x + 1] += w * v.y;
    }
  }
  const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
  const int i = static_cast<int>(p.divG.div(r));
  const size_t orow = (static_cast<size_t>(d.x) * p.T + i) * p.H + kvh * p.divG.d + (r - i * p.divG.d);
#pragma unroll
  for (int x = 0; x < V; x += 2)
    *reinterpret_cast<uint32_t*>(p.out + orow * D + lane * V + x) = ptx::pack_bf16x2(acc[x] * inv, acc[x + 1] * inv);
  if (p.lse && lane == 0) p.lse[orow] = sum > 0.f || sum != sum ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace mla
