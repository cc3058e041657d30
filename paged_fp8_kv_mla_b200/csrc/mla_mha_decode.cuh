// Decode attention over a paged cache with separate keys and values per kv head (sm_100a): kv plane 0
// holds K, plane 1 holds V, in bf16 or in e4m3 with one fp32 scale per token and head.  With G = H / HKV
// query heads per kv head, for request b, query token i and query head h (kv head h / G):
//   x[t] = softmax_scale <q[b,i,h,:], K[t]>  for t <= L_b + i,
//   lse  = ln sum_t exp(x[t]),   out[b,i,h,:] = sum_t exp(x[t] - lse) V[t].
//
// What bounds it.  A kv head's key and value are 4 D bytes (bf16) for 4 D flop per query row, so up to
// some hundred rows per kv head the cache's bytes set the time: every K and V byte is to cross HBM once,
// at full rate, and the arithmetic has to stay out of the way.  The rows that share a kv head
// (R = T * G of them) are few, so the products run on the warp-level 16 x 8 x 16 MMA with 16 rows per
// warp: a tcgen05 tile has 128 rows, most of them empty here, and its accumulator would have to come
// back from tensor memory for every rescale.
//
// Who does what.  Eight consumer warps per CTA (one CTA per SM).  A warp owns 16 rows of one kv head
// (its scores, weights and O stay in its registers; no exchange within a tile) and, where fewer than
// eight (head, row tile) pairs exist, every kw-th group of 16 keys; those kw warps merge once, at the
// end of a piece.  All warps read the same tile, so K and V are loaded once for all of up to 128 rows,
// and a tile's rows are read as whole contiguous runs of the page over the CTA's heads.  A ninth warp
// keeps a ring of tiles full by TMA: one box per page run and plane, [column of 128 (64) bytes][key],
// in the matching shared-memory swizzle, so that ldmatrix reads rows without bank conflicts.
//
// e4m3.  The values are converted to f16, exactly, as they leave shared memory (two per instruction),
// and never to anything wider: q is brought to f16 with a power of two per row (exact down to 2^-30 of
// the row's largest value), K's scale multiplies the score, and V's scale goes into the weight, relative
// to a running power-of-two bound of V's scales so that f16 holds it with 11 bits.  A thread's four
// consecutive bytes serve as the two k pairs of its MMA fragment, which only permutes the order of the
// sum over dims (q is permuted the same way).
//
// Work split.  The tiles of all (request, head group, row group) items laid end to end are cut into
// equal contiguous ranges, one per CTA.  An item cut by a range's end leaves normalised fp32 partials
// and their log-sum-exp in the workspace and a second kernel joins them; each CTA names the item whose
// head it holds and the last CTA of it, so the join needs no plan and nothing has to start at zero.
// Where all requests are short (one or two tiles), each CTA takes one item and the second launch is
// left out.
#pragma once
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

constexpr int MHA_WARPS = 8;                      // consumer warps
constexpr int MHA_THREADS = 32 * (MHA_WARPS + 4);   // consumers, and a warpgroup for the producer warp
constexpr int MHA_ROWS = 16 * MHA_WARPS;          // rows of a CTA at most
constexpr int MHA_MAX_STAGES = 8;
constexpr int MHA_MAX_RUNS = 16;                  // page runs of a tile
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
  int head_groups, row_groups;     // of a request: its items
  int tile, box_rows, box_shift, stages;   // keys per tile, keys per box (a power of two) and its log2, ring depth
  uint32_t plane_bytes, stage_bytes;   // of a tile's K (or V); of a ring stage
  int one_item;                    // 1: CTA c computes item c alone
  FastDiv divP, divG;              // by the page size and by G = H / HKV
  float scale_log2;                // softmax_scale * log2(e)
};

__device__ __forceinline__ void mma_16816_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_bf16(float2 (&c)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0].x), "+f"(c[0].y), "+f"(c[1].x), "+f"(c[1].y)
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_f16(float2 (&c)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0].x), "+f"(c[0].y), "+f"(c[1].x), "+f"(c[1].y)
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float warp_max(float v) {   // v >= 0
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t mha_length(const MhaParams& p, int b) {
  return min(p.cache_lengths[b], p.max_cache_length);
}
__device__ __forceinline__ int mha_tiles(const MhaParams& p, int b) {   // of one item of request b
  return static_cast<int>((mha_length(p, b) + p.T + p.tile - 1) / p.tile);
}

// A CTA's piece of an item: tiles [ta, tb) of nt.
struct MhaPiece {
  int b, item, ta, tb, nt;
};
// Walks the pieces of a CTA's range [r0, r1) of the items' tiles laid end to end.
struct MhaWalker {
  int b, item, t0;
  long long left;
  __device__ __forceinline__ bool next(const MhaParams& p, MhaPiece& u) {
    if (left <= 0 || b >= p.B) return false;
    u.b = b;
    u.item = item;
    u.nt = mha_tiles(p, b);
    u.ta = t0;
    u.tb = static_cast<int>(min(static_cast<long long>(u.nt), t0 + left));
    left -= u.tb - u.ta;
    t0 = 0;
    if (++item == p.head_groups * p.row_groups) {
      item = 0;
      ++b;
    }
    return true;
  }
};

// Shared memory after the ring: the warps' merge buffers (kw > 1), then the barriers.
template <int D>
__host__ __device__ constexpr uint32_t mha_merge_bytes() { return (MHA_WARPS / 2) * 16 * (D + 2) * 4; }
constexpr uint32_t MHA_MISC_BYTES = 8 * 4 * MHA_MAX_STAGES + 4 * MHA_MAX_STAGES + 64 + 8 * (MHA_WARPS + 4) + 64;

// One warp's state: 16 rows (thread: rows lane / 4 and lane / 4 + 8) of one kv head.
template <int D, bool FP8>
struct MhaRows {
  static constexpr int CW = D * (FP8 ? 1 : 2) < 128 ? D * (FP8 ? 1 : 2) : 128;   // bytes of a column
  uint32_t qa[D / 16][4];          // q as A fragments (bf16, or f16 times a power of two per row)
  float o[D / 8][4];
  float m[2];                      // reference maximum (base 2) of the thread's two rows
  float2 l[2];                     // this thread's part of the sum (even, odd keys)
  float xs;                        // score factor
  uint32_t koff, voff;             // this lane's place in a 16-key block of K and V
  uint32_t last[2];                // last visible key of each row
  float vref;                      // e4m3: power-of-two bound of V's scales so far (0: none yet)

  static __device__ __forceinline__ uint32_t swizzle(uint32_t r) { return CW == 128 ? (r & 7u) << 4 : ((r >> 1) & 3u) << 4; }

  // Query rows row0 .. row0 + 15 of kv head kvh (rows past the last one are zero).  For e4m3 caches q is
  // brought to f16 by one power of two for the 16 rows (largest value into [2^12, 2^13)).
  __device__ __forceinline__ void load_q(const MhaParams& p, int b, int kvh, int row0, int lane) {
    const int t = lane & 3;
    uint32_t m2 = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = row0 + (lane >> 2) + 8 * u;
      const bool have = r < p.R;
      const int i = have ? static_cast<int>(p.divG.div(r)) : 0;
      const int h = kvh * p.divG.d + (r - i * p.divG.d);
      last[u] = mha_length(p, b) + i;
      const uint16_t* src = p.q + ((static_cast<size_t>(b) * p.T + i) * p.H + h) * D;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if (!FP8) {
          qa[k][u] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * t) : 0u;
          qa[k][u + 2] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8 + 2 * t) : 0u;
        } else {
          const uint2 v = have ? *reinterpret_cast<const uint2*>(src + 16 * k + 4 * t) : make_uint2(0, 0);
          qa[k][u] = v.x;
          qa[k][u + 2] = v.y;
          m2 = __vmaxu2(__vmaxu2(m2, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
        }
      }
      m[u] = -INFINITY;
      l[u] = make_float2(0.f, 0.f);
    }
    xs = p.scale_log2;
    if (FP8) {
      const uint32_t big = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
      const int e = big == 0 ? 0 : min(max(12 - (static_cast<int>(big >> 7) - 127), -115), 126);
      const float f = pow2(e);
      xs = big >= 0x7F80u ? __uint_as_float(0x7FC00000u) : p.scale_log2 * pow2(-e);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          qa[k][x] = ptx::pack_f16x2(__uint_as_float(qa[k][x] << 16) * f, __uint_as_float(qa[k][x] & 0xFFFF0000u) * f);
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
    vref = 0.f;
    // ldmatrix rows and 16-byte units of this lane: K by keys (lane & 7) + 8 (lane / 16), V by keys lane & 15;
    // a row's swizzle depends on the key's low bits only, which a step's multiple of 16 does not change
    const uint32_t kr = (lane & 7) + ((lane >> 4) << 3), vr = lane & 15;
    koff = kr * CW + ((((lane >> 3) & 1) * 16) ^ swizzle(kr));
    voff = vr * CW + (((lane >> 4) * 16) ^ swizzle(vr));
  }

  // A step takes 16 KS keys, at rows row .. of a page run.  KS = 2 halves the rescales and reductions per
  // key and gives the MMAs four independent accumulators instead of two.
  // Products q K^T: s[8-key group][row lane / 4: keys 2t, 2t + 1; row lane / 4 + 8: the same], t = lane % 4.
  // kcol: the head's first column at the step's first row; pitch: bytes from column to column.
  template <int KS>
  __device__ __forceinline__ void scores(uint32_t kcol, uint32_t pitch, float2 (&s)[2 * KS][2]) const {
#pragma unroll
    for (int x = 0; x < 2 * KS; ++x) s[x][0] = s[x][1] = make_float2(0.f, 0.f);
    const uint32_t a0 = kcol + koff, a1 = a0 + pitch;
    if (!FP8) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t kb[4];
          ldsm4(((k * 32 < CW ? a0 : a1) ^ ((k * 32) % CW)) + y * 16 * CW, kb);
          mma_16816_bf16(s[2 * y], qa[k], kb[0], kb[1]);
          mma_16816_bf16(s[2 * y + 1], qa[k], kb[2], kb[3]);
        }
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2)
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t kb[4];
          ldsm4((a0 ^ (k * 16)) + y * 16 * CW, kb);
#pragma unroll
          for (int x = 0; x < 4; ++x)   // x & 1: k step, x >> 1: key half
            mma_16816_f16(s[2 * y + (x >> 1)], qa[k + (x & 1)], ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[x])),
                          ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(kb[x] >> 16)));
        }
    }
  }

  // Scores to weights (pa: A fragments of the value product) against a reference maximum that trails the
  // running one by at most LAZY (log2): weights stay below 2^LAZY and O is rescaled rarely.  ks, vs: the
  // scales of the step's first key, sstep bytes from key to key; key0: the first key, n: stored keys.
  static constexpr float LAZY = 6.f;
  template <int KS>
  __device__ __forceinline__ void weights(const MhaParams& p, float2 (&s)[2 * KS][2], uint32_t ks, uint32_t vs, uint32_t sstep,
                                          uint32_t key0, uint32_t n, int lane, uint32_t (&pa)[KS][4]) {
    const int t = lane & 3;
    float2 sv[2 * KS];
    if (FP8) {
      ks += 2 * t * sstep;
      vs += 2 * t * sstep;
    }
#pragma unroll
    for (int x = 0; x < 2 * KS; ++x) {  // keys 8 x + 2 t, + 1
      float2 f = make_float2(xs, xs);
      if (FP8) {
        f = __fmul2_rn(make_float2(ptx::ld_shared_f32(ks), ptx::ld_shared_f32(ks + sstep)), f);
        sv[x] = make_float2(ptx::ld_shared_f32(vs), ptx::ld_shared_f32(vs + sstep));
        ks += 8 * sstep;
        vs += 8 * sstep;
      }
      s[x][0] = __fmul2_rn(s[x][0], f);
      s[x][1] = __fmul2_rn(s[x][1], f);
    }
    if (key0 + 16 * KS - 1 > n - p.T) {   // some row may not see some of the keys
#pragma unroll
      for (int x = 0; x < 2 * KS; ++x) {
        const uint32_t key = key0 + 8 * x + 2 * t;
        if (key > last[0]) s[x][0].x = -INFINITY;
        if (key + 1 > last[0]) s[x][0].y = -INFINITY;
        if (key > last[1]) s[x][1].x = -INFINITY;
        if (key + 1 > last[1]) s[x][1].y = -INFINITY;
        if (FP8 && key >= n) sv[x].x = 0.f;
        if (FP8 && key + 1 >= n) sv[x].y = 0.f;
      }
    }
    float m0 = s[0][0].x, m1 = s[0][1].x, top = 0.f;
#pragma unroll
    for (int x = 0; x < 2 * KS; ++x) {
      m0 = fmaxf(m0, fmaxf(s[x][0].x, s[x][0].y));
      m1 = fmaxf(m1, fmaxf(s[x][1].x, s[x][1].y));
      if (FP8) top = fmaxf(top, fmaxf(fabsf(sv[x].x), fabsf(sv[x].y)));
    }
    // (the row's own lanes may disagree on whether a rescale is due: the vote decides for the warp)
    if (__any_sync(0xffffffffu, m0 > m[0] + LAZY || m1 > m[1] + LAZY || (FP8 && top > vref))) {
      m0 = fmaxf(m[0], quad_max(m0));
      m1 = fmaxf(m[1], quad_max(m1));
      float ref = vref;
      if (FP8) {
        top = warp_max(top);
        if (top > vref) ref = pow2(min(max(static_cast<int>(__float_as_uint(top) >> 23) - 126, -126), 126));
      }
      // ex2(-inf) = 0; a row that has seen no key yet keeps -inf
      const float c0 = m0 == -INFINITY ? 0.f : ptx::ex2_approx(m[0] - m0);
      const float c1 = m1 == -INFINITY ? 0.f : ptx::ex2_approx(m[1] - m1);
      const float vc = FP8 && ref != vref ? vref / ref : 1.f;
      l[0] = make_float2(l[0].x * c0, l[0].y * c0);
      l[1] = make_float2(l[1].x * c1, l[1].y * c1);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        o[k][0] *= c0 * vc;
        o[k][1] *= c0 * vc;
        o[k][2] *= c1 * vc;
        o[k][3] *= c1 * vc;
      }
      m[0] = m0;
      m[1] = m1;
      vref = ref;
    }
    const float r0 = m[0] == -INFINITY ? 0.f : -m[0], r1 = m[1] == -INFINITY ? 0.f : -m[1];
    // 1 / vref: a power of two's reciprocal has the mirrored exponent
    const float inv = FP8 && vref > 0.f ? __uint_as_float(0x7F000000u - __float_as_uint(vref)) : 0.f;
#pragma unroll
    for (int x = 0; x < 2 * KS; ++x) {
      uint32_t* a = &pa[x >> 1][(x & 1) * 2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2 e = __fadd2_rn(s[x][u], u ? make_float2(r1, r1) : make_float2(r0, r0));
        float2 w = make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
        l[u] = __fadd2_rn(l[u], w);
        if (FP8) {
          w = __fmul2_rn(w, __fmul2_rn(sv[x], make_float2(inv, inv)));
          a[u] = ptx::pack_f16x2(w.x, w.y);
        } else {
          a[u] = ptx::pack_bf16x2(w.x, w.y);
        }
      }
    }
  }

  // O += weights * V; vcol, pitch as for scores.
  template <int KS>
  __device__ __forceinline__ void values(uint32_t vcol, uint32_t pitch, const uint32_t (&pa)[KS][4]) {
    const uint32_t a0 = vcol + voff, a1 = a0 + pitch;
    if (!FP8) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t vb[4];
          ldsm4_t(((k * 32 < CW ? a0 : a1) ^ ((k * 32) % CW)) + y * 16 * CW, vb);
          mma_16816_bf16(o[2 * k], pa[y], vb[0], vb[1]);
          mma_16816_bf16(o[2 * k + 1], pa[y], vb[2], vb[3]);
        }
    } else {
#pragma unroll
      for (int k = 0; k < D / 32; ++k)          // 32 dims: two blocks of 16, an even and an odd tile each
#pragma unroll
        for (int y = 0; y < KS; ++y) {
          uint32_t vb[4];
          ldsm4_t((a0 ^ (k * 32)) + y * 16 * CW, vb);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a = vb[2 * x], b = vb[2 * x + 1];
            mma_16816_f16(o[4 * k + 2 * x], pa[y], ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(a, 0, 0x4420))),
                          ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(b, 0, 0x4420))));
            mma_16816_f16(o[4 * k + 2 * x + 1], pa[y], ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(a, 0, 0x4431))),
                          ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(b, 0, 0x4431))));
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

  // Adds another warp's state over other keys of the same rows (l already summed over the quad).
  __device__ __forceinline__ void put(float* buf, int lane) const {
    float* mine = buf + lane;
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x) mine[(4 * k + x) * 32] = o[k][x];
    if ((lane & 3) == 0) {
      float* ml = buf + 16 * D + (lane >> 2) * 2;
      ml[0] = m[0];
      ml[1] = l[0].x;
      ml[16] = m[1];
      ml[17] = l[1].x;
    }
  }
  __device__ __forceinline__ void add(const float* buf, int lane) {
    const float* ml = buf + 16 * D + (lane >> 2) * 2;
    float mine[2], theirs[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float om = ml[16 * u], ol = ml[16 * u + 1], mm = fmaxf(m[u], om), ref = mm == -INFINITY ? 0.f : mm;
      mine[u] = ptx::ex2_approx(m[u] - ref);
      theirs[u] = ptx::ex2_approx(om - ref);
      l[u].x = l[u].x * mine[u] + ol * theirs[u];
      m[u] = mm;
    }
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        o[k][x] = o[k][x] * mine[x >> 1] + buf[lane + (4 * k + x) * 32] * theirs[x >> 1];
  }
  __device__ __forceinline__ void finish_sums() {
    l[0].x = quad_sum(l[0].x + l[0].y);
    l[1].x = quad_sum(l[1].x + l[1].y);
    if (FP8) {
#pragma unroll
      for (int k = 0; k < D / 8; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[k][x] *= vref;
    }
  }
};

template <int D, bool FP8, int KS>
__global__ void __launch_bounds__(MHA_THREADS, 1) mla_mha_decode_kernel(const __grid_constant__ MhaParams p) {
  using Rows = MhaRows<D, FP8>;
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
    r1 = mha_tiles(p, blockIdx.x / items);
    __syncthreads();
  } else {
    long long mine = 0;
    for (int b = threadIdx.x; b < p.B; b += MHA_THREADS) mine += static_cast<long long>(mha_tiles(p, b)) * items;
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
      const int nt = b < p.B ? mha_tiles(p, b) : 0;
      const long long n = static_cast<long long>(nt) * items;
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
        start[1] = static_cast<int>(in / nt);
        start[2] = static_cast<int>(in % nt);
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
      const int kvh = hgi * p.hg + hl, row0 = (rgi * p.mt + rt) * 16;
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
      float2 s[2 * KS][2];
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
          uint32_t pa[KS][4];
          if (cur.ok) w.template weights<KS>(p, s, cur.sc, cur.sc + vscales, sstep, cur.key0, stored, lane, pa);
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
            w.template values<KS>(v, pitch, pa);
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
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int r = row0 + (lane >> 2) + 8 * v, t = lane & 3;
          if (r >= p.R) continue;
          const float inv = w.l[v].x > 0.f || w.l[v].x != w.l[v].x ? 1.f / w.l[v].x : 0.f;
          const float lse2 = w.l[v].x > 0.f || w.l[v].x != w.l[v].x ? w.m[v] + log2f(w.l[v].x) : -INFINITY;
          if (whole) {
            const int i = static_cast<int>(p.divG.div(r));
            const size_t row = (static_cast<size_t>(u.b) * p.T + i) * p.H + kvh * p.divG.d + (r - i * p.divG.d);
            uint16_t* out = p.out + row * D;
            if (!FP8) {
#pragma unroll
              for (int k = 0; k < D / 8; ++k)
                *reinterpret_cast<uint32_t*>(out + 8 * k + 2 * t) = ptx::pack_bf16x2(w.o[k][2 * v] * inv, w.o[k][2 * v + 1] * inv);
            } else {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                *reinterpret_cast<uint2*>(out + 16 * k + 4 * t) =
                    make_uint2(ptx::pack_bf16x2(w.o[2 * k][2 * v] * inv, w.o[2 * k + 1][2 * v] * inv),
                               ptx::pack_bf16x2(w.o[2 * k][2 * v + 1] * inv, w.o[2 * k + 1][2 * v + 1] * inv));
            }
            if (p.lse && t == 0) p.lse[row] = lse2 * 0.6931471805599453f;
          } else {
            const size_t row = (static_cast<size_t>(2 * blockIdx.x + (head ? 1 : 0)) * MHA_ROWS) + pair * 16 + (lane >> 2) + 8 * v;
            float* out = p.part_o + row * D;
            if (!FP8) {
#pragma unroll
              for (int k = 0; k < D / 8; ++k)
                *reinterpret_cast<float2*>(out + 8 * k + 2 * t) = make_float2(w.o[k][2 * v] * inv, w.o[k][2 * v + 1] * inv);
            } else {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                *reinterpret_cast<float4*>(out + 16 * k + 4 * t) =
                    make_float4(w.o[2 * k][2 * v] * inv, w.o[2 * k + 1][2 * v] * inv,
                                w.o[2 * k][2 * v + 1] * inv, w.o[2 * k + 1][2 * v + 1] * inv);
            }
            if (t == 0) p.part_lse[row] = lse2;
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
  const int pair = row >> 4, hl = pair / p.mt, rt = pair - hl * p.mt;
  const int hgi = d.y / p.row_groups, rgi = d.y - hgi * p.row_groups;
  const int kvh = hgi * p.hg + hl, r = (rgi * p.mt + rt) * 16 + (row & 15);
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
