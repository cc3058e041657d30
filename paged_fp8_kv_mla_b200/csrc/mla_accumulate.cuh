// Accumulated attention weight of every cached key (sm_100a): the quantity that cache eviction ranks
// keys by.  With lse the log-sum-exp the decode of the same step returned, for key t of request b
//   out[b][t] = (t < L_b ? scores[b][t] : 0)
//             + sum_{i : t <= L_b + i} sum_h exp(softmax_scale s_t <q[b,i,h,:], e4m3(code_t)> - lse[b,i,h]).
//
// What bounds it.  A key is 580 bytes and, at 128 heads, 2 * 128 * 576 flop: 88 ps of HBM time and
// 88 ps of bf16 tensor time per key at a B200's measured rates, so bytes and tensor work weigh the
// same and neither may be done twice.
//
// No conversion of the cache.  The keys go from HBM to the tensor core as the e4m3 bytes they are
// (kind::f8f6f4) and it is q that is brought to e4m3, without loss: a bf16 value has 8 significant
// bits and an e4m3 value 4, so after scaling a head's row by a power of two (largest value into
// [128, 256)) x = hi + lo with hi = e4m3_rn(x) and lo = x - hi, an integer multiple m 2^(e-7) with
// |m| <= 8, which e4m3 holds exactly while 2^e >= 2^-2.  Smaller elements are off by at most 2^-10,
// i.e. 2^-17 of the row's largest element.  8-bit MMAs run at twice the 16-bit rate, so the two terms
// cost what one bf16 product would, and no thread touches the keys.  (The accumulation of
// kind::f8f6f4 was measured to be that of fp32 sums: 4e-8 relative on K = 576.)
//
// A = K, B = Q.  D has one key per tensor-memory lane and one head per column, so the sum over heads
// is a sum over a thread's own registers; the per-key factors (scale, mask, running sum) are thread
// constants and the per-head factors (scale, lse) come from shared memory as broadcasts.  hi and lo
// are stacked along N (N = 2 x heads <= 256): one instruction reads the K tile once for both, which
// keeps the shared-memory operand reads (12 KB per 128 cycles of MMA) within the port.  The epilogue
// adds the two column blocks.
//
// Work split.  All requests' tiles of 128 keys laid end to end are cut into equal contiguous ranges,
// one per CTA (one CTA per SM).  A key belongs to one CTA for all query tokens and head groups, so
// sums are formed in a fixed order by one thread: no atomics, and the result does not depend on the
// launch.  K moves through a ring of ten 8 KB slots, one 64-dim column of a tile each, filled by TMA
// (one box per page run) and released by tcgen05.commit, so loads, MMAs and the exponentials of the
// tile before overlap.
//
// Warps: 0 producer, 1 MMA issuer and TMEM owner, 4-7 epilogue (lane quadrants 0-3), 8-15 q split.
#pragma once
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

struct AccumulateParams {
  CUtensorMap tmap_k;              // blocks as {64 bytes, rows, 9 columns}, box = box_rows rows of a column
  const uint16_t* q;               // bf16 bits [B, T, H, 576]
  const float* lse;                // [B, T, H], natural log
  const float* scales;             // [NSB, KVD, NL, P, 1, 1]
  const uint32_t* cache_lengths;   // [B]
  const uint32_t* lut;             // [B, max_pages]
  const uint32_t* slut;            // [B, max_pages] or null
  const float* scores;             // row stride scores_stride; may be null (all zero)
  float* out;                      // row stride out_stride; may be scores itself
  long long scores_stride, out_stride;
  unsigned int* status;
  unsigned long long wait_limit_ns;
  int B, T, H, G, P, KVD, NL, layer, NB, NSB, max_pages, box_rows;
  unsigned int max_cache_length;
  FastDiv divP, divG;
  float softmax_scale;
};

constexpr int ACC_BN = 128;                       // keys per tile (MMA M)
constexpr int ACC_HEADS = 128;                    // heads per item (MMA N = 2 x heads)
constexpr int ACC_COLS = HEAD_DIM / 64;           // 9 columns of 64 dims
constexpr int ACC_THREADS = 512;
constexpr int ACC_EPI_WARP0 = 4;
constexpr int ACC_Q_WARP0 = 8;
constexpr int ACC_Q_WARPS = 8;
constexpr int ACC_SLOTS = 10;
constexpr uint32_t ACC_SLOT_BYTES = ACC_BN * 64;
constexpr uint32_t ACC_SQ = 0;                    // [9 columns][2 x heads rows (hi, then lo)][64 B]
constexpr uint32_t ACC_SK = ACC_COLS * 2 * ACC_HEADS * 64;
constexpr uint32_t ACC_SH = ACC_SK + ACC_SLOTS * ACC_SLOT_BYTES;   // [128] {factor, -lse log2 e}
constexpr uint32_t ACC_SBAR = ACC_SH + ACC_HEADS * 8;
constexpr uint32_t ACC_SMISC = ACC_SBAR + 256;
constexpr uint32_t ACC_SMEM = ACC_SMISC + 64;
constexpr uint32_t ACC_SMEM_ALLOC = ACC_SMEM + 1024;
static_assert(ACC_SMEM_ALLOC <= 232448, "shared memory map exceeds 227 KB");

enum AccBar : uint32_t {
  AB_K_FULL = 0,                    // [10] producer's expect_tx arrival + the column's bytes
  AB_K_EMPTY = ACC_SLOTS,           // [10] commit: the column's MMAs have read it
  AB_ACC_FULL = 2 * ACC_SLOTS,      // [2] commit: a tile's products are in tensor memory
  AB_ACC_EMPTY = AB_ACC_FULL + 2,   // [2] 128 epilogue threads have read them
  AB_Q_FULL = AB_ACC_EMPTY + 2,     // 256 q threads: an item's q and head factors are written
  AB_Q_EMPTY = AB_Q_FULL + 1,       // commit: an item's last MMA is done
  AB_ITEM_DONE = AB_Q_EMPTY + 1,    // 128 epilogue threads: the item's head factors have been read
  AB_DRAIN = AB_ITEM_DONE + 1,      // commit at exit
  ACC_BARS
};
static_assert(8 * ACC_BARS <= 256, "barrier block overlaps what follows");

// D[tmem] (+)= A B^T with e4m3 operands in shared memory (one CTA).
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// Cached tokens of request b, and the keys stored once the step's tokens are in.  A length above
// max_cache_length is clamped (and flagged by the caller that owns the request's first tile).
__device__ __forceinline__ uint32_t acc_length(const AccumulateParams& p, int b) {
  return min(p.cache_lengths[b], p.max_cache_length);
}
__device__ __forceinline__ int acc_tiles(const AccumulateParams& p, int b) {
  return static_cast<int>((acc_length(p, b) + p.T + ACC_BN - 1) / ACC_BN);
}

// Walks a CTA's (request, query token x head group, tile) triples, tiles innermost.
struct AccWalker {
  int b, item, j, ta, tb;          // request, i * G + g, tile, the CTA's tile range of the request
  long long left;                  // tiles of the CTA's range in later requests (after this one)
  __device__ __forceinline__ AccWalker(int b0, int t0, long long tiles) : b(b0 - 1), item(0), j(t0), ta(0), tb(0), left(tiles) {}
  __device__ __forceinline__ bool start(const AccumulateParams& p, int t0) {
    if (left <= 0) return false;
    ++b;
    return open(p, t0);
  }
  __device__ __forceinline__ bool open(const AccumulateParams& p, int t0) {
    if (b >= p.B) return false;
    const int nt = acc_tiles(p, b);
    ta = t0;
    tb = static_cast<int>(min(static_cast<long long>(nt), t0 + left));
    left -= tb - ta;
    item = 0;
    j = ta;
    return true;
  }
  __device__ __forceinline__ bool first_of_item() const { return j == ta; }
  __device__ __forceinline__ bool last_of_item() const { return j + 1 == tb; }
  __device__ __forceinline__ bool next(const AccumulateParams& p) {   // next tile
    if (++j < tb) return true;
    return next_item(p);
  }
  __device__ __forceinline__ bool next_item(const AccumulateParams& p) {
    j = ta;
    if (++item < p.T * p.G) return true;
    if (left <= 0) return false;
    ++b;
    return open(p, 0);
  }
};

// The key a thread owns in tile j of request b: its place, its scale and its running sum.
struct AccKey {
  float scale, base;
  float* dst;                      // null: past the request's end, or in a page that does not exist
};
__device__ __forceinline__ AccKey acc_key(const AccumulateParams& p, int b, int item, int j, int r) {
  AccKey k;
  k.scale = 0.f;
  k.base = 0.f;
  k.dst = nullptr;
  const uint32_t L = acc_length(p, b), t = static_cast<uint32_t>(j) * ACC_BN + r;
  if (t >= L + p.T) return k;
  const uint32_t page = p.divP.div(t), slot = t - page * p.P;
  const size_t e = static_cast<size_t>(b) * p.max_pages + page;
  const uint32_t blk = p.lut[e];
  const uint32_t sblk = p.slut ? p.slut[e] : blk;
  if (blk >= static_cast<uint32_t>(p.NB) || sblk >= static_cast<uint32_t>(p.NSB)) {
    raise_status(p.status, STATUS_BOUNDS);
    return k;
  }
  k.scale = p.scales[((static_cast<size_t>(sblk) * p.KVD) * p.NL + p.layer) * p.P + slot];
  k.dst = p.out + b * p.out_stride + t;
  if (item == 0 && p.scores && t < L) k.base = p.scores[b * p.scores_stride + t];
  return k;
}

// Sum over W heads: the thread's hi and lo columns, its scale, and each head's factor and -lse.
template <int W>
__device__ __forceinline__ void acc_heads(const uint32_t (&hi)[W], const uint32_t (&lo)[W], float s, uint32_t hf,
                                          float (&sum)[4]) {
#pragma unroll
  for (int x = 0; x < W; x += 2) {
    const uint4 f = ptx::ld_shared_v4(hf + x * 8);       // {factor, -lse} of two heads
    const float x0 = (__uint_as_float(hi[x]) + __uint_as_float(lo[x])) * s;
    const float x1 = (__uint_as_float(hi[x + 1]) + __uint_as_float(lo[x + 1])) * s;
    sum[x & 2] += ptx::ex2_approx(fmaf(x0, __uint_as_float(f.x), __uint_as_float(f.y)));
    sum[(x & 2) + 1] += ptx::ex2_approx(fmaf(x1, __uint_as_float(f.z), __uint_as_float(f.w)));
  }
}

// One 16-byte chunk (8 bf16 values, scaled by m1 * m2, a power of two) as 8 hi and 8 lo codes.
__device__ __forceinline__ void acc_split8(uint4 v, float m1, float m2, uint2& hi, uint2& lo) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = __uint_as_float(in[k] << 16) * m1 * m2, b = __uint_as_float(in[k] & 0xFFFF0000u) * m1 * m2;
    h[k] = ptx::e4m3x2_rn_satfinite(a, b);
    const uint32_t back = ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(h[k]));
    l[k] = ptx::e4m3x2_rn_satfinite(a - ptx::f16_lo_to_f32(back), b - ptx::f16_hi_to_f32(back));
  }
  hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" :: "r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// Writes one item's q (hi and lo rows, 64-byte swizzled columns) and head factors.  Each warp takes
// every eighth head row, four rows at a time so that their loads overlap.
__device__ __forceinline__ void acc_write_q(const AccumulateParams& p, const AccWalker& w, uint32_t base, int wq, int lane,
                                            int heads, int hpad, uint4 (&v)[4][3], int r0) {
  const uint32_t col_bytes = static_cast<uint32_t>(hpad) * 128u;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = r0 + u * ACC_Q_WARPS;
    if (r >= hpad) break;
    uint32_t m2 = 0;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      m2 = __vmaxu2(m2, v[u][c].x & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, v[u][c].y & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, v[u][c].z & 0x7FFF7FFFu);
      m2 = __vmaxu2(m2, v[u][c].w & 0x7FFF7FFFu);
    }
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    // the row's power of two, 2^(7 - e) with e the exponent of its largest element; as a product of
    // two factors, since it can be 2^126 (tiny rows: the clamp keeps its reciprocal normal)
    const int e = static_cast<int>(m >> 7) - 127;
    const int k = m == 0 ? 0 : min(max(7 - e, -120), 126);
    const float f1 = __uint_as_float(static_cast<uint32_t>(127 + (k >> 1)) << 23);
    const float f2 = __uint_as_float(static_cast<uint32_t>(127 + (k - (k >> 1))) << 23);
#pragma unroll
    for (int c = 0; c < 3; ++c) {
      const int ch = lane + 32 * c;
      if (ch >= HEAD_DIM / 8) break;
      uint2 hi, lo;
      acc_split8(v[u][c], f1, f2, hi, lo);
      const uint32_t a = base + ACC_SQ + (ch >> 3) * col_bytes + (ch & 1) * 8;
      const uint32_t unit = static_cast<uint32_t>(ch & 7) >> 1;
      // hpad is a multiple of 8, so the lo row hpad + r has the same swizzle phase as row r
      const uint32_t off = r * 64u + ((unit ^ ((static_cast<uint32_t>(r) >> 1) & 3u)) << 4);
      st_shared_v2(a + off, hi);
      st_shared_v2(a + hpad * 64u + off, lo);
    }
    // non-finite rows: a NaN factor makes the request's sums NaN (the codes above would saturate)
    if (lane == 0) {
      const int i = static_cast<int>(p.divG.div(w.item)), g = w.item - i * p.G;
      const float lse = r < heads ? p.lse[(static_cast<size_t>(w.b) * p.T + i) * p.H + g * ACC_HEADS + r] : -INFINITY;
      float f = 0.f, nl = -INFINITY;                     // no such head, or a row without keys: weight 0
      if (lse != -INFINITY) {
        f = m >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                         : p.softmax_scale * 1.4426950408889634f *
                               __uint_as_float(static_cast<uint32_t>(127 - (k >> 1)) << 23) *
                               __uint_as_float(static_cast<uint32_t>(127 - (k - (k >> 1))) << 23);
        nl = -lse * 1.4426950408889634f;
      }
      st_shared_v2(base + ACC_SH + r * 8, make_uint2(__float_as_uint(f), __float_as_uint(nl)));
    }
  }
}

__global__ void __launch_bounds__(ACC_THREADS, 1) mla_accumulate_kernel(const __grid_constant__ AccumulateParams p) {
  extern __shared__ uint8_t acc_smem_raw[];
  const uint32_t raw = ptx::smem_u32(acc_smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = acc_smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + ACC_SMISC + 4);
  int* range = reinterpret_cast<int*>(smem + ACC_SMISC + 16);     // first request, its first tile
  long long* tot = reinterpret_cast<long long*>(smem + ACC_SQ);   // scan scratch (before q is written)
  auto bar = [&](uint32_t i) { return base + ACC_SBAR + 8 * i; };

  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < ACC_SLOTS; ++i) {
      ptx::mbar_init(bar(AB_K_FULL + i), 1);
      ptx::mbar_init(bar(AB_K_EMPTY + i), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(AB_ACC_FULL + i), 1);
      ptx::mbar_init(bar(AB_ACC_EMPTY + i), 128);
    }
    ptx::mbar_init(bar(AB_Q_FULL), 32 * ACC_Q_WARPS);
    ptx::mbar_init(bar(AB_Q_EMPTY), 1);
    ptx::mbar_init(bar(AB_ITEM_DONE), 128);
    ptx::mbar_init(bar(AB_DRAIN), 1);
    *abort = 0u;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap_k);
  }
  if (warp == 1) {
    ptx::tmem_alloc(base + ACC_SMISC, 512);
    ptx::tmem_relinquish();
  }
  // This CTA's range [r0, r1) of the requests' tiles laid end to end, and the request r0 falls in.
  long long mine = 0;
  for (int b = threadIdx.x; b < p.B; b += ACC_THREADS) mine += acc_tiles(p, b);
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) tot[warp] = mine;
  __syncthreads();
  long long all = 0;
  for (int w = 0; w < ACC_THREADS / 32; ++w) all += tot[w];
  const long long r0 = all * blockIdx.x / gridDim.x, r1 = all * (blockIdx.x + 1ll) / gridDim.x;
  __syncthreads();
  long long before = 0;                                  // tiles of the requests before this chunk
  for (int b0 = 0; b0 < p.B && before <= r0; b0 += ACC_THREADS) {
    const int b = b0 + threadIdx.x;
    const long long n = b < p.B ? acc_tiles(p, b) : 0;
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
      range[0] = b;
      range[1] = static_cast<int>(r0 - (off + inc - n));
    }
    for (int w = 0; w < ACC_THREADS / 32; ++w) before += tot[w];
    __syncthreads();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(smem + ACC_SMISC);
  const uint64_t lim = p.wait_limit_ns;
  const int t0 = range[1];
  AccWalker w(range[0], t0, r1 - r0);
  auto wait = [&](uint32_t b, uint32_t parity) {         // whole warp, all or none
    return __all_sync(0xffffffffu, wait_bar(b, parity, abort, p.status, 0, lim)) != 0;
  };
  auto poll = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, poll_bar(b, parity, abort, p.status, 0, lim)) != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    uint32_t n = 0;                                      // columns issued
    const int runs = ACC_BN / p.box_rows;
    bool live = w.start(p, t0);
    while (live) {
      const uint32_t t = static_cast<uint32_t>(w.j) * ACC_BN + lane * p.box_rows;
      bool have = lane < runs && t < acc_length(p, w.b) + p.T;
      int row = 0;
      if (have) {
        const uint32_t page = p.divP.div(t);
        const uint32_t blk = p.lut[static_cast<size_t>(w.b) * p.max_pages + page];
        have = blk < static_cast<uint32_t>(p.NB);        // the epilogue flags it and leaves its keys
        row = static_cast<int>((static_cast<uint64_t>(blk) * p.KVD * p.NL + p.layer) * p.P + (t - page * p.P));
      }
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, have)) * p.box_rows * 64u;
      for (int c = 0; c < ACC_COLS; ++c, ++n) {
        const uint32_t s = n % ACC_SLOTS, use = n / ACC_SLOTS;
        if (!wait(bar(AB_K_EMPTY + s), (use & 1) ^ 1)) { live = false; break; }
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar(AB_K_FULL + s), bytes);
        __syncwarp();
        if (have)
          ptx::tma_load_3d(base + ACC_SK + s * ACC_SLOT_BYTES + lane * p.box_rows * 64u, &p.tmap_k, 0, row, c,
                           bar(AB_K_FULL + s));
      }
      live = live && w.next(p);
    }
    // no copy may land after the CTA is gone (also on an aborted call)
    for (uint32_t s = 0; s < ACC_SLOTS && s < n; ++s)
      drain_bar(bar(AB_K_FULL + s), ((n - 1 - s) / ACC_SLOTS) & 1, lim);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    uint32_t n = 0, tile = 0, items = 0;
    bool live = w.start(p, t0);
    while (live) {
      const int g = w.item - static_cast<int>(p.divG.div(w.item)) * p.G;
      const int hpad = (min(p.H - g * ACC_HEADS, ACC_HEADS) + 7) & ~7;
      const uint32_t idesc = ptx::idesc_e4m3_f32(ACC_BN, 2 * hpad, false, false);
      const uint32_t col_bytes = static_cast<uint32_t>(hpad) * 128u;
      if (w.first_of_item()) {
        if (!poll(bar(AB_Q_FULL), items & 1)) break;
        ++items;
      }
      const uint32_t d = tbase + (tile & 1) * 256;
      if (!poll(bar(AB_ACC_EMPTY + (tile & 1)), ((tile >> 1) & 1) ^ 1)) break;
      ptx::tc_fence_after();
      for (int c = 0; c < ACC_COLS; ++c, ++n) {
        const uint32_t s = n % ACC_SLOTS;
        if (!poll(bar(AB_K_FULL + s), (n / ACC_SLOTS) & 1)) { live = false; break; }
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t a = ptx::smem_desc(base + ACC_SK + s * ACC_SLOT_BYTES, 16, 512, ptx::SW_64B);
          const uint64_t b = ptx::smem_desc(base + ACC_SQ + c * col_bytes, 16, 512, ptx::SW_64B);
          mma_ss_e4m3(d, a, b, idesc, c > 0);
          mma_ss_e4m3(d, a + 2, b + 2, idesc, 1);        // the column's second 32 dims: + 32 bytes
          ptx::mma_commit(bar(AB_K_EMPTY + s));
        }
        __syncwarp();
      }
      if (!live) break;
      if (ptx::elect_one()) {
        ptx::mma_commit(bar(AB_ACC_FULL + (tile & 1)));
        if (w.last_of_item()) ptx::mma_commit(bar(AB_Q_EMPTY));
      }
      __syncwarp();
      ++tile;
      live = w.next(p);
    }
    if (ptx::elect_one()) ptx::mma_commit(bar(AB_DRAIN));
    __syncwarp();
    drain_bar(bar(AB_DRAIN), 0, lim);
  } else if (warp >= ACC_EPI_WARP0 && warp < ACC_EPI_WARP0 + 4) {
    // ------------------------------------------------------------------ epilogue
    const int r = threadIdx.x - 32 * ACC_EPI_WARP0;      // the tile's key = tensor-memory lane
    const uint32_t quad = static_cast<uint32_t>(warp - ACC_EPI_WARP0) << 21;
    uint32_t tile = 0, items = 0;
    bool live = w.start(p, t0);
    if (live && r == 0 && p.cache_lengths[w.b] > p.max_cache_length) raise_status(p.status, STATUS_BOUNDS);
    AccKey key = live ? acc_key(p, w.b, w.item, w.j, r) : AccKey{0.f, 0.f, nullptr};
    while (live) {
      const AccWalker cur = w;
      live = w.next(p);
      if (live && w.b != cur.b && r == 0 && p.cache_lengths[w.b] > p.max_cache_length)
        raise_status(p.status, STATUS_BOUNDS);
      // the next tile's scale and running sum are on their way while this tile is summed
      const AccKey nxt = live ? acc_key(p, w.b, w.item, w.j, r) : AccKey{0.f, 0.f, nullptr};
      const int i = static_cast<int>(p.divG.div(cur.item)), g = cur.item - i * p.G;
      const int hpad = (min(p.H - g * ACC_HEADS, ACC_HEADS) + 7) & ~7;
      if (cur.first_of_item() && !wait(bar(AB_Q_FULL), items & 1)) break;   // head factors are written
      if (!wait(bar(AB_ACC_FULL + (tile & 1)), (tile >> 1) & 1)) break;
      ptx::tc_fence_after();
      const uint32_t d = tbase + quad + (tile & 1) * 256, hf = base + ACC_SH;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      int h = 0;
      for (; h + 32 <= hpad; h += 32) {
        uint32_t hi[32], lo[32];
        ptx::tmem_ld32(d + h, hi);
        ptx::tmem_ld32(d + hpad + h, lo);
        ptx::tmem_wait_ld();
        acc_heads<32>(hi, lo, key.scale, hf + h * 8, sum);
      }
      for (; h < hpad; h += 8) {
        uint32_t hi[8], lo[8];
        tmem_ld8(d + h, hi);
        tmem_ld8(d + hpad + h, lo);
        ptx::tmem_wait_ld();
        acc_heads<8>(hi, lo, key.scale, hf + h * 8, sum);
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(AB_ACC_EMPTY + (tile & 1)));
      if (cur.last_of_item()) {
        ptx::mbar_arrive(bar(AB_ITEM_DONE));
        ++items;
      }
      if (key.dst) {
        const uint32_t t = static_cast<uint32_t>(cur.j) * ACC_BN + r;
        const float add = t <= acc_length(p, cur.b) + i ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
        *key.dst = (cur.item == 0 ? key.base : *key.dst) + add;
      }
      key = nxt;
      ++tile;
    }
  } else if (warp >= ACC_Q_WARP0) {
    // ------------------------------------------------------------------ q split
    const int wq = warp - ACC_Q_WARP0;
    uint32_t items = 0;
    bool live = w.start(p, t0);
    while (live) {
      const int i = static_cast<int>(p.divG.div(w.item)), g = w.item - i * p.G;
      const int heads = min(p.H - g * ACC_HEADS, ACC_HEADS), hpad = (heads + 7) & ~7;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((static_cast<size_t>(w.b) * p.T + i) * p.H + g * ACC_HEADS) * HEAD_DIM);
      bool freed = items == 0;
      for (int r0 = wq; r0 < hpad; r0 += 4 * ACC_Q_WARPS) {
        uint4 v[4][3];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = r0 + u * ACC_Q_WARPS;
#pragma unroll
          for (int c = 0; c < 3; ++c)
            v[u][c] = r < heads && lane + 32 * c < HEAD_DIM / 8 ? src[static_cast<size_t>(r) * (HEAD_DIM / 8) + lane + 32 * c]
                                                               : make_uint4(0, 0, 0, 0);
        }
        if (!freed) {   // the last item's MMAs have read q, and its epilogue the head factors
          if (!wait(bar(AB_Q_EMPTY), (items - 1) & 1) || !wait(bar(AB_ITEM_DONE), (items - 1) & 1)) { live = false; break; }
          freed = true;
        }
        acc_write_q(p, w, base, wq, lane, heads, hpad, v, r0);
      }
      if (!live) break;
      if (!freed && (!wait(bar(AB_Q_EMPTY), (items - 1) & 1) || !wait(bar(AB_ITEM_DONE), (items - 1) & 1))) break;
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(bar(AB_Q_FULL));
      ++items;
      live = w.next_item(p);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tbase, 512);
}

}  // namespace mla
