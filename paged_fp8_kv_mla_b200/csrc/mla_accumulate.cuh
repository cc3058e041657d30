// Accumulated attention weight of every cached key (sm_100a): the quantity that cache eviction ranks
// keys by.  With lse the log-sum-exp the decode of the same step returned, for key t of request b
//   out[b][t] = (t < L_b ? scores[b][t] : 0)
//             + sum_{i : t <= L_b + i} sum_h exp(softmax_scale s_t <q[b,i,h,:], e4m3(code_t)> - lse[b,i,h]).
//
// What bounds it.  A key is 580 bytes and, at 128 heads, 2 * 128 * 576 flop: 88 ps of HBM time and
// 88 ps of bf16 tensor time per key at a B200's measured rates, so for one new token and up to 128 heads
// bytes and tensor work weigh the same and neither is done twice.  Each further (query token, group of 128
// heads) is an item of its own: q of one item takes 147 KB of shared memory, so a CTA walks its tiles once per
// item and the keys come again each time, from HBM where its range is long (64 ragged requests, 2 tokens: 302 MB
// read for 144 MB of keys).  Every item also walks to the end of its request, past the last key that its
// token sees, so a prompt does up to twice the products that it needs.
//
// No conversion of the cache.  The keys go from HBM to the tensor core as the e4m3 bytes they are
// (kind::f8f6f4) and it is q that is brought to e4m3, without loss: a bf16 value has 8 significant
// bits and an e4m3 value 4, so after scaling a head's row by a power of two (largest value into
// [128, 256)) x = hi + lo / 16 with hi = e4m3_rn(x) and lo = 16 (x - hi).  x - hi is m 2^(e-7) with an
// integer |m| <= 8, which e4m3 holds exactly down to 2^e = 2^-6, i.e. 2^-13 of the row's largest
// element; smaller elements are off by at most 2^-14, 2^-21 of it.  8-bit MMAs run at twice the 16-bit
// rate, so the two terms cost what one bf16 product would, and no thread touches the keys.  (The
// accumulation of kind::f8f6f4 was measured to be that of fp32 sums: 4e-8 relative on K = 576.)
// The split is a kernel of its own, once per (request, token, head): inside the main kernel every CTA
// that meets a request would repeat it (measured: 10 us per request and CTA, 20 of 183 us at 128 x 8k).
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
// launch.  K moves column by column, four of 128 dims (128-byte swizzle) and one of 64 per tile, through
// two rings of slots filled by TMA (one box per page run) and released by tcgen05.commit, so loads, MMAs
// and the exponentials of the tile before overlap.  A column's hand-over costs the producer about 330
// cycles whatever its width (traced), and a tile takes 3200 at HBM rate: five columns fit, nine of 64
// dims did not.  q is replaced column by column as the last MMAs of an item release it.  Two groups of
// epilogue warps take the even and the odd tiles of a request (one takes 3000 cycles a tile).
//
// Measured (floor): 128 requests of 8k keys, 128 heads, 149 us a call in short runs and 166 to 183 in long
// ones (97), 16 heads 113 (94), 2 tokens 297 in short runs (185); 64 requests of 1 to 32k, 2 tokens, 79 and 88 to
// 94 (44); 2 short requests 7; a prompt of 2048 with nothing cached, 16 CTAs of work, 6.3 ms (0.18).
// What bounds one token of many requests is the part's 1000 W: HBM at this rate and the 8-bit MMAs beside it bring
// the SM clock down to 1.1 GHz (the main kernel takes 127 us at full clock), so a form on CTA pairs, with half of
// the K reads from shared memory, took the same time and was not kept.  With two tokens it is the keys' second
// pass as well: in short runs, where the cap does not act, the 8-bit pipe is at 0.55 of its rate.
//
// Warps: 0 K producer, 1 MMA issuer and TMEM owner, 2 q producer, 4-7 and 8-11 epilogue (each the lane
// quadrants 0-3, for tiles of one parity).
#pragma once
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

struct AccumulateParams {
  CUtensorMap tmap_k;              // dims 0..511 of blocks as {128 bytes, rows, 4 columns}, box = box_rows rows of one
  CUtensorMap tmap_r;              // dims 512..575 as {64 bytes, rows, 1}
  const uint16_t* q;               // bf16 bits [B, T, H, 576]
  const float* lse;                // [B, T, H], natural log
  uint8_t* split;                  // workspace: per item, q's columns as the MMA reads them, then head factors
  const float* scales;             // [NSB, KVD, NL, P, 1, 1]
  const uint32_t* cache_lengths;   // [B]
  const uint32_t* lut;             // [B, max_pages]
  const uint32_t* slut;            // [B, max_pages] or null
  const float* scores;             // row stride scores_stride; may be null (all zero)
  float* out;                      // row stride out_stride; may be scores itself
  long long scores_stride, out_stride;
  unsigned int* status;
  unsigned long long wait_limit_ns;
  uint32_t item_bytes;             // of `split`
  int B, T, H, G, P, KVD, NL, layer, NB, NSB, max_pages, box_rows;
  int i0, ni;                      // the query tokens of this launch
  unsigned int max_cache_length;
  FastDiv divP, divG;
  float softmax_scale;
};

constexpr int ACC_BN = 128;                       // keys per tile (MMA M)
constexpr int ACC_HEADS = 128;                    // heads per item (MMA N = 2 x heads)
constexpr int ACC_COLS = 5;                       // columns of a key: 4 of 128 dims, 1 of 64
constexpr int ACC_THREADS = 384;
constexpr int ACC_Q_WARP = 2;
constexpr int ACC_EPI_WARP0 = 4;
constexpr int ACC_MAX_WIDE = 12, ACC_MAX_NARROW = 4;   // slots of the two rings
constexpr uint32_t ACC_WIDE_BYTES = ACC_BN * 128, ACC_NARROW_BYTES = ACC_BN * 64;
// Shared memory: head factors, barriers, scalars; then q, each column [2 x heads rows (hi, then lo)], and
// the rings in what is left (4 and 2 slots at 128 heads, up to 12 and 4 for few heads).
constexpr uint32_t ACC_SH = 0;                    // [2][64] {2^-k, 2^-k, -lse, -lse} of two heads
constexpr uint32_t ACC_SBAR = ACC_SH + 2 * ACC_HEADS * 8;
constexpr uint32_t ACC_SMISC = ACC_SBAR + 512;
constexpr uint32_t ACC_SQ = 3 * 1024;
constexpr uint32_t ACC_SMEM_ALLOC = 232448;
static_assert(ACC_SMISC + 256 <= ACC_SQ && ACC_SQ % 1024 == 0, "scalars overlap q");
__host__ __device__ constexpr uint32_t acc_wide_slots(uint32_t hpad) {
  uint32_t n = ACC_MAX_WIDE;
  while (n * ACC_WIDE_BYTES + (n / 4 + 1) * ACC_NARROW_BYTES > ACC_SMEM_ALLOC - ACC_SQ - hpad * 2 * HEAD_DIM) --n;
  return n;
}
static_assert(acc_wide_slots(ACC_HEADS) == 4 && ACC_MAX_WIDE / 4 + 1 == ACC_MAX_NARROW, "rings of K slots");

enum AccBar : uint32_t {
  // slot x of the wide ring, then slot x - ACC_MAX_WIDE of the narrow one:
  AB_K_FULL = 0,                    // producer's expect_tx arrival + the column's bytes
  AB_K_EMPTY = ACC_MAX_WIDE + ACC_MAX_NARROW,   // commit: the column's MMAs have read it
  AB_ACC_FULL = 2 * AB_K_EMPTY,     // [2] commit: a tile's products are in tensor memory (by tile parity)
  AB_ACC_EMPTY = AB_ACC_FULL + 2,   // [2] 128 epilogue threads have read them
  AB_Q_FULL = AB_ACC_EMPTY + 2,     // [5] a column of an item's q is in (bytes)
  AB_Q_EMPTY = AB_Q_FULL + ACC_COLS,   // [5] commit: the item's last MMAs on the column are done
  AB_H_FULL = AB_Q_EMPTY + ACC_COLS,   // [2] an item's head factors are in (bytes)
  AB_H_EMPTY = AB_H_FULL + 2,       // [2] 256 epilogue threads have read them
  AB_DRAIN = AB_H_EMPTY + 2,        // commit at exit
  ACC_BARS
};
static_assert(8 * ACC_BARS <= 512, "barrier block overlaps what follows");

// D[tmem] (+)= A B^T with e4m3 operands in shared memory (one CTA).
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bounded wait on an mbarrier phase in try_wait, which suspends the thread: threads that poll with
// test_wait keep the barrier unit busy (14 cycles a poll, several times that where the lanes of a warp
// poll different barriers) and made every other role's waits four times as long (210 instead of 50
// cycles on a phase that was complete).  The clock and the abort flag are looked at every 64 tries.
__device__ __forceinline__ bool try_bar(uint32_t addr, uint32_t parity, volatile uint32_t* abort, unsigned int* status,
                                        uint64_t limit) {
  if (ptx::mbar_try_wait(addr, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (ptx::mbar_try_wait(addr, parity)) return true;
    if (n & 63u) continue;
    if (*abort) return false;
    const uint64_t t = ptx::globaltimer();
    if (t0 == 0) t0 = t;
    if (t - t0 > limit) return wait_gave_up(abort, status, 0);
  }
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

// What a request costs a CTA beside its tiles (bringing q in), in tiles: the ranges are cut by this cost, the
// first ACC_ITEM_COST units of a request holding no tile (64 ragged requests of 2 tokens: 85 us with 0, 79 with
// 1, 82 with 2).
constexpr int ACC_ITEM_COST = 1;

// Walks a CTA's (request, query token x head group, tile) triples, tiles innermost.
struct AccWalker {
  int b, item, j, ta, tb;          // request, i * G + g, tile, the CTA's tile range of the request
  long long left;                  // units of the CTA's range in later requests (after this one)
  __device__ __forceinline__ AccWalker(int b0, int t0, long long tiles) : b(b0 - 1), item(0), j(t0), ta(0), tb(0), left(tiles) {}
  __device__ __forceinline__ bool start(const AccumulateParams& p, int t0) {
    if (left <= 0) return false;
    ++b;
    return open(p, t0);
  }
  // Opens request b, or the next one of which the range holds a tile; t0: first unit in request b.
  __device__ __forceinline__ bool open(const AccumulateParams& p, int t0) {
    for (;; ++b, t0 = 0) {
      if (b >= p.B) return false;
      const int end = static_cast<int>(min(static_cast<long long>(acc_tiles(p, b) + ACC_ITEM_COST), t0 + left));
      ta = max(t0 - ACC_ITEM_COST, 0);
      tb = max(end - ACC_ITEM_COST, 0);
      left -= end - t0;
      if (ta < tb) break;
      if (left <= 0) return false;
    }
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
    if (++item < p.ni * p.G) return true;
    if (left <= 0) return false;
    ++b;
    return open(p, 0);
  }
};

// The key a thread owns in tile j of request b: its place, its scale and its running sum.
struct AccKey {
  float2 scale;                    // softmax_scale times the key's scale, and what that rounding left
  float base;
  float* dst;                      // null: past the request's end, or in a page that does not exist
};
__device__ __forceinline__ AccKey acc_key(const AccumulateParams& p, int b, int item, int j, int r) {
  AccKey k;
  k.scale = make_float2(0.f, 0.f);
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
  const float s = p.scales[((static_cast<size_t>(sblk) * p.KVD) * p.NL + p.layer) * p.P + slot];
  k.scale.x = s * p.softmax_scale;
  k.scale.y = fmaf(s, p.softmax_scale, -k.scale.x);
  k.dst = p.out + b * p.out_stride + t;
  if (item == 0 && p.i0 == 0 && p.scores && t < L) k.base = p.scores[b * p.scores_stride + t];
  return k;
}

// Sum over W heads, two at a time: the thread's hi and lo columns, its scale, and each pair's powers of two and
// -lse.  A rounding of the score, relative to its size, would be a relative error of the weight several times
// as large, the same for all heads or all keys where it is a factor's: so the factor has two terms, the score
// meets the lse before it is rounded, and log2 e multiplies what is left.
template <int W>
__device__ __forceinline__ void acc_heads(const uint32_t (&hi)[W], const uint32_t (&lo)[W], float2 s, uint32_t hf,
                                          float2 (&sum)[2]) {
  const float2 s0 = make_float2(s.x, s.x), s1 = make_float2(s.y, s.y);
#pragma unroll
  for (int x = 0; x < W; x += 2) {
    const uint4 f = ptx::ld_shared_v4(hf + x * 8);       // 2^-k of two heads, then their -lse
    const float2 k = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
    const float2 v = __ffma2_rn(make_float2(__uint_as_float(lo[x]), __uint_as_float(lo[x + 1])), make_float2(0.0625f, 0.0625f),
                                make_float2(__uint_as_float(hi[x]), __uint_as_float(hi[x + 1])));
    float2 e = __ffma2_rn(v, __fmul2_rn(k, s0), make_float2(__uint_as_float(f.z), __uint_as_float(f.w)));
    e = __ffma2_rn(v, __fmul2_rn(k, s1), e);
    e = __fmul2_rn(e, make_float2(1.4426950408889634f, 1.4426950408889634f));
    sum[(x >> 1) & 1] = __fadd2_rn(sum[(x >> 1) & 1], make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y)));
  }
}

// ------------------------------------------------------------------ q split
// Workspace of an item ((b * ni + i) * G + g): 4 columns of 2 hpad rows (hi of each head, then lo) of
// 128 bytes in the 128-byte swizzle, one of 64 bytes in the 64-byte swizzle, then for every two heads the
// powers of two that undo their scaling and their -lse; hpad heads, a multiple of 8.
__device__ __forceinline__ uint32_t acc_hpad(const AccumulateParams& p, int g) {
  return (min(p.H - g * ACC_HEADS, ACC_HEADS) + 7) & ~7;
}

// One warp per head row.
__global__ void __launch_bounds__(256) mla_split_q_kernel(const __grid_constant__ AccumulateParams p) {
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t per_item = (min(p.H, ACC_HEADS) + 7) & ~7;   // rows of an item's workspace
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const long long item = w / per_item;
  const uint32_t r = static_cast<uint32_t>(w - item * per_item);
  if (item >= static_cast<long long>(p.B) * p.ni * p.G) return;
  const long long bi = item / p.G;
  const int g = static_cast<int>(item - bi * p.G);
  const uint32_t hpad = acc_hpad(p, g);
  if (r >= hpad) return;
  const int b = static_cast<int>(bi / p.ni), i = p.i0 + static_cast<int>(bi - static_cast<long long>(b) * p.ni);
  const int h = g * ACC_HEADS + r;
  const bool have = h < p.H;
  const size_t row = (static_cast<size_t>(b) * p.T + i) * p.H + h;
  const uint4* src = reinterpret_cast<const uint4*>(p.q + row * HEAD_DIM);
  const float lse = have ? p.lse[row] : -INFINITY;
  uint4 v[3];
#pragma unroll
  for (int c = 0; c < 3; ++c)
    v[c] = have && lane + 32 * c < HEAD_DIM / 8 ? src[lane + 32 * c] : make_uint4(0, 0, 0, 0);
  uint32_t m2 = 0;
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    if (lse == -INFINITY) v[c] = make_uint4(0, 0, 0, 0);   // adds nothing, whatever it holds (a padded token)
    m2 = __vmaxu2(__vmaxu2(m2, v[c].x & 0x7FFF7FFFu), v[c].y & 0x7FFF7FFFu);
    m2 = __vmaxu2(__vmaxu2(m2, v[c].z & 0x7FFF7FFFu), v[c].w & 0x7FFF7FFFu);
  }
  const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  // 2^k with k = 7 - e, e the exponent of the row's largest element (tiny rows: at most 2^126, whose
  // reciprocal is normal)
  const int k = m == 0 ? 0 : min(max(7 - (static_cast<int>(m >> 7) - 127), -120), 126);
  const float f = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  uint8_t* dst = p.split + item * p.item_bytes;
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    const uint32_t ch = lane + 32 * c;                   // dims 8 ch .. 8 ch + 7
    if (ch >= HEAD_DIM / 8) break;
    const uint32_t in[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      // f16 holds the scaled values exactly down to 2^-17 (their 8 bits), far below what lo resolves
      const uint32_t y = ptx::pack_f16x2(__uint_as_float(in[x] << 16) * f, __uint_as_float(in[x] & 0xFFFF0000u) * f);
      hi[x] = ptx::e4m3x2_rn_satfinite_f16x2(y);
      const uint32_t rest = ptx::sub_f16x2(y, ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(hi[x])));
      lo[x] = ptx::e4m3x2_rn_satfinite_f16x2(mul_f16x2(rest, 0x4C004C00u));   // x 16
    }
    // hpad is a multiple of 8, so the lo row hpad + r has the same swizzle phase as row r
    const bool wide = ch < 64;
    const uint32_t unit = (ch >> 1) & 7, width = wide ? 128 : 64;
    uint8_t* at = dst + (ch >> 4) * hpad * 256 + r * width + ((unit ^ (wide ? r & 7 : (r >> 1) & 3)) << 4) + (ch & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
    *reinterpret_cast<uint2*>(at + hpad * width) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  }
  if (lane == 0) {
    // no such head, or a row without keys: weight 0.  A non-finite row gets a NaN factor (its codes
    // would saturate) and makes the request's sums NaN.
    float* hf = reinterpret_cast<float*>(dst + hpad * 2 * HEAD_DIM) + (r >> 1) * 4 + (r & 1);
    hf[0] = lse == -INFINITY ? 0.f : m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    hf[2] = lse == -INFINITY ? -INFINITY : -lse;
  }
}

__global__ void __launch_bounds__(ACC_THREADS, 1) mla_accumulate_kernel(const __grid_constant__ AccumulateParams p) {
  extern __shared__ uint8_t acc_smem_raw[];
  const uint32_t base = ptx::smem_u32(acc_smem_raw);
  uint8_t* smem = acc_smem_raw;
  const uint32_t col = acc_hpad(p, 0) * 256;             // a q column's place is the same for every head group
  const uint32_t wides = acc_wide_slots(acc_hpad(p, 0)), narrows = wides / 4 + 1;
  const uint32_t ring = ACC_SQ + acc_hpad(p, 0) * 2 * HEAD_DIM, ring_n = ring + wides * ACC_WIDE_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + ACC_SMISC + 4);
  int* range = reinterpret_cast<int*>(smem + ACC_SMISC + 16);     // first request, its first tile
  long long* tot = reinterpret_cast<long long*>(smem + ACC_SMISC + 64);   // scan scratch
  auto bar = [&](uint32_t i) { return base + ACC_SBAR + 8 * i; };
  if (base & 1023u) {                                    // the swizzled columns start at multiples of 1 KB
    if (threadIdx.x == 0) raise_status(p.status, STATUS_LAYOUT);
    return;
  }
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < ACC_BARS; ++i) {
      const bool acc = i >= AB_ACC_EMPTY && i < AB_ACC_EMPTY + 2, heads = i >= AB_H_EMPTY && i < AB_H_EMPTY + 2;
      ptx::mbar_init(bar(i), acc ? 128 : heads ? 256 : 1);
    }
    *abort = 0u;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap_k);
    ptx::prefetch_tmap(&p.tmap_r);
  }
  if (warp == 1) {
    ptx::tmem_alloc(base + ACC_SMISC, 512);
    ptx::tmem_relinquish();
  }
  // This CTA's range [r0, r1) of the requests' tiles laid end to end, and the request r0 falls in.
  long long mine = 0;
  for (int b = threadIdx.x; b < p.B; b += ACC_THREADS) mine += acc_tiles(p, b) + ACC_ITEM_COST;
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
    const long long n = b < p.B ? acc_tiles(p, b) + ACC_ITEM_COST : 0;
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
  // Every thread waits for itself: a wait that gives up marks the CTA, and the other roles' waits end.
  auto wait = [&](uint32_t b, uint32_t parity) { return try_bar(b, parity, abort, p.status, lim); };

  if (warp == 0) {
    // ------------------------------------------------------------------ K producer: lane r, page run r
    uint32_t wide = 0, wide_use = 0, narrow = 0, narrow_use = 0;   // the rings' next slots
    const uint32_t runs = ACC_BN / p.box_rows;
    auto find = [&](int b, int j, int& row) {            // where this lane's run of tile j lies
      const uint32_t t = static_cast<uint32_t>(j) * ACC_BN + lane * p.box_rows;
      if (static_cast<uint32_t>(lane) >= runs || t >= acc_length(p, b) + p.T) return false;
      const uint32_t page = p.divP.div(t);
      const uint32_t blk = p.lut[static_cast<size_t>(b) * p.max_pages + page];
      row = static_cast<int>((static_cast<uint64_t>(blk) * p.KVD * p.NL + p.layer) * p.P + (t - page * p.P));
      return blk < static_cast<uint32_t>(p.NB);          // else the epilogue flags it and leaves its keys
    };
    bool live = w.start(p, t0);
    int row = 0;
    bool have = live && find(w.b, w.j, row);
    while (live) {
      const bool more = w.next(p);
      int next_row = 0;
      const bool next_have = more && find(w.b, w.j, next_row);   // looked up while this tile is issued
      const uint32_t rows = __popc(__ballot_sync(0xffffffffu, have)) * p.box_rows;
      for (int c = 0; c < ACC_COLS; ++c) {
        const bool is_wide = c < ACC_COLS - 1;
        const uint32_t x = is_wide ? wide : ACC_MAX_WIDE + narrow;
        const uint32_t full = bar(AB_K_FULL + x);
        if (!__all_sync(0xffffffffu, wait(bar(AB_K_EMPTY + x), ((is_wide ? wide_use : narrow_use) & 1) ^ 1))) {
          live = false;
          break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(full, rows * (is_wide ? 128u : 64u));
        __syncwarp();
        if (is_wide) {
          if (have)
            ptx::tma_load_3d(base + ring + wide * ACC_WIDE_BYTES + lane * p.box_rows * 128u, &p.tmap_k, 0, row, c, full);
          if (++wide == wides) {
            wide = 0;
            ++wide_use;
          }
        } else {
          if (have)
            ptx::tma_load_3d(base + ring_n + narrow * ACC_NARROW_BYTES + lane * p.box_rows * 64u, &p.tmap_r, 0, row, 0, full);
          if (++narrow == narrows) {
            narrow = 0;
            ++narrow_use;
          }
        }
      }
      live = live && more;
      row = next_row;
      have = next_have;
    }
    // no copy may land after the CTA is gone (also on an aborted call)
    for (uint32_t x = 0; x < wides; ++x) {
      const uint32_t uses = wide_use + (x < wide);       // times slot x was filled
      if (uses) drain_bar(bar(AB_K_FULL + x), (uses - 1) & 1, lim);
    }
    for (uint32_t x = 0; x < narrows; ++x) {
      const uint32_t uses = narrow_use + (x < narrow);
      if (uses) drain_bar(bar(AB_K_FULL + ACC_MAX_WIDE + x), (uses - 1) & 1, lim);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (one thread)
    if (ptx::elect_one()) {
      uint32_t wide = 0, wide_use = 0, narrow = 0, narrow_use = 0, items = 0;
      uint32_t acc_use0 = 0, acc_use1 = 0;
      bool live = w.start(p, t0);
      while (live) {
        const int g = w.item - static_cast<int>(p.divG.div(w.item)) * p.G;
        const uint32_t hpad = acc_hpad(p, g);
        const uint32_t idesc = ptx::idesc_e4m3_f32(ACC_BN, 2 * hpad, false, false);
        const uint64_t aw = ptx::smem_desc(base + ring, 16, 1024, ptx::SW_128B);
        const uint64_t an = ptx::smem_desc(base + ring_n, 16, 512, ptx::SW_64B);
        uint64_t b = ptx::smem_desc(base + ACC_SQ, 16, 1024, ptx::SW_128B);
        const uint64_t bn = ptx::smem_desc(base + ACC_SQ + 4 * col, 16, 512, ptx::SW_64B);
        const bool first = w.first_of_item(), last = w.last_of_item();
        const uint32_t buf = w.j & 1, d = tbase + buf * 256;
        if (!wait(bar(AB_ACC_EMPTY + buf), ((buf ? acc_use1 : acc_use0) & 1) ^ 1)) break;
        ptx::tc_fence_after();
#pragma unroll
        for (int c = 0; c < ACC_COLS; ++c) {
          const bool is_wide = c < ACC_COLS - 1;
          const uint32_t x = is_wide ? wide : ACC_MAX_WIDE + narrow;
          if (first && !wait(bar(AB_Q_FULL + c), items & 1)) { live = false; break; }
          if (!wait(bar(AB_K_FULL + x), (is_wide ? wide_use : narrow_use) & 1)) { live = false; break; }
          ptx::tc_fence_after();
          if (is_wide) {
            const uint64_t a = aw + wide * (ACC_WIDE_BYTES >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_ss_e4m3(d, a + 2 * k, b + 2 * k, idesc, c + k > 0);   // 32 dims each
            b += col >> 4;
            if (++wide == wides) {
              wide = 0;
              ++wide_use;
            }
          } else {
            const uint64_t a = an + narrow * (ACC_NARROW_BYTES >> 4);
            mma_ss_e4m3(d, a, bn, idesc, 1);
            mma_ss_e4m3(d, a + 2, bn + 2, idesc, 1);
            if (++narrow == narrows) {
              narrow = 0;
              ++narrow_use;
            }
          }
          ptx::mma_commit(bar(AB_K_EMPTY + x));
          if (last) ptx::mma_commit(bar(AB_Q_EMPTY + c));
        }
        if (!live) break;
        ptx::mma_commit(bar(AB_ACC_FULL + buf));
        acc_use0 += !buf;
        acc_use1 += buf;
        items += last;
        live = w.next(p);
      }
      ptx::mma_commit(bar(AB_DRAIN));
      drain_bar(bar(AB_DRAIN), 0, lim);
    }
    __syncwarp();
  } else if (warp == ACC_Q_WARP) {
    // ------------------------------------------------------------------ q producer (one thread)
    if (ptx::elect_one()) {
      ptx::griddep_wait();                               // the split kernel has written the workspace
      uint32_t items = 0, cols = 0;
      bool live = w.start(p, t0);
      while (live) {
        const int i = static_cast<int>(p.divG.div(w.item)), g = w.item - i * p.G;
        const uint32_t hpad = acc_hpad(p, g);
        const uint8_t* src = p.split + ((static_cast<long long>(w.b) * p.ni + i) * p.G + g) * p.item_bytes;
        if (!wait(bar(AB_H_EMPTY + (items & 1)), ((items >> 1) & 1) ^ 1)) break;
        ptx::mbar_arrive_expect_tx(bar(AB_H_FULL + (items & 1)), hpad * 8);
        ptx::bulk_load(base + ACC_SH + (items & 1) * ACC_HEADS * 8, src + hpad * 2 * HEAD_DIM, hpad * 8,
                       bar(AB_H_FULL + (items & 1)));
        cols = 0;
        ++items;
        for (; cols < ACC_COLS; ++cols) {
          if (!wait(bar(AB_Q_EMPTY + cols), (items & 1))) { live = false; break; }
          const uint32_t bytes = cols < ACC_COLS - 1 ? hpad * 256 : hpad * 128;
          ptx::mbar_arrive_expect_tx(bar(AB_Q_FULL + cols), bytes);
          ptx::bulk_load(base + ACC_SQ + cols * col, src + cols * hpad * 256, bytes, bar(AB_Q_FULL + cols));
        }
        live = live && w.next_item(p);
      }
      // the copies of the last item (and, of columns not reached, of the one before) have landed
      for (uint32_t c = 0; c < ACC_COLS; ++c) {
        const uint32_t done = items - (c < cols ? 0 : 1);   // times column c was loaded
        if (items > 0 && done > 0) drain_bar(bar(AB_Q_FULL + c), (done - 1) & 1, lim);
      }
      for (uint32_t x = 0; x < 2 && x < items; ++x) drain_bar(bar(AB_H_FULL + ((items - 1 - x) & 1)), ((items - 1 - x) >> 1) & 1, lim);
    }
    __syncwarp();
  } else if (warp >= ACC_EPI_WARP0) {
    // ------------------------------------------------------------------ epilogue
    const int r = threadIdx.x & 127;                     // the tile's key = tensor-memory lane
    const uint32_t buf = (warp - ACC_EPI_WARP0) >> 2;    // this group's tiles: those of this parity
    const uint32_t d = tbase + (static_cast<uint32_t>(warp & 3) << 21) + buf * 256;
    uint32_t use = 0, items = 0;
    bool live = w.start(p, t0);
    AccKey key{}, nxt{};
    if (live && (w.j & 1) == static_cast<int>(buf)) key = acc_key(p, w.b, w.item, w.j, r);
    while (live) {
      const AccWalker cur = w;
      const bool own = (cur.j & 1) == static_cast<int>(buf);
      if (cur.item == 0 && cur.j == 0 && buf == 0 && r == 0 && p.cache_lengths[cur.b] > p.max_cache_length)
        raise_status(p.status, STATUS_BOUNDS);
      if (cur.first_of_item() && !__all_sync(0xffffffffu, wait(bar(AB_H_FULL + (items & 1)), (items >> 1) & 1))) break;
      live = w.next(p);
      const bool next_own = live && (w.j & 1) == static_cast<int>(buf);
      const int i = static_cast<int>(p.divG.div(cur.item)), g = cur.item - i * p.G;
      const uint32_t hpad = acc_hpad(p, g), hf = base + ACC_SH + (items & 1) * ACC_HEADS * 8;
      // the scale and running sum of this group's next tile are on their way while others are summed
      if (next_own) nxt = acc_key(p, w.b, w.item, w.j, r);
      if (own) {
        if (!__all_sync(0xffffffffu, wait(bar(AB_ACC_FULL + buf), use & 1))) break;
        ++use;
        ptx::tc_fence_after();
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t h = 0;
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
        ptx::mbar_arrive(bar(AB_ACC_EMPTY + buf));
        if (key.dst) {
          const uint32_t t = static_cast<uint32_t>(cur.j) * ACC_BN + r;
          const float add = t <= acc_length(p, cur.b) + p.i0 + i ? (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y) : 0.f;
          *key.dst = (cur.item == 0 && p.i0 == 0 ? key.base : *key.dst) + add;
        }
      }
      if (cur.last_of_item()) {
        ptx::mbar_arrive(bar(AB_H_EMPTY + (items & 1)));
        ++items;
      }
      if (next_own) key = nxt;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tbase, 512);
}

}  // namespace mla
