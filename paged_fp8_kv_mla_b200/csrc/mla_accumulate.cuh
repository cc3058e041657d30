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
// launch.  K moves through a ring of ten 8 KB slots, one 64-dim column of a tile each, filled by TMA
// (one box per page run) and released by tcgen05.commit, so loads, MMAs and the exponentials of the
// tile before overlap.  q is replaced column by column as the last MMAs of an item release it.
//
// Warps: 0 K producer, 1 MMA issuer and TMEM owner, 2 q producer, 4-7 epilogue (lane quadrants 0-3).
#pragma once
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

struct AccumulateParams {
  CUtensorMap tmap_k;              // blocks as {64 bytes, rows, 9 columns}, box = box_rows rows of a column
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
constexpr int ACC_COLS = HEAD_DIM / 64;           // 9 columns of 64 dims
constexpr int ACC_THREADS = 256;
constexpr int ACC_Q_WARP = 2;
constexpr int ACC_EPI_WARP0 = 4;
constexpr int ACC_SLOTS = 10;
constexpr uint32_t ACC_SLOT_BYTES = ACC_BN * 64;
constexpr uint32_t ACC_SQ = 0;                    // [9 columns][2 x heads rows (hi, then lo)][64 B]
constexpr uint32_t ACC_SK = ACC_COLS * 2 * ACC_HEADS * 64;
constexpr uint32_t ACC_SH = ACC_SK + ACC_SLOTS * ACC_SLOT_BYTES;   // [2][128] {factor, -lse log2 e}
constexpr uint32_t ACC_SBAR = ACC_SH + 2 * ACC_HEADS * 8;
constexpr uint32_t ACC_SMISC = ACC_SBAR + 512;
constexpr uint32_t ACC_SMEM = ACC_SMISC + 256;
constexpr uint32_t ACC_SMEM_ALLOC = 232448;
static_assert(ACC_SMEM + 255 <= ACC_SMEM_ALLOC, "shared memory map exceeds 227 KB");

enum AccBar : uint32_t {
  AB_K_FULL = 0,                    // [10] producer's expect_tx arrival + the column's bytes
  AB_K_EMPTY = ACC_SLOTS,           // [10] commit: the column's MMAs have read it
  AB_ACC_FULL = 2 * ACC_SLOTS,      // [2] commit: a tile's products are in tensor memory
  AB_ACC_EMPTY = AB_ACC_FULL + 2,   // [2] 128 epilogue threads have read them
  AB_Q_FULL = AB_ACC_EMPTY + 2,     // [9] a column of an item's q is in (bytes)
  AB_Q_EMPTY = AB_Q_FULL + ACC_COLS,   // [9] commit: the item's last MMAs on the column are done
  AB_H_FULL = AB_Q_EMPTY + ACC_COLS,   // [2] an item's head factors are in (bytes)
  AB_H_EMPTY = AB_H_FULL + 2,       // [2] 128 epilogue threads have read them
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

// Bounded wait on an mbarrier phase that polls without sleeping: for roles whose every wait sits on the
// path of a tile (a thread suspended in try_wait resumes hundreds of cycles late).  Looks at the clock
// and at the abort flag every 256 polls only.
__device__ __forceinline__ bool spin_bar(uint32_t addr, uint32_t parity, volatile uint32_t* abort, unsigned int* status,
                                         uint64_t limit) {
  if (ptx::mbar_test_wait(addr, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t n = 1;; ++n) {
    if (ptx::mbar_test_wait(addr, parity)) return true;
    if ((n & 255u) == 0) {
      if (*abort) return false;
      if (ptx::globaltimer() - t0 > limit) return wait_gave_up(abort, status, 0);
    }
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
    if (++item < p.ni * p.G) return true;
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
  if (item == 0 && p.i0 == 0 && p.scores && t < L) k.base = p.scores[b * p.scores_stride + t];
  return k;
}

// Sum over W heads: the thread's hi and lo columns, its scale, and each head's factor and -lse.
template <int W>
__device__ __forceinline__ void acc_heads(const uint32_t (&hi)[W], const uint32_t (&lo)[W], float s, uint32_t hf,
                                          float (&sum)[4]) {
#pragma unroll
  for (int x = 0; x < W; x += 2) {
    const uint4 f = ptx::ld_shared_v4(hf + x * 8);       // {factor, -lse} of two heads
    const float x0 = fmaf(__uint_as_float(lo[x]), 0.0625f, __uint_as_float(hi[x])) * s;
    const float x1 = fmaf(__uint_as_float(lo[x + 1]), 0.0625f, __uint_as_float(hi[x + 1])) * s;
    sum[x & 2] += ptx::ex2_approx(fmaf(x0, __uint_as_float(f.x), __uint_as_float(f.y)));
    sum[(x & 2) + 1] += ptx::ex2_approx(fmaf(x1, __uint_as_float(f.z), __uint_as_float(f.w)));
  }
}

// ------------------------------------------------------------------ q split
// Workspace of an item ((b * ni + i) * G + g): 9 columns of 2 hpad rows (hi of each head, then lo) of
// 64 bytes in the 64-byte swizzle, then {factor, -lse log2 e} of each head; hpad heads, a multiple of 8.
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
  uint32_t m2 = 0;
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    v[c] = have && lane + 32 * c < HEAD_DIM / 8 ? src[lane + 32 * c] : make_uint4(0, 0, 0, 0);
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
    uint8_t* at = dst + (ch >> 3) * hpad * 128 + r * 64 + ((((ch & 7) >> 1) ^ ((r >> 1) & 3)) << 4) + (ch & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
    *reinterpret_cast<uint2*>(at + hpad * 64) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  }
  if (lane == 0) {
    // no such head, or a row without keys: weight 0.  A non-finite row gets a NaN factor (its codes
    // would saturate) and makes the request's sums NaN.
    float2 hf = make_float2(0.f, -INFINITY);
    if (lse != -INFINITY) {
      hf.x = m >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                          : p.softmax_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      hf.y = -lse * 1.4426950408889634f;
    }
    reinterpret_cast<float2*>(dst + ACC_COLS * hpad * 128)[r] = hf;
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
  long long* tot = reinterpret_cast<long long*>(smem + ACC_SMISC + 64);   // scan scratch
  auto bar = [&](uint32_t i) { return base + ACC_SBAR + 8 * i; };
  if (base - raw > ACC_SMEM_ALLOC - ACC_SMEM) {          // the map needs a base within 255 bytes of 1 KB
    if (threadIdx.x == 0) raise_status(p.status, STATUS_LAYOUT);
    return;
  }
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < ACC_BARS; ++i) {
      const bool many = (i >= AB_ACC_EMPTY && i < AB_ACC_EMPTY + 2) || (i >= AB_H_EMPTY && i < AB_H_EMPTY + 2);
      ptx::mbar_init(bar(i), many ? 128 : 1);
    }
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
  // Every thread waits for itself: a wait that gives up marks the CTA, and the other roles' waits end.
  auto wait = [&](uint32_t b, uint32_t parity) { return spin_bar(b, parity, abort, p.status, lim); };

  if (warp == 0) {
    // ------------------------------------------------------------------ K producer: lane r, page run r
    uint32_t n = 0;                                      // columns issued
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
      const bool next_have = more && find(w.b, w.j, next_row);   // in flight while this tile is issued
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, have)) * p.box_rows * 64u;
      for (int c = 0; c < ACC_COLS && live; ++c, ++n) {
        const uint32_t s = n % ACC_SLOTS, use = n / ACC_SLOTS;
        const bool ok = wait(bar(AB_K_EMPTY + s), (use & 1) ^ 1);
        if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
        if (lane == 0) ptx::mbar_arrive_expect_tx(bar(AB_K_FULL + s), bytes);
        __syncwarp();
        if (have)
          ptx::tma_load_3d(base + ACC_SK + s * ACC_SLOT_BYTES + lane * p.box_rows * 64u, &p.tmap_k, 0, row, c,
                           bar(AB_K_FULL + s));
      }
      live = live && more;
      row = next_row;
      have = next_have;
    }
    // no copy may land after the CTA is gone (also on an aborted call)
    for (uint32_t s = 0; s < ACC_SLOTS && s < n; ++s)
      drain_bar(bar(AB_K_FULL + s), ((n - 1 - s) / ACC_SLOTS) & 1, lim);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (one thread)
    if (ptx::elect_one()) {
      const uint32_t col = acc_hpad(p, 0) * 128;         // a column's place is the same for every head group
      uint32_t s = 0, use = 0, tile = 0, items = 0;
      bool live = w.start(p, t0);
      while (live) {
        const int g = w.item - static_cast<int>(p.divG.div(w.item)) * p.G;
        const uint32_t hpad = acc_hpad(p, g);
        const uint32_t idesc = ptx::idesc_e4m3_f32(ACC_BN, 2 * hpad, false, false);
        const uint64_t a0 = ptx::smem_desc(base + ACC_SK, 16, 512, ptx::SW_64B);
        uint64_t b = ptx::smem_desc(base + ACC_SQ, 16, 512, ptx::SW_64B);
        const bool first = w.first_of_item(), last = w.last_of_item();
        const uint32_t d = tbase + (tile & 1) * 256;
        if (!wait(bar(AB_ACC_EMPTY + (tile & 1)), ((tile >> 1) & 1) ^ 1)) break;
        ptx::tc_fence_after();
        for (int c = 0; c < ACC_COLS; ++c) {
          if (first && !wait(bar(AB_Q_FULL + c), items & 1)) { live = false; break; }
          if (!wait(bar(AB_K_FULL + s), use & 1)) { live = false; break; }
          ptx::tc_fence_after();
          const uint64_t a = a0 + s * (ACC_SLOT_BYTES >> 4);
          mma_ss_e4m3(d, a, b, idesc, c > 0);
          mma_ss_e4m3(d, a + 2, b + 2, idesc, 1);        // the column's second 32 dims: + 32 bytes
          ptx::mma_commit(bar(AB_K_EMPTY + s));
          if (last) ptx::mma_commit(bar(AB_Q_EMPTY + c));
          b += col >> 4;
          if (++s == ACC_SLOTS) { s = 0; ++use; }
        }
        if (!live) break;
        ptx::mma_commit(bar(AB_ACC_FULL + (tile & 1)));
        items += last;
        ++tile;
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
      const uint32_t col = acc_hpad(p, 0) * 128;
      uint32_t items = 0, cols = 0;
      bool live = w.start(p, t0);
      while (live) {
        const int i = static_cast<int>(p.divG.div(w.item)), g = w.item - i * p.G;
        const uint32_t hpad = acc_hpad(p, g);
        const uint8_t* src = p.split + ((static_cast<long long>(w.b) * p.ni + i) * p.G + g) * p.item_bytes;
        if (!wait(bar(AB_H_EMPTY + (items & 1)), ((items >> 1) & 1) ^ 1)) break;
        ptx::mbar_arrive_expect_tx(bar(AB_H_FULL + (items & 1)), hpad * 8);
        ptx::bulk_load(base + ACC_SH + (items & 1) * ACC_HEADS * 8, src + ACC_COLS * hpad * 128, hpad * 8,
                       bar(AB_H_FULL + (items & 1)));
        cols = 0;
        ++items;
        for (; cols < ACC_COLS; ++cols) {
          if (!wait(bar(AB_Q_EMPTY + cols), (items & 1))) { live = false; break; }
          ptx::mbar_arrive_expect_tx(bar(AB_Q_FULL + cols), hpad * 128);
          ptx::bulk_load(base + ACC_SQ + cols * col, src + cols * hpad * 128, hpad * 128, bar(AB_Q_FULL + cols));
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
      const uint32_t hpad = acc_hpad(p, g);
      bool ok = !cur.first_of_item() || wait(bar(AB_H_FULL + (items & 1)), (items >> 1) & 1);
      ok = ok && wait(bar(AB_ACC_FULL + (tile & 1)), (tile >> 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      ptx::tc_fence_after();
      const uint32_t d = tbase + quad + (tile & 1) * 256, hf = base + ACC_SH + (items & 1) * ACC_HEADS * 8;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
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
      ptx::mbar_arrive(bar(AB_ACC_EMPTY + (tile & 1)));
      if (cur.last_of_item()) {
        ptx::mbar_arrive(bar(AB_H_EMPTY + (items & 1)));
        ++items;
      }
      if (key.dst) {
        const uint32_t t = static_cast<uint32_t>(cur.j) * ACC_BN + r;
        const float add = t <= acc_length(p, cur.b) + p.i0 + i ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
        *key.dst = (cur.item == 0 && p.i0 == 0 ? key.base : *key.dst) + add;
      }
      key = nxt;
      ++tile;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) ptx::tmem_dealloc(tbase, 512);
}

}  // namespace mla
