// Which keys a request keeps (sm_100a).  Request b holds n_b keys with accumulated weights
// scores[b][0 .. n_b); when n_b exceeds the budget it keeps its first `num_sink` keys, its last
// `num_recent` keys and, of those between, the budget - num_sink - num_recent with the largest
// weights; ties go to the lowest index.  A request within the budget keeps everything.  The kept
// indices come out ascending.
//
// The weights between the two protected ends are mapped to unsigned keys that order like the numbers
// (-0 as +0, NaN below every number) and the smallest kept key is found by a radix selection over
// digits of 11, 11 and 10 bits: three histograms, no sort.  A second pass over the keys writes the
// indices in order, with counts from warp ballots.
//
// What bounds it.  4 bytes per key are read once; at these sizes (a few MB at most) that is under a
// microsecond of HBM time, and the time goes to the chain of passes: load, three histograms, output.
// So a request is spread over a thread-block cluster: every CTA holds its share of the keys in shared
// memory (read from HBM once), histograms are added up through distributed shared memory, and the passes
// are separated by cluster barriers instead of kernel launches.  Such an access takes some 700 cycles, so
// they are made in few rounds, all of a round in flight: in clusters of up to 4 every CTA reads all bins of
// all; in larger ones CTA r adds slice r and hands the sums to all, another barrier later.  Measured (20 or
// more calls in a graph): 4 requests of 128k keys 15.6 us, 128 of 8k 12.5 us, 32 of up to 4k 8.3 us (of which
// the launch is about 3); a digit costs 2 us of the last.  (With the bins added one by one: 17.0, 15.6, 11.1.)
#pragma once
#include <cstddef>
#include <cstdint>
#include "mla_kernels.cuh"

namespace mla {

struct SelectParams {
  const float* scores;             // row stride scores_stride
  const uint32_t* lengths;         // [B]
  int32_t* kept;                   // row stride kept_stride
  int32_t* kept_lengths;           // [B]
  unsigned int* status;
  long long scores_stride, kept_stride;
  unsigned int max_length;
  int budget, recent, sink;
};

constexpr int SEL_MAX_WARPS = 32;
constexpr int SEL_BINS = 2048;
constexpr int SEL_MAX_CLUSTER = 16;
constexpr int SEL_CACHE = 36864;   // keys a CTA holds in shared memory; keys past these are read again

// Shared memory: three histograms and the cluster-wide sums, then the keys.
struct SelectShared {
  uint32_t hist0[SEL_BINS][4];     // the first digit's counts, in four copies by lane (its few bins are
                                   // exponents, which the lanes of a warp share)
  uint32_t hist[3][SEL_BINS];
  uint32_t total[SEL_BINS];
  uint32_t cta_gt[SEL_MAX_CLUSTER], cta_eq[SEL_MAX_CLUSTER];   // kept and tied keys of each CTA of the cluster
  uint32_t warp_gt[SEL_MAX_WARPS], warp_eq[SEL_MAX_WARPS];
  uint32_t scan[SEL_MAX_WARPS];
  uint32_t bin, need;
};
constexpr uint32_t SEL_KEYS_OFF = (sizeof(SelectShared) + 15) / 16 * 16;
static_assert(SEL_KEYS_OFF + SEL_CACHE * 4 <= 232448, "shared memory map exceeds 227 KB");
static_assert(offsetof(SelectShared, hist) == sizeof(SelectShared::hist0), "the histograms are cleared as one");

__device__ __forceinline__ uint32_t select_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);           // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// c[0 .. n) += n words (4, 2 or 1) at an address of the cluster's shared memory.
template <int N>
__device__ __forceinline__ void add_cluster_words(uint32_t (&c)[N], int n, uint32_t cluster_addr) {
  uint32_t v[4] = {};
  if (N >= 4 && n == 4)
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(cluster_addr) : "memory");
  else if (N >= 2 && n == 2)
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(cluster_addr) : "memory");
  else
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v[0]) : "r"(cluster_addr) : "memory");
#pragma unroll
  for (int x = 0; x < N; ++x) c[x] += v[x];
}
__device__ __forceinline__ void st_cluster_v4(uint32_t cluster_addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};"
               :: "r"(cluster_addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// Sum of the words before `below` of a warp-sized table (n <= 32 of them used), the same for every lane.
__device__ __forceinline__ uint32_t sum_below(const uint32_t* table, int n, int below, int lane) {
  return __reduce_add_sync(0xffffffffu, lane < n && lane < below ? table[lane] : 0u);
}

template <int SEL_THREADS>
__global__ void __launch_bounds__(SEL_THREADS, 1) mla_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int SEL_WARPS = SEL_THREADS / 32;
  extern __shared__ __align__(16) uint8_t sel_smem[];
  SelectShared& s = *reinterpret_cast<SelectShared*>(sel_smem);
  uint32_t* cache = reinterpret_cast<uint32_t*>(sel_smem + SEL_KEYS_OFF);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t ncta;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ncta));
  const uint32_t rank = ptx::cluster_ctarank();
  const int b = static_cast<int>(ptx::cluster_id_x());
  const uint32_t given = p.lengths[b];                   // (on its way while the histograms are cleared)
  for (uint32_t i = tid; i < 7 * SEL_BINS / 4; i += SEL_THREADS) reinterpret_cast<uint4*>(&s.hist0[0][0])[i] = make_uint4(0, 0, 0, 0);
  const uint32_t n = min(given, p.max_length);
  const uint32_t count = min(n, static_cast<uint32_t>(p.budget));
  int32_t* out = p.kept + b * p.kept_stride;
  // kept_lengths may be lengths: it is written behind a barrier that every CTA reaches with the length read
  auto write_count = [&]() {
    if (rank == 0 && tid == 0) {
      if (given > p.max_length) raise_status(p.status, STATUS_BOUNDS);
      p.kept_lengths[b] = static_cast<int32_t>(count);
    }
  };
  // the protected ends (and, within the budget, every key)
  const bool all = n <= static_cast<uint32_t>(p.budget);
  const uint32_t head = all ? n : p.sink, tail = all ? 0 : p.recent;
  const uint32_t gtid = rank * SEL_THREADS + tid, gthreads = ncta * SEL_THREADS;
  for (uint32_t j = gtid; j < head; j += gthreads) out[j] = static_cast<int32_t>(j);
  for (uint32_t j = gtid; j < tail; j += gthreads) out[count - tail + j] = static_cast<int32_t>(n - tail + j);
  const uint32_t need0 = count - head - tail;            // keys to choose from the middle
  if (need0 == 0) {                                      // the same for every CTA of the cluster
    ptx::cluster_sync();
    write_count();
    return;
  }

  // this CTA's share [lo, hi) of the middle, and each warp's share of that (multiples of 32 keys, so
  // that indices ascend over lanes, steps, warps and CTAs)
  const uint32_t mid = n - head - tail;
  const uint32_t per = (mid + ncta - 1) / ncta;
  const uint32_t lo = min(rank * per, mid), hi = min(lo + per, mid), m = hi - lo;
  const float* src = p.scores + b * p.scores_stride + head + lo;
  __syncthreads();

  // Each pass counts the keys that agree with the digits found so far by their next digit.
  constexpr int shift[3] = {21, 10, 0};
  constexpr uint32_t bins[3] = {2048, 2048, 1024};
  uint32_t prefix = 0, need = need0;
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    constexpr int U = 8;                                 // keys in flight per thread
    for (uint32_t i0 = 0; i0 < m; i0 += U * SEL_THREADS) {
      uint32_t k[U];
      if (d == 0) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t i = i0 + u * SEL_THREADS + tid;
          x[u] = i < m ? src[i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t i = i0 + u * SEL_THREADS + tid;
          k[u] = select_key(x[u]);
          if (i < m && i < SEL_CACHE) cache[i] = k[u];
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t i = i0 + u * SEL_THREADS + tid;
          k[u] = i >= m ? 0u : i < SEL_CACHE ? cache[i] : select_key(src[i]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * SEL_THREADS >= m) break;
        const bool in = i0 + u * SEL_THREADS + tid < m && (d == 0 || (k[u] >> shift[d > 0 ? d - 1 : 0]) == prefix);
        if (!__any_sync(0xffffffffu, in)) continue;
        // one addition per warp where all its keys fall into one bin (equal weights, zeros)
        const uint32_t bin = in ? (k[u] >> shift[d]) & (bins[d] - 1) : bins[d];
        int same;
        __match_all_sync(0xffffffffu, bin, &same);
        uint32_t* at = d == 0 ? &s.hist0[bin & (SEL_BINS - 1)][lane & 3] : &s.hist[d][bin & (SEL_BINS - 1)];
        if (same) {
          if (lane == 0) atomicAdd(at, 32u);
        } else if (in) {
          atomicAdd(at, 1u);
        }
      }
    }
    if (d == 0) {
      __syncthreads();
      for (uint32_t i = tid; i < SEL_BINS; i += SEL_THREADS)
        s.hist[0][i] = s.hist0[i][0] + s.hist0[i][1] + s.hist0[i][2] + s.hist0[i][3];
    }
    ptx::cluster_sync();                                 // every CTA's histogram is complete
    if (d == 0) write_count();
    // the bin of the need-th largest key: thread t owns `each` bins, counted from the top
    constexpr int MOST = SEL_BINS / SEL_THREADS;
    const int each = bins[d] / SEL_THREADS;              // 4, 2 or 1
    const uint32_t first = bins[d] - (tid + 1) * each;   // the lowest of them
    uint32_t c[MOST] = {};                               // the cluster's counts of bins first ..
    if (ncta <= 4) {                                     // read from every CTA, all reads in flight together
#pragma unroll
      for (uint32_t u = 0; u < 4; ++u)
        if (u < ncta) add_cluster_words(c, each, ptx::mapa(ptx::smem_u32(&s.hist[d][first]), (rank + u) & (ncta - 1)));
    } else {
      // CTA r adds up slice r of the bins and hands the sums to all: four lanes share four bins, each reading
      // and writing a quarter of the CTAs (2 or 4)
      const uint32_t slice = bins[d] / ncta;             // at most 256, a multiple of 32
      if (tid < static_cast<int>(slice)) {
        const uint32_t bin = rank * slice + (tid & ~3u), q0 = rank + (tid & 3u);
        const uint32_t from = ptx::smem_u32(&s.hist[d][bin]), to = ptx::smem_u32(&s.total[bin]);
        uint32_t sum[4] = {};
#pragma unroll
        for (uint32_t u = 0; u < SEL_MAX_CLUSTER / 4; ++u)
          if (4 * u < ncta) add_cluster_words(sum, 4, ptx::mapa(from, (q0 + 4 * u) & (ncta - 1)));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
          sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        }
        for (uint32_t u = 0; 4 * u < ncta; ++u) st_cluster_v4(ptx::mapa(to, (q0 + 4 * u) & (ncta - 1)), sum);
      }
      ptx::cluster_sync();                               // every CTA holds the sums
#pragma unroll
      for (int x = 0; x < MOST; ++x)
        if (x < each) c[x] = s.total[first + x];
    }
    uint32_t own = 0;
#pragma unroll
    for (int x = 0; x < MOST; ++x) own += c[x];
    uint32_t inc = own;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) s.scan[warp] = inc;
    __syncthreads();
    uint32_t above = inc - own + sum_below(s.scan, SEL_WARPS, warp, lane);
#pragma unroll
    for (int x = MOST - 1; x >= 0; --x) {                // (c[x] of bins that are not its own is 0)
      if (above < need && need <= above + c[x]) {
        s.bin = first + x;
        s.need = need - above;
      }
      above += c[x];
    }
    __syncthreads();
    prefix = d == 2 ? (prefix << 10) | s.bin : (prefix << 11) | s.bin;
    need = s.need;                                       // keys still to take among those equal so far
    // (s.total is written again only after the next pass's first cluster barrier)
  }
  const uint32_t cut = prefix;                           // keep keys > cut, and the first `need` equal to it

  const uint32_t wper = ((m + SEL_WARPS - 1) / SEL_WARPS + 31) / 32 * 32;
  const uint32_t w0 = min(warp * wper, m), w1 = min(w0 + wper, m);
  uint32_t gt = 0, eq = 0;
  for (uint32_t i0 = w0; i0 < w1; i0 += 32) {
    const uint32_t i = i0 + lane;
    const uint32_t k = i >= w1 ? 0 : i < SEL_CACHE ? cache[i] : select_key(src[i]);
    gt += __popc(__ballot_sync(0xffffffffu, i < w1 && k > cut));
    eq += __popc(__ballot_sync(0xffffffffu, i < w1 && k == cut));
  }
  if (lane == 0) {
    s.warp_gt[warp] = gt;
    s.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t cg = sum_below(s.warp_gt, SEL_WARPS, SEL_WARPS, lane), ce = sum_below(s.warp_eq, SEL_WARPS, SEL_WARPS, lane);
    if (lane < static_cast<int>(ncta)) {
      ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(&s.cta_gt[rank]), lane), cg);
      ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(&s.cta_eq[rank]), lane), ce);
    }
  }
  ptx::cluster_sync();                                   // the last access to another CTA's memory
  // ties before this warp, its first output slot
  uint32_t ties = sum_below(s.cta_eq, ncta, rank, lane) + sum_below(s.warp_eq, SEL_WARPS, warp, lane);
  uint32_t at = head + sum_below(s.cta_gt, ncta, rank, lane) + sum_below(s.warp_gt, SEL_WARPS, warp, lane) + min(ties, need);
  const uint32_t below = (1u << lane) - 1;
  for (uint32_t i0 = w0; i0 < w1; i0 += 32) {
    const uint32_t i = i0 + lane;
    const uint32_t k = i >= w1 ? 0 : i < SEL_CACHE ? cache[i] : select_key(src[i]);
    const bool is_eq = i < w1 && k == cut;
    const uint32_t e = __ballot_sync(0xffffffffu, is_eq);
    const bool keep = (i < w1 && k > cut) || (is_eq && ties + __popc(e & below) < need);
    const uint32_t kb = __ballot_sync(0xffffffffu, keep);
    if (keep) out[at + __popc(kb & below)] = static_cast<int32_t>(head + lo + i);
    at += __popc(kb);
    ties += __popc(e);
  }
}

}  // namespace mla
