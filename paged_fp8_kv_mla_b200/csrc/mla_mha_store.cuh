// The KV-store step of the multi-head cache (sm_100a): the step's keys and values go into their pages,
// keys in kv plane 0 and values in plane 1, as bf16 or quantised to e4m3 with one fp32 scale per token
// and head (the per-token recipe of the latent cache's KV-store step, applied to each head's row):
//   scale = f32(max |x|) / 448 rounded to fp32 (1.0 for an all-zero row),
//   code_d = e4m3_rn_sat(f32_rn(x_d / scale)).
//
// HBM-bound: 2 bytes per value in, 2 or 1 out.  A group of D / 8 lanes holds one row (a token's head,
// 16 bytes per lane), so a warp reads and writes whole consecutive rows; the row's maximum is a shuffle
// within the group.
#pragma once
#include <cstdint>
#include "mla_kv_store.cuh"

namespace mla {

struct MhaStoreParams {
  const uint16_t* k;               // bf16 bits [B, T, HKV, D]
  const uint16_t* v;
  const uint32_t* cache_lengths;   // [B]
  const uint32_t* lut;             // [B, max_pages]
  const uint32_t* slut;            // [B, max_pages] or null
  uint8_t* blocks;                 // bf16 or e4m3 [NB, KVD, NL, P, HKV, D]
  float* scales;                   // fp32 [NSB, KVD, NL, P, HKV, 1] (e4m3 only)
  unsigned int* status;
  unsigned long long rows;         // B * T * HKV
  int B, T, HKV, P, KVD, NL, layer, NB, NSB, max_pages;
  FastDiv divH, divT;              // by HKV, by T
};

constexpr int MST_THREADS = 256;

template <int D, bool FP8>
__global__ void __launch_bounds__(MST_THREADS) mla_mha_store_kernel(const __grid_constant__ MhaStoreParams p) {
  constexpr int LANES = D / 8;
  const unsigned long long r =
      (static_cast<unsigned long long>(blockIdx.x) * MST_THREADS + threadIdx.x) / LANES;
  const int x = threadIdx.x & (LANES - 1), plane = blockIdx.y;
  bool ok = r < p.rows;
  size_t row = 0, srow = 0;
  if (ok) {
    const uint32_t tok = p.divH.div(static_cast<uint32_t>(r));
    const uint32_t h = static_cast<uint32_t>(r) - tok * p.HKV;
    const uint32_t b = p.divT.div(tok), i = tok - b * p.T;
    const uint64_t pos = static_cast<uint64_t>(p.cache_lengths[b]) + i, page = pos / static_cast<uint32_t>(p.P);
    const uint32_t slot = static_cast<uint32_t>(pos - page * p.P);
    if (page >= static_cast<uint64_t>(p.max_pages)) {
      ok = false;
    } else {
      const uint32_t blk = p.lut[static_cast<size_t>(b) * p.max_pages + page];
      const uint32_t sblk = FP8 && p.slut ? p.slut[static_cast<size_t>(b) * p.max_pages + page] : blk;
      ok = blk < static_cast<uint32_t>(p.NB) && (!FP8 || sblk < static_cast<uint32_t>(p.NSB));
      row = (((static_cast<size_t>(blk) * p.KVD + plane) * p.NL + p.layer) * p.P + slot) * p.HKV + h;
      srow = (((static_cast<size_t>(sblk) * p.KVD + plane) * p.NL + p.layer) * p.P + slot) * p.HKV + h;
    }
    if (!ok && x == 0) raise_status(p.status, STATUS_BOUNDS);
  }
  uint4 v = make_uint4(0, 0, 0, 0);
  if (ok) v = reinterpret_cast<const uint4*>((plane ? p.v : p.k) + r * D)[x];
  if (!FP8) {
    if (ok) reinterpret_cast<uint4*>(p.blocks + row * D * 2)[x] = v;
    return;
  }
  uint32_t m2 = absmax8_bits(v, 0u);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
  if (!ok) return;
  const float m = __uint_as_float(max(m2 & 0xFFFFu, m2 >> 16) << 16);
  const float s = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
  reinterpret_cast<uint2*>(p.blocks + row * D)[x] = s >= KVS_FAST_MIN_SCALE ? quant8(v, s, __frcp_rn(s)) : quant8_div(v, s);
  if (x == 0) p.scales[srow] = s;
}

}  // namespace mla
