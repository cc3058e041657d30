// The KV-store step of the multi-head cache (sm_100a): the step's keys and values go into their pages,
// keys in kv plane 0 and values in plane 1, as bf16 or quantised to e4m3 with one fp32 scale per token
// and head (the per-token recipe of the latent cache's KV-store step, applied to each head's row):
//   scale = f32(max |x|) / 448 rounded to fp32 (1.0 for an all-zero row),
//   code_d = e4m3_rn_sat(f32_rn(x_d / scale)).
//
// HBM-bound: 2 bytes per value in, 2 or 1 out.  LT lanes (8, 16 or 32) take one token of one plane: all
// its heads' values are one contiguous run on both sides, so the page is looked up once per token, and
// each lane moves 16-byte chunks x, x + LT, ... with four loads in flight.  A head row is D / 8
// neighbouring lanes; its maximum is a shuffle within them.  (One row per group, with its own look-up,
// was bound by instructions: 80 % of the issue slots at 0.34 of the copy rate.)
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
  unsigned int tokens;             // B * T
  int chunks;                      // 16-byte chunks of a token in one plane
  int B, T, HKV, P, KVD, NL, layer, NB, NSB, max_pages;
  FastDiv divT, divP;              // by T, by the page size
};

constexpr int MST_THREADS = 256;

template <int D, bool FP8, int LT>
__global__ void __launch_bounds__(MST_THREADS) mla_mha_store_kernel(const __grid_constant__ MhaStoreParams p) {
  constexpr int LANES = D / 8;                           // lanes of a head row
  constexpr int U = 4;
  const uint32_t tok = (blockIdx.x * MST_THREADS + threadIdx.x) / LT;
  const int x = threadIdx.x & (LT - 1), plane = blockIdx.y;
  bool ok = tok < p.tokens;
  size_t row = 0, srow = 0;
  if (ok) {
    const uint32_t b = p.divT.div(tok), i = tok - b * p.T;
    const uint32_t pos = p.cache_lengths[b] + i, page = p.divP.div(pos);
    const uint32_t slot = pos - page * p.P;
    ok = pos >= i && page < static_cast<uint32_t>(p.max_pages);   // (the sum has not wrapped)
    if (ok) {
      const uint32_t blk = p.lut[static_cast<size_t>(b) * p.max_pages + page];
      const uint32_t sblk = FP8 && p.slut ? p.slut[static_cast<size_t>(b) * p.max_pages + page] : blk;
      ok = blk < static_cast<uint32_t>(p.NB) && (!FP8 || sblk < static_cast<uint32_t>(p.NSB));
      row = ((static_cast<size_t>(blk) * p.KVD + plane) * p.NL + p.layer) * p.P + slot;
      srow = (((static_cast<size_t>(sblk) * p.KVD + plane) * p.NL + p.layer) * p.P + slot) * p.HKV;
    }
    if (!ok && x == 0) raise_status(p.status, STATUS_BOUNDS);
  }
  const uint4* src = reinterpret_cast<const uint4*>(plane ? p.v : p.k) + static_cast<size_t>(tok) * p.chunks;
  uint8_t* dst = p.blocks + row * p.chunks * (FP8 ? 8 : 16);
  // every lane of the warp takes part in every round (the shuffles below)
  for (int c0 = 0; c0 < p.chunks; c0 += U * LT) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * LT + x;
      v[u] = ok && c < p.chunks ? src[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * LT + x;
      const bool in = ok && c < p.chunks;
      if (!FP8) {
        if (in) reinterpret_cast<uint4*>(dst)[c] = v[u];
        continue;
      }
      uint32_t m2 = absmax8_bits(v[u], 0u);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
      if (!in) continue;
      const float m = __uint_as_float(max(m2 & 0xFFFFu, m2 >> 16) << 16);
      const float s = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
      reinterpret_cast<uint2*>(dst)[c] = s >= KVS_FAST_MIN_SCALE ? quant8(v[u], s, __frcp_rn(s)) : quant8_div(v[u], s);
      if (c % LANES == 0) p.scales[srow + c / LANES] = s;
    }
  }
}

}  // namespace mla
