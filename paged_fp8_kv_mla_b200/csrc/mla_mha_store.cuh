// The KV-store step of the multi-head cache (sm_100a): the step's keys and values go into their pages,
// keys in kv plane 0 and values in plane 1, as bf16 or quantised to e4m3 with one fp32 scale per token
// and head (the per-token recipe of the latent cache's KV-store step, applied to each head's row):
//   scale = f32(max |x|) / 448 rounded to fp32 (1.0 for an all-zero row),
//   code_d = e4m3_rn_sat(f32_rn(x_d / scale)).
//
// HBM-bound: 2 bytes per value in, 2 or 1 out.  LT lanes (8, 16 or 32, a divisor of the row's 16-byte
// chunks) take one token of one plane: all its heads' values are one contiguous run on both sides, so the
// page is looked up once per token (its first values are on their way meanwhile), and each lane moves chunks
// x, x + LT, ... with U (up to 4) loads in flight.  A head row is D / 8 neighbouring lanes; its maximum is a
// shuffle within them, two rows to a shuffle.  The e4m3 form is bound by its instructions as much as by HBM:
// one row per group, with its own look-up and division, ran at 0.34 of the copy rate with 80 % of the issue
// slots taken, both planes in one thread at 0.65.
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
  int steps;                       // a token's 16-byte chunks in one plane, per lane
  int B, T, HKV, P, KVD, NL, layer, NB, NSB, max_pages;
  FastDiv divT, divP;              // by T, by the page size
};

constexpr int MST_THREADS = 256;

// RN(m / 448) of a positive bf16 value m by one correction of the product with RN(1 / 448) (Markstein, as
// cited for quant8): compared with the IEEE quotient for every positive finite bf16 m, subnormals included.
__device__ __forceinline__ float mst_scale(float m) {
  constexpr float C = 1.f / 448.f;
  const float y0 = __fmul_rn(m, C);
  const float y = fmaf(fmaf(-448.f, y0, m), C, y0);
  return m > 0.f ? y : 1.f;
}

template <int D, bool FP8, int LT, int U>
__global__ void __launch_bounds__(MST_THREADS, 6) mla_mha_store_kernel(const __grid_constant__ MhaStoreParams p) {
  constexpr int LANES = D / 8;                           // lanes of a head row
  const uint32_t tok = (blockIdx.x * MST_THREADS + threadIdx.x) / LT;
  const int x = threadIdx.x & (LT - 1), plane = blockIdx.y;
  const bool live = tok < p.tokens;
  const uint4* src = reinterpret_cast<const uint4*>(plane ? p.v : p.k) + static_cast<size_t>(live ? tok : 0) * (p.steps * LT) + x;
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)                            // on their way while the page is looked up
    if (u < p.steps) v[u] = src[u * LT];
  bool ok = live;
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
  uint8_t* dst = p.blocks + (row * (p.steps * LT) + x) * (FP8 ? 8 : 16);
  float* scale = FP8 ? p.scales + srow + x / LANES : nullptr;
  for (int s = 0;;) {                                    // every lane of the warp takes part (the shuffles below)
    uint32_t top[(U + 1) / 2];                           // a row's maximum over its lanes, two rows to a register
    if (FP8) {
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        const uint32_t a = absmax8_bits(v[u], 0u), b = u + 1 < U ? absmax8_bits(v[u + 1 < U ? u + 1 : u], 0u) : 0u;
        uint32_t m2 = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        top[u / 2] = m2;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= p.steps || !ok) continue;
      if (!FP8) {
        *reinterpret_cast<uint4*>(dst + u * LT * 16) = v[u];
        continue;
      }
      const float f = mst_scale(__uint_as_float(u & 1 ? top[u / 2] & 0xFFFF0000u : top[u / 2] << 16));
      *reinterpret_cast<uint2*>(dst + u * LT * 8) = f >= KVS_FAST_MIN_SCALE ? quant8(v[u], f, __frcp_rn(f)) : quant8_div(v[u], f);
      if (x % LANES == 0) scale[u * LT / LANES] = f;
    }
    s += U;
    if (s >= p.steps) break;
    src += U * LT;
    dst += U * LT * (FP8 ? 8 : 16);
    if (FP8) scale += U * LT / LANES;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < p.steps) v[u] = src[u * LT];
  }
}

}  // namespace mla
