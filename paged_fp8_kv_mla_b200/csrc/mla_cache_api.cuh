// Host side of the cache operators' C ABI: eviction from the latent cache (accumulated weights,
// selection, compaction) and the multi-head cache (KV-store step, decode).  Part of the library's
// one translation unit (mla_lib.cu), after the decode's host side, whose helpers it uses.
#pragma once
#include "mla_accumulate.cuh"
#include "mla_compact.cuh"
#include "mla_mha_decode.cuh"
#include "mla_mha_store.cuh"
#include "mla_select.cuh"

namespace {

int gcd_int(int a, int b) { return b == 0 ? a : gcd_int(b, a % b); }

template <int D, bool FP8>
cudaError_t mha_smem() {
  auto set = [](auto* kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(mla::MHA_SMEM_LIMIT));
  };
  cudaError_t e = set(mla::mla_mha_decode_kernel<D, FP8, 1, 1>);
  if (e == cudaSuccess) e = set(mla::mla_mha_decode_kernel<D, FP8, 2, 1>);
  if (e == cudaSuccess) e = set(mla::mla_mha_decode_kernel<D, FP8, 1, 2>);
  if (e == cudaSuccess) e = set(mla::mla_mha_decode_kernel<D, FP8, 2, 2>);
  if constexpr (D == 64 && FP8) {
    if (e == cudaSuccess) e = set(mla::mla_mha_decode_kernel<64, true, 4, 1>);
    if (e == cudaSuccess) e = set(mla::mla_mha_decode_kernel<64, true, 4, 2>);
  }
  return e;
}

// The current device's SM count and status word, and (once per device) the shared-memory limits of the kernels here.
mla_status_t cache_device(int* sms, unsigned int** status, int* wide_clusters = nullptr) {
  static int g_sms[kMaxDevices], g_wide[kMaxDevices];
  static unsigned int* g_status[kMaxDevices];
  int dev = 0;
  MLA_CUDA(cudaGetDevice(&dev));
  if (dev >= kMaxDevices) return fail(MLA_ERR_UNSUPPORTED, "device index too large");
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[dev] == 0) {
    int n = 0;
    MLA_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    auto smem = [](auto* kernel, size_t bytes) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    };
    MLA_CUDA(smem(mla::mla_accumulate_kernel, mla::ACC_SMEM_ALLOC));
    MLA_CUDA(smem(mla::mla_select_kernel<512>, mla::SEL_KEYS_OFF + mla::SEL_CACHE * 4));
    MLA_CUDA(smem(mla::mla_select_kernel<1024>, mla::SEL_KEYS_OFF + mla::SEL_CACHE * 4));
    MLA_CUDA(smem(mla::mla_compact_kernel<64, 256, 4, 3, 3>, 3 * 4 * 256 * mla::CMP_SLOT));
    MLA_CUDA(smem(mla::mla_compact_kernel<32, 512, 2, 4, 2>, 4 * 2 * 512 * mla::CMP_SLOT));
    MLA_CUDA(smem(mla::mla_compact_kernel<32, 1024, 2, 5, 1>, 5 * 2 * 1024 * mla::CMP_SLOT));
    MLA_CUDA((mha_smem<64, false>()));
    MLA_CUDA((mha_smem<64, true>()));
    MLA_CUDA((mha_smem<128, false>()));
    MLA_CUDA((mha_smem<128, true>()));
    g_status[dev] = status_ptr();
    if (!g_status[dev]) return fail(MLA_ERR_CUDA, "status word address unavailable");
    // clusters of 16 (more than the portable size) of the selection that the device holds at once
    MLA_CUDA(cudaFuncSetAttribute(mla::mla_select_kernel<1024>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16 * 64);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = mla::SEL_KEYS_OFF + mla::SEL_CACHE * 4;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&g_wide[dev], mla::mla_select_kernel<1024>, &cfg) != cudaSuccess) {
      g_wide[dev] = 0;
      cudaGetLastError();
    }
    g_sms[dev] = n;
  }
  if (wide_clusters) *wide_clusters = g_wide[dev];
  *status = g_status[dev];
  *sms = g_sms[dev];
  return MLA_OK;
}

bool overlap(const void* a, uint64_t a_bytes, const void* b, uint64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A paged array's pool and page-table description, for any row width; the latent cache's own checks
// (check_cache) go further.
mla_status_t check_pages(const mla_paged_shape_t* s, uint32_t layer_idx) {
  if (s->batch < 0 || s->num_blocks < 1 || s->kv_dim < 1 || s->num_layers < 1 || s->page_size < 1 ||
      s->num_kv_heads < 1 || s->head_dim < 1 || s->num_scale_blocks < 1 || s->head_dim_granularity < 1 || s->max_pages < 1)
    return fail(MLA_ERR_INVALID_ARG, "non-positive dimension in shape");
  if (layer_idx >= static_cast<uint32_t>(s->num_layers))
    return fail(MLA_ERR_INVALID_ARG, "layer_idx %u >= num_layers %d", layer_idx, s->num_layers);
  const double rows = static_cast<double>(s->num_blocks) * s->kv_dim * s->num_layers * s->page_size;
  const double srows = static_cast<double>(s->num_scale_blocks) * s->kv_dim * s->num_layers * s->page_size;
  if (rows >= 2147483648.0 || srows >= 2147483648.0)
    return fail(MLA_ERR_UNSUPPORTED, "block pool too large (%.0f rows)", rows > srows ? rows : srows);
  if (static_cast<double>(s->max_pages) * s->page_size >= 1073741824.0)
    return fail(MLA_ERR_UNSUPPORTED, "max_pages * page_size too large");
  return MLA_OK;
}

// The multi-head cache: kv plane 0 keys, plane 1 values, head_dim 64 or 128, bf16 or e4m3 with one scale
// per token and head.
mla_status_t check_mha_shape(const mla_paged_shape_t* s, uint32_t layer_idx, int32_t element_bytes) {
  const mla_status_t st = check_pages(s, layer_idx);
  if (st != MLA_OK) return st;
  if (element_bytes != 1 && element_bytes != 2)
    return fail(MLA_ERR_INVALID_ARG, "element_bytes must be 1 (e4m3) or 2 (bf16), got %d", element_bytes);
  if (s->head_dim != 64 && s->head_dim != 128)
    return fail(MLA_ERR_UNSUPPORTED, "head_dim must be 64 or 128 (got %d)", s->head_dim);
  if (s->kv_dim < 2) return fail(MLA_ERR_INVALID_ARG, "kv_dim must be at least 2 (keys and values)");
  if (s->num_kv_heads > 256) return fail(MLA_ERR_UNSUPPORTED, "num_kv_heads must be at most 256 (got %d)", s->num_kv_heads);
  if (s->head_dim_granularity != 1)
    return fail(MLA_ERR_UNSUPPORTED, "only one scale per token and head (head_dim_granularity 1) is implemented");
  if (s->page_size % 16 != 0) return fail(MLA_ERR_UNSUPPORTED, "page_size must be a multiple of 16");
  return MLA_OK;
}

mla_status_t check_mha(const mla_paged_shape_t* s, uint32_t layer_idx, int32_t element_bytes, const void* blocks,
                       const void* scales, const uint32_t* cache_lengths, const uint32_t* lookup_table) {
  if (!s) return fail(MLA_ERR_INVALID_ARG, "shape is NULL");
  if (!blocks || !cache_lengths || !lookup_table)
    return fail(MLA_ERR_INVALID_ARG, "blocks, cache_lengths and lookup_table must be non-NULL");
  const mla_status_t st = check_mha_shape(s, layer_idx, element_bytes);
  if (st != MLA_OK) return st;
  if ((element_bytes == 1) != (scales != nullptr))
    return fail(MLA_ERR_INVALID_ARG, "an e4m3 cache needs scales and a bf16 cache takes none");
  if (!aligned16(blocks) || !aligned16(scales)) return fail(MLA_ERR_INVALID_ARG, "blocks and scales must be 16-byte aligned");
  return MLA_OK;
}

// Rows of row_bytes at `blocks` as {column bytes, rows, all_cols columns}: one box = `cols` columns of
// `box_rows` rows.
mla_status_t make_row_map(CUtensorMap* map, const void* blocks, uint64_t rows, uint64_t row_bytes, int col_bytes,
                          int all_cols, int box_rows, int cols) {
  EncodeTiledFn enc = nullptr;
  const mla_status_t st = get_encode_fn(&enc);
  if (st != MLA_OK) return st;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(col_bytes), rows, static_cast<cuuint64_t>(all_cols)};
  const cuuint64_t strides[2] = {row_bytes, static_cast<cuuint64_t>(col_bytes)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(col_bytes), static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(cols)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(blocks), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, col_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled(blocks) failed (%d)", static_cast<int>(r));
  return MLA_OK;
}

// The split q of the accumulated weights: an item's bytes, and the query tokens that one launch takes
// (long prompts run in several launches, so that the workspace stays at 256 MB unless one token of the
// batch needs more).
struct AccPlan {
  uint32_t item_bytes, heads;
  int tokens;
  uint64_t total;
};

mla_status_t acc_plan(int64_t B, int64_t T, int64_t H, AccPlan* out) {
  AccPlan a{};
  const int64_t G = (H + mla::ACC_HEADS - 1) / mla::ACC_HEADS;
  a.heads = static_cast<uint32_t>(((H < mla::ACC_HEADS ? H : mla::ACC_HEADS) + 7) / 8 * 8);
  a.item_bytes = a.heads * (2 * mla::HEAD_DIM + 8);
  if (B * G > (1ll << 24)) return fail(MLA_ERR_UNSUPPORTED, "too many (request, head group) items");
  const int64_t token = B * G * a.item_bytes;
  int64_t tokens = (256ll << 20) / token;
  tokens = tokens < 1 ? 1 : tokens > T ? T : tokens;
  a.tokens = static_cast<int>(tokens);
  a.total = static_cast<uint64_t>(token) * tokens;
  *out = a;
  return MLA_OK;
}

// How a multi-head decode is laid out (the rules the kernel's header comment describes).
struct MhaPlan {
  int R, nr, hg, mt, kw, ks, head_groups, row_groups, tile, box_rows, stages, NC, one_item;
  uint32_t plane_bytes, stage_bytes, smem;
  uint64_t part_lse_off, desc_off, total;
};

mla_status_t mha_plan(const mla_paged_shape_t* s, uint32_t T, uint32_t max_cache_length, int element_bytes, int sms,
                      MhaPlan* out) {
  MhaPlan m{};
  if (s->num_q_heads < 1 || s->num_q_heads % s->num_kv_heads != 0)
    return fail(MLA_ERR_INVALID_ARG, "num_q_heads %d must be a positive multiple of num_kv_heads %d", s->num_q_heads,
                s->num_kv_heads);
  if (T < 1) return fail(MLA_ERR_INVALID_ARG, "max_prompt_length must be >= 1");
  if (static_cast<uint64_t>(max_cache_length) + T + 256 >= (1ull << 30))
    return fail(MLA_ERR_UNSUPPORTED, "max_cache_length too large");
  const uint64_t need = (static_cast<uint64_t>(max_cache_length) + T + s->page_size - 1) / s->page_size;
  if (need > static_cast<uint64_t>(s->max_pages))
    return fail(MLA_ERR_INVALID_ARG, "lookup_table has %d pages per request, %llu needed for max_cache_length %u",
                s->max_pages, static_cast<unsigned long long>(need), max_cache_length);
  const uint64_t R = static_cast<uint64_t>(T) * (s->num_q_heads / s->num_kv_heads);
  if (R > (1u << 24)) return fail(MLA_ERR_UNSUPPORTED, "too many query rows per kv head");
  m.R = static_cast<int>(R);
  // Warps: first the row tiles of a head (they share its keys), then heads, then the keys of a tile.
  m.nr = m.R <= 8 ? 1 : 2;
  const int row_tiles = (m.R + 8 * m.nr - 1) / (8 * m.nr);
  m.mt = row_tiles < mla::MHA_WARPS ? row_tiles : mla::MHA_WARPS;
  m.row_groups = (row_tiles + m.mt - 1) / m.mt;
  const int most = mla::MHA_WARPS / m.mt;
  m.head_groups = (s->num_kv_heads + most - 1) / most;
  m.hg = (s->num_kv_heads + m.head_groups - 1) / m.head_groups;
  m.kw = 1;
  while (2 * m.kw * m.hg * m.mt <= mla::MHA_WARPS) m.kw *= 2;
  // Tile: 32 keys per warp at a time where a run of pages holds them and a ring stage of them takes at most
  // 72 KB (three stages), else 16; doubled while a stage stays within 72 KB (two steps per hand-over).  e4m3
  // heads of 64 take 64 keys at a time (128 x 8k, 8 kv heads: 194 us, 215 with 32, 244 in tiles of 32).
  const uint32_t per_key = 2u * m.hg * s->head_dim * element_bytes + (element_bytes == 1 ? 8u * s->num_kv_heads : 0u);
  m.ks = s->page_size % 32 == 0 && 32 * m.kw * per_key <= 73728 ? 2 : 1;
  if (s->head_dim == 64 && element_bytes == 1 && s->page_size % 64 == 0 && 64 * m.kw * per_key <= 73728) m.ks = 4;
  m.tile = 16 * m.ks * m.kw;
  while (m.tile < 128 && 2 * m.tile * per_key <= 73728) m.tile *= 2;
  m.box_rows = gcd_int(s->page_size, m.tile);
  if (m.box_rows > 256) m.box_rows = 256;                // (both are powers of two) a box's largest extent
  // (at most 8 boxes to a tile: a box holds at least 16 keys, 16 ks where ks > 1, or 256 of a tile's at most 512)
  m.plane_bytes = static_cast<uint32_t>(m.tile) * m.hg * s->head_dim * element_bytes;
  m.stage_bytes = static_cast<uint32_t>(align_up(m.tile * per_key, 1024));
  const uint32_t merge = m.kw > 1 ? (s->head_dim == 64 ? mla::mha_merge_bytes<64>() : mla::mha_merge_bytes<128>()) : 0;
  const uint32_t rest = merge + mla::MHA_MISC_BYTES + 1024;
  m.stages = static_cast<int>((mla::MHA_SMEM_LIMIT - rest) / m.stage_bytes);
  if (m.stages > mla::MHA_MAX_STAGES) m.stages = mla::MHA_MAX_STAGES;
  if (m.stages < 2) return fail(MLA_ERR_UNSUPPORTED, "%d kv heads: a tile's scales do not fit shared memory", s->num_kv_heads);
  m.smem = m.stages * m.stage_bytes + rest;
  const uint64_t items = static_cast<uint64_t>(s->batch) * m.head_groups * m.row_groups;
  const uint64_t max_tiles = (static_cast<uint64_t>(max_cache_length) + T + m.tile - 1) / m.tile;
  if (items > 0x7FFFFFFFull) return fail(MLA_ERR_UNSUPPORTED, "too many (request, head group, row group) items");
  // Items of a few tiles are not worth cutting: one CTA each, and no second launch.
  m.one_item = max_tiles <= 4;
  const uint64_t most_tiles = items * max_tiles;
  m.NC = m.one_item ? static_cast<int>(items) : static_cast<int>(most_tiles < static_cast<uint64_t>(sms) ? most_tiles : sms);
  if (!m.one_item) {
    uint64_t o = align_up(sizeof(float) * 2ull * m.NC * mla::MHA_ROWS * s->head_dim, 256);
    m.part_lse_off = o;
    o = align_up(o + sizeof(float) * 2ull * m.NC * mla::MHA_ROWS, 256);
    m.desc_off = o;
    m.total = align_up(o + sizeof(int4) * m.NC, 256);
  }
  *out = m;
  return MLA_OK;
}

template <int D, bool FP8>
mla_status_t mha_launch(const mla::MhaParams& p, const MhaPlan& m, cudaStream_t stream) {
  auto* kernel = m.nr == 1 ? (m.ks == 2 ? mla::mla_mha_decode_kernel<D, FP8, 2, 1> : mla::mla_mha_decode_kernel<D, FP8, 1, 1>)
                           : (m.ks == 2 ? mla::mla_mha_decode_kernel<D, FP8, 2, 2> : mla::mla_mha_decode_kernel<D, FP8, 1, 2>);
  if constexpr (D == 64 && FP8)
    if (m.ks == 4) kernel = m.nr == 1 ? mla::mla_mha_decode_kernel<64, true, 4, 1> : mla::mla_mha_decode_kernel<64, true, 4, 2>;
  kernel<<<m.NC, mla::MHA_THREADS, m.smem, stream>>>(p);
  MLA_CUDA(cudaGetLastError());
  if (m.one_item) return MLA_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(m.NC, static_cast<unsigned>(m.hg * m.mt * m.nr));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MLA_CUDA(cudaLaunchKernelEx(&cfg, mla::mla_mha_join_kernel<D>, p));
  return MLA_OK;
}

// A compaction kernel: slices, threads, rows per lane and chunk, chunks in shared memory, CTAs per SM.
template <int SLICE, int THREADS, int U, int S, int CTAS>
constexpr size_t compact_smem() { return static_cast<size_t>(S) * U * THREADS * mla::CMP_SLOT; }
template <int SLICE, int THREADS, int U, int S, int CTAS>
void compact_launch(const mla::CompactParams& p, dim3 grid, cudaStream_t stream) {
  mla::mla_compact_kernel<SLICE, THREADS, U, S, CTAS>
      <<<grid, THREADS, compact_smem<SLICE, THREADS, U, S, CTAS>(), stream>>>(p);
}

// Lanes per token: the largest power of two, up to a warp, that divides its 16-byte chunks in one plane;
// chunks per lane at a time: as many as a lane has, up to four.
template <int D, bool FP8, int LT>
void mha_store_kernel(const mla::MhaStoreParams& p, cudaStream_t stream) {
  auto* kernel = p.steps >= 3   ? mla::mla_mha_store_kernel<D, FP8, LT, 4>
                 : p.steps == 2 ? mla::mla_mha_store_kernel<D, FP8, LT, 2> : mla::mla_mha_store_kernel<D, FP8, LT, 1>;
  const uint64_t threads = static_cast<uint64_t>(p.tokens) * LT;
  const dim3 grid(static_cast<unsigned>((threads + mla::MST_THREADS - 1) / mla::MST_THREADS), 2);
  kernel<<<grid, mla::MST_THREADS, 0, stream>>>(p);
}

template <int D, bool FP8>
mla_status_t mha_store_launch(mla::MhaStoreParams& p, cudaStream_t stream) {
  if (static_cast<uint64_t>(p.tokens) * 32 > 0xFFFFFFFFull - mla::MST_THREADS)
    return fail(MLA_ERR_UNSUPPORTED, "too many new tokens (%u)", p.tokens);
  const int chunks = p.HKV * D / 8, lanes = gcd_int(chunks, 32);
  p.steps = chunks / lanes;
  if (lanes == 32)
    mha_store_kernel<D, FP8, 32>(p, stream);
  else if (lanes == 16)
    mha_store_kernel<D, FP8, 16>(p, stream);
  else if (D == 64)                                      // an odd number of heads of 64 values
    mha_store_kernel<64, FP8, 8>(p, stream);
  MLA_CUDA(cudaGetLastError());
  return MLA_OK;
}

}  // namespace

extern "C" {

mla_status_t mla_accumulate_weights_fp8(const void* q, const float* lse, const void* blocks, const float* scales,
                                        const uint32_t* cache_lengths, const uint32_t* lookup_table,
                                        const uint32_t* scales_lookup_table, uint32_t max_prompt_length,
                                        uint32_t max_cache_length, uint32_t layer_idx, float softmax_scale,
                                        const mla_paged_shape_t* shape, const float* scores, int64_t scores_stride,
                                        float* out, int64_t out_stride, void* workspace, uint64_t workspace_bytes,
                                        cudaStream_t stream) {
  mla::DecodeParams d{};
  uint64_t rows = 0;
  mla_status_t st = check_cache(blocks, scales, cache_lengths, lookup_table, max_prompt_length, max_cache_length,
                                layer_idx, shape, &d, &rows);
  if (st != MLA_OK) return st;
  if (d.SG != 1)
    return fail(MLA_ERR_UNSUPPORTED, "the accumulated weights take one scale per token (head_dim_granularity 1)");
  if (!q || !lse || !out) return fail(MLA_ERR_INVALID_ARG, "q, lse and out must be non-NULL");
  if (!aligned16(q)) return fail(MLA_ERR_INVALID_ARG, "q must be 16-byte aligned");
  if (!aligned4(lse) || !aligned4(scores) || !aligned4(out))
    return fail(MLA_ERR_INVALID_ARG, "lse, scores and out must be 4-byte aligned");
  if (!(softmax_scale == softmax_scale)) return fail(MLA_ERR_INVALID_ARG, "softmax_scale is NaN");
  const int64_t need = static_cast<int64_t>(max_cache_length) + max_prompt_length;
  if (out_stride < need || (scores && scores_stride < need))
    return fail(MLA_ERR_INVALID_ARG, "the rows of scores and out must hold max_cache_length + max_prompt_length = %lld values",
                static_cast<long long>(need));
  if (scores == out && scores_stride != out_stride)
    return fail(MLA_ERR_INVALID_ARG, "out may be scores only with the same stride");
  if (d.B == 0) return MLA_OK;
  if (static_cast<int64_t>(d.T) * d.G > 0x3FFFFFFF) return fail(MLA_ERR_UNSUPPORTED, "too many query tokens");
  int sms = 0;
  unsigned int* status = nullptr;
  st = cache_device(&sms, &status);
  if (st != MLA_OK) return st;
  mla::AccumulateParams p{};
  p.box_rows = gcd_int(d.P, mla::ACC_BN);
  st = make_row_map(&p.tmap_k, blocks, rows, mla::HEAD_DIM, 128, 4, p.box_rows, 1);
  if (st != MLA_OK) return st;
  st = make_row_map(&p.tmap_r, static_cast<const char*>(blocks) + 512, rows, mla::HEAD_DIM, 64, 1, p.box_rows, 1);
  if (st != MLA_OK) return st;
  AccPlan plan{};
  st = acc_plan(d.B, d.T, d.H, &plan);
  if (st != MLA_OK) return st;
  if (!workspace || workspace_bytes < plan.total)
    return fail(MLA_ERR_WORKSPACE, "the call needs a workspace of %llu bytes (mla_accumulate_workspace_bytes)",
                static_cast<unsigned long long>(plan.total));
  if (!aligned16(workspace)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  p.split = static_cast<uint8_t*>(workspace);
  p.item_bytes = plan.item_bytes;
  p.q = static_cast<const uint16_t*>(q);
  p.lse = lse;
  p.scales = scales;
  p.cache_lengths = cache_lengths;
  p.lut = lookup_table;
  p.slut = scales_lookup_table;
  p.scores = scores;
  p.out = out;
  p.scores_stride = scores_stride;
  p.out_stride = out_stride;
  p.status = status;
  p.B = d.B;
  p.T = d.T;
  p.H = d.H;
  p.G = d.G;
  p.P = d.P;
  p.KVD = d.KVD;
  p.NL = d.NL;
  p.layer = d.layer;
  p.NB = d.NB;
  p.NSB = d.NSB;
  p.max_pages = d.max_pages;
  p.max_cache_length = max_cache_length;
  p.divP = d.divP;
  p.divG = d.divG;
  p.softmax_scale = softmax_scale;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    p.wait_limit_ns = g_wait_limit_ns;
  }
  const uint64_t most = static_cast<uint64_t>(d.B) * ((need + mla::ACC_BN - 1) / mla::ACC_BN);
  const unsigned grid = static_cast<unsigned>(most < static_cast<uint64_t>(sms) ? most : sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(mla::ACC_THREADS);
  cfg.dynamicSmemBytes = mla::ACC_SMEM_ALLOC;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  for (p.i0 = 0; p.i0 < d.T; p.i0 += plan.tokens) {
    p.ni = d.T - p.i0 < plan.tokens ? d.T - p.i0 : plan.tokens;
    const uint64_t warps = static_cast<uint64_t>(d.B) * p.ni * d.G * plan.heads;
    mla::mla_split_q_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, stream>>>(p);
    MLA_CUDA(cudaGetLastError());
    MLA_CUDA(cudaLaunchKernelEx(&cfg, mla::mla_accumulate_kernel, p));
  }
  return MLA_OK;
}

mla_status_t mla_accumulate_workspace_bytes(uint32_t max_prompt_length, const mla_paged_shape_t* s, uint64_t* bytes) {
  if (!s || !bytes) return fail(MLA_ERR_INVALID_ARG, "shape and bytes must be non-NULL");
  *bytes = 0;
  if (s->batch < 0 || s->num_q_heads < 1 || max_prompt_length < 1)
    return fail(MLA_ERR_INVALID_ARG, "non-positive dimension in shape, or no query tokens");
  if (s->batch == 0) return MLA_OK;
  AccPlan plan{};
  const mla_status_t st = acc_plan(s->batch, static_cast<int64_t>(max_prompt_length), s->num_q_heads, &plan);
  if (st == MLA_OK) *bytes = plan.total;
  return st;
}

mla_status_t mla_select_keys(const float* scores, int64_t scores_stride, const uint32_t* lengths, int32_t batch,
                             uint32_t max_length, int32_t budget, int32_t num_recent, int32_t num_sink, int32_t* kept,
                             int64_t kept_stride, int32_t* kept_lengths, cudaStream_t stream) {
  if (batch < 0 || num_recent < 0 || num_sink < 0) return fail(MLA_ERR_INVALID_ARG, "batch, num_recent and num_sink must be >= 0");
  if (budget < 1) return fail(MLA_ERR_INVALID_ARG, "budget must be >= 1");
  if (static_cast<int64_t>(num_recent) + num_sink > budget)
    return fail(MLA_ERR_INVALID_ARG, "num_recent %d + num_sink %d exceed the budget %d", num_recent, num_sink, budget);
  if (!lengths || !kept_lengths || (max_length > 0 && (!scores || !kept)))
    return fail(MLA_ERR_INVALID_ARG, "scores, lengths, kept and kept_lengths must be non-NULL");
  if (!aligned4(scores) || !aligned4(kept)) return fail(MLA_ERR_INVALID_ARG, "scores and kept must be 4-byte aligned");
  if (max_length >= (1u << 30)) return fail(MLA_ERR_UNSUPPORTED, "max_length too large");
  if (scores_stride < static_cast<int64_t>(max_length))
    return fail(MLA_ERR_INVALID_ARG, "the rows of scores must hold max_length = %u values", max_length);
  const int64_t most = budget < static_cast<int64_t>(max_length) ? budget : static_cast<int64_t>(max_length);
  if (kept_stride < most) return fail(MLA_ERR_INVALID_ARG, "the rows of kept must hold %lld values", static_cast<long long>(most));
  if (batch == 0) return MLA_OK;
  if (static_cast<const void*>(kept_lengths) != lengths && overlap(kept_lengths, 4ull * batch, lengths, 4ull * batch))
    return fail(MLA_ERR_INVALID_ARG, "kept_lengths must be lengths itself or not overlap it");
  int sms = 0, wide_clusters = 0;
  unsigned int* status = nullptr;
  mla_status_t st = cache_device(&sms, &status, &wide_clusters);
  if (st != MLA_OK) return st;
  mla::SelectParams p{};
  p.scores = scores;
  p.lengths = lengths;
  p.kept = kept;
  p.kept_lengths = kept_lengths;
  p.status = status;
  p.scores_stride = scores_stride;
  p.kept_stride = kept_stride;
  p.max_length = max_length;
  p.budget = budget;
  p.recent = num_recent;
  p.sink = num_sink;
  // CTAs per request: about 2048 keys each, up to the portable cluster size, while all of them fit on the
  // device at once (two of 512 threads to an SM, or one of 1024, which a CTA with more than 4096 keys gets):
  // 64 requests of 4k take 8.1 us with 2, 9.2 with 1, 11.8 with 4; 128 of 8k 12.5 with 2, 24 with 4 in two
  // waves; 32 of 40k 15.7, 18.3 with 512 threads; 16 of 16k 12.4, 21 with 1024.  A few long requests take
  // clusters of 16, where the device has room for all: 4 of 128k 15.6 us, 19.9 with 8.
  auto fits = [&](int n) {
    return static_cast<int64_t>(batch) * n <= (max_length > static_cast<uint32_t>(n) * 4096 ? sms : 2 * sms);
  };
  int ncta = 1;
  while (ncta < 8 && static_cast<uint32_t>(ncta) * 2048 < max_length && fits(2 * ncta)) ncta *= 2;
  if (ncta == 8 && max_length > 65536 && batch <= wide_clusters) ncta = 16;
  if (static_cast<int64_t>(batch) * ncta > 0x7FFFFFFF) return fail(MLA_ERR_UNSUPPORTED, "batch too large");
  const uint32_t per = (max_length + ncta - 1) / ncta;
  const uint32_t cached = per < static_cast<uint32_t>(mla::SEL_CACHE) ? per : mla::SEL_CACHE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(batch) * ncta);
  const bool large = per > 4096;
  cfg.blockDim = dim3(large ? 1024 : 512);
  cfg.dynamicSmemBytes = mla::SEL_KEYS_OFF + cached * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ncta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (large)
    MLA_CUDA(cudaLaunchKernelEx(&cfg, mla::mla_select_kernel<1024>, p));
  else
    MLA_CUDA(cudaLaunchKernelEx(&cfg, mla::mla_select_kernel<512>, p));
  return MLA_OK;
}

mla_status_t mla_compact_paged(const int32_t* kept, int64_t kept_stride, int32_t max_kept, const int32_t* kept_lengths,
                               const uint32_t* lookup_table, const uint32_t* scales_lookup_table, uint32_t layer_idx,
                               int32_t element_bytes, const mla_paged_shape_t* s, void* blocks, float* scales,
                               float* scores, int64_t scores_stride, int32_t scores_cols, cudaStream_t stream) {
  if (!s) return fail(MLA_ERR_INVALID_ARG, "shape is NULL");
  if (!kept || !kept_lengths || !lookup_table || !blocks)
    return fail(MLA_ERR_INVALID_ARG, "kept, kept_lengths, lookup_table and blocks must be non-NULL");
  mla_status_t st = check_pages(s, layer_idx);
  if (st != MLA_OK) return st;
  if (element_bytes != 1 && element_bytes != 2)
    return fail(MLA_ERR_INVALID_ARG, "element_bytes must be 1 (e4m3) or 2 (bf16), got %d", element_bytes);
  if (max_kept < 1 || kept_stride < max_kept) return fail(MLA_ERR_INVALID_ARG, "max_kept must be >= 1 and at most kept_stride");
  if (!aligned16(blocks)) return fail(MLA_ERR_INVALID_ARG, "blocks must be 16-byte aligned");
  if (!aligned4(scales) || !aligned4(scores)) return fail(MLA_ERR_INVALID_ARG, "scales and scores must be 4-byte aligned");
  const int64_t row_bytes = static_cast<int64_t>(s->num_kv_heads) * s->head_dim * element_bytes;
  const int64_t row_words = static_cast<int64_t>(s->num_kv_heads) * s->head_dim_granularity;
  if (row_bytes % 32 != 0 || row_bytes > (1 << 20))
    return fail(MLA_ERR_UNSUPPORTED, "a token's row (%lld bytes) must be a multiple of 32 bytes, at most 1 MB",
                static_cast<long long>(row_bytes));
  if (static_cast<int64_t>(max_kept) * row_words >= (1ll << 30) || max_kept >= (1 << 28))
    return fail(MLA_ERR_UNSUPPORTED, "too many rows to move");
  if (scores && (scores_cols < 1 || scores_stride < scores_cols))
    return fail(MLA_ERR_INVALID_ARG, "scores_cols must be >= 1 and at most scores_stride");
  if (s->batch == 0) return MLA_OK;
  if (s->batch > 65535) return fail(MLA_ERR_UNSUPPORTED, "batch must be at most 65535");
  int sms = 0;
  unsigned int* status = nullptr;
  st = cache_device(&sms, &status);
  if (st != MLA_OK) return st;
  mla::CompactParams p{};
  p.kept = kept;
  p.kept_lengths = kept_lengths;
  p.lut = lookup_table;
  p.slut = scales_lookup_table ? scales_lookup_table : lookup_table;
  p.blocks = static_cast<uint8_t*>(blocks);
  p.scales = scales;
  p.scores = scores;
  p.status = status;
  p.kept_stride = kept_stride;
  p.scores_stride = scores_stride;
  p.max_kept = max_kept;
  p.scores_cols = scores_cols;
  p.P = s->page_size;
  p.KVD = s->kv_dim;
  p.NL = s->num_layers;
  p.layer = static_cast<int>(layer_idx);
  p.NB = s->num_blocks;
  p.NSB = s->num_scale_blocks;
  p.max_pages = s->max_pages;
  p.row_bytes = static_cast<int>(row_bytes);
  p.row_words = static_cast<int>(row_words);
  p.divP = make_fastdiv(static_cast<uint32_t>(s->page_size));
  p.divW = make_fastdiv(static_cast<uint32_t>(row_words));
  // Slices of 64 bytes where they give every SM a CTA, else of 32 bytes; those in CTAs of 512 threads where
  // there are more of them than SMs, else of 1024.  (12 requests of 30k cut to 15k: 57 us; 4 of 128k to 64k:
  // 116, 167 with 64-byte slices, of which there are 36.)
  const int64_t planes = static_cast<int64_t>(s->batch) * s->kv_dim;
  const bool narrow = row_bytes % 64 != 0 || planes * (row_bytes / 64) < sms;
  p.slices = static_cast<int>(row_bytes / (narrow ? 32 : 64));
  const int64_t gx = static_cast<int64_t>(s->kv_dim) * (p.slices + 1) + 1;
  if (gx > 0x7FFFFFFF) return fail(MLA_ERR_UNSUPPORTED, "grid too large");
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(s->batch));
  if (!narrow)
    compact_launch<64, 256, 4, 3, 3>(p, grid, stream);
  else if (planes * p.slices > sms)
    compact_launch<32, 512, 2, 4, 2>(p, grid, stream);
  else
    compact_launch<32, 1024, 2, 5, 1>(p, grid, stream);
  MLA_CUDA(cudaGetLastError());
  return MLA_OK;
}

mla_status_t mla_mha_kv_store(const void* k, const void* v, const uint32_t* cache_lengths, const uint32_t* lookup_table,
                              const uint32_t* scales_lookup_table, uint32_t num_new_tokens, uint32_t layer_idx,
                              int32_t element_bytes, const mla_paged_shape_t* s, void* blocks, float* scales,
                              cudaStream_t stream) {
  mla_status_t st = check_mha(s, layer_idx, element_bytes, blocks, scales, cache_lengths, lookup_table);
  if (st != MLA_OK) return st;
  mla::MhaStoreParams p{};
  const uint64_t tokens = static_cast<uint64_t>(s->batch) * num_new_tokens;
  if (tokens == 0) return MLA_OK;
  if (!k || !v) return fail(MLA_ERR_INVALID_ARG, "k and v must be non-NULL");
  if (!aligned16(k) || !aligned16(v)) return fail(MLA_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  if (tokens >= (1ull << 31)) return fail(MLA_ERR_UNSUPPORTED, "too many new tokens (%llu)", static_cast<unsigned long long>(tokens));
  int sms = 0;
  unsigned int* status = nullptr;
  st = cache_device(&sms, &status);
  if (st != MLA_OK) return st;
  p.tokens = static_cast<unsigned int>(tokens);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.cache_lengths = cache_lengths;
  p.lut = lookup_table;
  p.slut = scales_lookup_table;
  p.blocks = static_cast<uint8_t*>(blocks);
  p.scales = scales;
  p.status = status;
  p.B = s->batch;
  p.T = static_cast<int>(num_new_tokens);
  p.HKV = s->num_kv_heads;
  p.P = s->page_size;
  p.KVD = s->kv_dim;
  p.NL = s->num_layers;
  p.layer = static_cast<int>(layer_idx);
  p.NB = s->num_blocks;
  p.NSB = s->num_scale_blocks;
  p.max_pages = s->max_pages;
  p.divT = make_fastdiv(num_new_tokens);
  p.divP = make_fastdiv(static_cast<uint32_t>(p.P));
  if (s->head_dim == 64)
    return element_bytes == 1 ? mha_store_launch<64, true>(p, stream) : mha_store_launch<64, false>(p, stream);
  return element_bytes == 1 ? mha_store_launch<128, true>(p, stream) : mha_store_launch<128, false>(p, stream);
}

mla_status_t mla_mha_decode_workspace_bytes(uint32_t max_prompt_length, uint32_t max_cache_length, int32_t element_bytes,
                                            const mla_paged_shape_t* s, uint64_t* bytes) {
  if (!s || !bytes) return fail(MLA_ERR_INVALID_ARG, "shape and bytes must be non-NULL");
  *bytes = 0;
  mla_status_t st = check_mha_shape(s, 0, element_bytes);
  if (st != MLA_OK) return st;
  MhaPlan m{};                                           // what it refuses does not depend on the device
  st = mha_plan(s, max_prompt_length, max_cache_length, element_bytes, 1, &m);
  if (st != MLA_OK || s->batch == 0) return st;
  int sms = 0;
  unsigned int* status = nullptr;
  st = cache_device(&sms, &status);
  if (st != MLA_OK) return st;
  st = mha_plan(s, max_prompt_length, max_cache_length, element_bytes, sms, &m);
  if (st == MLA_OK) *bytes = m.total;
  return st;
}

mla_status_t mla_mha_decode_paged(const void* q, const void* blocks, const float* scales, const uint32_t* cache_lengths,
                                  const uint32_t* lookup_table, const uint32_t* scales_lookup_table,
                                  uint32_t max_prompt_length, uint32_t max_cache_length, uint32_t layer_idx,
                                  float softmax_scale, int32_t element_bytes, const mla_paged_shape_t* s, void* out,
                                  float* lse, void* workspace, uint64_t workspace_bytes, cudaStream_t stream) {
  mla_status_t st = check_mha(s, layer_idx, element_bytes, blocks, scales, cache_lengths, lookup_table);
  if (st != MLA_OK) return st;
  if (!q || !out) return fail(MLA_ERR_INVALID_ARG, "q and out must be non-NULL");
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace))
    return fail(MLA_ERR_INVALID_ARG, "q, out and workspace must be 16-byte aligned");
  if (!aligned4(lse)) return fail(MLA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if (!(softmax_scale == softmax_scale)) return fail(MLA_ERR_INVALID_ARG, "softmax_scale is NaN");
  MhaPlan m{};
  if (s->batch == 0) return mha_plan(s, max_prompt_length, max_cache_length, element_bytes, 1, &m);
  const uint64_t q_bytes = 2ull * s->batch * max_prompt_length * s->num_q_heads * s->head_dim;
  if (overlap(q, q_bytes, out, q_bytes)) return fail(MLA_ERR_INVALID_ARG, "out must not be q, nor overlap it");
  int sms = 0;
  unsigned int* status = nullptr;
  st = cache_device(&sms, &status);
  if (st != MLA_OK) return st;
  st = mha_plan(s, max_prompt_length, max_cache_length, element_bytes, sms, &m);
  if (st != MLA_OK) return st;
  if (m.total > 0 && (!workspace || workspace_bytes < m.total))
    return fail(MLA_ERR_WORKSPACE, "the call needs a workspace of %llu bytes (mla_mha_decode_workspace_bytes)",
                static_cast<unsigned long long>(m.total));
  mla::MhaParams p{};
  const uint64_t rows = static_cast<uint64_t>(s->num_blocks) * s->kv_dim * s->num_layers * s->page_size;
  const int head_bytes = s->head_dim * element_bytes, col = head_bytes < 128 ? head_bytes : 128;
  st = make_row_map(&p.tmap, blocks, rows, static_cast<uint64_t>(s->num_kv_heads) * head_bytes, col,
                    s->num_kv_heads * (head_bytes / col), m.box_rows,
                    m.hg * (head_bytes / col));
  if (st != MLA_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.scales = scales;
  p.cache_lengths = cache_lengths;
  p.lut = lookup_table;
  p.slut = scales_lookup_table ? scales_lookup_table : lookup_table;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  if (m.total > 0) {
    char* w = static_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(w);
    p.part_lse = reinterpret_cast<float*>(w + m.part_lse_off);
    p.desc = reinterpret_cast<int4*>(w + m.desc_off);
  }
  p.status = status;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    p.wait_limit_ns = g_wait_limit_ns;
  }
  p.B = s->batch;
  p.T = static_cast<int>(max_prompt_length);
  p.H = s->num_q_heads;
  p.HKV = s->num_kv_heads;
  p.R = m.R;
  p.P = s->page_size;
  p.KVD = s->kv_dim;
  p.NL = s->num_layers;
  p.layer = static_cast<int>(layer_idx);
  p.NB = s->num_blocks;
  p.NSB = s->num_scale_blocks;
  p.max_pages = s->max_pages;
  p.max_cache_length = max_cache_length;
  p.hg = m.hg;
  p.mt = m.mt;
  p.kw = m.kw;
  p.row_tile = 8 * m.nr;
  p.head_groups = m.head_groups;
  p.row_groups = m.row_groups;
  p.tile = m.tile;
  p.box_rows = m.box_rows;
  while ((1 << p.box_shift) < m.box_rows) ++p.box_shift;
  p.stages = m.stages;
  p.plane_bytes = m.plane_bytes;
  p.stage_bytes = m.stage_bytes;
  p.one_item = m.one_item;
  p.divP = make_fastdiv(static_cast<uint32_t>(p.P));
  p.divG = make_fastdiv(static_cast<uint32_t>(s->num_q_heads / s->num_kv_heads));
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  if (s->head_dim == 64)
    return element_bytes == 1 ? mha_launch<64, true>(p, m, stream) : mha_launch<64, false>(p, m, stream);
  return element_bytes == 1 ? mha_launch<128, true>(p, m, stream) : mha_launch<128, false>(p, m, stream);
}

}  // extern "C"
