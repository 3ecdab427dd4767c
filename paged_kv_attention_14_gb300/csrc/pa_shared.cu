// pa_shared.cu -- host side of pa_decode_shared: workspace layout and the
// launches (pa_shared_kernels.cuh has the kernels and their design).
#include "pa_host_cache.h"
#include "pa_shared_kernels.cuh"

namespace pa {

namespace {

constexpr size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct Layout {
  size_t axis, groups, seqs, starts, pre_o, pre_lse, own_o, own_lse, cut_o, cut_lse, sums, total;
};

// Sequences of a tile: what the largest group needs, up to the kernel's rows
int tile_seqs_of(const pa_kv_desc &d, int32_t max_group_size) {
  const int cap = shd::MAXROWS / (d.num_q_heads / d.num_kv_heads);
  return max_group_size < 1 ? 1 : max_group_size > cap ? cap : max_group_size;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn enc = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return enc;
}

// The cache as TMA sees it.  8-bit: rows of (block, kv head, token) triples, a
// box is the 16 rows of one block and kv head as they are (they are widened).
// 16-bit: the rows in groups of 8, each row in halves of 64 columns, a box is
// a block's two groups as [group][half][8 rows][128 B] (128-byte swizzle),
// one copy of 4 KB at head_dim 128 where plain rows would take one per half.
bool make_map(CUtensorMap *map, const void *base, const pa_kv_desc &d) {
  const bool kv8 = d.kv_dtype == PA_KV_FP8_E4M3 || d.kv_dtype == PA_KV_FP8_E5M2;
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t D = d.head_dim, rows = static_cast<cuuint64_t>(d.num_blocks) * d.num_kv_heads * 16;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  if (kv8) {
    const cuuint64_t dims[2] = {D, rows}, strides[1] = {D};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(D), 16};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[4] = {64, 8, D / 64, rows / 8}, strides[3] = {D * 2, 128, D * 16};
  const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(D / 64), 2};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q: rows as [sequence][half][head][64 columns], a box is a half of one kv
// head's rows of `seqs` sequences, [sequence][head][128 B].
bool make_q_map(CUtensorMap *map, const void *q, const pa_kv_desc &d, int32_t num_seqs, uint32_t seqs) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t D = d.head_dim, Hq = d.num_q_heads;
  const cuuint64_t dims[4] = {64, Hq, D / 64, static_cast<cuuint64_t>(num_seqs)}, strides[3] = {D * 2, 128, Hq * D * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(Hq / d.num_kv_heads), 1, seqs}, estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Layout layout(const pa_kv_desc &d, int32_t num_seqs, int32_t num_groups, int32_t max_group_size, int ctas) {
  Layout w;
  const size_t rows = static_cast<size_t>(num_seqs) * d.num_q_heads;
  const size_t cut = static_cast<size_t>(ctas) * 2 * tile_seqs_of(d, max_group_size) * (d.num_q_heads / d.num_kv_heads);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += up256(bytes);
    return x;
  };
  // (the parts first: the join counts their places from cut_o)
  w.cut_o = take(cut * d.head_dim * 4);
  w.pre_o = take(rows * d.head_dim * 4);
  w.own_o = take(rows * d.head_dim * 4);
  w.cut_lse = take(cut * 4);
  w.pre_lse = take(rows * 4);
  w.own_lse = take(rows * 4);
  w.axis = take(sizeof(shd::Axis));
  w.groups = take(sizeof(shd::GroupInfo) * num_groups);
  w.seqs = take(sizeof(shd::SeqInfo) * num_seqs);
  w.starts = take(sizeof(shd::CtaStart) * ctas);
  w.sums = take(static_cast<size_t>(ctas) * shd::MAXROWS * d.head_dim * 4);
  w.total = at;
  return w;
}

}  // namespace

size_t shared_workspace_bytes(const pa_kv_desc &d, int32_t num_seqs, int32_t num_groups, int32_t max_group_size) {
  return layout(d, num_seqs, num_groups, max_group_size, device_sm_count()).total;
}

cudaError_t launch_shared(const pa_kv_desc &d, float *out, float *lse, const void *q, const void *k_cache,
                          const void *v_cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                          const int32_t *context_lens, int32_t num_seqs, const int32_t *group_start,
                          const int32_t *prefix_lens, int32_t num_groups, int32_t max_group_size, float scale,
                          void *workspace, cudaStream_t stream) {
  const bool b16 = d.kv_dtype == PA_KV_BF16 || d.kv_dtype == PA_KV_F16;
  const shd::KernelInfo k = b16 ? shd::pick_attend_16(d.head_dim, d.kv_dtype) : shd::pick_attend_8(d.head_dim, d.kv_dtype);
  if (prepare_kernel(k.fn, k.threads, k.smem) < 1) return cudaErrorInvalidConfiguration;
  shd::Args a;
  memset(&a, 0, sizeof a);
  const int seqs = tile_seqs_of(d, max_group_size);
  if (!make_map(&a.kmap, k_cache, d) || !make_map(&a.vmap, v_cache, d) ||
      !make_q_map(&a.qmap, q, d, num_seqs, 1) ||
      (seqs >= shd::kQBox && !make_q_map(&a.qmap_box, q, d, num_seqs, shd::kQBox)))
    return cudaErrorInvalidValue;
  a.ctas = device_sm_count();
  a.narrow_units = b16 ? shd::kNarrowUnits16 : shd::kNarrowUnits8;
  a.wide_units = shd::kWideUnits;
  const Layout w = layout(d, num_seqs, num_groups, max_group_size, a.ctas);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.out = out;
  a.lse = lse;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.group_start = group_start;
  a.prefix_lens = prefix_lens;
  a.max_blocks = max_blocks_per_seq;
  a.num_seqs = num_seqs;
  a.num_groups = num_groups;
  a.num_kv = d.num_kv_heads;
  a.num_q = d.num_q_heads;
  a.g = d.num_q_heads / d.num_kv_heads;
  a.tile_seqs = seqs;
  a.slot_rows = a.tile_seqs * a.g;
  const float ks = (!b16 && d.k_scale != 0.f) ? d.k_scale : 1.f;
  a.qscale = scale * ks * shd::kLog2e;
  a.qscale0 = scale * shd::kLog2e;
  a.vscale = (!b16 && d.v_scale != 0.f) ? d.v_scale : 1.f;
  a.k_scales = b16 ? nullptr : d.k_scales;
  a.v_scales = b16 ? nullptr : d.v_scales;
  a.num_blocks = d.num_blocks;
  a.checked = d.check_indices;
  const TestHooks hooks = test_hooks();
  a.stall = hooks.stall;
  a.wait_ns = static_cast<uint32_t>(hooks.wait_ns < 0x7fffffffull ? hooks.wait_ns : 0x7fffffffull);
  a.err = d.error_word;
  a.axis = reinterpret_cast<shd::Axis *>(ws + w.axis);
  a.groups = reinterpret_cast<shd::GroupInfo *>(ws + w.groups);
  a.seqs = reinterpret_cast<shd::SeqInfo *>(ws + w.seqs);
  a.starts = reinterpret_cast<shd::CtaStart *>(ws + w.starts);
  a.pre_o = reinterpret_cast<float *>(ws + w.pre_o);
  a.pre_lse = reinterpret_cast<float *>(ws + w.pre_lse);
  a.own_o = reinterpret_cast<float *>(ws + w.own_o);
  a.own_lse = reinterpret_cast<float *>(ws + w.own_lse);
  a.cut_o = reinterpret_cast<float *>(ws + w.cut_o);
  a.cut_lse = reinterpret_cast<float *>(ws + w.cut_lse);
  a.sums = reinterpret_cast<float *>(ws + w.sums);

  // each launch overlaps the tail of the one before it (programmatic
  // dependent launch); every kernel waits for that one's writes first
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  void *args[] = {&a};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(shd::PLAN_THREADS);
  cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&shd::shared_plan_kernel), args);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(k.threads);
  cfg.dynamicSmemBytes = k.smem;
  e = cudaLaunchKernelExC(&cfg, k.fn, args);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(num_seqs), static_cast<unsigned>((d.num_q_heads + 1) / 2 * (d.head_dim / 64) + 1) / 2);
  cfg.blockDim = dim3(64);
  cfg.dynamicSmemBytes = 0;
  const void *join = d.head_dim == 64 ? reinterpret_cast<const void *>(&shd::shared_join_kernel<64>)
                                      : reinterpret_cast<const void *>(&shd::shared_join_kernel<128>);
  return cudaLaunchKernelExC(&cfg, join, args);
}

}  // namespace pa
