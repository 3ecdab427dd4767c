// pa_shared.cu -- pa_decode_shared: the plan, the join, workspace layout and
// the launches (pa_shared_kernels.cuh has the attention and the design).
#include <string.h>

#include "pa_host_cache.h"
#include "pa_shared_kernels.cuh"

namespace pa {
namespace shd {

// ------------------------------------------------------------------ planning

constexpr int PLAN_THREADS = 512;
constexpr int PLAN_CAP = 512;  // sequences / groups planned in shared memory

// n / d: 32 bits where they do (a 64-bit division is some 100 instructions)
static __device__ __noinline__ long long divide64(long long n, long long d) { return n / d; }
__device__ __forceinline__ long long divide(long long n, long long d) {
  if (((n | d) >> 31) == 0) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
  return divide64(n, d);
}

// Units of an item of nb blocks.
__device__ __forceinline__ int item_units(int nb, int extra) { return nb > 0 ? nb + extra : 0; }

// Exclusive prefix sums of two values over the CTA's threads; total gets the sums.
__device__ __forceinline__ void scan2(long long (&v)[2], long long (&total)[2], long long (*s_warp)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long in[2] = {v[0], v[1]};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long t = __shfl_up_sync(0xffffffffu, in[i], o);
      if (lane >= o) in[i] += t;
    }
  __syncthreads();  // s_warp may still be read from the last call
  if (lane == 31) {
    s_warp[warp][0] = in[0];
    s_warp[warp][1] = in[1];
  }
  __syncthreads();
  long long before[2] = {0, 0}, sum[2] = {0, 0};
#pragma unroll 4
  for (int w = 0; w < PLAN_THREADS / 32; ++w)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long x = s_warp[w][i];
      if (w < warp) before[i] += x;
      sum[i] += x;
    }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    total[i] = sum[i];
    v[i] = before[i] + in[i] - v[i];
  }
}

// The last entry whose base is <= u (entries without work share the base of
// the next one, so it is the entry that holds unit u).
template <class T>
__device__ __forceinline__ int find_base(const T *v, int n, long long u) {
  int lo = 0, hi = n - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (v[mid].base <= u)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The plan, by one CTA: a thread per group and per sequence (in rounds of
// PLAN_THREADS).  Up to PLAN_CAP of each are worked on in shared memory.
static __global__ void __launch_bounds__(PLAN_THREADS) shared_plan_kernel(const __grid_constant__ Args a) {
  __shared__ long long s_warp[PLAN_THREADS / 32][2];
  __shared__ SeqInfo s_seqs[PLAN_CAP];
  __shared__ GroupInfo s_groups[PLAN_CAP];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int S = a.num_seqs, G = a.num_groups;
  const int cap = min(a.max_blocks, 0x7ffffff) * 16;
  const bool small = S <= PLAN_CAP && G <= PLAN_CAP;
  SeqInfo *seqs = small ? s_seqs : a.seqs;
  GroupInfo *groups = small ? s_groups : a.groups;
  // the first round's lengths are in flight beside the groups'
  int len0 = tid < S ? __ldg(a.context_lens + tid) : 0;
#pragma unroll 1
  for (int j = tid; j < G; j += PLAN_THREADS) {
    const int r0 = __ldg(a.group_start + j), r1 = __ldg(a.group_start + j + 1), r2 = __ldg(a.prefix_lens + j);
    // whatever the arrays hold, no access leaves the batch
    GroupInfo q = {};
    q.first = min(max(r0, 0), S);
    q.n = min(max(r1, q.first), S) - q.first;
    if (a.checked && (r0 != q.first || r1 != q.first + q.n || r2 < 0 || r2 > cap))
      report_error(a.err, nullptr, kErrBadIndex);
    q.P = q.n < 2 ? 0 : min(max(r2, 0), cap) & ~15;  // a group of one shares with nobody
    q.row = 0x7fffffff;
    // tiles of equal numbers of sequences
    const int t = max(1, (q.n + a.tile_seqs - 1) / a.tile_seqs);
    q.tile_seqs = max(1, (q.n + t - 1) / t);
    q.tiles = (q.n + q.tile_seqs - 1) / q.tile_seqs;
    q.extra = is_narrow(q.tile_seqs * a.g) ? a.narrow_units : a.wide_units;
    groups[j] = q;
  }
  __syncthreads();
  // each sequence's group (a binary search over the first sequences), and
  // whether it holds the group's whole prefix
#pragma unroll 1
  for (int s = tid; s < S; s += PLAN_THREADS) {
    int L = s == tid ? len0 : __ldg(a.context_lens + s);
    if (a.checked) L = checked_len(L, cap, a.err, nullptr);
    SeqInfo q = {};
    q.len = min(max(L, 0), cap);
    int lo = 0, hi = G - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (groups[mid].first <= s)
        lo = mid;
      else
        hi = mid - 1;
    }
    q.group = G > 0 && s >= groups[lo].first && s < groups[lo].first + groups[lo].n ? lo : -1;
    if (q.group >= 0 && groups[lo].P > 0 && q.len >= groups[lo].P) {
      q.fb = groups[lo].P >> 4;
      atomicMin(&groups[lo].row, s);
    }
    q.nb = max(0, ((q.len + 15) >> 4) - q.fb);
    seqs[s] = q;
  }
  __syncthreads();
  // places on the axis: prefix items, then own parts
  long long at[2] = {0, 0};
#pragma unroll 1
  for (int i0 = 0; i0 < max(S, G); i0 += PLAN_THREADS) {
    const int i = i0 + tid;
    long long v[2] = {0, 0}, sum[2];
    if (i < G) {
      const int nb = groups[i].row != 0x7fffffff ? groups[i].P >> 4 : 0;
      groups[i].nb = nb;
      v[0] = static_cast<long long>(item_units(nb, groups[i].extra)) * (groups[i].tiles * a.num_kv);
    }
    if (i < S) v[1] = static_cast<long long>(item_units(seqs[i].nb, a.narrow_units)) * a.num_kv;
    scan2(v, sum, s_warp);
    if (i < G) groups[i].base = at[0] + v[0];
    if (i < S) seqs[i].base = at[1] + v[1];
    at[0] += sum[0];
    at[1] += sum[1];
  }
  const long long own = at[0], U = at[0] + at[1];  // the own parts' first unit, and the end
  const long long per = max(divide(U + a.ctas - 1, a.ctas), static_cast<long long>((is_narrow(a.slot_rows) ? a.narrow_units : a.wide_units) + BPT));
  if (tid == 0) {
    const uint32_t magic = U >> 32 ? 0u : static_cast<uint32_t>(divide64(1LL << 32, per));
    *a.axis = Axis{U, per, magic, {0, 0, 0}};
  }
  __syncthreads();
  // each CTA's first item
#pragma unroll 1
  for (int c = tid; c < a.ctas; c += PLAN_THREADS) {
    const long long u = c * per;
    CtaStart st = {2, 0, 0, 0};
    if (u < U) {
      st.kind = u < own ? 0 : 1;
      st.idx = st.kind == 0 ? find_base(groups, G, u) : find_base(seqs, S, u - own);
      const int n = st.kind == 0 ? item_units(groups[st.idx].nb, groups[st.idx].extra)
                                 : item_units(seqs[st.idx].nb, a.narrow_units);
      const long long r = st.kind == 0 ? u - groups[st.idx].base : u - own - seqs[st.idx].base;
      st.sub = static_cast<int>(divide(r, n));
      st.off = static_cast<int>(r - static_cast<long long>(st.sub) * n);
    }
    a.starts[c] = st;
  }
  if (!small) __syncthreads();  // the searches above read what is completed below
#pragma unroll 1
  for (int s = tid; s < S; s += PLAN_THREADS) {
    SeqInfo q = seqs[s];
    q.base += own;
    if (q.fb > 0) {
      const GroupInfo &gi = groups[q.group];
      const int i = s - gi.first, tile = i / gi.tile_seqs, t0 = tile * gi.tile_seqs;
      q.pnb = gi.nb;
      q.pbase = gi.base + static_cast<long long>(tile * a.num_kv) * item_units(gi.nb, gi.extra);
      q.prow = static_cast<short>((i - t0) * a.g);
      q.prows = static_cast<short>(min(gi.tile_seqs, gi.n - t0) * a.g);
      q.pextra = gi.extra;
      q.pseq = gi.first + t0;
    }
    a.seqs[s] = q;
  }
  if (small)
#pragma unroll 1
    for (int j = tid; j < G; j += PLAN_THREADS) a.groups[j] = s_groups[j];
}

// --------------------------------------------------------------------- join

// The CTA that holds unit u of the axis.  With 32 bits the product's high word
// is the quotient or one less.
__device__ __forceinline__ int axis_cta(long long u, const Axis &x) {
  if (x.magic == 0) return static_cast<int>(divide64(u, x.per));
  const uint32_t n = static_cast<uint32_t>(u), d = static_cast<uint32_t>(x.per), q = __umulhi(n, x.magic);
  return static_cast<int>(q + (n - q * d >= d ? 1u : 0u));
}

// 64 columns of two rows (sequence, head) per warp, a row on the lanes of one
// parity, 16 bytes of it a lane: two neighbouring rows of a tile fill a
// 32-byte sector of its [4 columns][row] parts.  Each row's pieces are weighed
// by their log-sum-exps.  Rows that the attention wrote itself (one uncut
// part) are left alone.  What bounds it is latency, so the loads come in two
// dependent rounds: the sequence's record, then 16 pieces' log-sum-exps and
// columns at once.  Places in the workspace are counted in 16 bytes from cut_o.
template <int D>
__global__ void __launch_bounds__(64) shared_join_kernel(const __grid_constant__ Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x;
  constexpr int C4 = D / 4, PARTS = D / 64;  // warps of a pair of rows
  const int w0 = blockIdx.y * 2 + (threadIdx.x >> 5);
  int h = w0 / PARTS * 2 + (lane & 1);
  // every lane stays for the shuffles
  bool mine = h < a.num_q;
  if (!mine) h = a.num_q - 1;
  const int64_t row = static_cast<int64_t>(s) * a.num_q + h;
  const int l = lane >> 1, c0 = l + 16 * (w0 % PARTS);  // this lane's columns: 4 c0 ..
  const SeqInfo q = a.seqs[s];
  const Axis ax = *a.axis;
  const int kvh = static_cast<int>(static_cast<uint32_t>(h) / static_cast<uint32_t>(a.g)), hg = h - kvh * a.g;
  // the pieces of the prefix part (0) and of the own part (1): piece i of a
  // part is CTA c1 + i's slot (1 where the item begins inside that CTA's
  // range), or the part's own place if one CTA holds all its blocks
  int c1[2], np[2], s0[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int nb = p ? q.nb : q.pnb, extra = p ? a.narrow_units : q.pextra, n = nb + extra;
    const long long u0 = (p ? q.base : q.pbase) + static_cast<long long>(kvh) * n;
    int c = axis_cta(u0, ax);
    if ((c + 1) * ax.per - u0 <= extra) ++c;  // that CTA's range holds none of its blocks
    c1[p] = c;
    np[p] = nb > 0 ? axis_cta(u0 + n - 1, ax) - c + 1 : 0;
    s0[p] = u0 > c * ax.per;
  }
  if (q.fb == 0 && np[1] == 1) mine = false;
  const int n = mine ? np[0] + np[1] : 0;
  const float4 *base = reinterpret_cast<const float4 *>(a.cut_o);
  const int64_t p_at = static_cast<int64_t>(q.pseq) * a.num_q + static_cast<int64_t>(kvh) * q.prows;  // its tile
  float M = -INFINITY, W = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int most = max(n, __shfl_xor_sync(0xffffffffu, n, 1));
#pragma unroll 1
  for (int i0 = 0; i0 < most; i0 += 16) {
    // each of a row's 16 lanes finds a piece's place (past the row's pieces:
    // the first one's again, with no weight)
    const bool there = i0 + l < n;
    const int i = there ? i0 + l : 0;
    const bool pre = i < np[0];
    int at = 0, stride = 0;
    float v = -INFINITY;
    if (n > 0) {
      const float *x;
      if (pre ? np[0] == 1 : np[1] == 1) {
        const int64_t r = pre ? p_at : row;
        at = static_cast<int>(reinterpret_cast<const float4 *>(pre ? a.pre_o : a.own_o) - base) +
             static_cast<int>(r) * C4 + (pre ? q.prow + hg : 0);
        stride = pre ? q.prows : 1;
        x = (pre ? a.pre_lse + q.prow + hg : a.own_lse) + r;
      } else {
        const int k = pre ? i : i - np[0], r = pre ? q.prow + hg : hg;
        const int slot = ((c1[pre ? 0 : 1] + k) * 2 + (k == 0 ? s0[pre ? 0 : 1] : 0)) * a.slot_rows;
        at = slot * C4 + r;
        stride = a.slot_rows;
        x = a.cut_lse + slot + r;
      }
      if (there) v = __ldcg(x);
    }
    // all the pieces' columns, four pieces to a branch
    float4 y[16];
#pragma unroll
    for (int k0 = 0; k0 < 16; k0 += 4) {
      if (i0 + k0 >= most) break;
#pragma unroll
      for (int k = k0; k < k0 + 4; ++k) {
        const int from = 2 * k + (lane & 1);
        const int ai = __shfl_sync(0xffffffffu, at, from), st = __shfl_sync(0xffffffffu, stride, from);
        y[k] = __ldcg(base + ai + c0 * st);
      }
    }
    float mn = fmaxf(M, v);
#pragma unroll
    for (int b = 2; b < 32; b <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, b));
    const float f = M == mn ? 1.f : ex2_approx(M - mn);
    const float w = v == -INFINITY ? 0.f : ex2_approx(v - mn);  // a NaN stays one
    M = mn;
    float ws = w;
#pragma unroll
    for (int b = 2; b < 32; b <<= 1) ws += __shfl_xor_sync(0xffffffffu, ws, b);
    W = W * f + ws;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int k0 = 0; k0 < 16; k0 += 4) {
      if (i0 + k0 >= most) break;
#pragma unroll
      for (int k = k0; k < k0 + 4; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, 2 * k + (lane & 1));
        acc.x += wk * y[k].x;
        acc.y += wk * y[k].y;
        acc.z += wk * y[k].z;
        acc.w += wk * y[k].w;
      }
    }
  }
  if (!mine) return;
  const float inv = (a.v_scales ? __ldg(a.v_scales + kvh) : a.vscale) / W;
  *reinterpret_cast<float4 *>(a.out + row * D + 4 * c0) =
      W == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
               : make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (a.lse && c0 == 0) a.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * kLn2;
}

}  // namespace shd

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
