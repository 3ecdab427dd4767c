// pa_rope.cu -- per-head RMS norm of queries and keys with their position
// rotation in one pass, and the same pass writing the keys and values into
// the paged cache.
//
// For a row x of head_dim D (one token, one head) with weight w:
//   y_i = x_i * rsqrt(mean_j x_j^2 + eps) * w_i            (y = x without a weight)
// and for the first rd = rotary_dim dims, with c, s the cosine and sine of
// the token's position for frequency i (a row of the caller's fp32 table,
// [max_position][rd] = rd / 2 cosines, then rd / 2 sines):
//   half split:   y_i' = y_i c_i - y_{i+rd/2} s_i,   y_{i+rd/2}' = y_{i+rd/2} c_i + y_i s_i
//   interleaved:  the same with the pairs (2i, 2i+1).
// The sum of squares, the norm and the rotation are fp32; each result is
// rounded once, to the activation type or to the 8-bit cache type (a key of
// an 8-bit cache is encoded from its fp32 value, not from a 16-bit copy).
//
// What bounds it: every element is read once and written once (4 bytes of a
// 16-bit row's element) for about ten operations, so HBM for long chunks and
// the launch for a decode step's few rows.
//
// Layout: a row belongs to D / 16 neighbouring lanes, each holding two
// 16-byte chunks that rotate with each other (half split: chunk l and chunk
// l + rd / 16), so a rotation never leaves its lane and the norm takes
// log2(D / 16) shuffles.
#include "pa_device.cuh"
#include "pa_host_cache.h"
#include "pa_internal.h"

namespace pa {

namespace {

struct RopeArgs {
  const uint16_t *q;
  const uint16_t *k;
  const uint16_t *v;
  int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
  uint16_t *q_out;                       // dense
  uint16_t *k_out;                       // dense (no cache)
  uint8_t *k_cache;
  uint8_t *v_cache;
  const int64_t *slots;
  const int32_t *positions;
  const float *table;
  const uint16_t *q_weight;
  const uint16_t *k_weight;
  const float *k_scales;
  const float *v_scales;
  float k_scale, v_scale, eps;
  int num_q, num_kv;  // query heads (0: no queries), kv heads (0: no keys)
  int heads;          // rows of a token: num_q + num_kv (+ num_kv values)
  int max_position;
  int rd;
  int64_t total;      // rows (few tokens), tokens (many)
  int64_t num_slots;
  int checked;
  int32_t *err;
};

// 8 values of the activation type (16-bit pairs) to fp32
template <int ACT>
__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo16<ACT>(w[i]);
    f[2 * i + 1] = hi16<ACT>(w[i]);
  }
}

template <int ACT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack16x2<ACT>(f[0], f[1]), pack16x2<ACT>(f[2], f[3]), pack16x2<ACT>(f[4], f[5]),
                    pack16x2<ACT>(f[6], f[7]));
}

// 8 values to 8 bytes of an 8-bit cache: x / s in fp32, then the cache
// write's rounding (nearest even, finite saturation)
template <int KVT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t lo = pack_fp8x2_satfinite<KVT>(__fdiv_rn(f[4 * i], s), __fdiv_rn(f[4 * i + 1], s));
    const uint16_t hi = pack_fp8x2_satfinite<KVT>(__fdiv_rn(f[4 * i + 2], s), __fdiv_rn(f[4 * i + 3], s));
    r[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint2(r[0], r[1]);
}

// A lane's share of a row: two chunks of 8 elements that rotate with each
// other, ca and cb, and for half split the 8 frequencies they share, for
// interleaved 4 of each.
template <int D, bool INTER>
struct Lane {
  static constexpr int LPR = D / 16;  // lanes of a row
  int ca, cb;
  bool rot;  // half split: lanes past rd / 16 hold unrotated dims
  __device__ __forceinline__ Lane(int l, int rd) {
    const int nr = rd / 16;
    rot = INTER || l < nr;
    ca = INTER ? l : (l < nr ? l : 2 * l);
    cb = INTER ? l + LPR : (l < nr ? l + nr : 2 * l + 1);
  }
  // the cosines and sines of a table row (1 and 0 past rd)
  __device__ __forceinline__ void angles(const float *row, int rd, float (&cs)[8], float (&sn)[8]) const {
    auto four = [&](float *dst, const float *src) { *reinterpret_cast<float4 *>(dst) = *reinterpret_cast<const float4 *>(src); };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
    if constexpr (INTER) {
      if (ca * 8 < rd) {
        four(cs, row + ca * 4);
        four(sn, row + rd / 2 + ca * 4);
      }
      if (cb * 8 < rd) {
        four(cs + 4, row + cb * 4);
        four(sn + 4, row + rd / 2 + cb * 4);
      }
    } else if (rot) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        four(cs + i, row + ca * 8 + i);
        four(sn + i, row + rd / 2 + ca * 8 + i);
      }
    }
  }
  __device__ __forceinline__ void rotate(float (&fa)[8], float (&fb)[8], const float (&cs)[8],
                                         const float (&sn)[8]) const {
    if constexpr (INTER) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a0 = fa[2 * e], a1 = fa[2 * e + 1], b0 = fb[2 * e], b1 = fb[2 * e + 1];
        fa[2 * e] = a0 * cs[e] - a1 * sn[e];
        fa[2 * e + 1] = a1 * cs[e] + a0 * sn[e];
        fb[2 * e] = b0 * cs[4 + e] - b1 * sn[4 + e];
        fb[2 * e + 1] = b1 * cs[4 + e] + b0 * sn[4 + e];
      }
    } else if (rot) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x0 = fa[e], x1 = fb[e];
        fa[e] = x0 * cs[e] - x1 * sn[e];
        fb[e] = x1 * cs[e] + x0 * sn[e];
      }
    }
  }
};

// rsqrt(mean square + eps) of a row over its lanes (all of the warp's lanes call it)
template <int D>
__device__ __forceinline__ float row_rsqrt(const float (&fa)[8], const float (&fb)[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss += fa[e] * fa[e] + fb[e] * fb[e];
#pragma unroll
  for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return rsqrtf(ss * (1.f / D) + eps);
}

// A finished row to where it goes: q_out or k_out, or the cache row of the
// token's slot (values as they came, xa and xb).
template <int D, int KVT, bool APPEND>
__device__ __forceinline__ void store_row(const RopeArgs &a, int64_t token, int h, int64_t slot, int ca, int cb,
                                          const float (&fa)[8], const float (&fb)[8], const uint4 &xa,
                                          const uint4 &xb) {
  constexpr int ACT = KVT == kKvF16 ? kKvF16 : kKvBf16;
  const bool is_q = h < a.num_q, is_v = APPEND && h >= a.num_q + a.num_kv;
  if (!APPEND || is_q) {
    uint16_t *dst = is_q ? a.q_out + (token * a.num_q + h) * D : a.k_out + (token * a.num_kv + h - a.num_q) * D;
    reinterpret_cast<uint4 *>(dst)[ca] = pack8<ACT>(fa);
    reinterpret_cast<uint4 *>(dst)[cb] = pack8<ACT>(fb);
  } else if (slot >= 0) {
    // cache row (slot / 16, kv head, slot % 16) of [num_blocks][num_kv_heads][16][D]
    const int kvh = h - a.num_q - (is_v ? a.num_kv : 0);
    const int64_t row = ((slot >> 4) * a.num_kv + kvh) * 16 + (slot & 15);
    uint8_t *cache = is_v ? a.v_cache : a.k_cache;
    if constexpr (kv16(KVT)) {
      uint4 *dst = reinterpret_cast<uint4 *>(cache + row * (2 * D));
      dst[ca] = is_v ? xa : pack8<ACT>(fa);  // values: bit copies
      dst[cb] = is_v ? xb : pack8<ACT>(fb);
    } else {
      const float *hs = is_v ? a.v_scales : a.k_scales;
      const float s = hs ? __ldg(hs + kvh) : (is_v ? a.v_scale : a.k_scale);
      uint2 *dst = reinterpret_cast<uint2 *>(cache + row * D);
      dst[ca] = encode8<KVT>(fa, s);
      dst[cb] = encode8<KVT>(fb, s);
    }
  }
}

// A token's position (0 in place of one out of range), and its cache slot
// (-1: none; with checked indices also for one out of range).  Checked, both
// are reported, but for the position of a padding token (one with a negative
// slot), which may be anything.
template <bool APPEND>
__device__ __forceinline__ int position_of(const RopeArgs &a, int64_t token, bool report) {
  const int pos = __ldg(a.positions + token);
  if (static_cast<uint32_t>(pos) < static_cast<uint32_t>(a.max_position)) return pos;
  if (a.checked && report && !(APPEND && __ldg(a.slots + token) < 0)) report_error(a.err, nullptr, kErrBadIndex);
  return 0;
}
__device__ __forceinline__ int64_t slot_of(const RopeArgs &a, int64_t token, bool report) {
  const int64_t slot = __ldg(a.slots + token);
  if (a.checked && slot >= a.num_slots) {
    if (report) report_error(a.err, nullptr, kErrBadIndex);
    return -1;
  }
  return slot;
}

// The kernel of few tokens: a row per D / 16 lanes, one pass.  One token's
// 40 rows take 2.1 us in a captured graph, the launch; 128 tokens of 48 heads
// 2.8 us.  KVT: the cache type (its activation type is fp16 for kKvF16, else
// bf16); APPEND: keys and values go to the cache.
template <int D, int KVT, bool APPEND, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  constexpr int ACT = KVT == kKvF16 ? kKvF16 : kKvBf16;
  constexpr int LPR = D / 16;
  // a programmatic dependent launched after this one waits for these writes;
  // this one waits for the writes of the kernel before it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  // every lane stays for the shuffles; lanes past the end touch no memory
  const bool live = unit < a.total;
  const int64_t token = !live             ? 0
                        : a.total >> 32 ? unit / a.heads
                                        : static_cast<uint32_t>(unit) / static_cast<uint32_t>(a.heads);
  const int h = live ? static_cast<int>(unit - token * a.heads) : 0;
  const Lane<D, INTER> ln(l, a.rd);
  const bool is_q = h < a.num_q, is_v = APPEND && h >= a.num_q + a.num_kv;
  uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
  float cs[8], sn[8];
  int64_t slot = -1;
  if (live) {
    const uint16_t *src = is_q  ? a.q + token * a.q_stride + static_cast<int64_t>(h) * D
                          : is_v ? a.v + token * a.v_stride + static_cast<int64_t>(h - a.num_q - a.num_kv) * D
                                 : a.k + token * a.k_stride + static_cast<int64_t>(h - a.num_q) * D;
    xa = reinterpret_cast<const uint4 *>(src)[ln.ca];
    xb = reinterpret_cast<const uint4 *>(src)[ln.cb];
    ln.angles(a.table + static_cast<int64_t>(position_of<APPEND>(a, token, l == 0)) * a.rd, a.rd, cs, sn);
    if constexpr (APPEND) slot = slot_of(a, token, l == 0);
  }
  float fa[8], fb[8];
  unpack8<ACT>(xa, fa);
  unpack8<ACT>(xb, fb);
  if (a.q_weight != nullptr || a.k_weight != nullptr) {  // the same for every lane: all reach the shuffles
    const float r = row_rsqrt<D>(fa, fb, a.eps);
    const uint16_t *w = is_q ? a.q_weight : a.k_weight;
    if (w != nullptr && !is_v) {
      float wa[8], wb[8];
      unpack8<ACT>(__ldg(reinterpret_cast<const uint4 *>(w) + ln.ca), wa);
      unpack8<ACT>(__ldg(reinterpret_cast<const uint4 *>(w) + ln.cb), wb);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        fa[e] *= r * wa[e];
        fb[e] *= r * wb[e];
      }
    }
  }
  if (!live) return;
  if (!is_v) ln.rotate(fa, fb, cs, sn);
  store_row<D, KVT, APPEND>(a, token, h, slot, ln.ca, ln.cb, fa, fb, xa, xb);
}

// The kernel of many tokens, one persistent CTA per SM: a producer warp brings
// the tokens' rows (one bulk copy each of its queries, keys and values, which
// lie together) and their table rows into a ring of stages, and 20 warps work
// through a stage's rows, so that some 200 KB per SM are in flight whatever
// registers the arithmetic takes.  16381 tokens of 32 q / 8 kv heads with
// norms: the kernel above 77.8 us, this one 57.4 us (5,990 GB/s, 90% of the
// measured copy rate) with 20 warps, 63.5 with 16, 60.3 with 28.  8192 tokens
// of 40 q / 8 kv heads into an E4M3 cache: 55.3 and 42.6 us; there the exact
// divisions by the scale still show.
constexpr int kStreamWarps = 20;

struct StreamPlan {
  int tokens;      // of a stage
  int stages;
  int token_bytes; // a token's rows and table row
  int blocks;      // stages of work
  unsigned long long wait_ns;
};

template <int D, int KVT, bool APPEND, bool INTER>
__global__ void __launch_bounds__((kStreamWarps + 1) * 32, 1) rope_stream_kernel(const RopeArgs a, const StreamPlan p) {
  constexpr int ACT = KVT == kKvF16 ? kKvF16 : kKvBf16;
  constexpr int LPR = D / 16;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint64_t full[16], empty[16];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kStreamWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row_bytes = D * 2, q_bytes = a.num_q * row_bytes, kv_bytes = a.num_kv * row_bytes;
  const int tab_at = a.heads * row_bytes;  // a token: q, k (and v) rows, then its table row
  const int64_t num_tokens = a.total;
  int st = 0;
  uint32_t par = 0;
  if (warp == kStreamWarps) {
    // ---- producer: a lane per (token, part)
    bool ok = true;
    int issued = 0;
    for (int b = blockIdx.x; b < p.blocks; b += gridDim.x) {
      const int64_t t0 = static_cast<int64_t>(b) * p.tokens;
      const int n = static_cast<int>(min(static_cast<int64_t>(p.tokens), num_tokens - t0));
      const int i = lane >> 2, part = lane & 3;  // up to 8 tokens x (q, k, v, table)
      int pos = 0;
      if (i < n && part == 3) pos = position_of<APPEND>(a, t0 + i, true);
      if (!mbar_wait(&empty[st], par ^ 1, p.wait_ns)) {
        ok = false;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[st], n * p.token_bytes);
      __syncwarp();
      if (i < n) {
        uint8_t *dst = ring + static_cast<size_t>(st) * p.tokens * p.token_bytes + i * p.token_bytes;
        const int64_t t = t0 + i;
        if (part == 0 && q_bytes) bulk_g2s(dst, a.q + t * a.q_stride, q_bytes, &full[st]);
        if (part == 1 && kv_bytes) bulk_g2s(dst + q_bytes, a.k + t * a.k_stride, kv_bytes, &full[st]);
        if (APPEND && part == 2) bulk_g2s(dst + q_bytes + kv_bytes, a.v + t * a.v_stride, kv_bytes, &full[st]);
        if (part == 3) bulk_g2s(dst + tab_at, a.table + static_cast<int64_t>(pos) * a.rd, a.rd * 4, &full[st]);
      }
      ++issued;
      if (++st == p.stages) {
        st = 0;
        par ^= 1;
      }
    }
    if (!ok) {
      if (lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
      // the copies already issued land before the CTA can exit
      for (int k = 1; k <= min(issued, p.stages); ++k) {
        const int s2 = st - k < 0 ? st - k + p.stages : st - k;
        mbar_wait(&full[s2], st - k < 0 ? par ^ 1 : par, p.wait_ns);
      }
    }
    return;
  }
  // ---- consumers: a lane keeps its chunks, and with them its norm weights
  const int l = threadIdx.x % LPR;
  const Lane<D, INTER> ln(l, a.rd);
  constexpr int ROWS = kStreamWarps * 32 / LPR;  // rows at once
  for (int b = blockIdx.x; b < p.blocks; b += gridDim.x) {
    const int64_t t0 = static_cast<int64_t>(b) * p.tokens;
    const int n = static_cast<int>(min(static_cast<int64_t>(p.tokens), num_tokens - t0));
    if (!mbar_wait(&full[st], par, p.wait_ns)) {
      if (lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
      return;
    }
    const uint8_t *stage = ring + static_cast<size_t>(st) * p.tokens * p.token_bytes;
    const int rows = n * a.heads;
    int i = (threadIdx.x / LPR) / a.heads, h = (threadIdx.x / LPR) - i * a.heads;
    // (whole warps go round: every lane reaches the shuffles)
    for (int r0 = (warp * 32) / LPR; r0 < rows; r0 += ROWS) {
      const bool live = i < n;
      const bool is_q = h < a.num_q, is_v = APPEND && h >= a.num_q + a.num_kv;
      uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
      const uint8_t *tok = stage + i * p.token_bytes;
      if (live) {
        const uint4 *src = reinterpret_cast<const uint4 *>(tok + h * row_bytes);
        xa = src[ln.ca];
        xb = src[ln.cb];
      }
      float fa[8], fb[8];
      unpack8<ACT>(xa, fa);
      unpack8<ACT>(xb, fb);
      if (a.q_weight != nullptr || a.k_weight != nullptr) {
        const float r = row_rsqrt<D>(fa, fb, a.eps);
        const uint16_t *w = is_q ? a.q_weight : a.k_weight;
        if (w != nullptr && !is_v) {
          float wa[8], wb[8];
          unpack8<ACT>(__ldg(reinterpret_cast<const uint4 *>(w) + ln.ca), wa);
          unpack8<ACT>(__ldg(reinterpret_cast<const uint4 *>(w) + ln.cb), wb);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            fa[e] *= r * wa[e];
            fb[e] *= r * wb[e];
          }
        }
      }
      if (live) {
        if (!is_v) {
          float cs[8], sn[8];
          ln.angles(reinterpret_cast<const float *>(tok + tab_at), a.rd, cs, sn);
          ln.rotate(fa, fb, cs, sn);
        }
        int64_t slot = -1;
        if (APPEND && !is_q) slot = slot_of(a, t0 + i, l == 0);
        store_row<D, KVT, APPEND>(a, t0 + i, h, slot, ln.ca, ln.cb, fa, fb, xa, xb);
      }
      for (h += ROWS; h >= a.heads; h -= a.heads) ++i;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (++st == p.stages) {
      st = 0;
      par ^= 1;
    }
  }
}

// The kernels of a call: of few and of many tokens.
struct RopeKernels {
  void (*few)(const RopeArgs);
  void (*many)(const RopeArgs, const StreamPlan);
};

template <int D, int KVT, bool APPEND>
RopeKernels pick_inter(bool inter) {
  if (inter) return {&rope_kernel<D, KVT, APPEND, true>, &rope_stream_kernel<D, KVT, APPEND, true>};
  return {&rope_kernel<D, KVT, APPEND, false>, &rope_stream_kernel<D, KVT, APPEND, false>};
}

template <int KVT, bool APPEND>
RopeKernels pick_dim(int d, bool inter) {
  return d == 64 ? pick_inter<64, KVT, APPEND>(inter) : pick_inter<128, KVT, APPEND>(inter);
}

RopeKernels pick(const pa_kv_desc &d, bool append, bool inter) {
  if (!append)  // the cache type only gives the activation type
    return d.kv_dtype == PA_KV_F16 || d.kv_dtype == PA_KV_INT4_F16
               ? pick_dim<kKvF16, false>(d.head_dim, inter)
               : pick_dim<kKvBf16, false>(d.head_dim, inter);
  switch (d.kv_dtype) {
    case PA_KV_F16: return pick_dim<kKvF16, true>(d.head_dim, inter);
    case PA_KV_FP8_E4M3: return pick_dim<kKvFp8, true>(d.head_dim, inter);
    case PA_KV_FP8_E5M2: return pick_dim<kKvE5M2, true>(d.head_dim, inter);
    default: return pick_dim<kKvBf16, true>(d.head_dim, inter);
  }
}

// The kernel of many tokens is taken from this many bytes of rows on.  2048
// tokens of 48 heads (25 MB): 13.3 us against 13.9 us; 1024 (13 MB): 8.3
// against 6.4 us.
constexpr int64_t kStreamBytes = 20 << 20;

bool plan_stream(const RopeArgs &a, int head_dim, int64_t num_tokens, StreamPlan *p) {
  if (num_tokens * a.heads * head_dim * 2 < kStreamBytes) return false;
  p->token_bytes = a.heads * head_dim * 2 + a.rd * 4;
  const int room = 216 * 1024;
  p->tokens = 49152 / p->token_bytes;
  p->tokens = p->tokens < 1 ? 1 : p->tokens > 8 ? 8 : p->tokens;
  // a stage's rows have to occupy the warps (8 tokens of 8 heads of 64: 12.5
  // us against 4.0 us for 8000 tokens)
  if (p->tokens * a.heads < kStreamWarps * 32 / (head_dim / 16)) return false;
  p->stages = room / (p->tokens * p->token_bytes);
  p->stages = p->stages > 16 ? 16 : p->stages;
  const int64_t blocks = (num_tokens + p->tokens - 1) / p->tokens;
  if (p->stages < 3 || blocks > 0x7fffffff) return false;
  p->blocks = static_cast<int>(blocks);
  p->wait_ns = test_hooks().wait_ns;
  return true;
}

}  // namespace

cudaError_t launch_rope(const pa_kv_desc &d, const pa_rope_desc &r, void *q_out, void *k_out, const void *q,
                        int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                        const int32_t *positions, void *k_cache, void *v_cache, const int64_t *slot_mapping,
                        int32_t num_tokens, cudaStream_t stream) {
  const bool append = k_cache != nullptr;
  RopeArgs a = {};
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.num_q = q ? d.num_q_heads : 0;
  a.num_kv = k ? d.num_kv_heads : 0;
  a.q_stride = q_stride ? q_stride : static_cast<int64_t>(d.num_q_heads) * d.head_dim;
  a.k_stride = k_stride ? k_stride : static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
  a.v_stride = v_stride ? v_stride : static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
  a.q_out = static_cast<uint16_t *>(q_out);
  a.k_out = static_cast<uint16_t *>(k_out);
  a.k_cache = static_cast<uint8_t *>(k_cache);
  a.v_cache = static_cast<uint8_t *>(v_cache);
  a.slots = slot_mapping;
  a.positions = positions;
  a.table = r.cos_sin;
  a.q_weight = static_cast<const uint16_t *>(r.q_weight);
  a.k_weight = static_cast<const uint16_t *>(r.k_weight);
  a.k_scales = d.k_scales;
  a.v_scales = d.v_scales;
  a.k_scale = d.k_scale == 0.f ? 1.f : d.k_scale;
  a.v_scale = d.v_scale == 0.f ? 1.f : d.v_scale;
  a.eps = r.eps;
  a.heads = a.num_q + a.num_kv * (append ? 2 : 1);
  a.max_position = r.max_position;
  a.rd = r.rotary_dim ? r.rotary_dim : d.head_dim;
  a.num_slots = static_cast<int64_t>(d.num_blocks) * d.block_size;
  a.checked = d.check_indices;
  a.err = d.error_word;
  const RopeKernels kern = pick(d, append, r.interleaved != 0);
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  StreamPlan p;
  if (plan_stream(a, d.head_dim, num_tokens, &p)) {
    const size_t smem = static_cast<size_t>(p.stages) * p.tokens * p.token_bytes;
    // (the limit is set for the largest ring once, not for every size)
    if (prepare_kernel(reinterpret_cast<const void *>(kern.many), (kStreamWarps + 1) * 32, 216 * 1024) < 1)
      return cudaErrorInvalidConfiguration;
    a.total = num_tokens;
    const int sms = device_sm_count();
    cfg.gridDim = dim3(p.blocks < sms ? p.blocks : sms);
    cfg.blockDim = dim3((kStreamWarps + 1) * 32);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, kern.many, a, p);
  }
  a.total = static_cast<int64_t>(num_tokens) * a.heads;
  const int threads = 256;
  const int64_t blocks = (a.total * (d.head_dim / 16) + threads - 1) / threads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  return cudaLaunchKernelEx(&cfg, kern.few, a);
}

}  // namespace pa
