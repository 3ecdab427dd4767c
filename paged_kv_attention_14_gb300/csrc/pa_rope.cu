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
// log2(D / 16) shuffles.  A lane's HPT rows are consecutive heads of one
// token: they share the lane's cosines, sines and position, and their loads
// are all in flight before the first use.
#include "pa_device.cuh"
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
  int slices;         // ceil(heads / HPT)
  int max_position;
  int rd;
  int64_t total;      // tokens * slices
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

// KVT: the cache type (its activation type is fp16 for kKvF16, else bf16);
// APPEND: keys and values go to the cache.
template <int D, int KVT, bool APPEND, bool INTER, int HPT>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  constexpr int ACT = KVT == kKvF16 ? kKvF16 : kKvBf16;
  constexpr int LPR = D / 16;  // lanes of a row
  // a programmatic dependent launched after this one waits for these writes;
  // this one waits for the writes of the kernel before it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / LPR;
  const int l = threadIdx.x % LPR;
  // every lane stays for the shuffles; lanes past the end touch no memory
  const bool live = unit < a.total;
  const int64_t token = live ? unit / a.slices : 0;
  const int h0 = live ? static_cast<int>(unit - token * a.slices) * HPT : 0;
  // this lane's chunks of 8 elements: ca and cb rotate with each other
  const int nr = a.rd / 16;
  const bool rot = INTER || l < nr;  // half split: lanes nr .. hold unrotated dims
  const int ca = INTER ? l : (l < nr ? l : 2 * l);
  const int cb = INTER ? l + LPR : (l < nr ? l + nr : 2 * l + 1);

  // ---- every load first
  uint4 xa[HPT], xb[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int h = h0 + i;
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (live && h < a.heads) {
      const uint16_t *src;
      if (h < a.num_q)
        src = a.q + token * a.q_stride + static_cast<int64_t>(h) * D;
      else if (!APPEND || h < a.num_q + a.num_kv)
        src = a.k + token * a.k_stride + static_cast<int64_t>(h - a.num_q) * D;
      else
        src = a.v + token * a.v_stride + static_cast<int64_t>(h - a.num_q - a.num_kv) * D;
      xa[i] = *reinterpret_cast<const uint4 *>(src + ca * 8);
      xb[i] = *reinterpret_cast<const uint4 *>(src + cb * 8);
    }
  }
  // cosines and sines: half split, 8 frequencies shared by both chunks;
  // interleaved, 4 of each chunk (1 and 0 past rd)
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  int64_t slot = -1;
  if (live) {
    int pos = __ldg(a.positions + token);
    if (a.checked && (pos < 0 || pos >= a.max_position)) {
      if (l == 0) report_error(a.err, nullptr, kErrBadIndex);
      pos = 0;
    }
    const float *row = a.table + static_cast<int64_t>(pos) * a.rd;
    if constexpr (INTER) {
      if (ca * 8 < a.rd) {
        *reinterpret_cast<float4 *>(cs) = __ldg(reinterpret_cast<const float4 *>(row + ca * 4));
        *reinterpret_cast<float4 *>(sn) = __ldg(reinterpret_cast<const float4 *>(row + a.rd / 2 + ca * 4));
      }
      if (cb * 8 < a.rd) {
        *reinterpret_cast<float4 *>(cs + 4) = __ldg(reinterpret_cast<const float4 *>(row + cb * 4));
        *reinterpret_cast<float4 *>(sn + 4) = __ldg(reinterpret_cast<const float4 *>(row + a.rd / 2 + cb * 4));
      }
    } else if (rot) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<float4 *>(cs + 4 * i) = __ldg(reinterpret_cast<const float4 *>(row + ca * 8) + i);
        *reinterpret_cast<float4 *>(sn + 4 * i) = __ldg(reinterpret_cast<const float4 *>(row + a.rd / 2 + ca * 8) + i);
      }
    }
    if constexpr (APPEND) {
      slot = __ldg(a.slots + token);
      if (a.checked && slot >= a.num_slots) {
        if (l == 0) report_error(a.err, nullptr, kErrBadIndex);
        slot = -1;
      }
    }
  }

#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int h = h0 + i;
    const bool is_q = h < a.num_q;
    const bool is_v = APPEND && h >= a.num_q + a.num_kv;
    float fa[8], fb[8];
    unpack8<ACT>(xa[i], fa);
    unpack8<ACT>(xb[i], fb);
    const uint16_t *w = is_q ? a.q_weight : a.k_weight;
    if (a.q_weight != nullptr || a.k_weight != nullptr) {  // the same for every lane: all reach the shuffles
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += fa[e] * fa[e] + fb[e] * fb[e];
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w != nullptr && !is_v) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        float wa[8], wb[8];
        unpack8<ACT>(__ldg(reinterpret_cast<const uint4 *>(w) + ca), wa);
        unpack8<ACT>(__ldg(reinterpret_cast<const uint4 *>(w) + cb), wb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          fa[e] *= r * wa[e];
          fb[e] *= r * wb[e];
        }
      }
    }
    if (!live || h >= a.heads) continue;
    if (!is_v) {
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
        dst[ca] = is_v ? xa[i] : pack8<ACT>(fa);  // values: bit copies
        dst[cb] = is_v ? xb[i] : pack8<ACT>(fb);
      } else {
        const float *hs = is_v ? a.v_scales : a.k_scales;
        const float s = hs ? __ldg(hs + kvh) : (is_v ? a.v_scale : a.k_scale);
        uint2 *dst = reinterpret_cast<uint2 *>(cache + row * D);
        dst[ca] = encode8<KVT>(fa, s);
        dst[cb] = encode8<KVT>(fb, s);
      }
    }
  }
}

using RopeKernel = void (*)(const RopeArgs);

template <int D, int KVT, bool APPEND, int HPT>
RopeKernel pick_inter(bool inter) {
  return inter ? &rope_kernel<D, KVT, APPEND, true, HPT> : &rope_kernel<D, KVT, APPEND, false, HPT>;
}

template <int KVT, bool APPEND, int HPT>
RopeKernel pick_dim(int d, bool inter) {
  return d == 64 ? pick_inter<64, KVT, APPEND, HPT>(inter) : pick_inter<128, KVT, APPEND, HPT>(inter);
}

template <int HPT>
RopeKernel pick(const pa_kv_desc &d, bool append, bool inter) {
  if (!append)  // the cache type only gives the activation type
    return d.kv_dtype == PA_KV_F16 ? pick_dim<kKvF16, false, HPT>(d.head_dim, inter)
                                   : pick_dim<kKvBf16, false, HPT>(d.head_dim, inter);
  switch (d.kv_dtype) {
    case PA_KV_F16: return pick_dim<kKvF16, true, HPT>(d.head_dim, inter);
    case PA_KV_FP8_E4M3: return pick_dim<kKvFp8, true, HPT>(d.head_dim, inter);
    case PA_KV_FP8_E5M2: return pick_dim<kKvE5M2, true, HPT>(d.head_dim, inter);
    default: return pick_dim<kKvBf16, true, HPT>(d.head_dim, inter);
  }
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
  const int hpt = 1;
  a.slices = (a.heads + hpt - 1) / hpt;
  a.total = static_cast<int64_t>(num_tokens) * a.slices;
  const int threads = 256;
  const int64_t blocks = (a.total * (d.head_dim / 16) + threads - 1) / threads;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const RopeKernel kern = pick<1>(d, append, r.interleaved != 0);
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace pa
