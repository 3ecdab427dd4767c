// pa_int4_pages.cu -- rows into a 4-bit cache, and its pages back to 16 bits.
//
// A group of 64 dims x of a row is stored as m = fp16(min x), s = fp16((max x
// - min x) / 15) and codes n = clamp(rint((x - m) * (1 / s)), 0, 15), 1 / s
// being the correctly rounded fp32 reciprocal; it reads as s n + m.  s = 0 (all
// dims alike) stores n = 0.  A group with a value that is not finite, or whose
// minimum or scale passes fp16, stores NaN for both and reads as NaN.
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

template <bool F16>
struct Act2;
template <>
struct Act2<true> {
  using T = __half2;
  static __device__ float2 f(T x) { return __half22float2(x); }
};
template <>
struct Act2<false> {
  using T = __nv_bfloat162;
  static __device__ float2 f(T x) { return __bfloat1622float2(x); }
};

// The codes (8 bytes) of 16 dims of a group held by four neighbouring lanes,
// and the group's (scale, minimum) pair.  range: the group's values are finite
// but pass fp16.
template <bool F16>
__device__ __forceinline__ uint2 encode16(const uint4 &a, const uint4 &b, uint32_t &pair, bool &range) {
  using A = Act2<F16>;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  typename A::T x[8], lo, hi;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const typename A::T *>(&w[i]);
  lo = hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = __hmin2_nan(lo, x[i]);
    hi = __hmax2_nan(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = __hmin2_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = __hmax2_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float2 l2 = A::f(lo), h2 = A::f(hi);
  const bool nan = l2.x != l2.x || l2.y != l2.y || h2.x != h2.x || h2.y != h2.y;
  const float mn = fminf(l2.x, l2.y), mx = fmaxf(h2.x, h2.y);
  __half s16 = __float2half_rn(__fdiv_rn(mx - mn, 15.f)), m16 = __float2half_rn(mn);
  const bool ok = !nan && fabsf(__half2float(s16)) <= 65504.f && fabsf(__half2float(m16)) <= 65504.f;
  range = !ok && !nan && fabsf(mn) <= 3.4e38f && fabsf(mx) <= 3.4e38f;
  if (!ok) s16 = m16 = __ushort_as_half(0x7fff);
  pair = static_cast<uint32_t>(__half_as_ushort(s16)) | (static_cast<uint32_t>(__half_as_ushort(m16)) << 16);
  const float s = __half2float(s16), m = __half2float(m16);
  const float r = s > 0.f ? __frcp_rn(s) : 0.f;
  // rounded to the nearest even whole number by the addition of 1.5 * 2^23, in
  // pairs; four codes at a time are put together as an fp32 number below 2^16
  const uint64_t m2 = f2_pack(-m, -m), r2 = f2_pack(r, r);
  const uint64_t big = f2_pack(12582912.f, 12582912.f), w256 = f2_pack(256.f, 256.f);
  // the codes grow with x, so its ends say whether any leaves [0, 15] (a
  // minimum far from 0 is rounded by more than a step); NaN says so too
  const bool inside = __fmul_rn(mn - m, r) > -0.5f && __fmul_rn(mx - m, r) < 15.5f;
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint64_t n[4];  // pairs of codes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = A::f(x[4 * h + i]);
      uint64_t t = f2_mul(f2_add(f2_pack(f.x, f.y), m2), r2);
      if (!inside) {  // (fmaxf takes the 0 of a NaN)
        const float2 u = f2_unpack(t);
        t = f2_pack(fminf(fmaxf(u.x, 0.f), 15.f), fminf(fmaxf(u.y, 0.f), 15.f));
      }
      n[i] = f2_sub(f2_add(t, big), big);
    }
    const float2 lo4 = f2_unpack(f2_fma(n[1], w256, n[0])), hi4 = f2_unpack(f2_fma(n[3], w256, n[2]));
    const float a4 = fmaf(lo4.y, 16.f, lo4.x) + 8388608.f, b4 = fmaf(hi4.y, 16.f, hi4.x) + 8388608.f;
    c[h] = __byte_perm(__float_as_uint(a4), __float_as_uint(b4), 0x5410);
  }
  return make_uint2(c[0], c[1]);
}

// One thread moves 16 dims of K and of V: 32 bytes read, 8 bytes of codes
// written; the first of a group's four threads writes its pair.  Bound by the
// issue slots: 16 instructions a dim (68.4 million warp instructions for 65536
// tokens of 8 heads of 128, issued in 82% of the cycles, the ALU busy in 68%), 1.36
// times the bytes' time (2 (2 D + 9 D / 16) per token and kv head): 68.7 us of a
// floor of 51.2; 16381 tokens 17.9 of 12.8 (86 MB).
template <int D, bool F16>
__global__ void __launch_bounds__(256) int4_write_kernel(const uint4 *__restrict__ k, const uint4 *__restrict__ v,
                                                         uint8_t *__restrict__ k_cache, uint8_t *__restrict__ v_cache,
                                                         const int64_t *__restrict__ slot_mapping, uint32_t rows,
                                                         uint32_t num_kv_heads, int64_t num_slots, int checked,
                                                         int32_t *err) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kParts = D / 16;
  // a row of 2^32 would be one of 550 GB of keys: 32 bits, whose division is short
  const uint32_t row = blockIdx.x * (256u / kParts) + threadIdx.x / kParts;  // token * num_kv_heads + head
  const int part = threadIdx.x % kParts;
  const int64_t i = static_cast<int64_t>(row) * kParts + part;
  const uint32_t token = row / num_kv_heads, head = row - token * num_kv_heads;
  int64_t slot = -1;
  if (row < rows) slot = __ldg(slot_mapping + token);
  if (checked && slot >= num_slots) {
    if (part == 0) report_error(err, nullptr, kErrBadIndex);
    slot = -1;
  }
  // a group's four lanes share a row, so they all have work or none has; the
  // shuffles take all lanes of the warp
  const bool live = slot >= 0;
  const uint4 z = make_uint4(0, 0, 0, 0);
  const uint4 k0 = live ? __ldg(k + 2 * i) : z, k1 = live ? __ldg(k + 2 * i + 1) : z;
  const uint4 v0 = live ? __ldg(v + 2 * i) : z, v1 = live ? __ldg(v + 2 * i + 1) : z;
  uint32_t kp, vp;
  bool kr, vr;
  const uint2 kc = encode16<F16>(k0, k1, kp, kr);
  const uint2 vc = encode16<F16>(v0, v1, vp, vr);
  if (!live) return;
  const int64_t tile = ((slot >> 4) * num_kv_heads + head) * i4::tile_bytes(D);
  const int off = static_cast<int>(slot & 15);
  const int64_t at = tile + off * (D / 2) + part * 8;
  *reinterpret_cast<uint2 *>(k_cache + at) = kc;
  *reinterpret_cast<uint2 *>(v_cache + at) = vc;
  if ((part & 3) == 0) {
    const int64_t pat = tile + i4::code_bytes(D) + (off * i4::groups(D) + part / 4) * 4;
    *reinterpret_cast<uint32_t *>(k_cache + pat) = kp;
    *reinterpret_cast<uint32_t *>(v_cache + pat) = vp;
    if (kr || vr) report_error(err, nullptr, kErrFp16Range);
  }
}

// Eight dims (one word of codes) as s n + m, rounded once to the activation type.
template <bool F16>
__device__ __forceinline__ uint4 widen8dims(uint32_t w, uint32_t pair) {
  const float s = f16lo(pair), m = f16hi(pair);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 2^23 + n, less 2^23: n as an fp32 number
    const float a = __uint_as_float(0x4B000000u | ((w >> (8 * i)) & 15u)) - 8388608.f;
    const float b = __uint_as_float(0x4B000000u | ((w >> (8 * i + 4)) & 15u)) - 8388608.f;
    r[i] = F16 ? pack_f16x2(fmaf(s, a, m), fmaf(s, b, m)) : pack_bf16x2(fmaf(s, a, m), fmaf(s, b, m));
    if constexpr (F16) {
      // the scale's rounding may carry the top of a group past fp16's largest
      __half2 h = *reinterpret_cast<const __half2 *>(&r[i]);
      const __half2 top = __half2half2(__ushort_as_half(0x7BFF));
      h = __hmax2_nan(__hmin2_nan(h, top), __hneg2(top));
      r[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// One warp widens one tile (a page of a kv head) of K or V: every lane has D /
// 16 words of codes in flight and stores 16 bytes for each, neighbouring lanes
// neighbouring bytes.  Bound by the bytes (9 D read, 32 D written a tile): 131072
// tokens of 8 heads of 128 take 112.5 us, 91% of the copy rate (32 CTAs an SM
// against 8: 57.7 us against 60.4 for 65536).
template <int D, bool F16>
__global__ void __launch_bounds__(256) int4_widen_kernel(const uint8_t *__restrict__ k_cache,
                                                         const uint8_t *__restrict__ v_cache,
                                                         const int32_t *__restrict__ src_blocks,
                                                         uint8_t *__restrict__ k_out, uint8_t *__restrict__ v_out,
                                                         const int32_t *__restrict__ dst_blocks, uint32_t tiles,
                                                         uint32_t num_kv_heads, int num_blocks, int num_out_blocks,
                                                         int checked, int32_t *err) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kWords = D / 16;  // per lane: 16 rows of D / 8 words
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * (blockDim.x / 32);
  // (2^31 tiles would be 4 TB of pages)
  for (uint32_t i = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; i < tiles; i += warps) {
    // tile order: page, K or V, kv head
    const uint32_t pair = i / (2 * num_kv_heads), r = i - pair * 2 * num_kv_heads;
    const bool is_v = r >= num_kv_heads;
    const uint32_t head = is_v ? r - num_kv_heads : r;
    const int sb = __ldg(src_blocks + pair), db = __ldg(dst_blocks + pair);
    if (checked && (sb < 0 || sb >= num_blocks || db < 0 || db >= num_out_blocks)) {
      if (r == 0 && lane == 0) report_error(err, nullptr, kErrBadIndex);
      continue;
    }
    const uint8_t *src =
        (is_v ? v_cache : k_cache) + (static_cast<int64_t>(sb) * num_kv_heads + head) * i4::tile_bytes(D);
    uint8_t *dst = (is_v ? v_out : k_out) + (static_cast<int64_t>(db) * num_kv_heads + head) * (32 * D);
    const uint32_t *codes = reinterpret_cast<const uint32_t *>(src);
    const uint32_t *pairs = reinterpret_cast<const uint32_t *>(src + i4::code_bytes(D));
    uint32_t w[kWords], p[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int at = j * 32 + lane;  // word of the tile: eight dims, a 64-dim group has eight words
      w[j] = __ldg(codes + at);
      p[j] = __ldg(pairs + at / 8);
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j)
      *reinterpret_cast<uint4 *>(dst + (j * 32 + lane) * 16) = widen8dims<F16>(w[j], p[j]);
  }
}

}  // namespace

cudaError_t launch_int4_write(const pa_kv_desc &d, const void *k, const void *v, void *k_cache, void *v_cache,
                              const int64_t *slot_mapping, int32_t num_tokens, cudaStream_t stream) {
  const bool f16 = d.kv_dtype == PA_KV_INT4_F16;
  const int64_t rows = static_cast<int64_t>(num_tokens) * d.num_kv_heads;
  const int threads = 256, per_cta = threads / (d.head_dim / 16);
  const int64_t blocks = (rows + per_cta - 1) / per_cta;
  if (rows > 0xffffffffLL || blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto kern = d.head_dim == 128 ? (f16 ? &int4_write_kernel<128, true> : &int4_write_kernel<128, false>)
                                : (f16 ? &int4_write_kernel<64, true> : &int4_write_kernel<64, false>);
  kern<<<static_cast<unsigned>(blocks), threads, 0, stream>>>(
      static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), static_cast<uint8_t *>(k_cache),
      static_cast<uint8_t *>(v_cache), slot_mapping, static_cast<uint32_t>(rows),
      static_cast<uint32_t>(d.num_kv_heads), static_cast<int64_t>(d.num_blocks) * 16, d.check_indices, d.error_word);
  return cudaGetLastError();
}

cudaError_t launch_int4_widen(const pa_kv_desc &d, const void *k_cache, const void *v_cache,
                              const int32_t *src_blocks, void *k_out, void *v_out, const int32_t *dst_blocks,
                              int32_t num_out_blocks, int32_t num_pairs, cudaStream_t stream) {
  const bool f16 = d.kv_dtype == PA_KV_INT4_F16;
  const int64_t tiles = static_cast<int64_t>(num_pairs) * d.num_kv_heads * 2;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  const int threads = 256;
  const int64_t want = (tiles + threads / 32 - 1) / (threads / 32);
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 32;
  const unsigned blocks = static_cast<unsigned>(want < cap ? want : cap);
  auto kern = d.head_dim == 128 ? (f16 ? &int4_widen_kernel<128, true> : &int4_widen_kernel<128, false>)
                                : (f16 ? &int4_widen_kernel<64, true> : &int4_widen_kernel<64, false>);
  kern<<<blocks, threads, 0, stream>>>(static_cast<const uint8_t *>(k_cache), static_cast<const uint8_t *>(v_cache),
                                       src_blocks, static_cast<uint8_t *>(k_out), static_cast<uint8_t *>(v_out),
                                       dst_blocks, static_cast<uint32_t>(tiles), static_cast<uint32_t>(d.num_kv_heads),
                                       d.num_blocks, num_out_blocks,
                                       d.check_indices, d.error_word);
  return cudaGetLastError();
}

}  // namespace pa
