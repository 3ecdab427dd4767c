// pa_int4_decode.cu -- decode attention over a 4-bit cache.
//
// With a row's dims x_d = s n_d + m per group of 64 (s and m per row and
// group), a score is
//   q . k_t = sum_groups s_t (q . n_t) + m_t (sum q),
// and an output
//   sum_t p_t v_t = sum_t (p_t s_t) n_t + (sum_t p_t m_t),
// so the codes go to the tensor cores as they are and the scales and minima are
// applied in fp32: to the scores' accumulators and to the weights.
//
// Work.  A unit is one 16-token block of one (sequence, kv head); the units of
// all of them in a row are cut into equal ranges, one per warp.  A warp fetches
// its blocks by 16-byte asynchronous copies into a ring of its own in shared
// memory, two blocks a stage, and never waits for another warp.  A (sequence,
// kv head) cut between warps is joined by the warp that finishes its last
// piece, in two steps (16 neighbouring pieces, then those), always in the same
// order.
//
// Codes as operands.  A code of 4 bits in the lowest bits of an fp16 number is
// the subnormal n 2^-24, exactly; in the next four it is 16 n 2^-24.  So a word
// of 8 codes becomes four operand registers by a shift and four masks, and the
// powers of two are taken out of the queries (scores) and of the results
// (outputs).  The queries are used in fp16, scaled by a power of two so that
// their largest is in [1, 2): exact for bf16 and fp16 down to 2^-10 of the
// largest, 2^-21 of it below.  The weights times the scales go in as a hi + lo
// pair of fp16 (22 bits): rows 8..15 of the operand are the lo halves of rows
// 0..7 (more than 8 query heads per kv head: a second product).
//
// The sums of the tensor cores round towards zero, so they run for 16 stages at
// most and are then added to fp32 registers.
#include <cuda.h>

#include "pa_host_cache.h"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kWarps = 8;
constexpr int kMinUnits = 4;   // units a warp gets at least, where there are few
constexpr int kFan = 16;       // pieces joined in one step
constexpr int kFlush = 16;     // stages between additions to the fp32 sums
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
  float *out, *lse;
  const uint16_t *q;
  const uint8_t *kc, *vc;
  const int32_t *tables, *lens;
  int max_blocks, num_seqs, hkv, hq, g;
  float qscale;  // scale * log2(e)
  int window, chunk;
  int32_t *err, *user_err;
  int checked, num_blocks, f16;
  int32_t *count1, *count2;  // pieces arrived: [2 workers] and [workers]
  float2 *slot_ml;           // [2 workers][g]: reference exponent, sum
  float *slot_o;             // [2 workers][g][D]
};

template <int D>
struct Cfg {
  static constexpr int TB = i4::tile_bytes(D);
  static constexpr int STAGE = 4 * TB;  // K and V of two blocks
  static constexpr int NST = D == 128 ? 6 : 8;
  static constexpr int RING = NST * STAGE;
  static constexpr int SMEM = kWarps * RING;
  static constexpr int NG = D / 64;
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Where byte `b` of row `r`'s codes lies in a staged tile.  The rows are
// shuffled so that the lanes of one load (rows r, r + 4, r + 1, r + 5 for the
// keys, r .. r + 3 for the values) meet no bank twice.
template <int D>
__device__ __forceinline__ int staged(int r, int b) {
  if constexpr (D == 128) return r * 64 + (b ^ ((((r >> 1) ^ (r >> 2)) & 1) << 5));
  return (r ^ (((r >> 2) & 1) << 1)) * 32 + b;
}

// The blocks of a sequence that its query sees: nb of them from b0 on.
struct Span {
  int len, first, b0, nb;
};
__device__ __forceinline__ Span span_of(const Args &a, int raw) {
  Span s;
  s.len = a.checked ? checked_len(raw, a.max_blocks * 16, a.err, a.user_err) : raw;
  if (s.len <= 0) {
    s.len = s.first = s.b0 = s.nb = 0;
    return s;
  }
  s.first = local_first_key(s.len - 1, a.window, a.chunk);
  s.b0 = s.first >> 4;
  s.nb = ((s.len + 15) >> 4) - s.b0;
  return s;
}

// Joins n pieces of one (sequence, kv head), slot_of(i) in turn; to the outputs
// of query row `row0` on (final) or to slot `to`.
template <int D, typename F>
__device__ __forceinline__ void join(const Args &a, int n, F slot_of, int64_t row0, bool final, int to) {
  constexpr int LPR = D / 4;  // lanes per row, 4 dims each
  const int lane = threadIdx.x & 31;
  const int c = (lane % LPR) * 4;
  for (int r = lane / LPR; r < a.g; r += 32 / LPR) {
    float ref = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < n; ++i) ref = fmaxf(ref, __ldcg(&a.slot_ml[static_cast<int64_t>(slot_of(i)) * a.g + r].x));
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const int64_t at = static_cast<int64_t>(slot_of(i)) * a.g + r;
      const float2 ml = __ldcg(&a.slot_ml[at]);
      const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.slot_o + at * D + c));
      const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - ref);
      l = fmaf(w, ml.y, l);
      o.x = fmaf(w, x.x, o.x);
      o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z);
      o.w = fmaf(w, x.w, o.w);
    }
    if (final) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<float4 *>(a.out + (row0 + r) * D + c) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (a.lse && c == 0) a.lse[row0 + r] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
    } else {
      const int64_t at = static_cast<int64_t>(to) * a.g + r;
      *reinterpret_cast<float4 *>(a.slot_o + at * D + c) = o;
      if (c == 0) a.slot_ml[at] = make_float2(ref, l);
    }
  }
}

// Counts a piece whose data all lanes have written; true for the last of n.
__device__ __forceinline__ bool last_of(int32_t *counter, int n) {
  __threadfence();
  __syncwarp();
  int last = 0;
  if ((threadIdx.x & 31) == 0) {
    last = atom_add_acq_rel_gpu(counter, 1) == n - 1;
    if (last) st_relaxed_gpu(counter, 0);
  }
  last = __shfl_sync(0xffffffffu, last, 0);
  __threadfence();
  return last != 0;
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kWarps * 32, 1) int4_decode_kernel(const Args a) {
  using C = Cfg<D>;
  constexpr int NG = C::NG, NST = C::NST, TB = C::TB;
  constexpr int NR = WIDE ? 2 : 1;  // query rows a lane holds: lane / 4, and 8 more
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long pre[kWarps * 32];
  __shared__ long long warp_sum[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.wait;" ::: "memory");

  // --- the units before each thread's share of the sequences, and all of them
  const int cs = (a.num_seqs + kWarps * 32 - 1) / (kWarps * 32);
  long long total;
  {
    long long mine = 0;
    for (int s = tid * cs; s < min((tid + 1) * cs, a.num_seqs); ++s)
      mine += static_cast<long long>(span_of(a, __ldg(a.lens + s)).nb) * a.hkv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += warp_sum[w];
      total += warp_sum[w];
    }
    pre[tid] = base + incl - mine;
    __syncthreads();
  }

  // --- sequences without tokens
  for (int s = blockIdx.x * kWarps + warp; s < a.num_seqs; s += gridDim.x * kWarps) {
    if (span_of(a, __ldg(a.lens + s)).nb > 0) continue;
    for (int i = lane; i < a.hq * D; i += 32) a.out[static_cast<int64_t>(s) * a.hq * D + i] = 0.f;
    if (a.lse)
      for (int i = lane; i < a.hq; i += 32) a.lse[static_cast<int64_t>(s) * a.hq + i] = -INFINITY;
  }

  // --- this warp's range of units [u0, u1)
  const long long all = static_cast<long long>(gridDim.x) * kWarps;
  const long long want = (total + kMinUnits - 1) / kMinUnits;
  const long long workers = want < all ? want : all;
  const int wk = warp * gridDim.x + blockIdx.x;
  if (wk >= workers) return;
  const long long u0 = total * wk / workers, u1 = total * (wk + 1) / workers;

  // --- the sequence of its first unit
  int s0;
  long long at0;  // units before it
  {
    int i = 0;
#pragma unroll
    for (int step = kWarps * 16; step > 0; step >>= 1)
      if (pre[i + step] <= u0) i += step;
    s0 = i * cs;
    at0 = pre[i];
    for (;; s0 += 32) {
      const int s = s0 + lane;
      long long incl = s < a.num_seqs ? static_cast<long long>(span_of(a, __ldg(a.lens + s)).nb) * a.hkv : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned over = __ballot_sync(0xffffffffu, at0 + incl > u0);
      if (over) {
        const int j = __ffs(over) - 1;
        const long long before = __shfl_sync(0xffffffffu, incl, j > 0 ? j - 1 : 0);
        if (j > 0) at0 += before;
        s0 += j;
        break;
      }
      at0 += __shfl_sync(0xffffffffu, incl, 31);
      if (s0 + 32 >= a.num_seqs) return;  // lengths changed under way: nothing to do
    }
  }

  // --- the fetching side: where it stands
  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  int fs = s0, fh, fb;  // sequence, kv head, block of the (sequence, kv head)
  Span fsp = span_of(a, __ldg(a.lens + fs));
  {
    const long long off = u0 - at0;
    fh = static_cast<int>(off / fsp.nb);
    fb = static_cast<int>(off - static_cast<long long>(fh) * fsp.nb);
  }
  int next_len = fs + 1 < a.num_seqs ? __ldg(a.lens + fs + 1) : 0;
  long long fu = u0;
  int fslot = 0;
  // a window of 32 entries of the sequence's table, one per lane, and the next
  int win = 0, win_s = -1, win_b = 0, nxt = 0, nxt_s = -1, nxt_b = 0;
  auto entries = [&](int s, const Span &sp, int b) {
    int id = 0;
    if (b + lane < sp.nb) {
      id = __ldg(a.tables + static_cast<int64_t>(s) * a.max_blocks + sp.b0 + b + lane);
      if (a.checked) id = checked_block(id, a.num_blocks, a.err, a.user_err);
    }
    return id;
  };
  const int my_dst = staged<D>(lane / (D / 32), (lane % (D / 32)) * 16);
  constexpr int PC = D / 16;  // 16-byte chunks of a tile's pairs
  const int pt = lane / PC;   // the tile whose pairs this lane copies: block pt / 2, K or V
  const int64_t head_stride = TB, block_stride = static_cast<int64_t>(a.hkv) * TB;
  auto fetch = [&]() {
    if (fu < u1) {
      if (!(win_s == fs && fb >= win_b && fb < win_b + 32)) {
        win = nxt_s == fs && nxt_b == fb ? nxt : entries(fs, fsp, fb);
        win_s = fs;
        win_b = fb;
        // the window that follows, asked for now
        if (fb + 32 < fsp.nb || fh + 1 < a.hkv) {
          nxt_b = fb + 32 < fsp.nb ? fb + 32 : 0;
          nxt_s = fs;
          nxt = entries(fs, fsp, nxt_b);
        } else {
          nxt_s = fs + 1;
          nxt_b = 0;
          nxt = nxt_s < a.num_seqs ? entries(nxt_s, span_of(a, next_len), 0) : 0;
        }
      }
      const bool two = fb + 1 < fsp.nb && fu + 1 < u1;
      const int id0 = __shfl_sync(0xffffffffu, win, (fb - win_b) & 31);
      const int id1 = __shfl_sync(0xffffffffu, win, (fb - win_b + 1) & 31);
      const uint32_t dst = ring + fslot * C::STAGE;
      const int64_t o0 = id0 * block_stride + fh * head_stride, o1 = id1 * block_stride + fh * head_stride;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        copy16(dst + my_dst + i * 512, a.kc + o0 + lane * 16 + i * 512);
        copy16(dst + TB + my_dst + i * 512, a.vc + o0 + lane * 16 + i * 512);
      }
      if (two) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          copy16(dst + 2 * TB + my_dst + i * 512, a.kc + o1 + lane * 16 + i * 512);
          copy16(dst + 3 * TB + my_dst + i * 512, a.vc + o1 + lane * 16 + i * 512);
        }
      }
      if (pt < (two ? 4 : 2)) {
        const int off = i4::code_bytes(D) + (lane % PC) * 16;
        copy16(dst + pt * TB + off, (pt & 1 ? a.vc : a.kc) + (pt & 2 ? o1 : o0) + off);
      }
      fslot = fslot + 1 == NST ? 0 : fslot + 1;
      const int n = two ? 2 : 1;
      fu += n;
      fb += n;
      if (fb == fsp.nb && fu < u1) {
        fb = 0;
        if (++fh == a.hkv) {
          fh = 0;
          do {  // the next sequence with tokens (fu < u1: there is one)
            ++fs;
            fsp = span_of(a, next_len);
            next_len = fs + 1 < a.num_seqs ? __ldg(a.lens + fs + 1) : 0;
          } while (fsp.nb == 0 && fs + 1 < a.num_seqs);
        }
      }
    }
    cp_async_commit();
  };
  int cseq = fs, ch = fh, cb = fb;  // the computing side
  Span csp = fsp;
#pragma unroll 1
  for (int i = 0; i < NST - 1; ++i) fetch();

  // --- addresses of a lane's operands in a staged tile
  const int krow = (gq >> 1) + 4 * (gq & 1);
  int kat[NG], vat[2][NG];  // vat[i & 1] for row t + 4 i
#pragma unroll
  for (int p = 0; p < NG; ++p) {
    kat[p] = staged<D>(krow, 32 * p + 8 * t);
    vat[0][p] = staged<D>(t, 32 * p + 4 * gq);
    vat[1][p] = staged<D>(t + 4, 32 * p + 4 * gq);
  }
  constexpr int ROW8 = 8 * (D / 2);  // eight rows further

  int cslot = 0;
  long long cu = u0;
#pragma unroll 1
  while (cu < u1) {
    // --- one (sequence, kv head), or this warp's part of it
    const long long seg = cu - cb;
    const int b_end = static_cast<int>(min(static_cast<long long>(csp.nb), cb + (u1 - cu)));
    const int64_t row0 = static_cast<int64_t>(cseq) * a.hq + ch * a.g;

    uint32_t qf[NR][D / 16][2];
    float cs_[NR], cm[NR][NG], M[NR], l[NR], mz[NR][NG];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const bool has = gq + 8 * r < a.g;
      uint4 raw[NG][2];
      float amax = 0.f, sum[NG];
#pragma unroll
      for (int p = 0; p < NG; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          raw[p][j] = has ? __ldg(reinterpret_cast<const uint4 *>(a.q + (row0 + gq + 8 * r) * D + 64 * p + 16 * t) + j)
                          : make_uint4(0, 0, 0, 0);
      float f[NG][16];
#pragma unroll
      for (int p = 0; p < NG; ++p) {
        sum[p] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = j < 4 ? (&raw[p][0].x)[j] : (&raw[p][1].x)[j - 4];
          f[p][2 * j] = a.f16 ? f16lo(w) : bf16lo(w);
          f[p][2 * j + 1] = a.f16 ? f16hi(w) : bf16hi(w);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          amax = fmaxf(amax, fabsf(f[p][j]));
          sum[p] += f[p][j];
        }
        sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], 1);
        sum[p] += __shfl_xor_sync(0xffffffffu, sum[p], 2);
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // the largest's exponent; none for a row of zeros or one that is not finite
      int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
      if (e == -127 || e == 128) e = 0;
      e = e > 100 ? 100 : e;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int p = 0; p < NG; ++p)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float *x = &f[p][8 * w];
          qf[r][p * 4 + 2 * w][0] = pack_f16x2(x[0] * down, x[4] * down);
          qf[r][p * 4 + 2 * w][1] = pack_f16x2(x[1] * (down * 0.0625f), x[5] * (down * 0.0625f));
          qf[r][p * 4 + 2 * w + 1][0] = pack_f16x2(x[2] * down, x[6] * down);
          qf[r][p * 4 + 2 * w + 1][1] = pack_f16x2(x[3] * (down * 0.0625f), x[7] * (down * 0.0625f));
        }
      cs_[r] = a.qscale * __uint_as_float(static_cast<uint32_t>(127 + 24 + e) << 23);
#pragma unroll
      for (int p = 0; p < NG; ++p) {
        cm[r][p] = a.qscale * sum[p];
        mz[r][p] = 0.f;
      }
      M[r] = -INFINITY;
      l[r] = 0.f;
    }
    // weights are 2^(x - M + kexp): kexp keeps weight * scale within fp16
    float kexp = 60.f, kap = 1152921504606846976.f;  // 2^60
    float acc[NG][8][4], sum[NR][NG][8][2];
#pragma unroll
    for (int p = 0; p < NG; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[p][j][i] = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r) sum[r][p][j][0] = sum[r][p][j][1] = 0.f;
      }
    auto flush = [&](const float (&alpha)[NR]) {
#pragma unroll
      for (int p = 0; p < NG; ++p)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (WIDE) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int c = 0; c < 2; ++c) sum[r][p][j][c] = (sum[r][p][j][c] + acc[p][j][2 * r + c]) * alpha[r];
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) sum[0][p][j][c] = (sum[0][p][j][c] + (acc[p][j][c] + acc[p][j][2 + c])) * alpha[0];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[p][j][i] = 0.f;
        }
    };

    int since = 0;
#pragma unroll 1
    while (cb < b_end) {
      cp_async_wait<NST - 2>();
      __syncwarp();
      fetch();
      const int n = b_end - cb < 2 ? 1 : 2;
      const uint32_t st = ring + cslot * C::STAGE;
      const int pos0 = (csp.b0 + cb) * 16;
      const bool edge = n < 2 || pos0 < csp.first || pos0 + 32 > csp.len;

      // scores: x[r][tile][i] of token t + 4 i
      float x[NR][2][4];
      float ks[2][4][NG], km[2][4][NG];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const uint32_t kt = st + 2 * tt * TB;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pa_ = kt + i4::code_bytes(D) + (t + 4 * i) * (4 * NG);
          uint32_t w[2];
          if constexpr (NG == 2) {
            const uint2 u = lds64(pa_);
            w[0] = u.x;
            w[1] = u.y;
          } else {
            w[0] = lds32(pa_);
          }
#pragma unroll
          for (int p = 0; p < NG; ++p) {
            ks[tt][i][p] = f16lo(w[p]);
            km[tt][i][p] = f16hi(w[p]);
          }
        }
        float s[2][NG][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int p = 0; p < NG; ++p) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][p][i] = 0.f;
            const uint2 w = lds64(kt + kat[p] + nt * ROW8);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u = h ? w.y : w.x, u8 = u >> 8;
              const uint32_t *qa = qf[0][p * 4 + 2 * h], *qb = qf[0][p * 4 + 2 * h + 1];
              const uint32_t *ra = qf[NR - 1][p * 4 + 2 * h], *rb = qf[NR - 1][p * 4 + 2 * h + 1];
              mma_f16_16816(s[nt][p], qa[0], WIDE ? ra[0] : 0u, qa[1], WIDE ? ra[1] : 0u, u & 0x000F000Fu,
                            u & 0x00F000F0u);
              mma_f16_16816(s[nt][p], qb[0], WIDE ? rb[0] : 0u, qb[1], WIDE ? rb[1] : 0u, u8 & 0x000F000Fu,
                            u8 & 0x00F000F0u);
            }
          }
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y = s[i >> 1][0][2 * r + (i & 1)] * ks[tt][i][0], z = km[tt][i][0] * cm[r][0];
            if constexpr (NG == 2) {
              y = fmaf(s[i >> 1][NG - 1][2 * r + (i & 1)], ks[tt][i][NG - 1], y);
              z = fmaf(km[tt][i][NG - 1], cm[r][NG - 1], z);
            }
            x[r][tt][i] = fmaf(y, cs_[r], z);
          }
      }

      // the values' scales and minima; masked tokens have neither
      float vs[2][4][NG], vm[2][4][NG];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t pa_ = st + (2 * tt + 1) * TB + i4::code_bytes(D) + (t + 4 * i) * (4 * NG);
          uint32_t w[2];
          if constexpr (NG == 2) {
            const uint2 u = lds64(pa_);
            w[0] = u.x;
            w[1] = u.y;
          } else {
            w[0] = lds32(pa_);
          }
#pragma unroll
          for (int p = 0; p < NG; ++p) {
            vs[tt][i][p] = f16lo(w[p]);
            vm[tt][i][p] = f16hi(w[p]);
          }
        }
      if (edge) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pos = pos0 + 16 * tt + t + 4 * i;
            if (pos < csp.first || pos >= csp.len || tt >= n) {
#pragma unroll
              for (int r = 0; r < NR; ++r) x[r][tt][i] = -INFINITY;
#pragma unroll
              for (int p = 0; p < NG; ++p) vs[tt][i][p] = vm[tt][i][p] = 0.f;
            }
          }
      }

      // the running maximum is raised only when a score passes it by 2^8, and
      // kexp lowered only when a scale needs it: a vote, no shuffles
      float smax = 0.f, xmax[NR];
      bool raise = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        xmax[r] = fmaxf(fmax3(x[r][0][0], x[r][0][1], x[r][0][2]), fmax3(x[r][0][3], x[r][1][0], x[r][1][1]));
        xmax[r] = fmax3(xmax[r], x[r][1][2], x[r][1][3]);
        raise |= xmax[r] > M[r] + 8.f;
      }
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int p = 0; p < NG; ++p) smax = fmaxf(smax, vs[tt][i][p]);
      raise |= smax * kap > 128.f;
      if (__any_sync(0xffffffffu, raise)) {
        float alpha[NR];
        smax = warp_max_xor(smax, 1, 32);
        float nk = kexp;
        if (smax * kap > 128.f) {
          int e = static_cast<int>(__float_as_uint(smax) >> 23) - 127;  // smax in [2^e, 2^(e + 1))
          e = e > 16 ? 16 : e;
          nk = static_cast<float>(4 - e);
          kap = __uint_as_float(static_cast<uint32_t>(127 + 4 - e) << 23);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const float m = fmaxf(M[r], warp_max_xor(xmax[r], 1, 4));
          alpha[r] = M[r] == -INFINITY ? 0.f : ex2_approx((M[r] - m) + (nk - kexp));
          M[r] = m;
          l[r] *= alpha[r];
#pragma unroll
          for (int p = 0; p < NG; ++p) mz[r][p] *= alpha[r];
        }
        kexp = nk;
        flush(alpha);
        since = 0;
      }
      float shift[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) shift[r] = kexp - (M[r] == -INFINITY ? 0.f : M[r]);

#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        uint32_t hi[NR][NG][2], lo[NR][NG][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = ex2_approx(x[r][tt][i] + shift[r]);
            l[r] += w[i];
#pragma unroll
            for (int p = 0; p < NG; ++p) mz[r][p] = fmaf(w[i], vm[tt][i][p], mz[r][p]);
          }
#pragma unroll
          for (int p = 0; p < NG; ++p)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float y0 = w[2 * j] * vs[tt][2 * j][p], y1 = w[2 * j + 1] * vs[tt][2 * j + 1][p];
              hi[r][p][j] = pack_f16x2(y0, y1);
              lo[r][p][j] = pack_f16x2(y0 - f16lo(hi[r][p][j]), y1 - f16hi(hi[r][p][j]));
            }
        }
        const uint32_t vt = st + (2 * tt + 1) * TB;
#pragma unroll
        for (int p = 0; p < NG; ++p) {
          const uint32_t w0 = lds32(vt + vat[0][p]), w1 = lds32(vt + vat[1][p]);
          const uint32_t w2 = lds32(vt + vat[0][p] + ROW8), w3 = lds32(vt + vat[1][p] + ROW8);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t b0 = __byte_perm(w0, w1, h ? 0x7632 : 0x5410);
            uint32_t b1 = __byte_perm(w2, w3, h ? 0x7632 : 0x5410);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t mask = j & 1 ? 0x00F000F0u : 0x000F000Fu;
              if (j == 2) {
                b0 >>= 8;
                b1 >>= 8;
              }
              if constexpr (WIDE) {
                mma_f16_16816(acc[p][4 * h + j], hi[0][p][0], hi[1][p][0], hi[0][p][1], hi[1][p][1], b0 & mask,
                              b1 & mask);
                mma_f16_16816(acc[p][4 * h + j], lo[0][p][0], lo[1][p][0], lo[0][p][1], lo[1][p][1], b0 & mask,
                              b1 & mask);
              } else {
                mma_f16_16816(acc[p][4 * h + j], hi[0][p][0], lo[0][p][0], hi[0][p][1], lo[0][p][1], b0 & mask,
                              b1 & mask);
              }
            }
          }
        }
      }
      cslot = cslot + 1 == NST ? 0 : cslot + 1;
      cb += n;
      cu += n;
      if (++since == kFlush) {
        float one[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) one[r] = 1.f;
        flush(one);
        since = 0;
      }
    }

    // --- the end of the piece: to the outputs, or to a slot and perhaps the join
    {
      float one[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) one[r] = 1.f;
      flush(one);
    }
    const bool whole = seg >= u0 && seg + csp.nb <= u1;
    const int slot = 2 * wk + (seg >= u0 ? 1 : 0);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
#pragma unroll
      for (int p = 0; p < NG; ++p) {
        mz[r][p] += __shfl_xor_sync(0xffffffffu, mz[r][p], 1);
        mz[r][p] += __shfl_xor_sync(0xffffffffu, mz[r][p], 2);
      }
      const int row = gq + 8 * r;
      if (row < a.g) {
        const float ref = M[r] == -INFINITY ? -INFINITY : M[r] - kexp;
        const float inv = !whole ? 1.f : l[r] == 0.f ? 0.f : 1.f / l[r];
        float *dst = whole ? a.out + (row0 + row) * D : a.slot_o + (static_cast<int64_t>(slot) * a.g + row) * D;
#pragma unroll
        for (int p = 0; p < NG; ++p)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
              // 2^24 for the codes' place in fp16, a sixteenth of it for the odd dims
              float4 o;
              o.x = fmaf(sum[r][p][j][c], 16777216.f, mz[r][p]) * inv;
              o.y = fmaf(sum[r][p][j + 1][c], 1048576.f, mz[r][p]) * inv;
              o.z = fmaf(sum[r][p][j + 2][c], 16777216.f, mz[r][p]) * inv;
              o.w = fmaf(sum[r][p][j + 3][c], 1048576.f, mz[r][p]) * inv;
              *reinterpret_cast<float4 *>(dst + 64 * p + 16 * t + 8 * c + j) = o;
            }
        if (t == 0) {
          if (!whole)
            a.slot_ml[static_cast<int64_t>(slot) * a.g + row] = make_float2(ref, l[r]);
          else if (a.lse)
            a.lse[row0 + row] = l[r] == 0.f ? -INFINITY : (ref + log2f(l[r])) * kLn2;
        }
      }
    }
    if (!whole) {
      // the workers of this (sequence, kv head) are wa .. wz
      const int wa = static_cast<int>(((seg + 1) * workers - 1) / total);
      const int wz = static_cast<int>(((seg + csp.nb) * workers - 1) / total);
      auto slot_of_worker = [wa](int w) { return 2 * w + (w == wa ? 1 : 0); };
      const int first = max(wa, wk / kFan * kFan), n1 = min(wz, wk / kFan * kFan + kFan - 1) - first + 1;
      const int n2 = wz / kFan - wa / kFan + 1;
      bool on = n1 == 1 || last_of(a.count1 + slot_of_worker(first), n1);
      if (on && n1 > 1)
        join<D>(a, n1, [&](int i) { return slot_of_worker(first + i); }, row0, n2 == 1, slot_of_worker(first));
      if (on && n2 > 1 && last_of(a.count2 + wa, n2))
        join<D>(a, n2, [&](int i) { return slot_of_worker(max(wa, (wa / kFan + i) * kFan)); }, row0, true, 0);
    }

    if (cb == csp.nb && cu < u1) {
      cb = 0;
      if (++ch == a.hkv) {
        ch = 0;
        do {
          ++cseq;
          csp = span_of(a, __ldg(a.lens + cseq));
        } while (csp.nb == 0 && cseq + 1 < a.num_seqs);
      }
    }
  }
  cp_async_wait<0>();
}

using Kernel = void (*)(const Args);

Kernel kernel_of(const pa_kv_desc &d, size_t *smem) {
  const bool wide = d.num_q_heads / d.num_kv_heads > 8;
  if (d.head_dim == 128) {
    *smem = Cfg<128>::SMEM;
    return wide ? &int4_decode_kernel<128, true> : &int4_decode_kernel<128, false>;
  }
  *smem = Cfg<64>::SMEM;
  return wide ? &int4_decode_kernel<64, true> : &int4_decode_kernel<64, false>;
}

struct Layout {
  size_t count1, count2, ml, o, total;
};

Layout layout(int ctas, int g, int d) {
  const size_t workers = static_cast<size_t>(ctas) * kWarps;
  Layout w;
  w.count1 = 256;
  w.count2 = w.count1 + 2 * workers * sizeof(int32_t);
  w.ml = (w.count2 + workers * sizeof(int32_t) + 255) / 256 * 256;
  w.o = (w.ml + 2 * workers * g * sizeof(float2) + 255) / 256 * 256;
  w.total = w.o + 2 * workers * g * d * sizeof(float);
  return w;
}

}  // namespace

pa_status plan_int4_decode(const pa_kv_desc &d, DecodePlan *plan, const char **why) {
  if (d.decode_impl != PA_DECODE_AUTO && d.decode_impl != PA_DECODE_MMA) {
    *why = "a 4-bit cache is decoded on the tensor cores (decode_impl AUTO or MMA)";
    return PA_ERR_UNSUPPORTED;
  }
  size_t smem = 0;
  const Kernel fn = kernel_of(d, &smem);
  const int occ = prepare_kernel(reinterpret_cast<const void *>(fn), kWarps * 32, smem);
  if (occ < 1) {
    *why = "the decode kernel does not fit on this device";
    return PA_ERR_CUDA;
  }
  plan->impl = PA_DECODE_MMA;
  plan->slot_heads = d.num_q_heads / d.num_kv_heads;
  plan->num_groups = d.num_kv_heads;
  plan->num_ctas = device_sm_count();
  const Layout w = layout(plan->num_ctas, plan->slot_heads, d.head_dim);
  plan->workspace_bytes = w.total;
  plan->zero_bytes = w.ml;
  return PA_OK;
}

cudaError_t launch_int4_decode(const pa_kv_desc &d, const DecodePlan &plan, float *out, float *lse, const void *q,
                               const void *k_cache, const void *v_cache, const int32_t *block_tables,
                               int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs, float scale,
                               void *workspace, cudaStream_t stream) {
  size_t smem = 0;
  const Kernel fn = kernel_of(d, &smem);
  const Layout w = layout(plan.num_ctas, plan.slot_heads, d.head_dim);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  Args a;
  a.out = out;
  a.lse = lse;
  a.q = static_cast<const uint16_t *>(q);
  a.kc = static_cast<const uint8_t *>(k_cache);
  a.vc = static_cast<const uint8_t *>(v_cache);
  a.tables = block_tables;
  a.lens = context_lens;
  a.max_blocks = max_blocks_per_seq;
  a.num_seqs = num_seqs;
  a.hkv = d.num_kv_heads;
  a.hq = d.num_q_heads;
  a.g = plan.slot_heads;
  a.qscale = scale * kLog2e;
  a.window = d.sliding_window;
  a.chunk = d.attention_chunk;
  a.err = reinterpret_cast<int32_t *>(ws);
  a.user_err = d.error_word;
  a.checked = d.check_indices;
  a.num_blocks = d.num_blocks;
  a.f16 = d.kv_dtype == PA_KV_INT4_F16;
  a.count1 = reinterpret_cast<int32_t *>(ws + w.count1);
  a.count2 = reinterpret_cast<int32_t *>(ws + w.count2);
  a.slot_ml = reinterpret_cast<float2 *>(ws + w.ml);
  a.slot_o = reinterpret_cast<float *>(ws + w.o);
  // programmatic dependent launch: it waits for the preceding kernel's writes
  // (the cache write) before reading anything
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.num_ctas);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  void *args[] = {&a};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(fn), args);
}

}  // namespace pa
