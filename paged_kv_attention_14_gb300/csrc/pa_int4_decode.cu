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
// all of them in a row are cut into equal ranges, one per CTA, and those into
// one per warp.  A warp fetches its blocks by 16-byte asynchronous copies into
// a ring of its own in shared memory, two blocks a stage, and never waits for
// another warp.  (Bulk copies issued by one lane: 17% slower.)  A (sequence, kv
// head) cut between warps is joined by the CTA from pieces in shared memory,
// one cut between CTAs by the CTA that counts in last, always in the same order.
// Where all sequences are short the CTAs' ranges end at whole (sequence, kv
// head)s, so that there is nothing to join between them (kWhole).
//
// Codes as operands.  A code of 4 bits in bits 2..5 of an fp16 number is the
// subnormal n 2^-22, exactly; in bits 6..9 it is n 2^-18.  So a word of 8 codes
// becomes four operand registers by two shifts and four masks, and the
// powers of two are taken out of the queries (scores) and of the results
// (outputs).  The queries are used in fp16, scaled by a power of two so that
// their largest is in [1, 2): exact for bf16 and fp16 down to 2^-10 of the
// largest, 2^-21 of it below.  The weights times the scales go in as a hi + lo
// pair of fp16, times a power of two per query and group of dims that follows the
// largest such product so far: 22 bits down to 2^-18 of it, 2^-29 of it below.
// (One power of two for a warp's piece, from the largest scale, loses groups and
// tokens of small scales beside large ones, and is 2 to 4% faster.)  Scores are
// keys (16 rows) times queries (8 columns), outputs are values (16 dims) times
// weights (8 columns); with up to 4 query heads per kv head the columns of
// queries 4..7 take the lo halves, with more there is a product for each half.
//
// Bounded by latency at two warps a scheduler, which is what the registers allow:
// a block of a kv head takes a warp about 335 instructions (codes to operands 105,
// products 16, weights and scales 135, fetching 30), three quarters of what the
// SMs could issue while its bytes come at the copy rate, and they issue in 54%
// of the cycles.  32 sequences of 8192, 32 / 8 heads of 128: 70.3 us, 4.3 TB/s; 128
// sequences of 1024 to 8192, 40 heads: 157 us.  Farthest from the bytes are 9 to
// 16 query heads a kv head (32 sequences of 4096, 16 / 1 heads: 22.5 us for 2.8):
// four products an operand, a ring of two stages, no queries asked for ahead.  The
// smallest call takes 7.4 us: lengths, tables and blocks one after the other from
// memory, launch, outputs.
//
// The sums of the tensor cores round towards zero, so they run over one stage
// and are then added to fp32 registers.
#include <cuda.h>

#include "pa_host_cache.h"
#include "pa_int4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// Units a CTA gets at least, where there are few: with more, warps take two one
// after the other (5 sequences of 1 to 33 tokens: 7.5 us; 16: 7.8).
constexpr int kMinUnits = 8;
// Blocks of the longest sequence up to which CTAs get whole (sequence, kv
// head)s: joining between CTAs costs about 3 us, a CTA's surplus at most as many
// blocks.  32 sequences, 32 / 8 heads of 128, whole against cut: of 128 tokens
// 8.2 us and 11.5, of 1024 15.3 and 17.5, of 2048 23.5 both, of 4096 41.8 and
// 40.7 (ragged to 4096: 40.1 and 28.1).
constexpr int kWhole = 64;
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
  int32_t *count;   // [CTAs]: pieces arrived of what begins in a CTA and goes on
  // what a CTA has of a (sequence, kv head) that began before it, and of one
  // that goes on behind it
  float2 *slot_ml;  // [CTAs][2][g]: reference exponent, sum
  float *slot_o;    // [CTAs][2][g][D]
};

template <int D, int NQ>
struct Cfg {
  // warps: what the registers allow without spilling (128 dims and more than 8
  // queries: 12 words of a lane spill).  64 dims, up to 8 queries: 12 (128
  // sequences of 1024 to 8192, 32 / 8 heads: 89 us; 8 warps about a tenth more).
  static constexpr int W = D == 64 && NQ <= 8 ? 12 : 8;
  static constexpr int TB = i4::tile_bytes(D);
  static constexpr int STAGE = 4 * TB;  // K and V of two blocks
  static constexpr int NST = W == 12 ? 4 : D == 64 ? 8 : NQ == 4 ? 5 : NQ == 8 ? 4 : 2;
  static constexpr int RING = NST * STAGE;
  static constexpr int OFF_ML = W * RING;                       // the pieces of the CTA's warps, two each:
  static constexpr int OFF_O = OFF_ML + 2 * W * NQ * 8;        // [2 W][g] reference exponent, sum, and
  static constexpr int SMEM = OFF_O + 2 * W * NQ * D * 4;      // [2 W][g][D]
  static constexpr int NG = D / 64;
};

// A word's bytes 0 and 2 (odd: 1 and 3) with their codes where the masks are:
// even dims n 2^-22, odd dims n 2^-18.  (The tensor cores lose what lies far
// below an operand's exponent, and a subnormal's counts as 2^-14.  Codes in bits
// 0..3 and 4..7 need a shift a word less and are 2 to 5% faster, but the outputs'
// errors, against 64 bits, are then 2.3e-6 to 2.8e-6 instead of 4.6e-7 to 8.7e-7;
// all codes in bits 6..9: 3.9e-7 to 7.4e-7, 5% slower.)
constexpr uint32_t kLowCodes = 0x003C003Cu, kHighCodes = 0x03C003C0u;
constexpr int kCodeExp = 22;
__device__ __forceinline__ uint32_t place(uint32_t w, int odd) { return odd ? w >> 6 : w << 2; }

__device__ __forceinline__ uint32_t lds32(const uint8_t *a) { return *reinterpret_cast<const uint32_t *>(a); }
__device__ __forceinline__ uint2 lds64(const uint8_t *a) { return *reinterpret_cast<const uint2 *>(a); }
// the pairs of a row: one word a group
template <int NG>
__device__ __forceinline__ void load_pairs(const uint8_t *at, uint32_t (&w)[2]) {
  if constexpr (NG == 2) {
    const uint2 u = lds64(at);
    w[0] = u.x;
    w[1] = u.y;
  } else {
    w[0] = lds32(at);
  }
}
// D = A(16x16, row) * B(16x8, col) + C, f16 inputs, fp32 accumulate; free to
// be scheduled (a function of its operands)
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// ... with C = 0
__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// the halves of an fp16 pair in fp32
__device__ __forceinline__ float2 halves(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }
// an 8 x 8 matrix of 16-bit values, one row's pair a lane, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
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
  s.len = a.checked ? checked_len(raw, table_tokens(a.max_blocks), a.err, a.user_err) : raw;
  if (s.len <= 0) {
    s.len = s.first = s.b0 = s.nb = 0;
    return s;
  }
  s.first = local_first_key(s.len - 1, a.window, a.chunk);
  s.b0 = s.first >> 4;
  s.nb = ((s.len + 15) >> 4) - s.b0;
  return s;
}

// D / 32 dims of a row: a lane's part.
template <int D>
struct Part {
  float x[D / 32];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = 0.f;
  }
  __device__ __forceinline__ void load(const float *p) {
    if constexpr (D == 128) {
      const float4 v = *reinterpret_cast<const float4 *>(p);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2 *>(p);
      x[0] = v.x, x[1] = v.y;
    }
  }
  __device__ __forceinline__ void load_l2(const float *p) {
    if constexpr (D == 128) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(p));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2 *>(p));
      x[0] = v.x, x[1] = v.y;
    }
  }
  __device__ __forceinline__ void store(float *p, float f) const {
    if constexpr (D == 128)
      *reinterpret_cast<float4 *>(p) = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
    else
      *reinterpret_cast<float2 *>(p) = make_float2(x[0] * f, x[1] * f);
  }
  __device__ __forceinline__ void add(float w, const Part &o) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = fmaf(w, o.x[i], x[i]);
  }
};

// A joined row (its reference, sum and dims) to the outputs.
template <int D>
__device__ __forceinline__ void store_row(const Args &a, int64_t row, float ref, float l, const Part<D> &o) {
  const int lane = threadIdx.x & 31;
  o.store(a.out + row * D + lane * (D / 32), l == 0.f ? 0.f : 1.f / l);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
}
constexpr float kNone = 3e38f;  // minus a running maximum that there is not yet
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ float weight_of(float2 ml, float ref) {
  return ml.x == -INFINITY ? 0.f * ml.y : ex2_approx(ml.x - ref);  // (a NaN stays one)
}

// A (sequence, kv head) of which a warp holds a piece.
struct Piece {
  long long seg;  // its first unit
  int64_t row0;   // its first query row
  int nb;         // its units; 0: no piece
};

// A (sequence, kv head) cut between n CTAs from CTA ca on, which this one joins;
// one of its pieces here (-1: nothing to join).
struct Join {
  int piece, ca, n;
};

// How the units are dealt out: CTA c of `ctas` has [first(c), first(c + 1)),
// its warp w of `warps` an equal part of that.  (total = each * ctas + rest;
// a CTA's part is below 2^27: of 2^31 tokens.)
struct Deal {
  long long each;
  int rest, ctas, warps;
  __device__ __forceinline__ Deal(long long total, int ctas_, int warps_) : ctas(ctas_), warps(warps_) {
    if (total < 0x7fffffffLL) {
      const int n = static_cast<int>(total), e = n / ctas;
      each = e;
      rest = n - e * ctas;
    } else {
      each = total / ctas;
      rest = static_cast<int>(total - each * ctas);
    }
  }
  __device__ __forceinline__ long long first(int c) const { return each * c + rest * c / ctas; }
  // the CTA that has unit u
  __device__ __forceinline__ int cta_of(long long u) const {
    const long long total = each * ctas + rest, x = (u + 1) * ctas - 1;
    if (total * ctas < 0xffffffffLL) return static_cast<int>(static_cast<unsigned>(x) / static_cast<unsigned>(total));
    return static_cast<int>(x / total);
  }
};

// NQ: query columns of the products of weights and values (4, 8 or 16).
template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::W * 32, 1) int4_decode_kernel(const Args a) {
  using C = Cfg<D, NQ>;
  constexpr int NG = C::NG, NST = C::NST, TB = C::TB, kWarps = C::W;
  constexpr int NR = NQ == 16 ? 2 : 1;  // eights of queries
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long pre[kWarps * 32];
  __shared__ long long warp_sum[kWarps];
  __shared__ int warp_longest[kWarps];
  __shared__ long long bounds[2];
  __shared__ Piece pieces[2 * kWarps];  // of each warp: one that began before its range, one that goes on behind it
  __shared__ long long starts[kWarps + 1];  // of the warps' ranges
  __shared__ Join joins[2];
  float2 *const part_ml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
  float *const part_o = reinterpret_cast<float *>(smem + C::OFF_O);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.wait;" ::: "memory");

  // --- the units before each thread's share of the sequences, and all of them
  const int cs = (a.num_seqs + kWarps * 32 - 1) / (kWarps * 32);
  long long total;
  int longest = 0;
  {
    long long mine = 0;
    for (int s = tid * cs; s < min((tid + 1) * cs, a.num_seqs); ++s) {
      const int nb = span_of(a, __ldg(a.lens + s)).nb;
      mine += static_cast<long long>(nb) * a.hkv;
      longest = max(longest, nb);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) {
      warp_sum[warp] = incl;
      warp_longest[warp] = longest;
    }
    __syncthreads();
    long long base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += warp_sum[w];
      total += warp_sum[w];
      longest = max(longest, warp_longest[w]);
    }
    pre[tid] = base + incl - mine;
    __syncthreads();
  }

  // --- this warp's range of units [u0, u1)
  const long long want = (total + kMinUnits - 1) / kMinUnits;
  const Deal deal(total, static_cast<int>(want < 1 ? 1 : want < gridDim.x ? want : gridDim.x), kWarps);
  const int cta = blockIdx.x;
  const bool idle = cta >= deal.ctas || total == 0;
  const bool whole_only = longest <= kWhole;
  long long r0 = 0, r1 = 0, u0 = 0, u1 = 0;  // the CTA's units, the warp's
  int s0 = 0;                                // the sequence of unit u0
  long long at0 = 0;                         // units before it
  if (!idle) {
    if (!whole_only) r0 = deal.first(cta), r1 = deal.first(cta + 1);
#pragma unroll 1
    for (int pass = whole_only ? 0 : 1; pass < 2; ++pass) {
      long long u;  // the unit whose sequence is looked for
      if (pass == 0) {
        u = deal.first(cta + (warp & 1));  // (total, for the last CTA's end: its last sequence or one behind it)
      } else {
        const unsigned n = static_cast<unsigned>(r1 - r0);
        u = u0 = r0 + n * warp / kWarps;
        u1 = r0 + n * (warp + 1) / kWarps;
        if (u0 >= u1) break;
      }
      // the last thread whose share begins at u or before it: of every
      // kWarps-th, then of those from there on
      int i = (__popc(__ballot_sync(0xffffffffu, pre[lane * kWarps] <= u)) - 1) * kWarps;
      i += __popc(__ballot_sync(0xffffffffu, lane < kWarps && pre[i + (lane < kWarps ? lane : 0)] <= u)) - 1;
      s0 = i * cs;
      at0 = pre[i];
#pragma unroll 1
      for (; cs > 1; s0 += 32) {  // (cs 1: a sequence a thread, it is the one)
        const int s = s0 + lane;
        long long incl = s < a.num_seqs ? static_cast<long long>(span_of(a, __ldg(a.lens + s)).nb) * a.hkv : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned over = __ballot_sync(0xffffffffu, at0 + incl > u);
        if (over) {
          const int j = __ffs(over) - 1;
          const long long before = __shfl_sync(0xffffffffu, incl, j > 0 ? j - 1 : 0);
          if (j > 0) at0 += before;
          s0 += j;
          break;
        }
        at0 += __shfl_sync(0xffffffffu, incl, 31);
        if (s0 + 32 >= a.num_seqs) break;  // (u is the total)
      }
      if (pass == 0) {
        // the nearest end of a (sequence, kv head)
        if (u < total) {
          const int nb = span_of(a, __ldg(a.lens + s0)).nb, in = static_cast<int>(u - at0) % nb;
          u += 2 * in < nb ? -in : nb - in;
        }
        if (warp < 2 && lane == 0) bounds[warp] = u;
        __syncthreads();
        r0 = bounds[0];
        r1 = bounds[1];
      }
    }
  }
  if (lane < 2) pieces[2 * warp + lane].nb = 0;
  if (lane == 0) starts[warp] = u0;
  if (tid == 0) starts[kWarps] = r1;

  if (u0 < u1) {  // (not indented: the whole of the warp's work)
  // --- the fetching side: where it stands
  const uint8_t *const ring = smem + warp * C::RING;
  const uint32_t ring_at = smem_u32(ring);
  int fs = s0, fh, fb;  // sequence, kv head, block of the (sequence, kv head)
  Span fsp = span_of(a, __ldg(a.lens + fs));
  {
    const long long off = u0 - at0;
    fh = total < 0x7fffffff ? static_cast<int>(off) / fsp.nb : static_cast<int>(off / fsp.nb);
    fb = static_cast<int>(off - static_cast<long long>(fh) * fsp.nb);
  }
  int next_len = fs + 1 < a.num_seqs ? __ldg(a.lens + fs + 1) : 0;
  int fleft = static_cast<int>(u1 - u0);  // units to fetch
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
  const int my_pair_dst = pt * TB + i4::code_bytes(D) + (lane % PC) * 16;
  const uint8_t *const my_k = a.kc + lane * 16, *const my_v = a.vc + lane * 16;
  const uint8_t *const my_pair = (pt & 1 ? a.vc : a.kc) + i4::code_bytes(D) + (lane % PC) * 16;
  const int64_t block_stride = static_cast<int64_t>(a.hkv) * TB;
  auto fetch = [&]() {
    if (fleft > 0) {
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
      const bool two = fb + 1 < fsp.nb && fleft > 1;
      const int id0 = __shfl_sync(0xffffffffu, win, (fb - win_b) & 31);
      const int id1 = __shfl_sync(0xffffffffu, win, (fb - win_b + 1) & 31);
      const uint32_t dst = ring_at + fslot * C::STAGE;
      const int64_t o0 = id0 * block_stride + fh * TB, o1 = id1 * block_stride + fh * TB;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        copy16(dst + my_dst + i * 512, my_k + o0 + i * 512);
        copy16(dst + TB + my_dst + i * 512, my_v + o0 + i * 512);
      }
      if (two) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          copy16(dst + 2 * TB + my_dst + i * 512, my_k + o1 + i * 512);
          copy16(dst + 3 * TB + my_dst + i * 512, my_v + o1 + i * 512);
        }
      }
      if (pt < (two ? 4 : 2)) copy16(dst + my_pair_dst, my_pair + (pt & 2 ? o1 : o0));
      fslot = fslot + 1 == NST ? 0 : fslot + 1;
      const int n = two ? 2 : 1;
      fleft -= n;
      fb += n;
      if (fb == fsp.nb && fleft > 0) {
        fb = 0;
        if (++fh == a.hkv) {
          fh = 0;
          do {  // the next sequence with tokens (units are left: there is one)
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
  // a lane's part of a piece's queries: with one eight of them asked for a
  // piece ahead, the first before the blocks
  constexpr bool kAhead = NR == 1;
  uint4 raw[NR][NG][2];
  auto ask_queries = [&](int seq, int head) {
    const int64_t row0 = static_cast<int64_t>(seq) * a.hq + head * a.g;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int query = (NQ == 4 ? gq & 3 : gq) + 8 * r;
#pragma unroll
      for (int p = 0; p < NG; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          raw[r][p][j] = query < a.g
                             ? __ldg(reinterpret_cast<const uint4 *>(a.q + (row0 + query) * D + 64 * p + 16 * t) + j)
                             : make_uint4(0, 0, 0, 0);
    }
  };
  if constexpr (kAhead) ask_queries(cseq, ch);
#pragma unroll 1
  for (int i = 0; i < NST - 1; ++i) fetch();

  // --- addresses of a lane's operands in a staged tile
  const int krow = (gq >> 1) + 4 * (gq & 1);
  const int kat = staged<D>(krow, 8 * t);                                    // group 1: ^ 32
  const int vat0 = staged<D>(t, 4 * gq), vat1 = staged<D>(t + 4, 4 * gq);  // rows t + 4 i: i even, odd
  constexpr int ROW8 = 8 * (D / 2);                                          // eight rows further

  const float low = t < 2 ? 0.f : -1.f;
  int cslot = 0;
  long long cu = u0;
#pragma unroll 1
  while (cu < u1) {
    // --- one (sequence, kv head), or this warp's part of it
    const long long seg = cu - cb;
    const int b_end = static_cast<int>(min(static_cast<long long>(csp.nb), cb + (u1 - cu)));
    cu += b_end - cb;
    const int64_t row0 = static_cast<int64_t>(cseq) * a.hq + ch * a.g;

    if constexpr (!kAhead) ask_queries(cseq, ch);

    // per lane: its part of query gq's dims, and the rest of queries 2 t, 2 t + 1
    uint32_t qf[NR][D / 16][2];
    float cs_[NR][2], cm[NR][NG][2], l[NR][2], mz[NR][NG][2];
    // Weights are 2^(x - M + k) with the running maximum M: k, per query and group
    // of dims, brings the largest weight times scale to about 2^4 (in fp16 the
    // hi + lo pair then has 22 bits down to 2^-18 of that, and 2^-29 of it below).
    // shift = k - M of group 0; rat = 2^(k - its k) of group 1; lim = 2^(7 - k).
    float shift[NR][2], lim[NR][2], rat[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float amax = 0.f, sum[NG];
      float f[NG][16];
#pragma unroll
      for (int p = 0; p < NG; ++p) {
        sum[p] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = j < 4 ? (&raw[r][p][0].x)[j] : (&raw[r][p][1].x)[j - 4];
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
      const float cq = a.qscale * __uint_as_float(static_cast<uint32_t>(127 + kCodeExp + e) << 23);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        cs_[r][c] = __shfl_sync(0xffffffffu, cq, 8 * t + 4 * c);
#pragma unroll
        for (int p = 0; p < NG; ++p) {
          cm[r][p][c] = a.qscale * __shfl_sync(0xffffffffu, sum[p], 8 * t + 4 * c);
          mz[r][p][c] = 0.f;
        }
        shift[r][c] = kNone;
        lim[r][c] = 128.f;
        rat[r][c] = 1.f;
        l[r][c] = 0.f;
      }
    }
    // the (sequence, kv head) of the next piece
    int nseq = cseq, nh = ch;
    Span nsp = csp;
    if (cu < u1) {
      if (++nh == a.hkv) {
        nh = 0;
        do {
          ++nseq;
          nsp = span_of(a, __ldg(a.lens + nseq));
        } while (nsp.nb == 0 && nseq + 1 < a.num_seqs);
      }
      if constexpr (kAhead) ask_queries(nseq, nh);
    }
    float sum[NR][NG][4][4];  // [queries 0..7, 8..15][group][16 dims]
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int p = 0; p < NG; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[r][p][j][i] = 0.f;
#pragma unroll 1
    while (cb < b_end) {
      cp_async_wait<NST - 2>();
      __syncwarp();
      fetch();
      const int n = b_end - cb < 2 ? 1 : 2;
      const uint8_t *const st = ring + cslot * C::STAGE;
      // Both blocks of the stage in step (where there is one only, the other's
      // tokens are masked).
      const int pos0 = (csp.b0 + cb) * 16;

      // scores: x[r][tt][i][c] of token krow + 8 i and query 2 t + c (+ 8 r)
      float x[NR][2][2][2];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const uint8_t *const kt = st + 2 * tt * TB;
        float s[NR][NG][4];
#pragma unroll
        for (int p = 0; p < NG; ++p) {
          const uint2 k0 = lds64(kt + (kat ^ (32 * p))), k8 = lds64(kt + (kat ^ (32 * p)) + ROW8);
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t u = place(h < 2 ? k0.x : k0.y, h & 1), v = place(h < 2 ? k8.x : k8.y, h & 1);
            const uint32_t a0 = u & kLowCodes, a1 = v & kLowCodes, a2 = u & kHighCodes, a3 = v & kHighCodes;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              if (h == 0)
                mma0(s[r][p], a0, a1, a2, a3, qf[r][p * 4 + h][0], qf[r][p * 4 + h][1]);
              else
                mma(s[r][p], a0, a1, a2, a3, qf[r][p * 4 + h][0], qf[r][p * 4 + h][1]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[2];
          load_pairs<NG>(kt + i4::code_bytes(D) + (krow + 8 * i) * (4 * NG), w);
          const float2 g0 = halves(w[0]), g1 = halves(w[NG - 1]);  // scale, minimum
#pragma unroll
          for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float y = s[r][0][2 * i + c] * g0.x, z = g0.y * cm[r][0][c];
              if constexpr (NG == 2) {
                y = fmaf(s[r][NG - 1][2 * i + c], g1.x, y);
                z = fmaf(g1.y, cm[r][NG - 1][c], z);
              }
              x[r][tt][i][c] = fmaf(y, cs_[r][c], z);
            }
        }
      }

      // the values' scales and minima; masked tokens have neither.  The weights
      // of a block's last eight tokens are negated and their codes taken from
      // 15, s n + m = (m + 15 s) - s (15 - n): codes are never negative, and
      // without this the two sums, of codes and of minima, would grow far past
      // their difference (131069 tokens: outputs off by 2e-4 of their norm).
      float vs[2][2][NG], vm[2][2][NG];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[2];
          load_pairs<NG>(st + (2 * tt + 1) * TB + i4::code_bytes(D) + (krow + 8 * i) * (4 * NG), w);
#pragma unroll
          for (int p = 0; p < NG; ++p) {
            const float2 g = halves(w[p]);
            vs[tt][i][p] = g.x;
            vm[tt][i][p] = i == 0 ? g.y : fmaf(15.f, g.x, g.y);
          }
        }
      if (n < 2 || pos0 < csp.first || csp.len - pos0 < 32) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int pos = pos0 + 16 * tt + krow + 8 * i;
            if (tt >= n || pos < csp.first || pos >= csp.len) {
#pragma unroll
              for (int r = 0; r < NR; ++r) x[r][tt][i][0] = x[r][tt][i][1] = -INFINITY;
#pragma unroll
              for (int p = 0; p < NG; ++p) vs[tt][i][p] = vm[tt][i][p] = 0.f;
            }
          }
      }

      // M and the k are set anew only when a weight passes 2^8 or a product of
      // weight and scale 2^15: a vote, no shuffles.  (The bound taken here is the
      // largest weight times the largest scale of a lane's tokens.  Pages from
      // elsewhere may have scales of either sign.)
      auto mag = [&](int tt, int i, int p) { return fabsf(vs[tt][i][p]); };
      float smax[NG];
#pragma unroll
      for (int p = 0; p < NG; ++p) smax[p] = fmaxf(fmax3(mag(0, 0, p), mag(0, 1, p), mag(1, 0, p)), mag(1, 1, p));
      bool raise = false;
      float w[NR][2][2][2];
      auto weigh = [&](int r, int c) {
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int i = 0; i < 2; ++i) w[r][tt][i][c] = ex2_approx(x[r][tt][i][c] + shift[r][c]);
      };
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          weigh(r, c);
          const float u = NG == 2 ? fmax3(smax[0], smax[NG - 1] * rat[r][c], lim[r][c]) : fmaxf(smax[0], lim[r][c]);
          raise |= fmaxf(fmax3(w[r][0][0][c], w[r][0][1][c], w[r][1][0][c]), w[r][1][1][c]) * u > 32768.f;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float k[2], n[2];  // of the groups, before and after
            k[0] = static_cast<float>(134 - static_cast<int>(__float_as_uint(lim[r][c]) >> 23));
            k[1] = k[0] + static_cast<float>(static_cast<int>(__float_as_uint(rat[r][c]) >> 23) - 127);
            const float xmax = fmaxf(fmax3(x[r][0][0][c], x[r][0][1][c], x[r][1][0][c]), x[r][1][1][c]);
            const float m0 = k[0] - shift[r][c], m = fmaxf(m0, warp_max_xor(xmax, 4, 32));
#pragma unroll
            for (int p = 0; p < NG; ++p) {
              // the largest weight times scale so far (within one binary place
              // per raise, from k) and of these tokens, relative to m
              float top = -INFINITY;
#pragma unroll
              for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int i = 0; i < 2; ++i) top = fmaxf(top, x[r][tt][i][c] + __log2f(mag(tt, i, p)));
              top = fmaxf(warp_max_xor(top, 4, 32) - m, (m0 - m) + (4.f - k[p]));
              n[p] = fminf(fmaxf(ceilf(4.f - top), -40.f), 60.f);
            }
            const float to = n[0] - m;
#pragma unroll
            for (int p = 0; p < NG; ++p) {
              const float alpha = ex2_approx((to - shift[r][c]) + ((n[p] - n[0]) - (k[p] - k[0])));
              if (p == 0) l[r][c] *= alpha;
              mz[r][p][c] *= alpha;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                sum[r][p][j][c] *= alpha;
                sum[r][p][j][2 + c] *= alpha;
              }
            }
            shift[r][c] = to;
            lim[r][c] = power_of_two(7 - static_cast<int>(n[0]));
            if constexpr (NG == 2) rat[r][c] = power_of_two(static_cast<int>(n[1] - n[0]));
            weigh(r, c);
          }
      }

      float acc[NR][NG][4][4];  // the stage's products
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const uint8_t *const vt = st + (2 * tt + 1) * TB;
        // weights times scales as hi + lo, turned into operands (token pairs of
        // a query) by 8 x 8 transposes
        uint32_t hi[NR][NG][2], lo[NR][NG][2];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w0 = w[r][tt][i][0], w1 = w[r][tt][i][1];
            l[r][0] += w0;
            l[r][1] += w1;
#pragma unroll
            for (int p = 0; p < NG; ++p) {
              const float2 u = p == 0 ? make_float2(w0, w1)
                                      : f2_unpack(f2_mul(f2_pack(w0, w1), f2_pack(rat[r][0], rat[r][1])));
              mz[r][p][0] = fmaf(u.x, vm[tt][i][p], mz[r][p][0]);
              mz[r][p][1] = fmaf(u.y, vm[tt][i][p], mz[r][p][1]);
              const float sv = i == 0 ? vs[tt][i][p] : -vs[tt][i][p];
              const float y0 = u.x * sv, y1 = u.y * sv;
              const uint32_t h = pack_f16x2(y0, y1);
              const float2 hf = halves(h);
              if constexpr (NQ == 4) {  // the lo halves in the columns of queries 4..7 (y - 0 h is y)
                hi[r][p][i] = transposed(pack_f16x2(fmaf(low, hf.x, y0), fmaf(low, hf.y, y1)));
              } else {
                hi[r][p][i] = transposed(h);
                lo[r][p][i] = transposed(pack_f16x2(y0 - hf.x, y1 - hf.y));
              }
            }
          }
#pragma unroll
        for (int p = 0; p < NG; ++p) {
          const uint32_t w0 = lds32(vt + (vat0 ^ (32 * p))), w1 = lds32(vt + (vat1 ^ (32 * p)));
          const uint32_t w2 = lds32(vt + (vat0 ^ (32 * p)) + ROW8), w3 = lds32(vt + (vat1 ^ (32 * p)) + ROW8);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t b0 = __byte_perm(w0, w1, h ? 0x7632 : 0x5410);
            const uint32_t b1 = __byte_perm(w2, w3, h ? 0x7632 : 0x5410);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t c0 = place(b0, j), c1 = place(b1, j);
              const uint32_t v0 = c0 & kLowCodes, v1 = c0 & kHighCodes, v2 = ~c1 & kLowCodes, v3 = ~c1 & kHighCodes;
#pragma unroll
              for (int r = 0; r < NR; ++r) {
                if (tt == 0)
                  mma0(acc[r][p][2 * h + j], v0, v1, v2, v3, hi[r][p][0], hi[r][p][1]);
                else
                  mma(acc[r][p][2 * h + j], v0, v1, v2, v3, hi[r][p][0], hi[r][p][1]);
                if constexpr (NQ != 4) mma(acc[r][p][2 * h + j], v0, v1, v2, v3, lo[r][p][0], lo[r][p][1]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int p = 0; p < NG; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[r][p][j][i] += acc[r][p][j][i];
      cslot = cslot + 1 == NST ? 0 : cslot + 1;
      cb += n;
    }

    // --- the end of the piece: to the outputs, or to a slot for the join
    const bool whole = seg >= u0 && seg + csp.nb <= u1;
    const int slot = 2 * warp + (seg >= u0 ? 1 : 0);
    float *dst = whole ? a.out + row0 * D : part_o + slot * a.g * D;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int query = 2 * t + c + 8 * r;
        const bool has = query < a.g && (NQ != 4 || t < 2);
        float lsum = l[r][c], z[NG];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
#pragma unroll
        for (int p = 0; p < NG; ++p) {
          z[p] = mz[r][p][c];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) z[p] += __shfl_xor_sync(0xffffffffu, z[p], o);
        }
        const float ref = shift[r][c] == kNone ? -INFINITY : -shift[r][c];
        const float inv = !whole ? 1.f : lsum == 0.f ? 0.f : 1.f / lsum;
        if (gq == 0 && has) {
          if (!whole)
            part_ml[slot * a.g + query] = make_float2(ref, lsum);
          else if (a.lse)
            a.lse[row0 + query] = lsum == 0.f ? -INFINITY : (ref + log2f(lsum)) * kLn2;
        }
#pragma unroll
        for (int p = 0; p < NG; ++p) {
          // 2^22 for the codes' place in fp16, a sixteenth of it for the odd dims;
          // 1 / rat
          const float by = p == 0 ? inv : inv * __uint_as_float((254u << 23) - __float_as_uint(rat[r][c]));
          float o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float e = sum[r][p][j][c], d = sum[r][p][j][2 + c];
            if constexpr (NQ == 4) {  // the lo halves, from the columns of queries 4..7
              e += __shfl_xor_sync(0xffffffffu, e, 2);
              d += __shfl_xor_sync(0xffffffffu, d, 2);
            }
            o[2 * j] = fmaf(e, static_cast<float>(1 << kCodeExp), z[p]) * by;
            o[2 * j + 1] = fmaf(d, static_cast<float>(1 << (kCodeExp - 4)), z[p]) * by;
          }
          if (has) {
            float4 *to = reinterpret_cast<float4 *>(dst + query * D + 64 * p + 8 * gq);
            to[0] = make_float4(o[0], o[1], o[2], o[3]);
            to[1] = make_float4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    if (!whole && lane == 0) pieces[slot] = Piece{seg, row0, csp.nb};

    cseq = nseq;
    ch = nh;
    csp = nsp;
    cb = 0;
  }
  cp_async_wait<0>();
  }  // u0 < u1

  // --- sequences without tokens
#pragma unroll 1
  for (int s = blockIdx.x * kWarps + warp; s < a.num_seqs; s += gridDim.x * kWarps) {
    if (span_of(a, __ldg(a.lens + s)).nb > 0) continue;
    for (int i = lane; i < a.hq * D; i += 32) a.out[static_cast<int64_t>(s) * a.hq * D + i] = 0.f;
    if (a.lse)
      for (int i = lane; i < a.hq; i += 32) a.lse[static_cast<int64_t>(s) * a.hq + i] = -INFINITY;
  }
  if (idle) return;

  // --- pieces of this CTA's warps joined
  __syncthreads();
  const long long c0 = starts[0], c1 = starts[kWarps];
  static_assert(2 * kWarps <= 32, "a lane a piece");
  // lane k: piece k; whether it is the first here of its (sequence, kv head),
  // and the warps (bits) that have its further pieces
  Piece pc = pieces[lane < 2 * kWarps ? lane : 0];
  if (lane >= 2 * kWarps) pc.nb = 0;
  const long long end = pc.seg + pc.nb;
  const bool lead = pc.nb > 0 && starts[lane >> 1] <= (pc.seg > c0 ? pc.seg : c0);
  const bool here = pc.seg >= c0 && end <= c1;
  const unsigned has0 = __ballot_sync(0xffffffffu, pc.nb > 0);  // bit 2 w: warp w has a piece that began before it
  unsigned more = 0;
#pragma unroll
  for (int x = 1; x < kWarps; ++x)
    more |= (x > lane >> 1 && starts[x] < end && (has0 >> (2 * x) & 1u)) ? 1u << x : 0u;
  unsigned todo = __ballot_sync(0xffffffffu, lead);
  // kRows rows at a time, in step: a warp for each such part of a (sequence, kv
  // head).  (A row at a time: 1,100 to 1,900 cycles each.)
  constexpr int kLanes = kWarps <= 8 ? 8 : 16, kRows = 32 / kLanes;
  for (int part = 0; todo; todo &= todo - 1) {
    const int k = __ffs(todo) - 1, w = k >> 1;
    const unsigned in = __shfl_sync(0xffffffffu, more, k) | 1u << w;
    const bool out = __shfl_sync(0xffffffffu, here, k);
    const bool second = __shfl_sync(0xffffffffu, pc.seg >= c0, k);
    const int64_t row0 = __shfl_sync(0xffffffffu, pc.row0, k);
#pragma unroll 1
    for (int r0 = 0; r0 < a.g; r0 += kRows, ++part) {
      if (part % kWarps != warp) continue;
      // lane: the piece of warp lane % kLanes, row r0 + lane / kLanes
      const int x = lane % kLanes, r = r0 + lane / kLanes;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (x < kWarps && (in >> x & 1u) && r < a.g) ml = part_ml[(x == w ? k : 2 * x) * a.g + r];
      float ref = ml.x;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
      const float f = weight_of(ml, ref);
      float l = f * ml.y;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      Part<D> o[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) o[j].clear();
#pragma unroll 1
      for (unsigned left = in; left; left &= left - 1) {
        const int y = __ffs(left) - 1;
        const float *from = part_o + ((y == w ? k : 2 * y) * a.g + r0) * D + lane * (D / 32);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          Part<D> v;
          v.clear();
          if (r0 + j < a.g) v.load(from + j * D);
          o[j].add(__shfl_sync(0xffffffffu, f, j * kLanes + y), v);
        }
      }
      const int64_t at = out ? row0 + r0 : (2 * static_cast<int64_t>(cta) + (second ? 1 : 0)) * a.g + r0;
      const float by = !out ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const float byj = __shfl_sync(0xffffffffu, by, j * kLanes);
        if (r0 + j < a.g) o[j].store((out ? a.out : a.slot_o) + (at + j) * D + lane * (D / 32), byj);
      }
      if (x == 0 && r < a.g) {
        if (!out)
          a.slot_ml[at + (r - r0)] = make_float2(ref, l);
        else if (a.lse)
          a.lse[at + (r - r0)] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
      }
    }
  }

  if (whole_only) return;

  // --- and what goes beyond this CTA, by the CTA that finishes its last piece.
  // Lane 0 of warp 0: what began before this CTA; lane 1: what begins here and
  // goes on.
  int mine = -1, ca = 0, n = 0;
  if (warp == 0) {
    const unsigned before = __ballot_sync(0xffffffffu, pc.nb > 0 && pc.seg < c0);
    const unsigned behind = __ballot_sync(0xffffffffu, pc.nb > 0 && pc.seg >= c0 && end > c1);
    mine = lane < 2 ? __ffs(lane == 0 ? before : behind) - 1 : -1;
    if (mine >= 0) {
      ca = deal.cta_of(pieces[mine].seg);
      n = deal.cta_of(pieces[mine].seg + pieces[mine].nb - 1) - ca + 1;
    }
  }
  __syncthreads();  // (the CTA's slots: released with the counts below)
  if (tid < 2) {
    if (mine >= 0 && atom_add_acq_rel_gpu(a.count + ca, 1) == n - 1) {
      st_relaxed_gpu(a.count + ca, 0);
    } else {
      mine = -1;
    }
    joins[tid] = Join{mine, ca, n};
  }
  __syncthreads();
#pragma unroll 1
  for (int i = warp; i < 2 * a.g; i += kWarps) {  // a row of one of the two a warp
    const Join jn = joins[i >= a.g];
    if (jn.piece < 0) continue;
    const int r = i >= a.g ? i - a.g : i;
    // slots, in the order of the units: the second of CTA ca, the first of those behind
    auto slot_of = [&](int i) { return 2 * static_cast<int64_t>(jn.ca + i) + (i == 0 ? 1 : 0); };
    float ref = -INFINITY, l = 0.f;
    Part<D> o;
    o.clear();
    for (int base = 0; base < jn.n; base += 32) {
      // a lane's piece's reference and sum; the dims come four pieces at a time
      const int m = min(32, jn.n - base);
      const float2 ml = lane < m ? __ldcg(&a.slot_ml[slot_of(base + lane) * a.g + r]) : make_float2(-INFINITY, 0.f);
      Part<D> v[4];
      auto ask = [&](int i0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i0 + i < m)
            v[i].load_l2(a.slot_o + (slot_of(base + i0 + i) * a.g + r) * D + lane * (D / 32));
          else
            v[i].clear();
        }
      };
      ask(0);
      const float up = fmaxf(ref, warp_max_xor(ml.x, 1, 32));
      const float f = weight_of(ml, up), keep = ref == -INFINITY ? 0.f : ex2_approx(ref - up);
      ref = up;
      l *= keep;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o.x[i] *= keep;
#pragma unroll 1
      for (int i0 = 0; i0 < m; i0 += 4) {
        if (i0) ask(i0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = (i0 + i) & 31;  // (lanes from m on have weight and sum 0)
          const float w = __shfl_sync(0xffffffffu, f, at);
          l = fmaf(w, __shfl_sync(0xffffffffu, ml.y, at), l);
          o.add(w, v[i]);
        }
      }
    }
    store_row<D>(a, pieces[jn.piece].row0 + r, ref, l, o);
  }
}

struct Kernel {
  const void *fn;
  int warps, smem;
};

template <int D, int NQ>
Kernel kernel_for() {
  return {reinterpret_cast<const void *>(&int4_decode_kernel<D, NQ>), Cfg<D, NQ>::W, Cfg<D, NQ>::SMEM};
}

template <int D>
Kernel kernel_of_dim(int g) {
  return g <= 4 ? kernel_for<D, 4>() : g <= 8 ? kernel_for<D, 8>() : kernel_for<D, 16>();
}

Kernel kernel_of(const pa_kv_desc &d) {
  const int g = d.num_q_heads / d.num_kv_heads;
  return d.head_dim == 128 ? kernel_of_dim<128>(g) : kernel_of_dim<64>(g);
}

// Of the workspace: the slots' statistics, their dims, and the end.
struct Layout {
  size_t ml, o, total;
};

Layout layout(int ctas, int g, int d) {
  const size_t slots = 2 * static_cast<size_t>(ctas);
  Layout w;
  w.ml = kWsSlots;
  w.o = (w.ml + slots * g * sizeof(float2) + 255) / 256 * 256;
  w.total = w.o + slots * g * d * sizeof(float);
  return w;
}

}  // namespace

pa_status plan_int4_decode(const pa_kv_desc &d, DecodePlan *plan, const char **why) {
  if (d.decode_impl != PA_DECODE_AUTO && d.decode_impl != PA_DECODE_MMA) {
    *why = "a 4-bit cache is decoded on the tensor cores (decode_impl AUTO or MMA)";
    return PA_ERR_UNSUPPORTED;
  }
  const Kernel k = kernel_of(d);
  const int occ = prepare_kernel(k.fn, k.warps * 32, k.smem);
  if (occ < 1) {
    *why = "the decode kernel does not fit on this device";
    return PA_ERR_CUDA;
  }
  plan->impl = PA_DECODE_MMA;
  plan->slot_heads = d.num_q_heads / d.num_kv_heads;
  plan->num_groups = d.num_kv_heads;
  plan->num_ctas = device_sm_count();
  if (kWsCtaCounters + plan->num_ctas * sizeof(int32_t) > kWsSlots) {
    *why = "more SMs than the workspace has counters for";
    return PA_ERR_UNSUPPORTED;
  }
  const Layout w = layout(plan->num_ctas, plan->slot_heads, d.head_dim);
  plan->slots = w.ml;
  plan->counters = kWsCtaCounters;
  plan->workspace_bytes = w.total;
  plan->zero_bytes = kWsCtaCounters + plan->num_ctas * sizeof(int32_t);
  return PA_OK;
}

cudaError_t launch_int4_decode(const pa_kv_desc &d, const DecodePlan &plan, float *out, float *lse, const void *q,
                               const void *k_cache, const void *v_cache, const int32_t *block_tables,
                               int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t num_seqs, float scale,
                               void *workspace, cudaStream_t stream) {
  const Kernel k = kernel_of(d);
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
  a.count = reinterpret_cast<int32_t *>(ws + plan.counters);
  a.slot_ml = reinterpret_cast<float2 *>(ws + w.ml);
  a.slot_o = reinterpret_cast<float *>(ws + w.o);
  // programmatic dependent launch: it waits for the preceding kernel's writes
  // (the cache write) before reading anything
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.num_ctas);
  cfg.blockDim = dim3(k.warps * 32);
  cfg.dynamicSmemBytes = k.smem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  void *args[] = {&a};
  return cudaLaunchKernelExC(&cfg, k.fn, args);
}

}  // namespace pa
