// pa_shared_kernels.cuh -- decode attention of a batch whose sequences share
// prefixes, each prefix read once for all the sequences of its group.
//
// For sequence s of group j, query head h and kv head h / g:
//   out[s][h] = sum_t softmax_t(scale * q[s][h] . K_t) V_t,   t < L_s.
// The first P_j tokens of a group's sequences are the same cache blocks, so
// the sum is cut at P_j: the queries of all the group's sequences attend the
// prefix together, each sequence attends its own rest, and the parts (each
// normalised by its own sum, with its log-sum-exp) are joined by weights
// 2^(lse_p - max lse).
//
// What bounds it: the K/V bytes (each prefix once per group and kv head, each
// own part once) while a group has up to about 64 (sequence, head) rows per
// kv head; with more rows the products of the prefix.
//
// Three launches:
//  * shared_plan_kernel (one CTA) turns the lengths into a list of items --
//    (group, tile of rows, kv head) over the prefix's blocks, and
//    (sequence, kv head) over its own blocks -- laid out on one axis of
//    work units (a block costs more units in a tile of many rows).
//  * shared_attend_kernel, one persistent CTA per SM: CTA c takes the units
//    [c U / G, (c + 1) U / G) of that axis, so every CTA has the same work
//    whatever the lengths.  A producer warp streams the blocks by TMA into a
//    ring; 8 consumer warps run m16n8k16 MMAs with the rows as M: a tile of
//    up to 128 rows is RG row groups of 16 x KG = 8 / RG key groups, so one
//    sequence's few heads spread their keys over all 8 warps and a wide tile
//    spreads its rows.  P enters P V as a hi + lo pair of 16-bit values
//    (near-fp32), 8-bit caches are widened to fp16 in registers.
//  * shared_join_kernel, one warp per (sequence, head): joins the parts.
#pragma once

#include <cuda.h>

#include "pa_decode_kernels.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace shd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int NC = 8;            // consumer warps; warp NC produces
constexpr int NTHREADS = (NC + 1) * 32;
constexpr int MAXROWS = 16 * NC;  // rows of a tile
constexpr int kMaxSeqs = 65535;   // sequences of a call (as pa_prefill_chunk)
// the running maximum of a row is only raised when a score exceeds it by
// more than this (log2 units), so that O is rarely rescaled
constexpr float kRaise = 8.f;

// One group's prefix on the work axis.
struct __align__(16) GroupInfo {
  long long base;  // first unit
  int first;       // first sequence
  int n;           // sequences
  int nb;          // blocks of the prefix that some sequence reads (0: nothing shared)
  int kend;        // keys of the prefix that some sequence reads
  int tile_seqs;   // sequences of a tile (the last tile may have fewer)
  int w;           // units of a block
  int row;         // a sequence whose table holds all of the prefix that is read
  int pad[3];
};
// One sequence's own part.
struct __align__(16) SeqInfo {
  long long base;
  int len;    // tokens
  int fb;     // first own block
  int nb;     // own blocks
  int group;  // its group, -1: none
  int pad[2];
};
// Where a CTA's range begins.
struct __align__(16) CtaStart {
  int kind;  // 0 prefix item, 1 own part, 2 nothing to do
  int idx;   // group or sequence
  int sub;   // tile * kv heads + kv head, or kv head
  int pad;
};

constexpr int kOwnUnits = 4;  // units of a block of an own part

// Units of a prefix block in a tile of `rows` rows: the stream bounds tiles of
// up to 64 rows, their MMAs the wider ones.
__host__ __device__ constexpr int tile_units(int rows) { return rows <= 64 ? 4 : (rows + 15) / 16; }

struct Args {
  CUtensorMap kmap;
  CUtensorMap vmap;
  float *out;
  float *lse;
  const uint16_t *q;
  const int32_t *block_tables;
  const int32_t *context_lens;
  const int32_t *group_start;
  const int32_t *prefix_lens;
  int max_blocks;
  int num_seqs;
  int num_groups;
  int num_kv;
  int num_q;
  int g;
  int tile_rows;  // rows a tile may have (a multiple of g, at most MAXROWS)
  int slot_rows;  // rows of a cut item's slot
  int ctas;       // CTAs that share the work axis
  float qscale;   // scale * k_scale * log2(e)
  float qscale0;  // scale * log2(e)
  float vscale;
  const float *k_scales;
  const float *v_scales;
  int num_blocks;
  int checked;
  int stall;
  unsigned long long wait_ns;
  int32_t *err;
  // workspace
  long long *units;     // [1] U
  GroupInfo *groups;
  SeqInfo *seqs;
  CtaStart *starts;
  float *pre_o;         // [S][Hq][D] prefix parts of uncut items, normalised
  float *pre_lse;       // [S][Hq], log2 units
  float *own_o;         // ... own parts
  float *own_lse;
  float *cut_o;         // [ctas][2][slot_rows][D] pieces of cut items
  float *cut_lse;
};

// CTA c's units are [first_unit(c), first_unit(c + 1)); cta_of(u) holds u.
__device__ __forceinline__ long long first_unit(long long c, long long U, int G) { return c * U / G; }
__device__ __forceinline__ int cta_of(long long u, long long U, int G) {
  return static_cast<int>(((u + 1) * G - 1) / U);
}
// Blocks [lo, hi) of an item of nb blocks, w units each, from unit u0, that
// the units [b0, b1) hold: those whose first unit lies there.
__device__ __forceinline__ void piece_blocks(long long u0, int nb, int w, long long b0, long long b1, int &lo,
                                             int &hi) {
  lo = b0 <= u0 ? 0 : static_cast<int>((b0 - u0 + w - 1) / w);
  hi = static_cast<int>(min((b1 - u0 + w - 1) / w, static_cast<long long>(nb)));
}

// ------------------------------------------------------------------ planning

constexpr int PLAN_THREADS = 1024;

// Exclusive prefix sum over the CTA's threads; *total gets the sum.
__device__ __forceinline__ long long scan_exclusive(long long v, long long *total, long long *s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  __syncthreads();  // s_warp may still be read from the last call
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  long long before = 0, sum = 0;
  for (int i = 0; i < PLAN_THREADS / 32; ++i) {
    const long long x = s_warp[i];
    if (i < warp) before += x;
    sum += x;
  }
  *total = sum;
  return before + incl - v;
}

static __global__ void __launch_bounds__(PLAN_THREADS) shared_plan_kernel(const __grid_constant__ Args a) {
  __shared__ long long s_warp[PLAN_THREADS / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.num_seqs, G = a.num_groups;
  const int cap = a.max_blocks * 16;
  for (int s = tid; s < S; s += PLAN_THREADS) {
    int L = __ldg(a.context_lens + s);
    if (a.checked) L = checked_len(L, cap, a.err, nullptr);
    SeqInfo &q = a.seqs[s];
    q.len = max(L, 0);
    q.fb = 0;
    q.group = -1;
  }
  for (int c = tid; c < a.ctas; c += PLAN_THREADS) a.starts[c] = CtaStart{2, 0, 0, 0};
  __syncthreads();
  // one warp per group: its sequences, and how much of the prefix they read
  const int tile_seqs = a.tile_rows / a.g;
  for (int j = warp; j < G; j += PLAN_THREADS / 32) {
    const int r0 = __ldg(a.group_start + j), r1 = __ldg(a.group_start + j + 1);
    int P = __ldg(a.prefix_lens + j);
    // whatever the arrays hold, no access leaves the batch
    const int s0 = min(max(r0, 0), S), s1 = min(max(r1, s0), S);
    if (a.checked && lane == 0 && (r0 != s0 || r1 != s1 || P < 0 || P > cap)) report_error(a.err, nullptr, kErrBadIndex);
    P = min(max(P, 0), cap) & ~15;
    if (s1 - s0 < 2) P = 0;  // nobody to share with
    int mine = -1, row = 0;
    for (int s = s0 + lane; s < s1; s += 32) {
      const int n = min(a.seqs[s].len, P);
      if (n > mine) {
        mine = n;
        row = s;
      }
      a.seqs[s].fb = P >> 4;
      a.seqs[s].group = j;
    }
    const int best = __reduce_max_sync(0xffffffffu, mine);
    row = __reduce_min_sync(0xffffffffu, mine == best ? row : 0x7fffffff);
    const int top = max(best, 0);
    if (lane == 0) {
      GroupInfo q;
      q.row = row;
      q.base = 0;
      q.first = s0;
      q.n = s1 - s0;
      q.kend = top;
      q.nb = (top + 15) >> 4;
      const int tiles = max(1, (q.n + tile_seqs - 1) / tile_seqs);
      q.tile_seqs = max(1, (q.n + tiles - 1) / tiles);
      q.w = tile_units(q.tile_seqs * a.g);
      a.groups[j] = q;
    }
  }
  __syncthreads();
  // places on the work axis: prefix items, then own parts
  long long at = 0;
  for (int j0 = 0; j0 < G; j0 += PLAN_THREADS) {
    const int j = j0 + tid;
    long long v = 0;
    if (j < G) {
      const GroupInfo &q = a.groups[j];
      const int tiles = (q.n + q.tile_seqs - 1) / q.tile_seqs;
      v = static_cast<long long>(q.nb) * q.w * tiles * a.num_kv;
    }
    long long sum;
    const long long e = scan_exclusive(v, &sum, s_warp);
    if (j < G) a.groups[j].base = at + e;
    at += sum;
  }
  for (int s0 = 0; s0 < S; s0 += PLAN_THREADS) {
    const int s = s0 + tid;
    long long v = 0;
    int nb = 0;
    if (s < S) {
      const SeqInfo &q = a.seqs[s];
      nb = max(0, ((q.len + 15) >> 4) - q.fb);
      v = static_cast<long long>(nb) * kOwnUnits * a.num_kv;
    }
    long long sum;
    const long long e = scan_exclusive(v, &sum, s_warp);
    if (s < S) {
      a.seqs[s].nb = nb;
      a.seqs[s].base = at + e;
    }
    at += sum;
  }
  const long long U = at;
  if (tid == 0) *a.units = U;
  if (U == 0) return;
  __syncthreads();
  // each item's owner names it to the CTAs whose first unit it holds
  auto name = [&](int kind, int idx, long long base, long long item, int items) {
    if (item == 0) return;
    const long long end = base + item * items;
    // the first CTA whose first unit is >= base: floor(c U / G) >= base
    for (long long c = (base * a.ctas + U - 1) / U; c < a.ctas; ++c) {
      const long long u = first_unit(c, U, a.ctas);
      if (u >= end) break;
      if (u >= base) a.starts[c] = CtaStart{kind, idx, static_cast<int>((u - base) / item), 0};
    }
  };
  for (int j = tid; j < G; j += PLAN_THREADS) {
    const GroupInfo &q = a.groups[j];
    name(0, j, q.base, static_cast<long long>(q.nb) * q.w, (q.n + q.tile_seqs - 1) / q.tile_seqs * a.num_kv);
  }
  for (int s = tid; s < S; s += PLAN_THREADS)
    name(1, s, a.seqs[s].base, static_cast<long long>(a.seqs[s].nb) * kOwnUnits, a.num_kv);
}

// ------------------------------------------------------------------- attend

constexpr int kFirst = 1;  // the stage begins a piece
constexpr int kLast = 2;   // ... ends it
constexpr int kToOut = 0;  // a piece's result: the output itself,
constexpr int kToPre = 1;  // the prefix parts, the own parts,
constexpr int kToOwn = 2;
constexpr int kToCut = 3;  // or a cut item's slot

struct __align__(16) Stage {
  int kind;    // 0 data, 1 end
  int flags;
  int seq0;    // first sequence of the tile
  int rows;    // rows of the tile (sequences x g)
  int kvh;
  int key0;    // position of the stage's first token
  int kend;    // keys from here on are not the item's
  int blk;     // the stage's first block within the piece
  int nblk;
  int to;
  int slot;    // kToCut: the slot
  int prefix;  // 1: rows have limits of their own (their lengths)
};

template <int D_, int KVT_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int KVT = KVT_;
  static constexpr int ESZ = kv16(KVT) ? 2 : 1;
  static constexpr int ROWB = D * ESZ;
  static constexpr int TILEB = 16 * ROWB;                // a block of one kv head
  static constexpr int BPS = 16384 / TILEB;              // blocks of a stage: 16 KB of K, 16 KB of V
  static constexpr int KVB = BPS * TILEB;
  static constexpr int STAGEB = 2 * KVB;
  static constexpr int REDW = (D / 2 + 4) * 32;          // floats of a warp's partial state
  static constexpr int NRED = NC / 2;                    // warps that write one at a time
  static constexpr int FIXED = NRED * REDW * 4 + 2048;
  static constexpr int NS = (230000 - 1024 - FIXED) / STAGEB;
  static constexpr size_t SMEM = 1024 + size_t(NS) * STAGEB + FIXED;
  // exponent offset of P: fp16 P keeps small probabilities out of its
  // subnormals; with kRaise the largest P is 2^(8 + 6), below fp16's range
  static constexpr float PB = KVT == kKvBf16 ? 0.f : 6.f;
  static_assert(NS >= 3 && SMEM <= 232448, "ring");
};

template <class C>
__device__ void produce(const Args &a, uint8_t *ring, Stage *hdr, uint64_t *full, uint64_t *empty, int lane) {
  constexpr int BPS = C::BPS;
  const int me = blockIdx.x, G = a.ctas;
  const long long U = *a.units;
  const uint64_t pol = l2_evict_first_policy();
  bool ok = true;
  int stage = 0, issued = 0;
  uint32_t par = 1;  // a fresh barrier counts its preceding phase as complete
  if (U > 0 && !a.stall) {
    const long long b0 = first_unit(me, U, G), b1 = first_unit(me + 1, U, G);
    const CtaStart st = a.starts[me];
    int kind = st.kind, idx = st.idx, sub = st.sub;
    if (b0 >= b1) kind = 2;
    while (kind < 2 && ok) {
      // the group's or sequence's items, from `sub` on
      int items, nb, w, fb, kend, seq0 = 0, nseq = 0, tile_seqs = 1, table_row;
      long long base;
      bool alone = false;
      if (kind == 0) {
        const GroupInfo q = a.groups[idx];
        items = q.nb > 0 ? (q.n + q.tile_seqs - 1) / q.tile_seqs * a.num_kv : 0;
        nb = q.nb;
        w = q.w;
        fb = 0;
        kend = q.kend;
        base = q.base;
        seq0 = q.first;
        nseq = q.n;
        tile_seqs = q.tile_seqs;
        table_row = q.row;
      } else {
        const SeqInfo q = a.seqs[idx];
        items = q.nb > 0 ? a.num_kv : 0;
        nb = q.nb;
        w = kOwnUnits;
        fb = q.fb;
        kend = q.len;
        base = q.base;
        table_row = idx;
        alone = q.fb == 0;
      }
      const int32_t *table = a.block_tables + static_cast<int64_t>(table_row) * a.max_blocks;
      auto entry = [&](int e) {  // physical block of the item's block e
        if (e >= nb) return 0;
        const int v = __ldg(table + fb + e);
        return a.checked ? checked_block(v, a.num_blocks, a.err, nullptr) : v;
      };
      for (; sub < items && ok; ++sub) {
        const long long u0 = base + static_cast<long long>(sub) * nb * w;
        const long long u1 = u0 + static_cast<long long>(nb) * w;
        if (u0 >= b1) {
          kind = 2;
          break;
        }
        int lo, hi;
        piece_blocks(u0, nb, w, b0, b1, lo, hi);
        const bool cut = b0 > u0 || b1 < u1;
        const int kvh = kind == 0 ? sub % a.num_kv : sub;
        const int t0 = kind == 0 ? sub / a.num_kv * tile_seqs : 0;
        // this lane's entry of the next 32, and of the 32 after them
        int win = lo, cur = entry(lo + lane), nxt = 0;
        if (hi - lo > 32) nxt = entry(lo + 32 + lane);
        for (int b = lo; b < hi; b += BPS) {
          const int n = min(BPS, hi - b);
          if (b - win >= 32) {
            win += 32;
            cur = nxt;
            nxt = win + 32 < hi ? entry(win + 32 + lane) : 0;
          }
          // BPS divides 32: a stage's entries are in one window
          const int phys = __shfl_sync(0xffffffffu, cur, (b - win + (lane % BPS)) & 31);
          if (!mbar_wait(&empty[stage], par, a.wait_ns)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            Stage h;
            h.kind = 0;
            h.flags = (b == lo ? kFirst : 0) | (b + BPS >= hi ? kLast : 0);
            h.seq0 = kind == 0 ? seq0 + t0 : idx;
            h.rows = (kind == 0 ? min(tile_seqs, nseq - t0) : 1) * a.g;
            h.kvh = kvh;
            h.key0 = (fb + b) * 16;
            h.kend = kend;
            h.blk = b - lo;
            h.nblk = n;
            h.to = cut ? kToCut : kind == 0 ? kToPre : alone ? kToOut : kToOwn;
            h.slot = me * 2 + (u0 <= b0 ? 0 : 1);
            h.prefix = kind == 0;
            hdr[stage] = h;
            mbar_arrive_expect_tx(&full[stage], 2u * n * C::TILEB);
          }
          __syncwarp();
          uint8_t *sk = ring + static_cast<size_t>(stage) * C::STAGEB;
          const int row = (phys * a.num_kv + kvh) * 16;
          // lanes 0 .. BPS - 1 copy K, the next BPS lanes V
          if (lane % BPS < n && lane < 2 * BPS) {
            const bool is_v = lane >= BPS;
            uint8_t *dst = sk + (is_v ? C::KVB : 0) + (lane % BPS) * C::TILEB;
            const CUtensorMap *map = is_v ? &a.vmap : &a.kmap;
            if constexpr (C::ROWB > 128)
              tma_load_3d(dst, map, 0, row, 0, &full[stage], pol);
            else
              tma_load_2d(dst, map, 0, row, &full[stage], pol);
          }
          ++issued;
          if (++stage == C::NS) {
            stage = 0;
            par ^= 1;
          }
        }
      }
      if (kind == 2 || !ok) break;
      // the next group with a prefix, after the last one the sequences with
      // an own part; the ones without work are passed over 32 at a time
      sub = 0;
      ++idx;
      auto next = [&](int n, auto blocks) {
        while (idx < n) {
          const unsigned some = __ballot_sync(0xffffffffu, idx + lane < n && blocks(idx + lane) > 0);
          if (some) {
            idx += __ffs(some) - 1;
            return true;
          }
          idx += 32;
        }
        return false;
      };
      if (kind == 0 && !next(a.num_groups, [&](int j) { return a.groups[j].nb; })) {
        kind = 1;
        idx = 0;
      }
      if (kind == 1 && !next(a.num_seqs, [&](int s) { return a.seqs[s].nb; })) kind = 2;
    }
  }
  if (ok && !a.stall) {
    if (mbar_wait(&empty[stage], par, a.wait_ns)) {
      if (lane == 0) {
        hdr[stage].kind = 1;
        mbar_arrive(&full[stage]);
      }
    } else {
      ok = false;
    }
  }
  if (!ok) {
    if (lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
    // the copies already issued land before the CTA can exit
    for (int i = 1; i <= min(issued, C::NS); ++i) {
      int st = stage - i;
      uint32_t p = par ^ 1;  // parity of the fill the ring index `stage` would get next, minus one lap
      if (st < 0) {
        st += C::NS;
        p ^= 1;
      }
      mbar_wait(&full[st], p, a.wait_ns);
    }
  }
}

template <class C>
__device__ void consume(const Args &a, uint8_t *ring, const Stage *hdr, uint64_t *full, uint64_t *empty, float *red,
                        uint64_t *join_bar, int warp, int lane) {
  constexpr int D = C::D;
  constexpr int KVT = C::KVT;
  constexpr int KS = D / 16;  // k-steps of Q K^T
  constexpr int NT = D / 8;   // n-tiles of P V
  const int r = lane >> 2, c = lane & 3;
  const int lm = lane >> 3, lr = lane & 7;
  uint32_t qa[KS][4];
  float o[NT][4];
  float m[2], l[2];
  int lim[2];
  float qsc = 0.f;
  int rg = 0, kg = 0, RG = 1, KG = 1;
  bool busy = false;
  uint32_t joins = 0;  // phases of join_bar so far
  int stage = 0;
  uint32_t par = 0;
  for (;;) {
    if (!mbar_wait(&full[stage], par, a.wait_ns)) {
      if (lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
      return;
    }
    const Stage h = hdr[stage];
    if (h.kind != 0) return;
    if (h.flags & kFirst) {
      RG = h.rows <= 16 ? 1 : h.rows <= 32 ? 2 : h.rows <= 64 ? 4 : 8;
      KG = NC / RG;
      rg = warp % RG;
      kg = warp / RG;
      busy = rg * 16 < h.rows;
      qsc = a.k_scales ? a.qscale0 * __ldg(a.k_scales + h.kvh) : a.qscale;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
        lim[e] = h.kend;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
      if (busy) {
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int R = rg * 16 + r + 8 * e;
          const bool live = R < h.rows;
          const int s = h.seq0 + (live ? R / a.g : 0);
          if (h.prefix) lim[e] = live ? min(h.kend, a.seqs[s].len) : 0;
          const uint16_t *src = a.q + (static_cast<int64_t>(s) * a.num_q + h.kvh * a.g + (live ? R % a.g : 0)) * D;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            if constexpr (kv16(KVT)) {
              // fragment columns 2c, 2c + 1 and 2c + 8, 2c + 9 are those dims
              qa[k][e] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 2 * c)) : 0u;
              qa[k][e + 2] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 2 * c + 8)) : 0u;
            } else {
              // an 8-bit K fragment's four bytes are dims 4c .. 4c + 3
              uint2 x = make_uint2(0, 0);
              if (live) x = __ldg(reinterpret_cast<const uint2 *>(src + 16 * k + 4 * c));
              const float f0 = bf16lo(x.x), f1 = bf16hi(x.x), f2 = bf16lo(x.y), f3 = bf16hi(x.y);
              big = fmaxf(big, fmaxf(fmaxf(fabsf(f0), fabsf(f1)), fmaxf(fabsf(f2), fabsf(f3))));
              qa[k][e] = pack_f16x2(f0, f1);
              qa[k][e + 2] = pack_f16x2(f2, f3);
            }
          }
        }
        // a finite query beyond fp16 does not fit the widened products
        if (!kv16(KVT) && big >= 65520.f && big <= FLT_MAX) report_error(a.err, nullptr, kErrFp16Range);
      }
    }
    if (busy) {
      const uint8_t *Ks = ring + static_cast<size_t>(stage) * C::STAGEB;
      for (int b = 0; b < h.nblk; ++b) {
        if ((h.blk + b) % KG != kg) continue;
        const uint32_t kt = smem_u32(Ks + b * C::TILEB);
        const uint32_t vt = smem_u32(Ks + C::KVB + b * C::TILEB);
        // ---- S (16 rows x 16 tokens, two n-tiles of 8) = Q K^T
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        if constexpr (kv16(KVT)) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t b0, b1, b2, b3;  // (tokens 0-7, dims 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
            ldmatrix_x4(b0, b1, b2, b3, kt + dec::swz_off<C::ROWB, 1>(lr + (lm >> 1) * 8, 2 * k + (lm & 1)));
            mma16_16816<KVT>(s[0], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b0, b1);
            mma16_16816<KVT>(s[1], qa[k][0], qa[k][1], qa[k][2], qa[k][3], b2, b3);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t x0, x1, x2, x3;  // 16-byte chunks k and k + 1 of tokens 0-7 and 8-15
            ldmatrix_x4(x0, x1, x2, x3, kt + dec::swz_off<C::ROWB, 1>(lr + (lm & 1) * 8, k + (lm >> 1)));
            const uint32_t w[4] = {x0, x1, x2, x3};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t lo = fp8x2_to_f16x2<KVT>(static_cast<uint16_t>(w[i] & 0xffffu));
              const uint32_t hi = fp8x2_to_f16x2<KVT>(static_cast<uint16_t>(w[i] >> 16));
              const int kk = k + (i >> 1);
              mma_f16_16816(s[i & 1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], lo, hi);
            }
          }
        }
        // ---- scores in log2 units, keys past a row's limit out
        const int key = h.key0 + 16 * b;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= qsc;
        if (h.prefix || key + 16 > h.kend) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + 8 * n + 2 * c + (e & 1) >= lim[e >> 1]) s[n][e] = -INFINITY;
        }
        // ---- the running maximum: raised only when a score is far above it
        const float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        const float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        if (__any_sync(0xffffffffu, t0 > m[0] + kRaise || t1 > m[1] + kRaise)) {
          float x[2] = {t0, t1};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 1));
            x[e] = fmaxf(x[e], __shfl_xor_sync(0xffffffffu, x[e], 2));
            const float mn = fmaxf(m[e], x[e]);
            const float f = mn == m[e] ? 1.f : exp2f(m[e] - mn);
            m[e] = mn;
            l[e] *= f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              o[t][2 * e] *= f;
              o[t][2 * e + 1] *= f;
            }
          }
        }
        // ---- P = 2^(s - m + PB), as a hi + lo pair
        uint32_t ph[4], pl[4];
        const float mu0 = (m[0] == -INFINITY ? 0.f : m[0]) - C::PB, mu1 = (m[1] == -INFINITY ? 0.f : m[1]) - C::PB;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2_approx(s[n][0] - mu0), p1 = ex2_approx(s[n][1] - mu0);
          const float p2 = ex2_approx(s[n][2] - mu1), p3 = ex2_approx(s[n][3] - mu1);
          l[0] += p0 + p1;
          l[1] += p2 + p3;
          constexpr int PT = KVT == kKvBf16 ? kKvBf16 : kKvF16;
          ph[2 * n] = pack16x2<PT>(p0, p1);
          ph[2 * n + 1] = pack16x2<PT>(p2, p3);
          pl[2 * n] = pack16x2<PT>(p0 - lo16<PT>(ph[2 * n]), p1 - hi16<PT>(ph[2 * n]));
          pl[2 * n + 1] = pack16x2<PT>(p2 - lo16<PT>(ph[2 * n + 1]), p3 - hi16<PT>(ph[2 * n + 1]));
        }
        // ---- O += P V.  Tokens past the item's keys may hold anything, NaN
        // included, which a zero probability does not cancel: zeroed in V
        const int vt0 = h.kend - key;
        auto keep = [&](int t) { return t < vt0; };
        uint32_t mk0 = 0xffffffffu, mk1 = 0xffffffffu;
        if (vt0 < 16) {
          mk0 = (keep(2 * c) ? 0xffffu : 0u) | (keep(2 * c + 1) ? 0xffff0000u : 0u);
          mk1 = (keep(2 * c + 8) ? 0xffffu : 0u) | (keep(2 * c + 9) ? 0xffff0000u : 0u);
        }
        if constexpr (kv16(KVT)) {
#pragma unroll
          for (int t = 0; t < NT; t += 2) {
            uint32_t b0, b1, b2, b3;  // n-tile t: tokens 0-7, 8-15; n-tile t + 1
            ldmatrix_x4_trans(b0, b1, b2, b3, vt + dec::swz_off<C::ROWB, 1>(lr + (lm & 1) * 8, t + (lm >> 1)));
            b0 &= mk0;
            b1 &= mk1;
            b2 &= mk0;
            b3 &= mk1;
            mma16_16816<KVT>(o[t], ph[0], ph[1], ph[2], ph[3], b0, b1);
            mma16_16816<KVT>(o[t + 1], ph[0], ph[1], ph[2], ph[3], b2, b3);
            mma16_16816<KVT>(o[t], pl[0], pl[1], pl[2], pl[3], b0, b1);
            mma16_16816<KVT>(o[t + 1], pl[0], pl[1], pl[2], pl[3], b2, b3);
          }
        } else {
#pragma unroll
          for (int j = 0; j < KS; j += 2) {
            uint32_t x0, x1, x2, x3;  // 16-byte chunks j, j + 1 of tokens 0-7 and 8-15
            ldmatrix_x4_trans(x0, x1, x2, x3, vt + dec::swz_off<C::ROWB, 1>(lr + (lm & 1) * 8, j + (lm >> 1)));
            const uint32_t w[4] = {x0, x1, x2, x3};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // bytes (token 2c: dims 2r, 2r + 1), (token 2c + 1: the same)
              // to token pairs: dims 16 j + 2r (even n-tile) and 2r + 1 (odd)
              const uint32_t y0 = __byte_perm(w[2 * i], 0, 0x3120), y1 = __byte_perm(w[2 * i + 1], 0, 0x3120);
              const uint32_t e0 = fp8x2_to_f16x2<KVT>(static_cast<uint16_t>(y0 & 0xffffu)) & mk0;
              const uint32_t e1 = fp8x2_to_f16x2<KVT>(static_cast<uint16_t>(y1 & 0xffffu)) & mk1;
              const uint32_t d0 = fp8x2_to_f16x2<KVT>(static_cast<uint16_t>(y0 >> 16)) & mk0;
              const uint32_t d1 = fp8x2_to_f16x2<KVT>(static_cast<uint16_t>(y1 >> 16)) & mk1;
              const int t = 2 * (j + i);
              mma_f16_16816(o[t], ph[0], ph[1], ph[2], ph[3], e0, e1);
              mma_f16_16816(o[t + 1], ph[0], ph[1], ph[2], ph[3], d0, d1);
              mma_f16_16816(o[t], pl[0], pl[1], pl[2], pl[3], e0, e1);
              mma_f16_16816(o[t + 1], pl[0], pl[1], pl[2], pl[3], d0, d1);
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[stage]);
    if (++stage == C::NS) {
      stage = 0;
      par ^= 1;
    }
    if (!(h.flags & kLast)) continue;

    // ---- the piece's result
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    // the key groups' states join pairwise: of 2 n RG warps the upper half
    // hands its states to the lower half.  In the first round warp i + n RG
    // writes slot i; later a warp writes the slot it read in the first round,
    // so that a slot has no reader when it is written.  Every round ends at
    // one barrier of all consumer warps, and the next join starts behind the
    // last one's end.
    if (KG > 1) {
      if (joins > 0 && !mbar_wait(join_bar, (joins - 1) & 1, a.wait_ns)) {
        if (lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
        return;
      }
      bool first = true;
      for (int half = NC / 2; half >= RG; half >>= 1, first = false) {  // half: off * RG warps read
        if (warp >= half && warp < 2 * half && busy) {
          float *x = red + (first ? warp - half : warp) * C::REDW + lane;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[(4 * t + e) * 32] = o[t][e];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[(4 * NT + e) * 32] = m[e];
            x[(4 * NT + 2 + e) * 32] = l[e];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(join_bar);
        if (!mbar_wait(join_bar, joins & 1, a.wait_ns)) {
          if (lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
          return;
        }
        ++joins;
        if (warp < half && busy) {
          const float *x = red + (first ? warp : warp + half) * C::REDW + lane;
          float f0[2], f1[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float m2 = x[(4 * NT + e) * 32], l2 = x[(4 * NT + 2 + e) * 32];
            const float mn = fmaxf(m[e], m2);
            f0[e] = m[e] == mn ? 1.f : exp2f(m[e] - mn);
            f1[e] = m2 == mn ? 1.f : exp2f(m2 - mn);
            l[e] = l[e] * f0[e] + l2 * f1[e];
            m[e] = mn;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = o[t][e] * f0[e >> 1] + x[(4 * t + e) * 32] * f1[e >> 1];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(join_bar);
      ++joins;
    }
    if (kg != 0 || !busy) continue;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int R = rg * 16 + r + 8 * e;
      if (R >= h.rows) continue;
      const int s = h.seq0 + R / a.g, hd = h.kvh * a.g + R % a.g;
      const int64_t row = static_cast<int64_t>(s) * a.num_q + hd;
      float *dst, *dl;
      if (h.to == kToCut) {
        const int64_t x = static_cast<int64_t>(h.slot) * a.slot_rows + R;
        dst = a.cut_o + x * D;
        dl = a.cut_lse + x;
      } else {
        dst = (h.to == kToOut ? a.out : h.to == kToPre ? a.pre_o : a.own_o) + row * D;
        dl = h.to == kToOut ? (a.lse ? a.lse + row : nullptr) : (h.to == kToPre ? a.pre_lse : a.own_lse) + row;
      }
      // no key (a sequence shorter than the prefix's first block): nothing to weigh
      const bool none = l[e] == 0.f;
      float inv = none ? 0.f : 1.f / l[e];
      if (h.to == kToOut) inv *= a.v_scales ? __ldg(a.v_scales + h.kvh) : a.vscale;
      const float ls = none ? -INFINITY : m[e] + log2f(l[e]) - C::PB;
      if (dl && c == 0) *dl = h.to == kToOut ? ls * kLn2 : ls;
      if constexpr (kv16(KVT)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          *reinterpret_cast<float2 *>(dst + 8 * t + 2 * c) =
              none ? make_float2(0.f, 0.f) : make_float2(o[t][2 * e] * inv, o[t][2 * e + 1] * inv);
      } else {
#pragma unroll
        for (int t = 0; t < NT; t += 2)  // columns 2c, 2c + 1 of the even and odd n-tiles: dims 4c .. 4c + 3
          *reinterpret_cast<float4 *>(dst + 8 * t + 4 * c) =
              none ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : make_float4(o[t][2 * e] * inv, o[t + 1][2 * e] * inv, o[t][2 * e + 1] * inv,
                                 o[t + 1][2 * e + 1] * inv);
      }
    }
  }
}

template <int D, int KVT>
__global__ void __launch_bounds__(NTHREADS, 1) shared_attend_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, KVT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *ring = smem;
  float *red = reinterpret_cast<float *>(smem + static_cast<size_t>(C::NS) * C::STAGEB);
  Stage *hdr = reinterpret_cast<Stage *>(red + C::NRED * C::REDW);
  uint64_t *full = reinterpret_cast<uint64_t *>(hdr + C::NS);
  uint64_t *empty = full + C::NS;
  uint64_t *join_bar = empty + C::NS;
  static_assert(C::NS * (sizeof(Stage) + 16) + 8 <= 2048, "headers and barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NC);
    }
    mbar_init(join_bar, NC);
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == NC)
    produce<C>(a, ring, hdr, full, empty, lane);
  else
    consume<C>(a, ring, hdr, full, empty, red, join_bar, warp, lane);
}

// --------------------------------------------------------------------- join

// One warp per (sequence, head): the parts' pieces by log-sum-exp weights.
// Rows that the attention wrote itself (one uncut part) are left alone.
template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const __grid_constant__ Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.num_seqs) * a.num_q) return;
  const int lane = threadIdx.x & 31;
  const int s = static_cast<int>(row / a.num_q), h = static_cast<int>(row % a.num_q), kvh = h / a.g;
  const SeqInfo q = a.seqs[s];
  constexpr int EPL = D / 32;
  float *out = a.out + row * D + lane * EPL;
  if (q.len == 0) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[e] = 0.f;
    if (a.lse && lane == 0) a.lse[row] = -INFINITY;
    return;
  }
  const long long U = *a.units;
  float M = -INFINITY, W = 0.f, acc[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
  auto add = [&](const float *o, float x) {
    if (x == -INFINITY) return;
    float v[EPL];
#pragma unroll
    for (int e = 0; e < EPL; e += 2) *reinterpret_cast<float2 *>(v + e) = __ldcg(reinterpret_cast<const float2 *>(o + lane * EPL + e));
    const float mn = fmaxf(M, x);
    const float f = M == -INFINITY ? 0.f : exp2f(M - mn), w = exp2f(x - mn);
    M = mn;
    W = W * f + w;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = acc[e] * f + w * v[e];
  };
  // an item's pieces: its own place if one CTA holds it, else the CTAs' slots
  auto pieces = [&](long long u0, int nb, int w, int r, const float *whole_o, const float *whole_lse) {
    const long long u1 = u0 + static_cast<long long>(nb) * w;
    const int c1 = cta_of(u0, U, a.ctas), c2 = cta_of(u1 - 1, U, a.ctas);
    if (c1 == c2) {
      add(whole_o + row * D, __ldcg(whole_lse + row));
      return;
    }
    for (int cc = c1; cc <= c2; ++cc) {
      const long long b0 = first_unit(cc, U, a.ctas), b1 = first_unit(cc + 1, U, a.ctas);
      int lo, hi;
      piece_blocks(u0, nb, w, b0, b1, lo, hi);
      if (lo >= hi) continue;  // a range that holds no block's first unit
      const int64_t x = (static_cast<int64_t>(cc) * 2 + (u0 <= b0 ? 0 : 1)) * a.slot_rows + r;
      add(a.cut_o + x * D, __ldcg(a.cut_lse + x));
    }
  };
  if (q.fb == 0 && q.nb > 0) {
    const long long u0 = q.base + static_cast<long long>(kvh) * q.nb * kOwnUnits;
    if (cta_of(u0, U, a.ctas) == cta_of(u0 + static_cast<long long>(q.nb) * kOwnUnits - 1, U, a.ctas)) return;
  }
  if (q.fb > 0) {
    const GroupInfo gi = a.groups[q.group];
    const int i = s - gi.first, tile = i / gi.tile_seqs;
    const long long u0 = gi.base + static_cast<long long>(tile * a.num_kv + kvh) * gi.nb * gi.w;
    pieces(u0, gi.nb, gi.w, (i - tile * gi.tile_seqs) * a.g + h % a.g, a.pre_o, a.pre_lse);
  }
  if (q.nb > 0)
    pieces(q.base + static_cast<long long>(kvh) * q.nb * kOwnUnits, q.nb, kOwnUnits, h % a.g, a.own_o, a.own_lse);
  const float inv = W == 0.f ? 0.f : (a.v_scales ? __ldg(a.v_scales + kvh) : a.vscale) / W;
#pragma unroll
  for (int e = 0; e < EPL; e += 2)
    *reinterpret_cast<float2 *>(out + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = W == 0.f ? -INFINITY : (M + log2f(W)) * kLn2;
}

// The attention kernel for a descriptor (pa_shared_bf16.cu and so on).
struct KernelInfo {
  const void *fn;
  size_t smem;
};
template <int D, int KVT>
KernelInfo attend_info() {
  return KernelInfo{reinterpret_cast<const void *>(&shared_attend_kernel<D, KVT>), Cfg<D, KVT>::SMEM};
}
KernelInfo pick_attend_16(int head_dim, int kv_dtype);
KernelInfo pick_attend_8(int head_dim, int kv_dtype);

}  // namespace shd
}  // namespace pa
