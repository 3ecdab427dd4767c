// pa_shared_kernels.cuh -- decode attention of a batch whose sequences share
// prefixes, each prefix read once for all the sequences of its group.
//
// For sequence s of group j, query head h and kv head h / g:
//   out[s][h] = sum_t softmax_t(scale * q[s][h] . K_t) V_t,   t < L_s.
// The first P_j tokens of a group's sequences are the same cache blocks, so
// the sum is cut at P_j: the queries of all the group's sequences attend the
// prefix together, each sequence attends its own rest, and the parts (each
// normalised by its own sum, with its log-sum-exp) are joined by weights
// 2^(lse_p - max lse).  A sequence with L_s < P_j attends all its tokens as its
// own: in a product a weight of 0 does not keep out a V row that is not finite,
// so a row of a prefix item has to read all of the item's keys.
//
// Three launches (the first and the last are in pa_shared.cu):
//  * shared_plan_kernel (one CTA) turns the lengths into a list of items --
//    (group, tile of up to 128 rows, kv head) over the prefix's blocks, and
//    (sequence, kv head) over its own blocks -- laid end to end on one axis
//    of units, a unit a block, with some units in front of every item for what
//    it costs besides its blocks.
//  * shared_attend_kernel, one persistent CTA per SM: CTA c takes the units
//    [c n, (c + 1) n) of that axis, so every CTA has the same work whatever
//    the lengths; an item cut between CTAs leaves a piece in each.
//  * shared_join_kernel, a warp per two (sequence, head) rows: joins the parts.
//
// The attention runs on tcgen05 for every item, a sequence's few heads
// included: an M 128 product costs the tensor cores the same whatever its
// live rows, 24 products of K 16 per 128 keys (8 for Q K^T, 16 for P V with P
// as a hi + lo pair) -- about 1,500 cycles (the tensor pipe's active time over
// the steps of 64 sequences on 16384 tokens), less than the 2,850 in which the
// SM's share of the measured HBM rate brings those 128 keys (64 KB of bf16).
// Roles (warps) of the attend kernel:
//   0  issues Q K^T (one thread), one step ahead of
//   2  P V (one thread), so that the softmax of one step runs behind the
//      products of the next;
//   1  walks the CTA's part of the axis, publishes its items, copies their
//      K and V (TMA);
//   3  Q tiles (TMA), in two slots, so that items overlap;
//   4-11  softmax, two threads per row (64 keys each), and each item's output;
//      items of up to 32 rows take one quarter of the lanes each, in turn, so
//      that four of them can be in their softmax or output at once;
//   12-15 (8-bit caches) widen the landed Q and bytes to fp16 tiles (exact).
// Scores and outputs are double-buffered in tensor memory (S 2 x 128, O 2 x D
// columns); P overwrites its scores.  Every wait is bounded.
//
// Measured, us a call in a captured graph (in brackets what the bytes take at
// the measured HBM rate, 6.69 TB/s), 32 / 8 heads of 128, bf16:
//   8 sequences on one document of 131072 tokens     97.3 (81.0)
//   four groups of 16 on 4096 tokens, own 16-511     36.9 (20.8)
//   64 sequences on 16384 tokens, own 16-511         47.5 (21.4)
//   E4M3, 40 / 8 heads, 128 sequences, own 1-1000    84.6 (23.0)
// What bounds it, from the clock read at the roles' phases (1.9 GHz):
//  * the document, HBM (75% of its peak rate inside the attention kernel); the
//    rest is the chain of three launches, 3.6 us of plan and 5 to 10 of join.
//  * 64 sequences on one prompt, the softmax: the 85 SMs with the prefix take 24
//    or 25 steps of 2,200 cycles, 1,810 of them from a step's scores to its P,
//    55,000 of the kernel's 72,000 cycles.  6,500 go by before the first product
//    (the plan is read, the first copies land, code is fetched cold), 4,000 in
//    the flush of the sums (kChain), 5,700 in the output.  The SMs with own
//    parts are done after 20 to 30 of the 38.8 us: a block weighs the same on
//    the axis in an item of either kind.
//  * the E4M3 batch, the latency of a step: 39 to 46 steps an SM, one every
//    2,970 cycles.  Two are in flight (two score buffers), each for some 5,900
//    from its Q K^T to the end of its P V, 2,400 of them in the softmax where a
//    16-bit cache's narrow items take 1,870: shared memory is busy.  Per 128
//    keys the products read 128 KB (Q, K, and V twice), the widening reads 32
//    and writes 64, the copies write 32, together 2,050 cycles at 128 bytes a
//    cycle.  The conversion itself costs nothing (E5M2 by byte moves instead:
//    no change), nor does its order (two warps for K and two for V: the same).
//  * short items, the same latency (16-bit narrow ones some 2,300 cycles a step)
//    and instruction fetch: the roles run different code at once, so their loops
//    are short and the waits' slow path is one function.
//
// Fewer bits than fp32, and why.  The products take 16-bit operands.  P as one
// such value would leave 2^-8 (bf16) or 2^-11 (fp16) of each weight; the pair
// leaves 2^-16 or 2^-22 and costs a second product, which the tensor cores have
// room for; a third part would cost as much again.  Queries of an 8-bit cache
// become fp16 (see widen).  Exponentials are ex2.approx, 2^-22.  O loses to the
// products' truncation (see kChain).  Error against 64 bits, relative in the
// 2-norm, and that of fp32 PyTorch operations: document 5.1e-6 (6.5e-6), one
// prompt 4.7e-6 (2.3e-6), four groups 4.6e-6 (1.2e-6), E4M3 batch 2.5e-6
// (8.6e-7), four sequences of some 30 tokens 2.1e-6 (1.1e-7).
#pragma once

#include <cuda.h>
#include <float.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace shd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int MAXROWS = 128;     // rows of a tile: one TMEM lane each
constexpr int KT = 128;          // keys of a step
constexpr int BPT = KT / 16;     // blocks of a step
// the running maximum of a row is only raised when a score exceeds it by
// more than this (log2 units), so that O is rarely rescaled
constexpr float kRaise = 8.f;
// An item costs its blocks and this many more (its Q tile, its first copies'
// latency, its output), so the axis gives it that many extra units in front;
// a wide item, which all eight softmax warps finish together, far more than a
// narrow one.  Measured, wide items' 4 / 10 / 16 / 24 / 32: an E4M3 batch with
// 16 short wide items among long ones 100.3 / 95.7 / 87.1 / 85.2 / 87.9 us,
// 64 sequences on one prompt of 16384 tokens (16-bit, from 6) 49.1 / 48.8 /
// 48.4 / 46.9 / 47.9 us; narrow ones' 4 / 6 / 8 / 10: four groups of 16 on
// 4096 tokens (16-bit) 39.4 / 37.3 / 36.3 / 38.0 us, the E4M3 batch 85.2 /
// 84.2 / 86.3 / 87.9 us.  (All at head_dim 128; own parts weigh as narrow items,
// and a tile as its group's fullest one.)
constexpr int kNarrowUnits16 = 8, kNarrowUnits8 = 6, kWideUnits = 24;

constexpr int kQBox = 8;  // sequences of a copy of queries

// One group's prefix on the axis.
struct __align__(8) GroupInfo {
  long long base;  // first unit
  int first;       // first sequence
  int n;           // sequences
  int nb;          // blocks of the prefix (0: nobody reads it)
  int tile_seqs;   // sequences of a tile (the last tile may have fewer)
  int tiles;
  int row;         // the first sequence that holds the whole prefix
  int P;           // the prefix, whole blocks
  int extra;       // units of an item besides its blocks
};
// One sequence: its own part, and its place in its group's prefix part.
struct __align__(16) SeqInfo {
  long long base;   // first unit of the own part
  int len;          // tokens
  int fb;           // first own block
  int nb;           // own blocks
  int group;        // its group, -1: none
  long long pbase;  // first unit of its tile of the prefix (kv head 0)
  int pnb;          // blocks of the prefix, 0: none
  short prow;       // first row in the tile
  short prows;      // rows of the tile
  int pextra;       // units of its items besides their blocks
  int pseq;         // first sequence of the tile
};
// Where a CTA's part of the axis begins.
struct __align__(16) CtaStart {
  int kind;  // 0 prefix item, 1 own part, 2 nothing to do
  int idx;   // group or sequence
  int sub;   // tile * kv heads + kv head, or kv head
  int off;   // first unit within the item
};
// The whole axis.
struct __align__(16) Axis {
  long long units;  // U
  long long per;    // units of a CTA
  uint32_t magic;   // floor(2^32 / per), 0 if U does not fit 32 bits
  uint32_t pad[3];
};

struct Args {
  CUtensorMap kmap;
  CUtensorMap vmap;
  CUtensorMap qmap;      // queries: a box is one sequence's rows of a kv head, half of their columns,
  CUtensorMap qmap_box;  // or those of kQBox sequences
  float *out;
  float *lse;
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
  int tile_seqs;  // sequences a tile may have
  int slot_rows;  // rows of a cut item's slot
  int ctas;       // CTAs that share the axis
  int narrow_units, wide_units;  // units of an item besides its blocks (own parts: narrow ones)
  float qscale;   // scale * k_scale * log2(e)
  float qscale0;  // scale * log2(e)
  float vscale;
  const float *k_scales;
  const float *v_scales;
  int num_blocks;
  int checked;
  int stall;
  uint32_t wait_ns;  // limit of every bounded wait
  int32_t *err;
  // workspace
  Axis *axis;
  GroupInfo *groups;
  SeqInfo *seqs;
  CtaStart *starts;
  float *pre_o;    // prefix parts of uncut items, normalised: tile after tile of [D / 4][rows][4]
  float *pre_lse;  // ... their log-sum-exps, log2 units
  float *own_o;    // own parts, [S][Hq][D]
  float *own_lse;
  float *cut_o;    // pieces of cut items, [ctas][2][D / 4][slot_rows][4]
  float *cut_lse;
  float *sums;     // O's sums over the chains of steps so far, [ctas][D / 4][MAXROWS][4]
};

// A tile of at most 32 rows needs one quarter of the TMEM lanes, and so only
// the two softmax warps of that quarter.  Such narrow items take the quarters
// in turn, so that four of them can be in their softmax or output at once.
__host__ __device__ __forceinline__ bool is_narrow(int rows) { return rows <= 32; }

// ------------------------------------------------------------------- attend

constexpr int kToOut = 0;  // a piece's result: the output itself,
constexpr int kToPre = 1;  // the prefix parts, the own parts,
constexpr int kToOwn = 2;
constexpr int kToCut = 3;  // or a cut item's slot

// A piece of an item, as the walking warp hands it to the other roles.
struct __align__(16) Item {
  int end;     // 1: nothing follows
  int seq0;    // first sequence of the tile
  int rows;    // rows of the tile (sequences x g)
  int kvh;
  int key0;    // position of the piece's first token
  int kend;    // keys from here on are not the piece's
  int nblk;    // blocks of the piece
  int lo;      // first block, counted from the item's
  int to;
  int slot;    // kToCut: the slot
  int pad[2];
};

constexpr int NIQ = 4;  // items in flight between the roles
// A product adds to O with its sum truncated, not rounded, so that O loses
// half a unit of its last place on average with every product, always towards
// zero.  After a chain of this many steps O goes to sums in the workspace,
// whose additions round, and starts again.  Relative error of a prefix of
// 131072 tokens, in pieces of some 55 steps, against 64 bits (and us a call):
// 1.6e-5 without chains (97.8), 7.1e-6 with 24 (99.3), 5.1e-6 with 16
// (100.1), 3.4e-6 with 8 (101.2); 64 sequences on 16384 tokens, pieces of some
// 20 steps: 7.3e-6 without (44.9), 4.7e-6 with 16 (46.9), 3.3e-6 with 8 (49.4).
constexpr int kChain = 16;

// Waits, with a whole warp, until the phase of `bar` with the given parity has
// completed; false (for all its lanes) if that does not happen within
// limit_ns (at most 2^31).  Its loop is not inlined: it is waited some forty
// times in the kernel, and the roles share the SM's instruction caches.
static __device__ __noinline__ bool wait_on(uint32_t addr, uint32_t parity, uint32_t limit_ns) {
  uint32_t t0, t1;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
  while (!__all_sync(0xffffffffu, mbar_test(addr, parity))) {
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t1));
    if (__any_sync(0xffffffffu, t1 - t0 > limit_ns)) return false;
  }
  return true;
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint32_t limit_ns) {
  const uint32_t addr = smem_u32(bar);
  return __all_sync(0xffffffffu, mbar_test(addr, parity)) || wait_on(addr, parity, limit_ns);
}

template <int D_, int KVT_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int KVT = KVT_;
  static constexpr bool KV8 = !kv16(KVT);
  static constexpr bool BF16 = KVT == kKvBf16;  // bf16 products (fp16 otherwise)
  static constexpr int NCONV = KV8 ? 4 : 0;     // widening warps
  static constexpr int NTHREADS = (12 + NCONV) * 32;
  static constexpr int HALVES = D / 64;         // 128-byte column halves of a 16-bit row
  // a 16-bit K or V tile: 8-key groups of [half][8 keys][128 B], 128-byte
  // swizzle.  A cache block's two groups are one TMA box, and both operand
  // forms (K: keys as N; V: keys as K) step through it evenly
  static constexpr int GB = HALVES * 1024;      // bytes of a group
  static constexpr int TB = KT / 8 * GB;
  // where TMA copies land: the tiles themselves, or byte tiles to be widened
  static constexpr int LB = KV8 ? KT * D : TB;
  static constexpr int BLOCKB = LB / BPT;       // one 16-token block
  static constexpr int NT = KV8 ? 2 : (D == 128 ? 3 : 6);      // 16-bit tiles of K, and of V
  static constexpr int NL = KV8 ? (D == 128 ? 2 : 6) : NT;     // landing slots of K, and of V
  static constexpr int QHALF = MAXROWS * 128;   // one half of a 128-row Q tile
  static constexpr int QB = HALVES * QHALF;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = OFF_K + NT * TB;
  static constexpr int OFF_V = OFF_Q + QB;
  static constexpr int OFF_LK = KV8 ? OFF_V + NT * TB : OFF_K;
  static constexpr int OFF_LV = KV8 ? OFF_LK + NL * LB : OFF_V;
  static constexpr int OFF_X = KV8 ? OFF_LV + NL * LB : OFF_V + NT * TB;  // [2][128] fp32: a row's halves exchange
  static constexpr int OFF_IQ = OFF_X + 2 * MAXROWS * 4;
  static constexpr int OFF_BAR = OFF_IQ + NIQ * static_cast<int>(sizeof(Item));
  static constexpr int BARB = D == 64 ? 768 : 512;
  static constexpr int SMEM = OFF_BAR + BARB + 1024;  // + alignment slack
  // an M 128 product reads 128 rows around a slot's: before and behind them
  // it reads whatever lies there, which only feeds dead rows
  static_assert(OFF_Q >= 96 * 128, "Q reads stay inside shared memory");
  static_assert(OFF_Q + QB / 2 + QB / 4 * (HALVES - 1) + QHALF <= OFF_X, "Q reads stay inside shared memory");
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static constexpr uint32_t S_COL = 0;            // two score tiles of KT columns
  static constexpr uint32_t O_COL = 2 * KT;       // two outputs of D columns
  static constexpr uint32_t TMEM_COLS = 512;
  static_assert(O_COL + 2 * D <= TMEM_COLS, "TMEM columns");
  static constexpr uint32_t IDESC_QK = umma_idesc_bf16(MAXROWS, KT, false, false, !BF16);
  static constexpr uint32_t IDESC_PV = umma_idesc_bf16(MAXROWS, D, false, true, !BF16);
  // exponent offset of P: fp16 P keeps small probabilities out of its
  // subnormals; with kRaise the largest P is 2^(8 + 6), inside fp16's range
  static constexpr float PB = BF16 ? 0.f : 6.f;
};

template <class C>
struct Bars {
  uint64_t iq_full[NIQ], iq_empty[NIQ];
  uint64_t lk_full[C::NL], lk_empty[C::NL], lv_full[C::NL], lv_empty[C::NL];  // landed copies
  static constexpr int NW = C::KV8 ? C::NT : 1;
  uint64_t k_full[NW], k_empty[NW], v_full[NW], v_empty[NW];  // 8-bit: widened tiles
  uint64_t q_land[2], q_full[2], q_empty[2], p_empty[2];  // q_land: Q's copies; q_full: ... in fp16 (8-bit caches)
  uint64_t sw_full[2], sn_full[4][2];    // scores of wide items, of narrow ones by quarter; [buffer]
  uint64_t ow_full[2], on_full[4];       // outputs (a quarter's items all use one buffer)
  uint64_t p_full[2][2], o_empty[2][2];  // [narrow][buffer]
  uint64_t drain[2];
  uint32_t tmem;
};

// First lane of item number `item` of the CTA
__device__ __forceinline__ int first_lane(int rows, uint32_t item) {
  return is_narrow(rows) ? static_cast<int>(item & 3) * 32 : 0;
}

// The Q slot of an item: tiles of up to 64 rows alternate between two
// half-size slots, larger ones take both.  Every role follows the items in
// order and so knows the slots and how often each was used.
struct QSlots {
  uint32_t par = 0;  // bit = slot: parity of its uses so far
  int turn = 0;
  bool big = false;
  int slot = 0;
  __device__ __forceinline__ void next(int rows) {
    big = rows > MAXROWS / 2;
    if (!big) {
      slot = turn;
      turn ^= 1;
    } else {
      slot = 0;
    }
  }
  __device__ __forceinline__ bool uses_slot(int i) const { return big || slot == i; }
  __device__ __forceinline__ uint32_t parity(int i) const { return (par >> i) & 1; }
  __device__ __forceinline__ void done() { par ^= big ? 3u : 1u << slot; }
};

// Block-table entries of a piece, 32 at a time, the next 32 requested while
// the current ones are used (one warp).
struct TableWindow {
  const int32_t *row;
  int n, win, cur, nxt;
  template <class A>
  __device__ __forceinline__ int entry(const A &a, int e, int lane) const {
    if (e + lane >= n) return 0;
    const int v = __ldg(row + e + lane);
    return a.checked ? checked_block(v, a.num_blocks, a.err, nullptr) : v;
  }
  template <class A>
  __device__ __forceinline__ void begin(const A &a, const int32_t *row_, int n_, int lane) {
    row = row_;
    n = n_;
    win = 0;
    cur = entry(a, 0, lane);
    nxt = n > 32 ? entry(a, 32, lane) : 0;
  }
  // the block id at b + k, b a multiple of BPT and k < BPT
  template <class A>
  __device__ __forceinline__ int at(const A &a, int b, int k, int lane) {
    if (b - win >= 32) {
      win += 32;
      cur = nxt;
      nxt = win + 32 < n ? entry(a, win + 32, lane) : 0;
    }
    return __shfl_sync(0xffffffffu, cur, (b - win + k) & 31);
  }
};

// One 4-D tile of a tensor map (TMA), completing on `bar`.
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint64_t *bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// An L2 policy that keeps what is read: every CTA on a tile reads its queries.
__device__ __forceinline__ uint64_t l2_evict_last_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// The copies of a piece's K and V blocks into the landing slots, a step at a
// time; `fill` counts the slots of each filled so far.
template <class C>
__device__ bool copy_piece(const Args &a, uint8_t *smem, Bars<C> &bar, const int32_t *table, int nblk, int kvh,
                           uint32_t &fill, uint64_t pol, int lane) {
  TableWindow tw;
  tw.begin(a, table, nblk, lane);
#pragma unroll 1
  for (int b = 0; b < nblk; b += BPT) {
    const int n = min(BPT, nblk - b);
    const int tile = tw.at(a, b, lane & (BPT - 1), lane) * a.num_kv + kvh;  // (block, kv head)
    const uint32_t st = fill % C::NL, ph = ((fill / C::NL) & 1) ^ 1;
    const int off = st * C::LB + lane * C::BLOCKB;
    auto copy = [&](int to, const CUtensorMap *map, uint64_t *full) {
      if (lane == 0) mbar_arrive_expect_tx(full, n * C::BLOCKB);
      __syncwarp();
      if (lane < n) {
        if constexpr (C::KV8)
          tma_load_2d(smem + to + off, map, 0, tile * 16, full, pol);
        else
          tma_load_4d(smem + to + off, map, 0, 0, 0, tile * 2, full, pol);
      }
    };
    if (!wait(&bar.lk_empty[st], ph, a.wait_ns)) return false;
    copy(C::OFF_LK, &a.kmap, &bar.lk_full[st]);
    if (!wait(&bar.lv_empty[st], ph, a.wait_ns)) {
      wait(&bar.lk_full[st], ph ^ 1, a.wait_ns);  // the K copies just issued land
      return false;
    }
    copy(C::OFF_LV, &a.vmap, &bar.lv_full[st]);
    ++fill;
  }
  return true;
}

// After a failed wait: the copies already issued land before the CTA exits.
template <class C>
__device__ void drain_copies(const Args &a, Bars<C> &bar, uint32_t fill) {
#pragma unroll 1
  for (uint32_t i = fill > C::NL ? fill - C::NL : 0; i < fill; ++i) {
    wait(&bar.lk_full[i % C::NL], (i / C::NL) & 1, a.wait_ns);
    wait(&bar.lv_full[i % C::NL], (i / C::NL) & 1, a.wait_ns);
  }
}

// Warp 1: the CTA's items, and their copies.
template <class C>
__device__ bool walk(const Args &a, uint8_t *smem, Bars<C> &bar, Item *iq, int lane) {
  if (a.stall) return true;  // test hook: nothing is issued, every wait runs out
  const int me = blockIdx.x;
  const Axis ax = *a.axis;
  const long long b0 = me * ax.per, b1 = min(b0 + ax.per, ax.units);
  const uint64_t pol = l2_evict_first_policy();
  uint32_t fill = 0, posted = 0;
  long long left = b1 - b0;
  CtaStart st = a.starts[me];
  if (left <= 0) st.kind = 2;
  int kind = -1, items = 0, nb = 0, extra = 0, fb = 0, first = 0, n = 1, tile_seqs = 1, kend = 0, row = 0, whole_to = 0;
  const int32_t *table = nullptr;
  bool ok = true;
  Item it = {};
#pragma unroll 1
  while (ok && !it.end) {
    if (left <= 0 || st.kind == 2) {
      it.end = 1;
    } else {
      if (kind < 0) {  // a group or sequence begins
        kind = st.kind;
        if (kind == 0) {
          const GroupInfo &q = a.groups[st.idx];
          items = q.tiles * a.num_kv;
          nb = q.nb;
          extra = q.extra;
          fb = 0;
          first = q.first;
          n = q.n;
          tile_seqs = q.tile_seqs;
          kend = q.nb * 16;
          row = q.row;
          whole_to = kToPre;
        } else {
          const SeqInfo &q = a.seqs[st.idx];
          items = a.num_kv;
          nb = q.nb;
          extra = a.narrow_units;
          fb = q.fb;
          first = row = st.idx;
          n = tile_seqs = 1;
          kend = q.len;
          whole_to = q.fb == 0 ? kToOut : kToOwn;
        }
        table = a.block_tables + static_cast<int64_t>(row) * a.max_blocks + fb;
      }
      const int tile = st.sub / a.num_kv;
      it.kvh = st.sub - tile * a.num_kv;
      it.seq0 = first + tile * tile_seqs;
      it.rows = min(tile_seqs, n - tile * tile_seqs) * a.g;
      // the part of the item's units in this CTA's range, and its blocks
      const int size = nb + extra;
      const int take = static_cast<int>(min(static_cast<long long>(size - st.off), left));
      const int lo = max(st.off - extra, 0);
      it.nblk = max(st.off + take - extra, 0) - lo;
      it.key0 = (fb + lo) * 16;
      it.kend = min(kend, it.key0 + it.nblk * 16);  // a cut piece ends before the item
      it.lo = lo;
      it.to = it.nblk == nb ? whole_to : kToCut;
      // a cut item that begins inside this CTA's range is its last one
      it.slot = me * 2 + (st.off == 0 && left < b1 - b0 ? 1 : 0);
      left -= take;
      st.off = 0;
      ++st.sub;
    }
    if (it.end || it.nblk > 0) {
      const uint32_t at = posted % NIQ;
      ok = wait(&bar.iq_empty[at], ((posted / NIQ) & 1) ^ 1, a.wait_ns);
      if (!ok) break;
      if (lane == 0) {
        iq[at] = it;
        mbar_arrive(&bar.iq_full[at]);
      }
      __syncwarp();
      ++posted;
      if (it.end) break;
      ok = copy_piece<C>(a, smem, bar, table + it.lo, it.nblk, it.kvh, fill, pol, lane);
    }
    if (st.sub == items && left > 0) {
      // the next group with a prefix, after the last one the sequences with
      // an own part; the ones without work are passed over 32 at a time
      st.sub = 0;
      kind = -1;
      ++st.idx;
#pragma unroll 1
      for (;;) {
        const int count = st.kind == 0 ? a.num_groups : a.num_seqs, i = st.idx + lane;
        const int work = i >= count ? 0 : st.kind == 0 ? a.groups[i].nb : a.seqs[i].nb;
        const unsigned some = __ballot_sync(0xffffffffu, work > 0);
        if (some) {
          st.idx += __ffs(some) - 1;
          break;
        }
        st.idx += 32;
        if (st.idx < count) continue;
        st.idx = 0;
        if (++st.kind == 2) break;
      }
    }
  }
  if (!ok) drain_copies<C>(a, bar, fill);
  return ok;
}

// The next item for one role (whole warp): false when the wait ran out.
template <class C>
__device__ __forceinline__ bool take_item(const Args &a, Bars<C> &bar, const Item *iq, uint32_t &taken, Item &it,
                                          int lane) {
  const uint32_t st = taken % NIQ;
  if (!wait(&bar.iq_full[st], (taken / NIQ) & 1, a.wait_ns)) return false;
  it = iq[st];
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar.iq_empty[st]);
  ++taken;
  return true;
}

// Warp 3: Q tiles, [half][row][128 B] with the 128-byte swizzle.  A copy is
// one half of kQBox sequences' rows of the kv head; what is left over goes one
// sequence at a time (a copy takes some 90 cycles to issue).
template <class C>
__device__ bool load_q(const Args &a, uint8_t *smem, Bars<C> &bar, const Item *iq, int lane) {
  const uint64_t pol = l2_evict_last_policy();
  uint32_t taken = 0;
  QSlots qs;
  Item it;
  bool ok = true;
#pragma unroll 1
  for (;;) {
    ok = take_item<C>(a, bar, iq, taken, it, lane);
    if (!ok || it.end) break;
    qs.next(it.rows);
    ok = (!qs.uses_slot(0) || wait(&bar.q_empty[0], qs.parity(0) ^ 1, a.wait_ns)) &&
         (!qs.uses_slot(1) || wait(&bar.q_empty[1], qs.parity(1) ^ 1, a.wait_ns));
    if (!ok) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bar.q_land[qs.slot], it.rows * C::HALVES * 128);
      if (qs.big) mbar_arrive(&bar.q_land[1]);
    }
    __syncwarp();
    const uint32_t half = qs.big ? C::QHALF : C::QHALF / 2;
    uint8_t *to = smem + C::OFF_Q + qs.slot * (C::QB / 2) + (lane % C::HALVES) * half;
    const int n = it.rows / a.g, boxes = n / kQBox;  // sequences
#pragma unroll 1
    for (int i = lane / C::HALVES; i < boxes + n % kQBox; i += 32 / C::HALVES) {
      const int s = i < boxes ? i * kQBox : boxes * kQBox + i - boxes;
      tma_load_4d(to + s * a.g * 128, i < boxes ? &a.qmap_box : &a.qmap, 0, it.kvh * a.g, lane % C::HALVES, it.seq0 + s,
                  &bar.q_land[qs.slot], pol);
    }
    __syncwarp();
    qs.done();
  }
  // the copies land before the CTA exits, whatever became of the others
  wait(&bar.q_land[0], qs.parity(0) ^ 1, a.wait_ns);
  wait(&bar.q_land[1], qs.parity(1) ^ 1, a.wait_ns);
  return ok;
}

// Warps 12-15 (8-bit caches): Q tiles to fp16, in place (both operands of a
// product have one type, and bytes fit fp16; bf16's 8 bits fit too, off by
// 2^-25 at most below 2^-14, and a finite |q| beyond fp16 does not fit and is
// reported); landed bytes to fp16 tiles, exact; V rows past
// the piece's keys zeroed (they may hold anything, and 0 * NaN is NaN).  A
// thread keeps its 16-byte column chunk and its row modulo 8, and with them
// its places in the swizzled tile, over all its rows.  Of the two 16-byte
// stores the threads of the second column half begin with the other one:
// equal places of the halves lie in the same banks.
template <class C>
__device__ bool widen(const Args &a, uint8_t *smem, Bars<C> &bar, const Item *iq, int ct, int lane) {
  constexpr int CPR = C::D / 16;                  // 16-byte chunks of a row of bytes
  constexpr int RSTEP = C::NCONV * 32 / CPR;      // rows between a thread's chunks (a multiple of 8)
  static_assert(RSTEP % 8 == 0 && KT % RSTEP == 0, "a thread's rows agree modulo 8");
  constexpr int PER = KT / RSTEP;
  const int c = ct % CPR, r0 = ct / CPR, r7 = r0 & 7;
  const int put = (r0 >> 3) * C::GB + (c >> 2) * 1024 + r7 * 128;
  const bool swap = (c & 4) != 0;
  const int x0 = ((2 * (c & 3) + swap) ^ r7) << 4, x1 = ((2 * (c & 3) + !swap) ^ r7) << 4;
  uint32_t taken = 0, step = 0;
  QSlots qs;
  Item it;
#pragma unroll 1
  for (;;) {
    if (!take_item<C>(a, bar, iq, taken, it, lane)) return false;
    if (it.end) return true;
    qs.next(it.rows);
    if (qs.uses_slot(0) && !wait(&bar.q_land[0], qs.parity(0), a.wait_ns)) return false;
    if (qs.uses_slot(1) && !wait(&bar.q_land[1], qs.parity(1), a.wait_ns)) return false;
    {
      constexpr int CH = C::D / 8, RPI = C::NCONV * 32 / CH;  // 16-byte chunks of a row; rows at once
      const int half = qs.big ? C::QHALF : C::QHALF / 2;
      uint8_t *at = smem + C::OFF_Q + qs.slot * (C::QB / 2) + (ct % CH >> 3) * half + (ct % CH & 7) * 16;
      float big = 0.f;
#pragma unroll 2
      for (int R = ct / CH; R < it.rows; R += RPI) {
        uint4 *p = reinterpret_cast<uint4 *>(at + R * 128);  // (any order: the swizzle stays as it is)
        const uint4 x = *p;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f0 = bf16lo(w[e]), f1 = bf16hi(w[e]);
          const float f = fmaxf(fabsf(f0), fabsf(f1));
          if (f <= FLT_MAX) big = fmaxf(big, f);
          o[e] = pack_f16x2(f0, f1);
        }
        *p = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (big >= 65520.f) report_error(a.err, nullptr, kErrFp16Range);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (qs.uses_slot(0)) mbar_arrive(&bar.q_full[0]);
        if (qs.uses_slot(1)) mbar_arrive(&bar.q_full[1]);
      }
      qs.done();
    }
#pragma unroll 1
    for (int b = 0; b < it.nblk; b += BPT, ++step) {
      const int rows = min(BPT, it.nblk - b) * 16;
      const int keep = it.kend - (it.key0 + b * 16);  // rows of the piece's keys
      const uint32_t ls = step % C::NL, lp = (step / C::NL) & 1, ts = step % C::NT, tp = ((step / C::NT) & 1) ^ 1;
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        if (!wait(v ? &bar.v_empty[ts] : &bar.k_empty[ts], tp, a.wait_ns)) return false;
        if (!wait(v ? &bar.lv_full[ls] : &bar.lk_full[ls], lp, a.wait_ns)) return false;
        const uint8_t *src = smem + (v ? C::OFF_LV : C::OFF_LK) + ls * C::LB + ct * 16;
        uint8_t *dst = smem + (v ? C::OFF_V : C::OFF_K) + ts * C::TB + put;
        constexpr int ILP = PER < 4 ? PER : 4;
#pragma unroll 1
        for (int k0 = 0; k0 < PER; k0 += ILP) {
          if (r0 + k0 * RSTEP >= rows) break;
          uint4 x[ILP];
#pragma unroll
          for (int k = 0; k < ILP; ++k) x[k] = *reinterpret_cast<const uint4 *>(src + (k0 + k) * RSTEP * C::D);
#pragma unroll
          for (int k = 0; k < ILP; ++k) {
            const uint32_t w[4] = {swap ? x[k].z : x[k].x, swap ? x[k].w : x[k].y, swap ? x[k].x : x[k].z,
                                   swap ? x[k].y : x[k].w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[2 * e] = fp8x2_to_f16x2<C::KVT>(static_cast<uint16_t>(w[e] & 0xffffu));
              o[2 * e + 1] = fp8x2_to_f16x2<C::KVT>(static_cast<uint16_t>(w[e] >> 16));
            }
            uint8_t *row = dst + (k0 + k) * (RSTEP / 8) * C::GB;
            *reinterpret_cast<uint4 *>(row + x0) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(row + x1) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        if (v && keep < rows) {
#pragma unroll 1
          for (int r = keep + (r0 - keep & RSTEP - 1); r < rows; r += RSTEP) {
            uint8_t *row = dst + (r - r0) / 8 * C::GB;
            *reinterpret_cast<uint4 *>(row + x0) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(row + x1) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v ? &bar.lv_empty[ls] : &bar.lk_empty[ls]);
          mbar_arrive(v ? &bar.v_full[ts] : &bar.k_full[ts]);
        }
      }
    }
  }
}

// Score scale of a kv head, log2 units.
__device__ __forceinline__ float score_scale(const Args &a, int kvh) {
  return a.k_scales ? a.qscale0 * __ldg(a.k_scales + kvh) : a.qscale;
}

// The products, from descriptors split in halves: along a tile only the low
// word changes (the start address), by constants, so that the one issuing
// thread takes few instructions per product and the tensor pipe stays fed.
constexpr uint32_t desc_high(uint32_t sbo) {  // stride, version, 128-byte swizzle
  return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29);
}
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) & 0x3FFFu) << 16;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// The value of lane 0, which the compiler may keep in a uniform register: the
// products' operands have to be in those, and descriptors that only differ by
// constants then cost one instruction each.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Warp 0, one thread: the scores, S[k % 2] = Q K^T of step k, once the step's
// K has landed and P V of step k - 2 has read the P that lay there.
template <class C>
__device__ bool issue_qk(const Args &a, uint32_t sbase, uint32_t tmem, Bars<C> &bar, const Item *iq, int lane) {
  // 16-bit caches: the landed tiles feed the products
  uint64_t *k_full = C::KV8 ? bar.k_full : bar.lk_full, *k_empty = C::KV8 ? bar.k_empty : bar.lk_empty;
  uint64_t *q_full = C::KV8 ? bar.q_full : bar.q_land;
  uint32_t taken = 0, k = 0;
  QSlots qs;
  Item it;
  for (;;) {
    if (!take_item<C>(a, bar, iq, taken, it, lane)) return false;
    if (it.end) return true;
    qs.next(it.rows);
    // the softmax takes maxima of the scores as they come, so a negative
    // scale's sign goes into the product (bit 13 negates A)
    const uint32_t idesc = uniform(C::IDESC_QK | (score_scale(a, it.kvh) < 0.f ? 1u << 13 : 0u));
    const uint32_t qhalf = qs.big ? C::QHALF : C::QHALF / 2;
    // row 0 of the slot is lane first_lane of the product
    const uint32_t qd0 = uniform(
        desc_low(sbase + C::OFF_Q + qs.slot * (C::QB / 2) - first_lane(it.rows, taken - 1) * 128, 16));
    const uint32_t qd1 = uniform(qd0 + (qhalf >> 4));  // the second column half
    if (qs.uses_slot(0) && !wait(&q_full[0], qs.parity(0), a.wait_ns)) return false;
    if (qs.uses_slot(1) && !wait(&q_full[1], qs.parity(1), a.wait_ns)) return false;
    uint64_t *s_full = is_narrow(it.rows) ? bar.sn_full[(taken - 1) & 3] : bar.sw_full;
#pragma unroll 1
    for (int b = 0; b < it.nblk; b += BPT, ++k) {
      if (!wait(&bar.p_empty[k & 1], ((k >> 1) & 1) ^ 1, a.wait_ns)) return false;
      if (!wait(&k_full[k % C::NT], (k / C::NT) & 1, a.wait_ns)) return false;
      tc_fence_after_sync();
      const uint32_t kd = uniform(desc_low(sbase + C::OFF_K + (k % C::NT) * C::TB, 16));
      const uint32_t s = uniform(tmem + C::S_COL + (k & 1) * KT);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < C::D / 16; ++kk)
          mma_ss(s, (kk < 4 ? qd0 : qd1) + (kk & 3) * 2, desc_high(1024),
                 kd + ((kk >> 2) * 1024 + (kk & 3) * 32) / 16, desc_high(C::GB), idesc, kk > 0);
        umma_commit(&s_full[k & 1]);
        umma_commit(&k_empty[k % C::NT]);
      }
      __syncwarp();
    }
    if (elect_one()) {
      if (qs.uses_slot(0)) umma_commit(&bar.q_empty[0]);
      if (qs.uses_slot(1)) umma_commit(&bar.q_empty[1]);
    }
    __syncwarp();
    qs.done();
  }
}

// Warp 2, one thread: O += P V of every step, hi and lo.
template <class C>
__device__ bool issue_pv(const Args &a, uint32_t sbase, uint32_t tmem, Bars<C> &bar, const Item *iq, int lane) {
  uint64_t *v_full = C::KV8 ? bar.v_full : bar.lv_full, *v_empty = C::KV8 ? bar.v_empty : bar.lv_empty;
  uint32_t taken = 0, k = 0;
  // the barriers of P and of O count the warps that work on the item, two for
  // a narrow one and eight else, so there is one of each kind per buffer:
  // bit 2 * narrow + buffer is the parity of its next phase
  uint32_t p_par = 0, o_par = 0;
  uint32_t used = 0, was = 0;  // bit = buffer: it has held an item; that was a narrow one
  Item it;
  for (;;) {
    if (!take_item<C>(a, bar, iq, taken, it, lane)) return false;
    if (it.end) return true;
    const int nar = is_narrow(it.rows), ob = (taken - 1) & 1;
    const uint32_t o = uniform(tmem + C::O_COL + ob * C::D);
    // the item's first product overwrites the output of the item two before
    if ((used >> ob) & 1) {
      const int kind = (was >> ob) & 1, i = 2 * kind + ob;
      if (!wait(&bar.o_empty[kind][ob], (o_par >> i) & 1, a.wait_ns)) return false;
      o_par ^= 1u << i;
    }
    used |= 1u << ob;
    was = (was & ~(1u << ob)) | (static_cast<uint32_t>(nar) << ob);
#pragma unroll 1
    for (int b = 0; b < it.nblk; b += BPT, ++k) {
      if (!wait(&v_full[k % C::NT], (k / C::NT) & 1, a.wait_ns)) return false;
      const int i = 2 * nar + (k & 1);
      if (!wait(&bar.p_full[nar][k & 1], (p_par >> i) & 1, a.wait_ns)) return false;
      p_par ^= 1u << i;
      tc_fence_after_sync();
      const uint32_t vd = uniform(desc_low(sbase + C::OFF_V + (k % C::NT) * C::TB, 1024));
      const uint32_t p = uniform(tmem + C::S_COL + (k & 1) * KT);
      const uint32_t n = uniform(it.nblk - b), more = uniform(b / BPT % kChain);
      if (elect_one()) {
        // keys 16 kk .. 16 kk + 15: hi at +0, lo at +16 of their 32-column chunk
#pragma unroll
        for (int kk = 0; kk < BPT; ++kk) {
          if (kk >= static_cast<int>(n)) break;
          const uint32_t bd = vd + kk * (2 * C::GB / 16), ap = p + (kk >> 1) * 32 + (kk & 1) * 8;
          mma_ts(o, ap, bd, desc_high(C::GB), C::IDESC_PV, kk > 0 || more != 0);
          mma_ts(o, ap + 16, bd, desc_high(C::GB), C::IDESC_PV, true);
        }
        umma_commit(&v_empty[k % C::NT]);
        umma_commit(&bar.p_empty[k & 1]);
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(nar ? &bar.on_full[(taken - 1) & 3] : &bar.ow_full[ob]);
    __syncwarp();
  }
}

// 16 consecutive TMEM columns of this warp's 32 lanes (one lane per thread).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Warps 4-11: softmax and outputs.  Warps 4-7 take keys 0-63 and warps 8-11
// keys 64-127 of every step; a thread holds lane 32 (warp % 4) + lane of the
// tile and its half h of the keys, later its half of the columns.  A narrow
// item's warps are those of its quarter.  Partner warps w and w + 4 agree at their named barrier on every wait, so
// that both go on or both stop.  The loops over 32 scores are not unrolled
// further: the roles' code shares the SM's instruction caches.
template <class C>
struct Softmax {
  static constexpr int D = C::D;
  static constexpr int PT = C::BF16 ? kKvBf16 : kKvF16;  // type of P
  const Args &a;
  uint8_t *smem;
  Bars<C> &bar;
  uint32_t trow;  // this warp's lanes in tensor memory
  float *xch;
  int warp, lane, h, row, pair;
  bool ok = true;
  // parities of the next phases of the barriers this warp waits on.  A warp
  // sees every phase of the wide items' barriers and of its own quarter's,
  // and no other's, so each parity names one phase.
  uint32_t sw = 0, sn = 0;  // scores: bit = buffer
  uint32_t ow = 0, on = 0;  // outputs: bit = buffer; bit 0

  // This thread's columns c .. c + 3 of the item's sum over the chains before
  // the current one.
  __device__ __forceinline__ float4 *sum_at(int c) const {
    uint32_t at = blockIdx.x * (D / 4) * MAXROWS + threadIdx.x % MAXROWS;  // (threadIdx.x % 128: the row)
    asm volatile("" : "+r"(at));  // not kept in a register from here to there
    return reinterpret_cast<float4 *>(a.sums) + at + c / 4 * MAXROWS;
  }

  // The end of a chain, the steps before k: O goes to the sums.  No other
  // thread adds to this one's, so they are taken in order.
  __device__ __forceinline__ void flush(uint32_t k, uint32_t num, bool live, bool first, uint64_t *v_empty) {
    ok = wait(&v_empty[(k - 1) % C::NT], ((k - 1) / C::NT) & 1, a.wait_ns) && ok;
    tc_fence_after_sync();
#pragma unroll 1
    for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 16) {
      float o[16];
      tmem_ld16(trow + C::O_COL + (num & 1) * D + c0, o);
      if (live) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 x = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          if (first)
            __stcg(sum_at(c0 + i), x);
          else
            atomicAdd(sum_at(c0 + i), x);
        }
      }
    }
  }

  // An item's output, once its last product is through.
  __device__ __forceinline__ void finish(const Item &it, uint32_t num, bool chains, float m, float l) {
    const int ob = num & 1;
    const int r = row - first_lane(it.rows, num);  // row of the tile
    const bool live = r >= 0 && r < it.rows;
    const bool mine = __any_sync(0xffffffffu, live);  // the same for both partners
    float lsum = l;
    if (mine) {
      named_bar_sync(pair, 64);  // the partner has read the last maxima
      xch[h * MAXROWS + row] = l;
      named_bar_sync(pair, 64);
      lsum += xch[(h ^ 1) * MAXROWS + row];
    }
    if (is_narrow(it.rows)) {
      ok = wait(&bar.on_full[warp & 3], on, a.wait_ns) && ok;
      on ^= 1;
    } else {
      ok = wait(&bar.ow_full[ob], (ow >> ob) & 1, a.wait_ns) && ok;
      ow ^= 1u << ob;
    }
    if (mine && ok) {
      tc_fence_after_sync();
      // outputs and own parts are rows; prefix parts and pieces are
      // [4 columns][row of the tile], so that a wide tile's lanes write
      // consecutive 16 bytes
      const int sq = live ? r / a.g : 0;
      const int64_t orow = static_cast<int64_t>(it.seq0 + sq) * a.num_q + it.kvh * a.g + (r - sq * a.g);
      float *o_dst = (it.to == kToOut ? a.out : a.own_o) + orow * D;
      float *l_dst = it.to == kToOut ? (a.lse ? a.lse + orow : nullptr) : a.own_lse + orow;
      int64_t stride = 4;
      if (it.to == kToCut) {
        o_dst = a.cut_o + static_cast<int64_t>(it.slot) * a.slot_rows * D + 4 * r;
        l_dst = a.cut_lse + static_cast<int64_t>(it.slot) * a.slot_rows + r;
        stride = 4 * a.slot_rows;
      } else if (it.to == kToPre) {
        const int64_t at = static_cast<int64_t>(it.seq0) * a.num_q + static_cast<int64_t>(it.kvh) * it.rows;
        o_dst = a.pre_o + at * D + 4 * r;
        l_dst = a.pre_lse + at + r;
        stride = 4 * it.rows;
      }
      // (no key has a weight: scores of -inf throughout)
      const bool none = lsum == 0.f;
      float inv = none ? 0.f : 1.f / lsum;
      if (it.to == kToOut) inv *= a.v_scales ? __ldg(a.v_scales + it.kvh) : a.vscale;
      if (live && h == 0 && l_dst) {
        const float ls = none ? -INFINITY : m + log2f(lsum) - C::PB;
        *l_dst = it.to == kToOut ? ls * kLn2 : ls;
      }
#pragma unroll 1
      for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 16) {
        float o[16];
        tmem_ld16(trow + C::O_COL + ob * D + c0, o);
        if (live) {
          if (chains) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 x = __ldcg(sum_at(c0 + i));
              o[i] += x.x;
              o[i + 1] += x.y;
              o[i + 2] += x.z;
              o[i + 3] += x.w;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4 *>(o_dst + (c0 + i) / 4 * stride) =
                none ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
        }
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0 && (mine || !is_narrow(it.rows))) mbar_arrive(&bar.o_empty[is_narrow(it.rows)][ob]);
  }

  __device__ bool run(const Item *iq) {
    uint64_t *v_full = C::KV8 ? bar.v_full : bar.lv_full, *v_empty = C::KV8 ? bar.v_empty : bar.lv_empty;
    uint32_t taken = 0, k = 0;
#pragma unroll 1
    for (;;) {
      Item it;
      const bool got = take_item<C>(a, bar, iq, taken, it, lane);
      if (!named_bar_and(pair, 64, got && ok)) return false;
      const uint32_t num = taken - 1;
      const bool nar = is_narrow(it.rows);
      if (it.end) return ok;
      const int r = row - first_lane(it.rows, num);
      const bool live = r >= 0 && r < it.rows;
      const bool mine = __any_sync(0xffffffffu, live);
      const int steps = (it.nblk + BPT - 1) / BPT;
      if (nar && !mine) {  // another quarter's
        k += steps;
        continue;
      }
      // (a negative scale's sign is in the scores; a zero one must not meet
      // the -inf of a masked score as a zero)
      const float qsc = fmaxf(fabsf(score_scale(a, it.kvh)), 1e-37f);
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int b = 0; b < it.nblk; b += BPT, ++k) {
        const int n = min(BPT, it.nblk - b);
        const int key0 = it.key0 + b * 16;
        bool there;
        if (nar) {
          there = wait(&bar.sn_full[warp & 3][k & 1], (sn >> (k & 1)) & 1, a.wait_ns);
          sn ^= 1u << (k & 1);
        } else {
          there = wait(&bar.sw_full[k & 1], (sw >> (k & 1)) & 1, a.wait_ns);
          sw ^= 1u << (k & 1);
        }
        tc_fence_after_sync();
        if (!C::KV8 && it.kend < key0 + n * 16) {
          // V rows past the item's keys may hold anything (0 * NaN is NaN)
          there = there && wait(&v_full[k % C::NT], (k / C::NT) & 1, a.wait_ns);
          const int keep = it.kend - key0;
          const int threads = nar ? 64 : 256, me = nar ? h * 32 + lane : static_cast<int>(threadIdx.x) - 128;
          uint8_t *v = smem + C::OFF_V + (k % C::NT) * C::TB;
#pragma unroll 1
          for (int i = me; there && i < (n * 16 - keep) * C::HALVES * 8; i += threads) {
            const int rr = keep + i / (C::HALVES * 8), c = i % (C::HALVES * 8);
            *reinterpret_cast<uint4 *>(v + (rr >> 3) * C::GB + (c >> 3) * 1024 + (rr & 7) * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (!named_bar_and(pair, 64, there && ok)) return false;
        if (mine) {
          // (counted from the step's first key: positions end at the end of 32 bits)
          step(k, it.kend - key0, b / BPT, live, qsc, num, v_empty, m, l);
          if (b > 0 && b / BPT % kChain == 0) flush(k, num, live, b / BPT == kChain, v_empty);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[nar][k & 1]);
      }
      finish(it, num, steps > kChain, m, l);
    }
  }

  // One step's scores (in tensor memory) to P over them; m and l follow.  The
  // keys from `keys` on are no row's.  (Rows of a sequence that does not hold the
  // whole prefix, in its group's tile, are computed, and read by nobody.)
  __device__ __forceinline__ void step(uint32_t k, int keys, int done, bool live, float qsc, uint32_t num,
                                       uint64_t *v_empty, float &m, float &l) {
    const uint32_t scol = trow + C::S_COL + (k & 1) * KT + 64 * h;
    const int mine = keys - 64 * h;
    // 32 scores, keys past the item's last out
    auto load = [&](int c, uint32_t(&x)[32]) {
      tmem_ld32_async(scol + 32 * c, x);
      tmem_wait_ld(x);
      if (32 * c + 32 > mine) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (32 * c + i >= mine) x[i] = __float_as_uint(-INFINITY);
      }
    };
    uint32_t sc[32];
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 1; c >= 0; --c) {
      load(c, sc);
      float t[11];  // a tree of three-input maxima
#pragma unroll
      for (int i = 0; i < 10; ++i)
        t[i] = fmax3(__uint_as_float(sc[3 * i]), __uint_as_float(sc[3 * i + 1]), __uint_as_float(sc[3 * i + 2]));
      t[10] = fmaxf(__uint_as_float(sc[30]), __uint_as_float(sc[31]));
      mx = fmax3(mx, fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmax3(t[6], t[7], t[8])),
                 fmaxf(t[9], t[10]));
    }
    // the row's maximum over both halves (the barrier behind the wait above
    // says that the partner has read the last exchange)
    xch[h * MAXROWS + row] = mx;
    named_bar_sync(pair, 64);
    mx = fmaxf(mx, xch[(h ^ 1) * MAXROWS + row]);
    mx = mx == -INFINITY ? mx : mx * qsc;
    const bool raise = live && mx > m + kRaise;  // m = -inf: any finite score
    if (__any_sync(0xffffffffu, raise && m != -INFINITY)) {
      // rare: this half of O's columns takes the new maximum; the product of
      // the step before, which releases its V tile, is through
      if (done) ok = wait(&v_empty[(k - 1) % C::NT], ((k - 1) / C::NT) & 1, a.wait_ns) && ok;
      tc_fence_after_sync();
      const float f = (raise && m != -INFINITY) ? exp2f(m - mx) : 1.f;
      l *= f;
#pragma unroll 1
      for (int c0 = h * (D / 2); c0 < (h + 1) * (D / 2); c0 += 32) {
        float o[32];
        tmem_ld32(trow + C::O_COL + (num & 1) * D + c0, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= f;
        tmem_st32(trow + C::O_COL + (num & 1) * D + c0, o);
      }
      if (done > kChain) {  // and its sums
#pragma unroll 1
        for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 4) {
          const float4 x = __ldcg(sum_at(c));
          __stcg(sum_at(c), make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
        }
      }
    }
    if (raise) m = mx;
    // P = 2^(score - m + PB) in pairs; 32 keys become 16 columns of hi pairs
    // and 16 of lo pairs over their own, loaded, scores (chunk 0's are still
    // in registers)
    const float off = C::PB - (m == -INFINITY ? 0.f : m);
    const uint64_t q2 = f2_pack(qsc, qsc), o2 = f2_pack(off, off);
    uint64_t ls[2] = {0, 0};
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      if (c == 1) load(1, sc);
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 y =
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sc[2 * e]), __uint_as_float(sc[2 * e + 1])), q2, o2));
        const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
        const uint64_t pp = f2_pack(p0, p1);
        ls[e & 1] = f2_add(ls[e & 1], pp);
        hi[e] = pack16x2<PT>(p0, p1);
        const float2 d = f2_unpack(f2_sub(pp, f2_pack(lo16<PT>(hi[e]), hi16<PT>(hi[e]))));
        lo[e] = pack16x2<PT>(d.x, d.y);
      }
      tmem_st16_async(scol + 32 * c, hi);
      tmem_st16_async(scol + 32 * c + 16, lo);
    }
    const float2 l2 = f2_unpack(f2_add(ls[0], ls[1]));
    l += l2.x + l2.y;
    tmem_wait_st();
  }
};

template <int D, int KVT>
__global__ void __launch_bounds__(Cfg<D, KVT>::NTHREADS, 1) shared_attend_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, KVT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars<C> &bar = *reinterpret_cast<Bars<C> *>(smem + C::OFF_BAR);
  static_assert(sizeof(Bars<C>) <= C::BARB, "barriers");
  Item *iq = reinterpret_cast<Item *>(smem + C::OFF_IQ);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NIQ; ++i) {
      mbar_init(&bar.iq_full[i], 1);
      mbar_init(&bar.iq_empty[i], 1 + 1 + 1 + 8 + C::NCONV);  // the warps that take items
    }
    for (int i = 0; i < C::NL; ++i) {
      mbar_init(&bar.lk_full[i], 1);
      mbar_init(&bar.lk_empty[i], C::KV8 ? C::NCONV : 1);
      mbar_init(&bar.lv_full[i], 1);
      mbar_init(&bar.lv_empty[i], C::KV8 ? C::NCONV : 1);
    }
    for (int i = 0; i < Bars<C>::NW; ++i) {
      mbar_init(&bar.k_full[i], C::KV8 ? C::NCONV : 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], C::KV8 ? C::NCONV : 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_land[i], 1);
      mbar_init(&bar.q_full[i], C::KV8 ? C::NCONV : 1);
      mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.sw_full[i], 1);
      mbar_init(&bar.ow_full[i], 1);
#pragma unroll 1
      for (int nar = 0; nar < 2; ++nar) {
        mbar_init(&bar.p_full[nar][i], nar ? 2 : 8);
        mbar_init(&bar.o_empty[nar][i], nar ? 2 : 8);
      }
      mbar_init(&bar.p_empty[i], 1);
      mbar_init(&bar.drain[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.sn_full[i][0], 1);
      mbar_init(&bar.sn_full[i][1], 1);
      mbar_init(&bar.on_full[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&bar.tmem, C::TMEM_COLS);
  // the maps are fetched while the plan is still made
  if (warp == 1 && lane < (a.tile_seqs < kQBox ? 3 : 4))
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.kmap + lane)) : "memory");
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bar.tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool ok = true;
  if (warp == 0) {
    ok = issue_qk<C>(a, smem_u32(smem), tmem, bar, iq, lane);
  } else if (warp == 1) {
    ok = walk<C>(a, smem, bar, iq, lane);
  } else if (warp == 2) {
    ok = issue_pv<C>(a, smem_u32(smem), tmem, bar, iq, lane);
  } else if (warp == 3) {
    ok = load_q<C>(a, smem, bar, iq, lane);
  } else if (warp < 12) {
    const int h = (warp - 4) >> 2;
    Softmax<C> sm{a,
                  smem,
                  bar,
                  tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16),
                  reinterpret_cast<float *>(smem + C::OFF_X),
                  warp,
                  lane,
                  h,
                  ((warp & 3) << 5) | lane,
                  1 + (warp & 3)};
    ok = sm.run(iq);
  } else if constexpr (C::KV8) {
    ok = widen<C>(a, smem, bar, iq, threadIdx.x - 12 * 32, lane);
  }
  if (!ok && lane == 0) report_error(a.err, nullptr, kErrWaitTimeout);
  // every product issued completes before the tensor memory is given back
  if (warp == 0 || warp == 2) {
    __syncwarp();
    if (elect_one()) umma_commit(&bar.drain[warp >> 1]);  // the lane that issued them
    wait(&bar.drain[warp >> 1], 0, a.wait_ns);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// The attention kernel for a descriptor (pa_shared_16.cu, pa_shared_8.cu).
struct KernelInfo {
  const void *fn;
  size_t smem;
  int threads;
};
template <int D, int KVT>
KernelInfo attend_info() {
  return KernelInfo{reinterpret_cast<const void *>(&shared_attend_kernel<D, KVT>), Cfg<D, KVT>::SMEM,
                    Cfg<D, KVT>::NTHREADS};
}
KernelInfo pick_attend_16(int head_dim, int kv_dtype);
KernelInfo pick_attend_8(int head_dim, int kv_dtype);

}  // namespace shd
}  // namespace pa
