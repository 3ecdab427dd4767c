// pa_prompt.cu -- causal attention of whole prompts from their own rows.
//
//   out_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j   within each prompt,
// prompts of different lengths packed one behind another, query head h using kv
// head h / g; sliding-window and chunked-local layers start at a later key.
//
// Work.  An item is up to 256 rows of one (prompt, kv head): the query tokens
// times the g heads that share the kv head, in two tiles of 128 rows (128 / g
// tokens each), so that every K / V tile of 128 keys feeds two products.  A CTA
// per SM runs its items through one pipeline: warp 0 issues the products, warp 1
// the copies (TMA, straight from the strided rows, into the next item while the
// last one's products run), warps 2-3 look over the V tiles that some row sees
// only in part, and a warpgroup per tile does the softmax, one row a thread.
// Items go to the CTAs in rows, longest key ranges first, every second row
// backwards.
//
// Per K tile and query tile: S = Q K^T into 128 columns of tensor memory; the
// softmax writes P, in the activation type, over them; O += P V takes P from
// tensor memory.  The tensor cores work on one tile while the other's softmax
// runs.  The running maximum is raised only when it grows by 2^8 (O is then
// rescaled in tensor memory), sums are fp32 of the unrounded weights.  P in 16
// bits is off by half a step of the type that the output is rounded to as well:
// outputs are off by 1.3 times what their own rounding costs (16384 tokens, bf16,
// against 64 bits: 2.1e-3 of their norm, 1.6e-3 with exact weights).  As a hi +
// lo pair, the low half in the columns of S beside the high half's, P costs
// nothing more of that but half as many products again: 1.88 ms for 1.26 (five
// prompts of 256 to 2048: 83 us for 65).  The caller's choice (prefill_impl).
//
// A weight of zero does not cancel an infinity or a NaN: in the V tiles that
// some row sees in part, rows behind the keys in use are zeroed, and a row with
// a value that is not finite is zeroed and noted; the epilogue adds it to
// the queries that do see it, in fp32.
//
// Bounded by the tensor cores: 4 D flops a (query head, key) pair.  A key tile
// takes 2,950 cycles for both query tiles, its products 2,600 of them (84 cycles a
// product with both operands in shared memory, 78 with one in tensor memory); an
// item's first and last tiles take about 9,000 cycles more.  16384 tokens, 32 / 8
// heads of 128: 1.26 ms, 1.75 PFLOP/s; five prompts of 256 to 2048: 60 us, 1.0.
// With 64 dims no unit is: a window of 1024 over prompts of 4096 and 3000, 32 / 8
// heads (85 us), has the products at 32% of the cycles, the exponentials at 32%, an
// instruction in 44%; the softmax of its tiles (1,270 cycles a tile and
// warpgroup) is a third of the time, the items' ends another.
#include <cuda.h>

#include "pa_device.cuh"
#include "pa_host_cache.h"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int KT = 128;                  // keys of a tile
constexpr float kRaise = 8.f;            // log2 units the maximum may be behind
constexpr int kNoted = 32;               // partly seen tiles with a mask of their own
constexpr int kAhead = 4;                // items found before they are needed

struct Args {
  CUtensorMap qmap, kmap, vmap;
  void *out;
  float *lse;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *starts;
  int num_seqs, num_tokens, max_q_len, hq, hkv, g;
  int rt;            // tokens of a tile: 128 / g
  int tiles;         // items of a prompt of the longest length (by position), 0: items packed
  int packed;        // ... and then their number
  int items;         // places for items of all kv heads
  float scale2;      // scale * log2(e)
  float qs, mul;     // its magnitude (1 for 0), and the factor (1, -1, 0) that is left
  int window, chunk;
  int32_t *err;
  int checked, stall;
  unsigned long long wait_ns;
};

template <int D, int NQT>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF = 128 * 128;  // bytes of 128 rows of 64 dims
  static constexpr int TILE = HALVES * HALF;
  static constexpr int NSK = NQT == 2 ? (D == 128 ? 2 : 4) : (D == 128 ? 1 : 2);
  static constexpr int NSV = NSK;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NQT * TILE;
  static constexpr int OFF_V = OFF_K + NSK * TILE;
  // 32 rows of a softmax warp on their way out: all dims, or 32 of them at a time
  static constexpr int STAGE_ROW = NQT == 2 ? 128 : 64;
  static constexpr int OFF_STAGE = OFF_V + NSV * TILE;
  static constexpr int OFF_NOTE = OFF_STAGE + NQT * 4 * 32 * STAGE_ROW;  // [2][kNoted][4] masks
  static constexpr int OFF_BAR = OFF_NOTE + 2 * kNoted * 16;
  static constexpr int OFF_ITEM = OFF_BAR + 384;
  static constexpr int SMEM = OFF_ITEM + kAhead * 64 + 1024;  // alignment slack
  static constexpr int THREADS = 128 + NQT * 128;
  static constexpr uint32_t COLS = NQT * 256;  // tensor memory: S of each tile, then O
  static constexpr uint32_t O_COL = NQT * KT;
  // barriers
  static constexpr int Q_FULL = 0, Q_EMPTY = 1, K_FULL = 2, K_EMPTY = K_FULL + NSK, V_FULL = K_EMPTY + NSK,
                       V_EMPTY = V_FULL + NSV, V_OK = V_EMPTY + NSV, S_FULL = V_OK + NSV, P_FULL = S_FULL + NQT,
                       P_REST = P_FULL + NQT, O_FULL = P_REST + NQT, NOTED = O_FULL + NQT, I_FULL = NOTED + 2,
                       I_EMPTY = I_FULL + kAhead, DRAIN = I_EMPTY + kAhead, NBAR = DRAIN + 1;
  static_assert(NBAR * 8 + 36 <= 384 && SMEM <= (NQT == 2 ? 232448 : 115 * 1024), "shared memory");
};

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}
template <bool F16>
__device__ __forceinline__ float val(uint16_t x) {
  return F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float(static_cast<uint32_t>(x) << 16);
}
// The signs' places of a pair of values: set where one is not finite (an
// exponent of all ones carries into the sign's place).
template <bool F16>
__device__ __forceinline__ uint32_t exponents_full(const uint4 &x) {
  const uint32_t m = F16 ? 0x7C007C00u : 0x7F807F80u, one = F16 ? 0x04000400u : 0x00800080u;
  return ((x.x & m) + one) | ((x.y & m) + one) | ((x.z & m) + one) | ((x.w & m) + one);
}
// x + a . b of two pairs
template <bool F16>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float x) {
  x = fmaf(val<F16>(static_cast<uint16_t>(a)), val<F16>(static_cast<uint16_t>(b)), x);
  return fmaf(val<F16>(static_cast<uint16_t>(a >> 16)), val<F16>(static_cast<uint16_t>(b >> 16)), x);
}

// An item.
struct Item {
  int start, len;        // the prompt's first token, its tokens
  int p0, p1;            // the item's first and last query
  int head;              // kv head
  int nt;                // tiles
  int j0, n_iter;        // tiles of keys
  int all_lo, all_hi;    // keys that all of its queries see
};
static_assert(sizeof(Item) <= 64, "an item's place in shared memory");

// The item at place b; all lanes of the calling warp.  False: none.
template <int NQT>
__device__ __forceinline__ bool find_item(const Args &a, int b, Item &it) {
  const int lane = threadIdx.x & 31, qt = NQT * a.rt;
  it.head = b % a.hkv;
  b /= a.hkv;
  int s, tile;
  if (a.tiles > 0) {  // the longest key ranges of all prompts first
    s = b % a.num_seqs;
    tile = a.tiles - 1 - b / a.num_seqs;
  } else {
    // items are numbered so that prompt s begins at start(s) / qt + s: room
    // for all of its items, and no sums over the prompts before it
    const int i = a.packed - 1 - b;
    int lo = 0, n = a.num_seqs;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const int x = lo + lane * step;
      const bool in = lane * step < n && __ldg(a.starts + x) / qt + x <= i;
      const int c = __popc(__ballot_sync(0xffffffffu, in));
      const int skip = (c > 0 ? c - 1 : 0) * step;
      lo += skip;
      n = min(step, n - skip);
    }
    s = lo;
    tile = i - (__ldg(a.starts + s) / qt + s);
  }
  it.start = __ldg(a.starts + s);
  int end = __ldg(a.starts + s + 1);
  if (a.checked) {
    if (it.start < 0 || end < it.start || end > a.num_tokens) return false;  // (reported by CTA 0)
  }
  it.len = end - it.start;
  if (tile < 0 || tile >= (it.len + qt - 1) / qt) return false;
  it.p0 = tile * qt;
  it.p1 = min(it.p0 + qt, it.len) - 1;
  it.nt = it.p1 - it.p0 < a.rt ? 1 : NQT;
  it.j0 = local_first_key(it.p0, a.window, a.chunk) / KT;
  it.n_iter = it.p1 / KT + 1 - it.j0;
  it.all_lo = local_first_key(it.p1, a.window, a.chunk);
  it.all_hi = it.p0 + 1;
  return true;
}

// The place of this CTA's i-th item: rows of a place per CTA, every second one
// backwards.
__device__ __forceinline__ int place(int i) {
  const int c = blockIdx.x, n = gridDim.x;
  return i * n + (i & 1 ? n - 1 - c : c);
}

template <int R>
__device__ __forceinline__ void set_registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

// Whether a row of D values (16-byte aligned) has one that is not finite.
template <int D, bool F16>
__device__ __forceinline__ bool not_finite(const uint16_t *row) {
  const uint4 *x = reinterpret_cast<const uint4 *>(row);
  uint32_t bad = 0;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) bad |= exponents_full<F16>(__ldg(x + c));
  return (bad & 0x80008000u) != 0;
}

// The outputs of a row (a lane of tensor memory, live or not; the whole warp
// calls it) of an item with noted V rows: the products' sums, and the noted rows
// that its query sees.  Partly seen tiles past the first kNoted are looked
// over here, a row a lane: a chunk of 2^20 keys then takes some 10 ms, far from the
// limit of the waits for this warp, and so does one whose rows are all noted.
template <int D, bool F16>
__device__ __noinline__ void store_noted(const Args &a, const uint32_t *notes, const Item &it, int pos, int head,
                                         int first, bool live, float inv, float lse2, uint32_t o_at) {
  const int lane = threadIdx.x & 31;
  const uint4 *q = reinterpret_cast<const uint4 *>(a.q + static_cast<int64_t>(it.start + pos) * a.q_stride + head * D);
  uint8_t *out = static_cast<uint8_t *>(a.out) + (static_cast<int64_t>(it.start + pos) * a.hq + head) * (D * 2);
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 64) {
    float o[2][32];
    tmem_ld32(o_at + c0, o[0]);
    tmem_ld32(o_at + c0 + 32, o[1]);
#pragma unroll
    for (int x = 0; x < 64; ++x) o[x >> 5][x & 31] *= inv;
    int e = 0;
#pragma unroll 1
    for (int jj = 0; jj < it.n_iter; ++jj) {
      const int k0 = (it.j0 + jj) * KT;
      if (k0 >= it.all_lo && k0 + KT <= it.all_hi) continue;
#pragma unroll 1
      for (int w = 0; w < KT; w += 32) {
        uint32_t bad;
        if (e < kNoted) {
          bad = notes[e * 4 + (w >> 5)];
        } else {
          const int key = k0 + w + lane;
          bad = __ballot_sync(0xffffffffu, key <= it.p1 && not_finite<D, F16>(a.v + static_cast<int64_t>(it.start + key) *
                                                                                       a.v_stride + it.head * D));
        }
#pragma unroll 1
        for (; bad; bad &= bad - 1) {
          const int key = k0 + w + __ffs(bad) - 1;
          if (!live || key < first || key > pos) continue;
          const uint4 *k =
              reinterpret_cast<const uint4 *>(a.k + static_cast<int64_t>(it.start + key) * a.k_stride + it.head * D);
          const uint4 *v = reinterpret_cast<const uint4 *>(a.v + static_cast<int64_t>(it.start + key) * a.v_stride +
                                                           it.head * D + c0);
          float x = 0.f;
#pragma unroll 2
          for (int d = 0; d < D / 8; ++d) {
            const uint4 qd = __ldg(q + d), kd = __ldg(k + d);
            x = dot2<F16>(qd.x, kd.x, x);
            x = dot2<F16>(qd.y, kd.y, x);
            x = dot2<F16>(qd.z, kd.z, x);
            x = dot2<F16>(qd.w, kd.w, x);
          }
          const float p = exp2f(x * a.scale2 - lse2);
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const uint4 vd = __ldg(v + d);
            const uint32_t u[4] = {vd.x, vd.y, vd.z, vd.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float *y = &o[d >> 2][(d & 3) * 8 + 2 * i];
              y[0] = fmaf(p, val<F16>(static_cast<uint16_t>(u[i])), y[0]);
              y[1] = fmaf(p, val<F16>(static_cast<uint16_t>(u[i] >> 16)), y[1]);
            }
          }
        }
      }
      ++e;
    }
    __syncwarp();
    if (live)
#pragma unroll
      for (int x = 0; x < 64; x += 2)
        *reinterpret_cast<uint32_t *>(out + (c0 + x) * 2) = pack2<F16>(o[x >> 5][x & 31], o[x >> 5][(x & 31) + 1]);
  }
}

// PAIR: the weights go to the products as a hi + lo pair.
template <int D, bool F16, int NQT, bool PAIR>
__global__ void __launch_bounds__(Cfg<D, NQT>::THREADS, NQT == 2 ? 1 : 2) prompt_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, NQT>;
  constexpr int KVT = F16 ? kKvF16 : kKvBf16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + C::NBAR);
  volatile int *s_abort = reinterpret_cast<int *>(tmem_slot + 1);
  int *s_noted = reinterpret_cast<int *>(tmem_slot + 2);  // [2][2]: of each of the warps that look over V
  int *s_last = reinterpret_cast<int *>(tmem_slot + 6);   // K and V tiles and Qs whose copies were issued
  uint32_t *notes = reinterpret_cast<uint32_t *>(smem + C::OFF_NOTE);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  if (tid == 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.qmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&a.vmap)) : "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < C::NSK; ++i) {
      mbar_init(&bar[C::K_FULL + i], 1);
      mbar_init(&bar[C::K_EMPTY + i], 1);
    }
    for (int i = 0; i < C::NSV; ++i) {
      mbar_init(&bar[C::V_FULL + i], 1);
      mbar_init(&bar[C::V_EMPTY + i], 1);
      mbar_init(&bar[C::V_OK + i], 2);
    }
    for (int t = 0; t < NQT; ++t) {
      mbar_init(&bar[C::S_FULL + t], 1);
      mbar_init(&bar[C::P_FULL + t], 4);
      mbar_init(&bar[C::P_REST + t], 4);
      mbar_init(&bar[C::O_FULL + t], 1);
    }
    mbar_init(&bar[C::Q_FULL], 1);
    mbar_init(&bar[C::Q_EMPTY], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&bar[C::NOTED + i], NQT * 4);
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&bar[C::I_FULL + i], 1);
      mbar_init(&bar[C::I_EMPTY + i], 3 + NQT * 4);
    }
    mbar_init(&bar[C::DRAIN], 1);
    *s_abort = 0;
    for (int i = 0; i < 4; ++i) s_noted[i] = 0;
    s_last[0] = s_last[1] = s_last[2] = 0;
    fence_mbar_init();
  }
  for (int i = tid; i < 2 * kNoted * 4; i += C::THREADS) notes[i] = 0;
  if (warp == 0) tmem_alloc(tmem_slot, C::COLS);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // the tensor memory of a kernel before this one is free by now, its results
  // are there after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.checked && blockIdx.x == 0)
    for (int s = tid; s < a.num_seqs; s += C::THREADS) {
      const int b = __ldg(a.starts + s), e = __ldg(a.starts + s + 1);
      if (b < 0 || e < b || e > a.num_tokens || e - b > a.max_q_len) report_error(a.err, nullptr, kErrBadIndex);
    }
  bool ok = true;
  Item it;
  int n_items = 0;
  const Item *ring = reinterpret_cast<const Item *>(smem + C::OFF_ITEM);  // 64 bytes apart
  // the next item that the copying warp found; false: no more, or a wait ran out
  auto next_item = [&]() {
    const int st = n_items % kAhead;
    if (!mbar_wait(&bar[C::I_FULL + st], (n_items / kAhead) & 1, a.wait_ns)) {
      ok = false;
      return false;
    }
    it = *reinterpret_cast<const Item *>(reinterpret_cast<const uint8_t *>(ring) + st * 64);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[C::I_EMPTY + st]);
    ++n_items;
    return it.nt > 0;
  };

  if (warp < 4) {
    set_registers_down<NQT == 2 ? 88 : 56>();
    if (warp == 1) {
      // ------------------------------------------------------- copies
      const uint64_t pol = l2_evict_first_policy();
      uint64_t keep;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
      int nq = 0, nk = 0;  // Qs, K (and V) tiles so far
      // hands an item (nt 0: the end) to the other warps
      auto publish = [&]() {
        const int st = n_items % kAhead, use = n_items / kAhead;
        if (use > 0 && !mbar_wait(&bar[C::I_EMPTY + st], (use - 1) & 1, a.wait_ns)) ok = false;
        if (ok && lane == 0) {
          *reinterpret_cast<Item *>(smem + C::OFF_ITEM + st * 64) = it;
          mbar_arrive(&bar[C::I_FULL + st]);
        }
        ++n_items;
      };
      for (int i = 0; i * gridDim.x < static_cast<unsigned>(a.items) && ok; ++i) {
        const int b = place(i);
        if (b >= a.items || !find_item<NQT>(a, b, it)) continue;
        publish();
        if (a.stall) continue;
        if (nq > 0 && !mbar_wait(&bar[C::Q_EMPTY], (nq - 1) & 1, a.wait_ns)) ok = false;
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&bar[C::Q_FULL], it.nt * C::HALVES * a.rt * a.g * 128);
          for (int t = 0; t < it.nt; ++t)
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_3d(smem + C::OFF_Q + t * C::TILE + h * C::HALF, &a.qmap, h * 64, it.head * a.g,
                          it.start + it.p0 + t * a.rt, &bar[C::Q_FULL], pol);
          s_last[2] = nq + 1;
        }
        ++nq;
        for (int jj = 0; jj < it.n_iter && ok; ++jj, ++nk) {
          const int row = it.start + (it.j0 + jj) * KT, st = nk % C::NSK, use = nk / C::NSK;
#pragma unroll
          for (int part = 0; part < 2; ++part) {  // K, V
            const int full = (part ? C::V_FULL : C::K_FULL) + st, empty = (part ? C::V_EMPTY : C::K_EMPTY) + st;
            if (ok && use > 0 && !mbar_wait(&bar[empty], (use - 1) & 1, a.wait_ns)) ok = false;
            if (*s_abort) ok = false;
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(&bar[full], C::TILE);
              for (int h = 0; h < C::HALVES; ++h)
                tma_load_3d(smem + (part ? C::OFF_V : C::OFF_K) + st * C::TILE + h * C::HALF, part ? &a.vmap : &a.kmap,
                            h * 64, it.head, row, &bar[full], keep);
              s_last[part] = nk + 1;
            }
          }
        }
      }
      it.nt = 0;
      if (ok) publish();
    } else if (warp == 0) {
      // ----------------------------------------------------- products
      // the warp stays together, so that the operands are in uniform registers
      // and a product is one instruction: with a lane's own registers the
      // issuing took 105 and 80 cycles a product and 300 between the tiles
      constexpr uint32_t IQK = umma_idesc_bf16(128, KT, false, false, F16);
      constexpr uint32_t IPV = umma_idesc_bf16(128, D, false, true, F16);
      const uint32_t q_lo = uniform(desc_low(sbase + C::OFF_Q, 16)), k_lo = uniform(desc_low(sbase + C::OFF_K, 16));
      const uint32_t v_lo = uniform(desc_low(sbase + C::OFF_V, C::HALF));
      const uint32_t tm = uniform(tmem);
      auto qk = [&](int t, int stage) {
        const uint32_t qd = uniform(q_lo + t * (C::TILE >> 4)), kd = uniform(k_lo + stage * (C::TILE >> 4));
        const uint32_t s = uniform(tm + t * KT);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4;
            mma_ss(s, qd + off, desc_high(1024), kd + off, desc_high(1024), IQK, kk > 0);
          }
        }
        __syncwarp();
      };
      auto pv = [&](int t, int stage, int half, bool more) {
        const uint32_t vd = uniform(v_lo + stage * (C::TILE >> 4)), p = uniform(tm + t * KT);
        const uint32_t o = uniform(tm + C::O_COL + t * D), acc = uniform(more ? 1u : 0u);
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kk = half * 4 + i;
            mma_ts(o, p + (kk >> 1) * 32 + (kk & 1) * 8, vd + kk * (2048 >> 4), desc_high(1024), IPV,
                   kk > 0 || acc != 0);
            if constexpr (PAIR)
              mma_ts(o, p + (kk >> 1) * 32 + 16 + (kk & 1) * 8, vd + kk * (2048 >> 4), desc_high(1024), IPV, true);
          }
        }
        __syncwarp();
      };
      auto commit = [&](int b) {
        if (elect_one()) umma_commit(&bar[b]);
        __syncwarp();
      };
      uint32_t nq = 0, p_par[2] = {0, 0};
      int vs = 0, ks = 0;  // stages of the next V and K tile, and their parities
      uint32_t v_par = 0, k_par = 0;
      while (ok && next_item()) {
        const int nt = it.nt, n_iter = it.n_iter;
        // S of a key tile, both query tiles; then its K is done with
        auto k_done = [&](bool last) {
          commit(C::K_EMPTY + ks);
          if (last) commit(C::Q_EMPTY);
          if (++ks == C::NSK) {
            ks = 0;
            k_par ^= 1;
          }
        };
        ok = mbar_wait(&bar[C::Q_FULL], nq & 1, a.wait_ns) && mbar_wait(&bar[C::K_FULL + ks], k_par, a.wait_ns);
        ++nq;
        if (!ok) break;
        tc_fence_after_sync();
        for (int t = 0; t < nt; ++t) {
          qk(t, ks);
          commit(C::S_FULL + t);
        }
        k_done(n_iter == 1);
        for (int jj = 0; jj < n_iter && ok; ++jj) {
          const bool next = jj + 1 < n_iter;
          ok = mbar_wait(&bar[C::V_OK + vs], v_par, a.wait_ns);
#pragma unroll
          for (int t = 0; t < NQT; ++t) {
            if (t >= nt || !ok) continue;
            if (!mbar_wait_hint(&bar[C::P_FULL + t], p_par[t], a.wait_ns)) {
              ok = false;
              continue;
            }
            tc_fence_after_sync();
            pv(t, vs, 0, jj > 0);
            if (!mbar_wait_hint(&bar[C::P_REST + t], p_par[t], a.wait_ns)) {
              ok = false;
              continue;
            }
            p_par[t] ^= 1;
            tc_fence_after_sync();
            pv(t, vs, 1, true);
            if (t == nt - 1) commit(C::V_EMPTY + vs);
            if (next) {
              if (t == 0 && !mbar_wait(&bar[C::K_FULL + ks], k_par, a.wait_ns)) {
                ok = false;
                continue;
              }
              tc_fence_after_sync();
              qk(t, ks);
              commit(C::S_FULL + t);  // S of the next key tile is there, and P V of this one done
            } else {
              commit(C::O_FULL + t);
            }
          }
          if (next && ok) k_done(jj + 2 == n_iter);
          if (++vs == C::NSV) {
            vs = 0;
            v_par ^= 1;
          }
        }
      }
    } else {
      // ------------------------------------------------- V tiles looked over
      // Warp 2 has rows 0..31 and 64..95 of a tile, warp 3 the others: each
      // has words of its own in a tile's mask (w, w + 2) and a flag of its own,
      // and so never waits for the other, which may be tiles ahead of it or
      // have given up.
      const int ct = tid - 64, w = warp - 2;
      int nv = 0;
      while (ok && next_item()) {
        const int buf = (n_items - 1) & 1;
        uint32_t *note = notes + buf * kNoted * 4;
        volatile int *noted = &s_noted[2 * buf + w];
        // the notes of the item before the last are read: this warp's are cleared
        if (n_items > 2) {
          if (!mbar_wait(&bar[C::NOTED + buf], (((n_items - 1) >> 1) - 1) & 1, a.wait_ns)) {
            ok = false;
            break;
          }
          const bool used = *noted != 0;  // (set by lanes of this warp)
          __syncwarp();
          if (used) {
            for (int x = lane; x < kNoted; x += 32) note[x * 4 + w] = note[x * 4 + w + 2] = 0;
            if (lane == 0) *noted = 0;
          }
          __syncwarp();
        }
        int e = 0;  // partly seen tiles so far
        for (int jj = 0; jj < it.n_iter; ++jj, ++nv) {
          const int st = nv % C::NSV, k0 = (it.j0 + jj) * KT;
          if (!mbar_wait(&bar[C::V_FULL + st], (nv / C::NSV) & 1, a.wait_ns)) {
            ok = false;
            break;
          }
          if (k0 < it.all_lo || k0 + KT > it.all_hi) {
            uint8_t *vt = smem + C::OFF_V + st * C::TILE;
#pragma unroll 1
            for (int r = ct; r < KT; r += 64) {
              const bool drop = k0 + r > it.p1;
              uint32_t bad = 0;
              if (!drop) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                  const uint4 x =
                      *reinterpret_cast<const uint4 *>(vt + (c >> 3) * C::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                  bad |= exponents_full<F16>(x);
                }
                bad &= 0x80008000u;
              }
              if (drop || bad) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                  *reinterpret_cast<uint4 *>(vt + (c >> 3) * C::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                      make_uint4(0, 0, 0, 0);
                if (!drop) {
                  if (e < kNoted) atomicOr(&note[e * 4 + (r >> 5)], 1u << (r & 31));
                  *noted = 1;
                }
              }
            }
            fence_proxy_async_smem();
            ++e;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C::V_OK + st]);
        }
      }
    }
  } else {
    // --------------------------------------------------------- softmax
    set_registers_up<NQT == 2 ? 208 : 200>();
    const int t = (warp - 4) >> 2, r = tid - 128 - t * 128;  // tile, row
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int tok = r / a.g, sub = r - tok * a.g;
    uint8_t *stage = smem + C::OFF_STAGE + (warp - 4) * 32 * C::STAGE_ROW;
    const unsigned g_inv = (65536 + a.g - 1) / a.g;  // x / g = x * g_inv >> 16 for x < 128
    uint32_t s_par = 0, o_par = 0;
    while (ok && next_item()) {
      const int buf = (n_items - 1) & 1;
      if (t < it.nt) {
        const int pos = min(it.p0 + t * a.rt + tok, it.p1);
        const int first = local_first_key(pos, a.window, a.chunk);
        // keys that every row of this warp sees
        const int w_hi = __reduce_min_sync(0xffffffffu, pos), w_lo = __reduce_max_sync(0xffffffffu, first);
        float ms = -INFINITY;  // the reference maximum, scaled
        float lsum = 0.f;
        for (int jj = 0; jj < it.n_iter; ++jj) {
          const int k0 = (it.j0 + jj) * KT;
          if (!mbar_wait(&bar[C::S_FULL + t], s_par, a.wait_ns)) {
            ok = false;
            break;
          }
          s_par ^= 1;
          tc_fence_after_sync();
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_async(trow + t * KT + c * 32, s[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
          if (a.mul != 1.f) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int x = 0; x < 32; ++x) s[c][x] = __float_as_uint(__uint_as_float(s[c][x]) * a.mul);
          }
          if (k0 + KT > w_hi + 1 || k0 < w_lo) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int c0 = k0 + c * 32;
              if (c0 + 31 > w_hi) {  // some row's last key is before the chunk's end
                const int hi = pos - c0;
#pragma unroll
                for (int x = 0; x < 32; ++x) s[c][x] = x > hi ? 0xff800000u : s[c][x];  // -inf
              }
              if (c0 < w_lo) {
                const int lo = first - c0;
#pragma unroll
                for (int x = 0; x < 32; ++x) s[c][x] = x < lo ? 0xff800000u : s[c][x];
              }
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float m4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t *x = &s[c][8 * k];
              m4[k] = fmax3(fmax3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2])),
                            fmax3(__uint_as_float(x[3]), __uint_as_float(x[4]), __uint_as_float(x[5])),
                            fmaxf(__uint_as_float(x[6]), __uint_as_float(x[7])));
            }
            mx[c] = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
          }
          const float mt = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * a.qs;
          if (__any_sync(0xffffffffu, mt > ms + kRaise)) {
            const float nm = fmaxf(ms, mt);
            const float alpha = ms == -INFINITY ? 0.f : ex2_approx(ms - nm);
            ms = nm;
            lsum *= alpha;
            if (jj > 0) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(trow + C::O_COL + t * D + c, o);
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= alpha;
                tmem_st32(trow + C::O_COL + t * D + c, o);
              }
            }
          }
          const float ref = ms == -INFINITY ? 0.f : ms;
          const uint64_t q2 = f2_pack(a.qs, a.qs), r2 = f2_pack(-ref, -ref);
          uint64_t l2[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16], lo[PAIR ? 16 : 1];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float2 y = f2_unpack(
                  f2_fma(f2_pack(__uint_as_float(s[c][2 * x]), __uint_as_float(s[c][2 * x + 1])), q2, r2));
              const float e0 = ex2_approx(y.x), e1 = ex2_approx(y.y);
              l2[x & 1] = f2_add(l2[x & 1], f2_pack(e0, e1));
              p[x] = pack16x2<KVT>(e0, e1);
              if constexpr (PAIR) lo[x] = pack16x2<KVT>(e0 - lo16<KVT>(p[x]), e1 - hi16<KVT>(p[x]));
            }
            tmem_st16_async(trow + t * KT + c * 32, p);
            if constexpr (PAIR) tmem_st16_async(trow + t * KT + c * 32 + 16, lo);  // (S is in registers)
            if (c & 1) {  // the first 64 keys' products need not wait for the rest
              tmem_wait_st();
              tc_fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar[(c == 1 ? C::P_FULL : C::P_REST) + t]);
            }
          }
          const float2 la = f2_unpack(f2_add(l2[0], l2[1]));
          lsum += la.x + la.y;
        }
        // the last products are done: out, through shared memory, so that a
        // warp's stores cover whole rows (a row a thread was 16 bytes of 32
        // rows a store: 64 lines each, 6000 cycles an item)
        if (ok && !mbar_wait(&bar[C::O_FULL + t], o_par, a.wait_ns)) ok = false;
        o_par ^= 1;
        if (!ok) break;
        tc_fence_after_sync();
        const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // (a NaN stays one)
        const float lse2 = lsum == 0.f ? -INFINITY : ms + log2f(lsum);
        const int tok0 = it.start + it.p0 + t * a.rt;
        const int left = min(a.rt, it.p1 + 1 - (it.p0 + t * a.rt)) * a.g;  // rows in use
        const int head = it.head * a.g + sub;
        if (r < left && a.lse) a.lse[static_cast<int64_t>(tok0 + tok) * a.hq + head] = lse2 * kLn2;
        volatile int *noted = &s_noted[2 * buf];
        if ((noted[0] | noted[1]) != 0) {
          store_noted<D, F16>(a, notes + buf * kNoted * 4, it, pos, head, first, r < left, inv, lse2,
                              trow + C::O_COL + t * D);
        } else {
          constexpr int PART = C::STAGE_ROW / 2;  // dims staged at a time
          constexpr int LPR = C::STAGE_ROW / 16;  // lanes of a staged row
          uint8_t *out = static_cast<uint8_t *>(a.out) + (static_cast<int64_t>(tok0) * a.hq + it.head * a.g) * (D * 2);
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += PART) {
#pragma unroll
            for (int h = 0; h < PART / 32; ++h) {
              float o[32];
              tmem_ld32(trow + C::O_COL + t * D + c0 + h * 32, o);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4 *>(stage + lane * C::STAGE_ROW + (((h * 4 + x) ^ (lane & (LPR - 1))) << 4)) =
                    make_uint4(pack2<F16>(o[8 * x] * inv, o[8 * x + 1] * inv),
                               pack2<F16>(o[8 * x + 2] * inv, o[8 * x + 3] * inv),
                               pack2<F16>(o[8 * x + 4] * inv, o[8 * x + 5] * inv),
                               pack2<F16>(o[8 * x + 6] * inv, o[8 * x + 7] * inv));
            }
            __syncwarp();
            const int ch = lane % LPR;
#pragma unroll
            for (int x = 0; x < LPR; ++x) {
              const int rr = x * (32 / LPR) + lane / LPR, q = (warp & 3) * 32 + rr;
              const uint4 v =
                  *reinterpret_cast<const uint4 *>(stage + rr * C::STAGE_ROW + ((ch ^ (rr & (LPR - 1))) << 4));
              const int qtok = static_cast<int>(q * g_inv >> 16);
              if (q < left)
                *reinterpret_cast<uint4 *>(out + (static_cast<int64_t>(qtok) * a.hq + (q - qtok * a.g)) * (D * 2) +
                                           c0 * 2 + ch * 16) = v;
            }
            __syncwarp();
          }
        }
      } else if (n_items > 2 && !mbar_wait(&bar[C::NOTED + buf], (((n_items - 1) >> 1) - 1) & 1, a.wait_ns)) {
        // (a tile without rows here could be items ahead of the other one, and
        // would count twice for the notes that the other still reads)
        ok = false;
        break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::NOTED + buf]);
    }
  }
  if (!ok) *s_abort = 1;

  // --- the end: copies in flight land, products complete, then the memory goes
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (*s_abort) {
    if (tid == 0) report_error(a.err, nullptr, kErrWaitTimeout);
    if (warp == 1) {
      if (s_last[2] > 0) mbar_wait(&bar[C::Q_FULL], (s_last[2] - 1) & 1, a.wait_ns);
      for (int j = max(0, s_last[0] - C::NSK); j < s_last[0]; ++j)
        mbar_wait(&bar[C::K_FULL + j % C::NSK], (j / C::NSK) & 1, a.wait_ns);
      for (int j = max(0, s_last[1] - C::NSV); j < s_last[1]; ++j)
        mbar_wait(&bar[C::V_FULL + j % C::NSV], (j / C::NSV) & 1, a.wait_ns);
    }
  }
  if (warp == 0) {
    if (elect_one()) umma_commit(&bar[C::DRAIN]);  // the lane that issued the products
    __syncwarp();
    mbar_wait(&bar[C::DRAIN], 0, a.wait_ns);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, C::COLS);
}

// Rows [tokens][heads][d], `stride` elements from token to token, box {64
// dims, `heads_box` heads, `tokens_box` tokens}; behind the last token zeros.
bool make_rows_map(CUtensorMap *map, const void *base, bool f16, int tokens, int heads, int d, int64_t stride,
                   int heads_box, int tokens_box) {
  thread_local MapCache<24> cache;
  const MapKey key = map_key(base, f16, tokens, heads, d, stride, heads_box, tokens_box);
  if (cache.find(key, map)) return true;
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads_box), static_cast<cuuint32_t>(tokens_box)};
  const cuuint32_t estr[3] = {1, 1, 1};
  if (enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base),
          dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  cache.put(key, *map);
  return true;
}

template <int D, bool F16, int NQT, bool PAIR>
cudaError_t launch(Args &a, int max_q_len, cudaStream_t stream) {
  using C = Cfg<D, NQT>;
  const void *fn = reinterpret_cast<const void *>(&prompt_kernel<D, F16, NQT, PAIR>);
  if (prepare_kernel(fn, C::THREADS, C::SMEM) < 1) return cudaErrorInvalidConfiguration;
  const int qt = NQT * a.rt;
  // by position, the longest key ranges first, unless that leaves too many
  // CTAs without an item (prompts much shorter than the longest)
  const int64_t by_pos = (static_cast<int64_t>(max_q_len) + qt - 1) / qt * a.num_seqs;
  const int64_t packed = a.num_tokens / qt + static_cast<int64_t>(a.num_seqs);
  a.tiles = by_pos <= 2 * packed ? (max_q_len + qt - 1) / qt : 0;
  a.packed = static_cast<int>(packed);
  a.items = static_cast<int>((a.tiles ? by_pos : packed) * a.hkv);
  const int ctas = device_sm_count() * (NQT == 2 ? 1 : 2);
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.items < ctas ? a.items : ctas));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  void *args[] = {&a};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int D, bool F16, bool PAIR>
cudaError_t launch_tiles(Args &a, int max_q_len, cudaStream_t stream) {
  // prompts of one tile: a smaller CTA, two to an SM
  return max_q_len <= a.rt ? launch<D, F16, 1, PAIR>(a, max_q_len, stream)
                           : launch<D, F16, 2, PAIR>(a, max_q_len, stream);
}

template <int D, bool F16>
cudaError_t launch_weights(Args &a, bool pair, int max_q_len, cudaStream_t stream) {
  return pair ? launch_tiles<D, F16, true>(a, max_q_len, stream) : launch_tiles<D, F16, false>(a, max_q_len, stream);
}

}  // namespace

cudaError_t launch_prompt(const pa_kv_desc &d, void *out, float *lse, const void *q, int64_t q_stride, const void *k,
                          int64_t k_stride, const void *v, int64_t v_stride, const int32_t *query_start_loc,
                          int32_t num_seqs, int32_t num_tokens, int32_t max_q_len, float scale, cudaStream_t stream) {
  Args a;
  memset(&a, 0, sizeof a);
  const bool f16 = d.kv_dtype == PA_KV_F16 || d.kv_dtype == PA_KV_INT4_F16;
  const int D = d.head_dim;
  a.g = d.num_q_heads / d.num_kv_heads;
  a.rt = 128 / a.g;
  a.q_stride = q_stride ? q_stride : static_cast<int64_t>(d.num_q_heads) * D;
  a.k_stride = k_stride ? k_stride : static_cast<int64_t>(d.num_kv_heads) * D;
  a.v_stride = v_stride ? v_stride : static_cast<int64_t>(d.num_kv_heads) * D;
  if (!make_rows_map(&a.qmap, q, f16, num_tokens, d.num_q_heads, D, a.q_stride, a.g, a.rt) ||
      !make_rows_map(&a.kmap, k, f16, num_tokens, d.num_kv_heads, D, a.k_stride, 1, KT) ||
      !make_rows_map(&a.vmap, v, f16, num_tokens, d.num_kv_heads, D, a.v_stride, 1, KT))
    return cudaErrorInvalidValue;
  a.out = out;
  a.lse = lse;
  a.q = static_cast<const uint16_t *>(q);
  a.k = static_cast<const uint16_t *>(k);
  a.v = static_cast<const uint16_t *>(v);
  a.starts = query_start_loc;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.max_q_len = max_q_len;
  a.hq = d.num_q_heads;
  a.hkv = d.num_kv_heads;
  a.scale2 = scale * kLog2e;
  a.qs = scale == 0.f ? 1.f : fabsf(a.scale2);
  a.mul = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
  a.window = d.sliding_window;
  a.chunk = d.attention_chunk;
  a.err = d.error_word;
  a.checked = d.check_indices;
  const TestHooks hooks = test_hooks();
  a.stall = hooks.stall;
  a.wait_ns = hooks.wait_ns;
  // the settings whose prefill multiplies by a pair too
  const bool pair = d.prefill_impl == PA_PREFILL_TCGEN05_PAIR || d.prefill_impl == PA_PREFILL_MMA_SYNC;
  if (D == 128)
    return f16 ? launch_weights<128, true>(a, pair, max_q_len, stream)
               : launch_weights<128, false>(a, pair, max_q_len, stream);
  return f16 ? launch_weights<64, true>(a, pair, max_q_len, stream)
             : launch_weights<64, false>(a, pair, max_q_len, stream);
}

}  // namespace pa
