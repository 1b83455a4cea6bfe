// Causal attention over whole prompts: rows and keys of many sequences packed one behind another, on the 5th-generation
// tensor cores.
//
//   o_i = sum_{j <= i + off} p_j v_j / sum p_j,  p_j = 2^(s_j - m),  s_j = q_i k_j scale log2(e),  off = keys - rows.
// 4 d operations for each (row, visible key, query head) against 2 d (2 nq + 2 nkv) bytes a token: bound by the tensor cores
// from a few hundred tokens on, by latency below.
//
// The query heads of a KV head read the same keys, so a tile of 128 query vectors is RB = 128 / G positions times the G
// heads: one TMA box lays them out so, and grouped heads need neither copies nor masks of their own. An item is a pair of such
// tiles (2 RB positions of one KV head) with all the keys that its rows see, KT at a time. A CTA an SM takes items in
// turn, the ones with the most keys first. 16 warps:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one thread a query vector (TMEM lane): S row -> weights as bf16 in TMEM, running sum;
//                   O is rescaled only when the maximum moves by more than 2^8; a tile's first warp brings its Q by TMA and gives
//                   the ring's stages back;
//   warps 8-11      results: O of both tiles from TMEM, divided by the sums;
//   warp 12         finds the items, brings the next one's Q into L2; TMA: K and V tiles through one ring;
//   warps 13, 14    tcgen05.mma of tile 0 / 1: S = Q K^T (operands in shared memory), O += P V (P in TMEM, V read MN-major);
//   warp 15         looks through value tiles that not all rows see (below).
//
// TMEM decides the tile. With S, then P over it, of 128 keys (256 columns for two tiles, 256 for their O) a tile's chain of
// S, softmax, P V, S ... has no overlap but the other tile's: 1.7 us for 128 keys of a pair, of them 1.06 of products and 0.54 of
// softmax; the hand-overs between softmax and products, some 0.6 us a round, are in nobody's shadow. So P has columns of its
// own: S of the next keys is computed as soon as the softmax warps hold this one in registers. For d = 128 that leaves
// 80 keys a tile (S 80, P 40 of a tile's 128 columns beside O), for d = 64 128 keys (O 64, S 128, P 64 of 256). A pair's 128 keys
// then take 1.43 us (1.21 of products: of 80 columns they are bound by reading Q from shared memory); without any softmax
// work 1.36: what is left is the way of S into the softmax warps and back, 1100 clocks beside its products. (Tiles of 64 keys with two
// P, so that no weights wait for a product: 1.79. A key tile takes its 0.9 us whatever its size.)
//
// The tiles are not kept in step: each has its own warps throughout, and one runs ahead of the other as far as the ring
// lets it. (In turn, key tile by key tile: 64 prompts of 128 to 2048 tokens of 32 heads over 8 928 us instead of 812.) Those take
// 740 us in a short burst (800 to 850 in a stream of calls, at the clocks of the power cap), the products of what rows see 404 (450):
// 96 are for keys behind the diagonal, and 59 items a CTA have some 4 us each until
// products follow without a pause: the last, masked softmax, then the issuing warp's way to the next item and its first S, 5100 clocks
// where a key tile's period is 1700, and 0.9 us for results that the next item waits for. (A first S ahead of the last value
// product: 852; what the issuing warp does besides slows every key tile. 110 KB of code instead of 80: 893.)
//
// Weights are rounded to bf16 (2^-8 relative at most, as the values that they meet); maxima, sums and outputs are fp32, the
// sum of the unrounded weights. That rounding is what results are off by beyond their own: 64-bit arithmetic with weights rounded
// as here is off the exact results by 0.0021 relative (1024 tokens of 32 heads; rounded results alone: 0.0016), the kernel off it by 0.00006.
//
// A weight of zero does not hide a value that is not finite (0 * inf = NaN). Warp 15 looks through the value tiles that some
// rows see only in part, beside the products. Where it finds such a value the CTA takes all its items again, now with the
// products behind its look: it replaces the values by zero and keeps, for each column, the first key that held a NaN, +inf and
// -inf; rows that see it get that value in their results, the others are left alone. (Every look in front of its products: 4 of
// 21 us for a prompt of 1024 tokens of 32 heads.)
#include "attn_tc.cuh"
#include "kernels.h"
#include "ops_ext.h"

#include <algorithm>
#include <cuda_bf16.h>

namespace eagle {
namespace {

constexpr int AT = 128;              // query vectors a tile
constexpr int AP_SOFT = 8;           // softmax warps, four a tile; behind them four that write results, then four single ones
constexpr int AP_TMA = AP_SOFT + 4, AP_MMA = AP_TMA + 1, AP_LOOK = AP_TMA + 3;
constexpr int AP_THREADS = (AP_SOFT + 8) * 32;
constexpr float AP_LAZY = 8.f;       // binary orders that a maximum may pass its reference by
// A wait gives up after EAGLE_WAIT_LIMIT_NS and this much for each key tile that there is: the warps that write results, and those
// of a tile without rows, wait for a whole item. (A key tile takes 0.9 to 1.2 us at the clocks seen, so 2^27 keys of one item 1.5 to 1.9 s.)
constexpr int AP_TILE_NS = 4000;
constexpr uint32_t AP_NONE = 0x3fffffffu;      // three fields of ten bits, "no key"

template <int D>
struct ApShape {
  static constexpr int KT = D == 128 ? 80 : 128;                          // keys a tile
  static constexpr int HALVES = D / 64, QHALF = AT * 128, KHALF = KT * 128;   // 64 dims of all rows
  static constexpr int QB = HALVES * QHALF, KB = HALVES * KHALF;          // a tile of Q, of K or V
  static constexpr int STAGES = 8;
  static constexpr int OFF_RING = 2 * QB, OFF_BAR = OFF_RING + STAGES * KB;
  static constexpr int OFF_ITEM = OFF_BAR + 448, OFF_BAD = OFF_ITEM + 2 * 48, OFF_INV = OFF_BAD + 2 * D * 4;
  static constexpr int BYTES = OFF_INV + 2 * AT * 4;
  // TMEM columns: O of both tiles, then S and P of each
  static constexpr int T_S = 2 * D, T_P = T_S + KT, T_STEP = (512 - 2 * D) / 2;
  static_assert(KT + KT / 2 <= T_STEP, "S and P of a tile beside O");
  // registers a thread of the softmax warps, the result warps, the single ones: together those of the launch, 128 each
  static constexpr int R_SOFT = 176, R_OUT = 88, R_ONE = 72;
  static_assert(2 * R_SOFT + R_OUT + R_ONE <= 4 * 128, "registers of the launch");
};

// What a CTA does next. lim0: the last key, from k0 on, that the first row sees (negative: none); rows of tile 0 and 1; key tiles
// of each; slot: where the sums of a piece of an item go, -1 for a whole one.
struct ApItem {
  int h, row0, rows[2], n[2], k0, lim0, slot;
};

struct ApArgs {
  int R, Rk, nq, nkv, G, RB, B;
  const int *start, *kstart;
  float sl2;                   // scale * log2(e)
  __nv_bfloat16* out;
  long long ldo;
  float* lse;
  int* err;
  unsigned long long wait_ns;  // what a wait may take (AP_TILE_NS)
  float *part_o, *part_ml;     // split: [slot][2 tiles][128][D], [slot][2 tiles][128][2]
  struct ApStart* starts;      // split: [CTA]
  struct ApJoin* joins;        // split: [CTA]
};

// One sequence's rows and keys; none where the starts are not in order or out of range.
struct ApSeq { int r0, lq, k0, lk; };
__device__ __forceinline__ ApSeq ap_seq(const ApArgs& a, int b, bool& bad) {
  const int r0 = __ldg(a.start + b), r1 = __ldg(a.start + b + 1), k0 = __ldg(a.kstart + b), k1 = __ldg(a.kstart + b + 1);
  bad = r0 < 0 || r1 < r0 || r1 > a.R || k0 < 0 || k1 < k0 || k1 > a.Rk;
  return bad ? ApSeq{0, 0, 0, 0} : ApSeq{r0, r1 - r0, k0, k1 - k0};
}

// The items' order. Pair t of a sequence has size t + off / (a pair's positions): proportional to its keys, nearly. A level
// holds the sizes that agree in their highest `bits` bits: as a rule one size each. Items go by falling level, then sequence, then
// falling size, then head: the last ones are the short ones, so the CTAs end together. A CTA goes through the sequences
// twice a level that has pairs, however many items it takes: it goes on where its last one was. (From
// the first sequence and the next level each time, 4096 prompts of 1 to 39 tokens of 32 heads took 5.7 ms instead of 0.93, 64 sequences
// of which one is 512 rows behind 100000 keys 2.4 instead of 1.2.)
//
// One pass is B / 32 rounds of a warp, 0.43 us each. Between two of its items a CTA may go through every level, and its
// other warps wait for that with a limit; so there are at most so many levels that their passes take AP_ROUNDS rounds, with
// fewer bits where sequences are many and sizes far apart. (2048 single rows of 8 heads over one behind up to 16000 keys:
// 2.1 ms, with a level for each of 1000 sizes 7.9. 2^20 sequences, all but 2000 empty, those of 2000 sizes: 42 ms, three passes.
// Up to 64 sequences have 2048 levels, so one for each size up to some 100000 keys.)
constexpr int AP_ROUNDS = 4096;
struct ApList {
  int bits;
  int lo, hi, next;            // the level at hand has sizes lo .. hi - 1; the largest size below it (-1: none)
  int above, upto;             // pairs of higher levels, of this and higher ones
  int b0, passed;              // the sequences that the search goes on from, pairs of this level before them
  int total;
};
constexpr int AP_MANY = 1 << 25;      // what sums over a lane's sequences stop at, so that a warp's stay in range
__device__ __forceinline__ int ap_pairs(const ApArgs& a, int lq) { return (lq + 2 * a.RB - 1) / (2 * a.RB); }
__device__ __forceinline__ int ap_first(const ApArgs& a, const ApSeq& s) { return s.lk > s.lq ? (s.lk - s.lq) / (2 * a.RB) : 0; }
// The pairs that rows in order have at most. (Starts out of order may seem to have more; what is past this is left out.)
__device__ __forceinline__ int ap_most(const ApArgs& a) { return a.R / (2 * a.RB) + a.B; }
// The low bits of a size that its level leaves out, and the number of levels up to that of a size.
__device__ __forceinline__ int ap_cut(int size, int bits) { return max(0, 32 - __clz(size) - bits); }
__device__ __forceinline__ int ap_levels(int size, int bits) {
  const int cut = ap_cut(size, bits);
  return bits ? (cut << (bits - 1)) + (size >> cut) + 1 : 1;
}
__device__ __forceinline__ ApList ap_begin(const ApArgs& a, bool latch) {
  int total = 0, top = -1;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    bool bad;
    const ApSeq s = ap_seq(a, b, bad);
    if (bad && latch) latch_error(a.err, DEVERR_BOUNDS);
    const int T = ap_pairs(a, s.lq);
    total = min(total + T, AP_MANY);
    if (T) top = max(top, ap_first(a, s) + T - 1);
  }
  ApList l{};
  l.total = min((int)__reduce_add_sync(0xffffffffu, total), ap_most(a));
  l.next = __reduce_max_sync(0xffffffffu, top);
  const int most = max(1, AP_ROUNDS / ((a.B + 31) / 32));
  l.bits = 30;
#pragma unroll 1
  while (l.next >= 0 && ap_levels(l.next, l.bits) > most) --l.bits;
  return l;
}
// The next level that has pairs (a converged warp).
__device__ __forceinline__ void ap_descend(const ApArgs& a, ApList& l) {
  const int cut = ap_cut(l.next, l.bits), lo = l.lo = l.next >> cut << cut, hi = l.hi = l.next + 1;
  int n = 0, next = -1;
#pragma unroll 1
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    bool bad;
    const ApSeq s = ap_seq(a, b, bad);
    const int T = ap_pairs(a, s.lq), first = ap_first(a, s);
    n = min(n + max(0, min(first + T, hi) - max(first, lo)), AP_MANY);
    if (T && first < lo) next = max(next, min(first + T, lo) - 1);
  }
  l.above = l.upto;
  l.upto += __reduce_add_sync(0xffffffffu, n);
  l.next = __reduce_max_sync(0xffffffffu, next);
  l.b0 = l.passed = 0;
}
// Item i; h = -1 behind the last one. i rises from call to call.
template <int KT>
__device__ __forceinline__ ApItem ap_item(const ApArgs& a, ApList& l, long long i) {
  ApItem it{};
  it.h = -1;
  const long long rank = i / a.nkv;
  if (rank >= l.total) return it;
#pragma unroll 1
  while (rank >= l.upto) {
    if (l.next < 0) return it;
    ap_descend(a, l);
  }
  const int k = (int)rank - l.above;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (; l.b0 < a.B; l.b0 += 32) {
    const int b = l.b0 + lane;
    ApSeq s{0, 0, 0, 0};
    bool bad;
    if (b < a.B) s = ap_seq(a, b, bad);
    const int first = ap_first(a, s), end = min(first + ap_pairs(a, s.lq), l.hi);
    const int here = min(max(0, end - max(first, l.lo)), AP_MANY);      // pairs of this level
    const int n = __reduce_add_sync(0xffffffffu, here);
    if (k - l.passed >= n) {
      l.passed += n;
      continue;
    }
    int upto = here;      // those of the sequences before this one with them
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, upto > k - l.passed)) - 1;
    const int t = end - 1 - (k - l.passed - (upto - here)) - first;      // (of that lane; the others' are of no account)
    const int p0 = t * 2 * a.RB, off = s.lk - s.lq;
    ApItem x;
    x.h = (int)(i - rank * a.nkv);
    x.row0 = s.r0 + p0;
    x.k0 = s.k0;
    x.lim0 = off + p0;
    const int left = s.lq - p0;
    x.rows[0] = min(a.RB, left);
    x.rows[1] = max(0, min(a.RB, left - a.RB));
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int last = x.lim0 + y * a.RB + x.rows[y] - 1;      // (a sequence's last row sees its last key, none further)
      x.n[y] = x.rows[y] > 0 && last >= 0 ? last / KT + 1 : 0;
    }
    it.h = __shfl_sync(0xffffffffu, x.h, src);
    it.row0 = __shfl_sync(0xffffffffu, x.row0, src);
    it.k0 = __shfl_sync(0xffffffffu, x.k0, src);
    it.lim0 = __shfl_sync(0xffffffffu, x.lim0, src);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      it.rows[y] = __shfl_sync(0xffffffffu, x.rows[y], src);
      it.n[y] = __shfl_sync(0xffffffffu, x.n[y], src);
    }
    return it;
  }
  return it;      // not reached
}

// ---- few items: their key tiles, laid end to end, cut into equal ranges, one a CTA -------------------------------------
// The items in order: pairs of tiles of the sequences one after another, the heads of a pair side by side. An item has as
// many units as key tiles, one where its rows see nothing. prompt_plan_k finds where each range starts.
struct ApStart { int b, t, h, j, units, pad[3]; };      // sequence, pair, head, key tile; units of the range
struct ApJoin { int row0, rows[2], h, first, last, pad[2]; };   // the item that starts in a range and ends behind it: its first
                                                       // piece's slot, the CTA of its last one; h = -1: none
constexpr int AP_LEAST = 4;         // units that a range has at least: its ends cost as much
constexpr int AP_PLAN = 512;        // threads of the plan: pairs, sequences and CTAs are fewer

template <int KT>
__device__ __forceinline__ int ap_tiles(const ApArgs& a, const ApSeq& s, int t) {
  const int last = s.lk - s.lq + min((t + 1) * 2 * a.RB, s.lq) - 1;
  return last >= 0 ? last / KT + 1 : 1;
}
__device__ __forceinline__ void ap_rows(const ApArgs& a, const ApSeq& s, int t, int* rows) {
  const int left = s.lq - t * 2 * a.RB;
  rows[0] = min(a.RB, left);
  rows[1] = max(0, min(a.RB, left - a.RB));
}

// Exclusive sums of a value a thread, and the total.
__device__ __forceinline__ int ap_block_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  const int w = lane < AP_PLAN / 32 ? sums[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, w);
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  __syncthreads();
  return before + x - v;
}
// The last of n rising values that is at most u.
__device__ __forceinline__ int ap_find(const int* v, int n, int u) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int KT>
__global__ void __launch_bounds__(AP_PLAN) prompt_plan_k(const ApArgs a, int grid) {
  __shared__ int sums[32], pair0[AP_PLAN], unit0[AP_PLAN];
  PDL_ENTRY();
  const int i = threadIdx.x;
  ApSeq s{0, 0, 0, 0};
  bool bad = false;
  if (i < a.B) s = ap_seq(a, i, bad);
  if (bad) latch_error(a.err, DEVERR_BOUNDS);
  int pairs, units;
  pair0[i] = ap_block_scan(ap_pairs(a, s.lq), sums, pairs);
  pairs = min(pairs, ap_most(a));      // (at most AP_PLAN, or the host does not split)
  __syncthreads();
  // (equal values: the last one, so the sequence that has the pair)
  int b = 0, t = 0, n = 0;
  if (i < pairs) {
    b = ap_find(pair0, a.B, i);
    t = i - pair0[b];
    s = ap_seq(a, b, bad);
    n = ap_tiles<KT>(a, s, t);
  }
  unit0[i] = ap_block_scan(n * a.nkv, sums, units);
  __syncthreads();
  const int shares = max(1, min(grid, units / AP_LEAST));
  if (i >= grid) return;
  ApStart st{};
  ApJoin jn{};
  jn.h = -1;
  if (i < shares && units > 0) {
    const int u0 = (int)((long long)units * i / shares), u1 = (int)((long long)units * (i + 1) / shares);
    int p = ap_find(unit0, pairs, u0);
    st.b = ap_find(pair0, a.B, p);
    st.t = p - pair0[st.b];
    s = ap_seq(a, st.b, bad);
    n = ap_tiles<KT>(a, s, st.t);
    st.h = (u0 - unit0[p]) / n;
    st.j = (u0 - unit0[p]) % n;
    st.units = u1 - u0;
    if (u1 > u0) {
      p = ap_find(unit0, pairs, u1 - 1);
      b = ap_find(pair0, a.B, p);
      t = p - pair0[b];
      s = ap_seq(a, b, bad);
      n = ap_tiles<KT>(a, s, t);
      const int h = (u1 - 1 - unit0[p]) / n, from = unit0[p] + h * n;
      if (from >= u0 && from + n > u1) {
        jn.h = h;
        jn.row0 = s.r0 + t * 2 * a.RB;
        ap_rows(a, s, t, jn.rows);
        jn.first = 2 * i + (from == u0 ? 0 : 1);
        int y = i + 1;
        while (y + 1 < shares && (int)((long long)units * (y + 1) / shares) < from + n) ++y;
        jn.last = y;
      }
    }
  }
  a.starts[i] = st;
  a.joins[i] = jn;
}

// Whether key tile j holds keys that a row of the tiles that use it does not see, and the last one that all of them see.
template <int KT>
__device__ __forceinline__ bool ap_partial(const ApItem& it, int RB, int j, int& seen) {
  seen = j < it.n[0] ? it.lim0 : it.lim0 + RB;
  return j * KT + KT - 1 > seen;
}

__device__ __forceinline__ void tma_prefetch_3d(const void* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c0),
               "r"(c1), "r"(c2)
               : "memory");
}

// D[tmem] (+)= A B, the operands' descriptors given by their low halves (128-byte swizzle, rows of eight 1024 bytes apart).
constexpr uint32_t AP_DESC_HIGH = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ void ap_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(AP_DESC_HIGH)
      : "memory");
}
__device__ __forceinline__ void ap_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(AP_DESC_HIGH)
      : "memory");
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait of a converged warp for an mbarrier phase, looking at the abort flag and the clock every 64th time. Gives up as
// mbar_wait does; every lane gets the same answer. (Short: it is inlined some twenty times, and the instruction cache is
// what bounds the ends of items.)
__device__ __forceinline__ bool ap_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, const ApArgs& a, bool honor_abort = true) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t tries = 1; !__all_sync(0xffffffffu, mbar_try(bar, parity)); ++tries) {
    if (tries & 63u) continue;
    if (honor_abort && __any_sync(0xffffffffu, *abort_flag)) return false;
    const uint64_t now = globaltimer();
    if (!t0) t0 = now;
    if (__any_sync(0xffffffffu, now - t0 > a.wait_ns)) {
      *abort_flag = 1;
      latch_error(a.err, DEVERR_MBAR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// 16 columns of this warp's lanes; the values are there after tmem_wait_ld_n.
__device__ __forceinline__ void tmem_ld16_async(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(t));
}
template <int N>
__device__ __forceinline__ void tmem_wait_ld_n(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_st8u(uint32_t t, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// A warp's 16 lanes of TMEM as fragments: thread t gets of row t / 4 and of row t / 4 + 8 the columns 2 (t % 4) and one more of
// every eight (v[4 i .. 4 i + 3]: the two of the first row, the two of the second).
__device__ __forceinline__ void frag_ld64(uint32_t t, float* v) {      // 64 columns
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t));
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// w[j]: word q of piece j (q = the thread's place among the four of its row) -> word j of piece q.
__device__ __forceinline__ void quad_transpose(uint32_t* w, int q) {
  const bool odd = q & 1, high = q & 2;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? w[j] : w[j + 1], 1);
    if (odd) w[j] = y;
    else w[j + 1] = y;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, high ? w[j] : w[j + 2], 2);
    if (high) w[j] = y;
    else w[j + 2] = y;
  }
}

// Values that are not finite in rows from r0 on of a value tile (16-byte pieces, 128-byte swizzle): replaced by zero, the
// first key (of those after the first row's last, 0: seen by all) kept for each column; only looked for without `mend`. By a
// converged warp.
template <int D>
__device__ __forceinline__ bool ap_clean(uint8_t* v, int r0, int key0, int lim0, uint32_t* bad, bool fresh, bool mend) {
  using Sh = ApShape<D>;
  const int lane = threadIdx.x & 31;
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 acc = zero;
  r0 &= ~3;      // (rows before the first that is hidden from some: seen by all, and looked at for nothing)
#pragma unroll 1
  for (int x = 0; x < Sh::HALVES; ++x)
#pragma unroll 2
    for (int i = r0 * 8 + lane; i < Sh::KT * 8; i += 32) {
      const uint4 w = *reinterpret_cast<const uint4*>(v + x * Sh::KHALF + i * 16);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[y]), zero, acc);   // inf * 0 = NaN
    }
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&acc);
  if (!__any_sync(0xffffffffu, (bits & 0x7fff7fffu) != 0)) return false;
  if (!mend) return true;
  if (fresh) {
    for (int c = lane; c < D; c += 32) bad[c] = AP_NONE;
    __syncwarp();
  }
#pragma unroll 1
  for (int x = 0; x < Sh::HALVES; ++x)
#pragma unroll 1
    for (int i = r0 * 8 + lane; i < Sh::KT * 8; i += 32) {
      const int row = i >> 3, piece = (i & 7) ^ (row & 7);
      __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(v + x * Sh::KHALF + i * 16);
      const int rel = max(0, key0 + row - lim0);
#pragma unroll 1
      for (int y = 0; y < 8; ++y) {
        const uint16_t h = reinterpret_cast<const uint16_t*>(p)[y];
        if ((h & 0x7f80) != 0x7f80) continue;
        reinterpret_cast<uint16_t*>(p)[y] = 0;
        if (rel > 1022) continue;
        const int shift = (h & 0x7f) ? 0 : (h & 0x8000) ? 20 : 10;
        uint32_t* at = bad + x * 64 + piece * 8 + y;
        uint32_t old = *reinterpret_cast<volatile uint32_t*>(at);
        while ((int)((old >> shift) & 1023) > rel) {
          const uint32_t now = (old & ~(1023u << shift)) | ((uint32_t)rel << shift);
          const uint32_t seen = atomicCAS(at, old, now);
          if (seen == old) break;
          old = seen;
        }
      }
    }
  return true;
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(AP_THREADS, 1)
    prompt_k(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const ApArgs a) {
  using Sh = ApShape<D>;
  constexpr int ST = Sh::STAGES, KT = Sh::KT;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::OFF_BAR);
  uint64_t *full = bars, *empty = bars + ST, *looked = bars + 2 * ST /* ring */, *q_full = bars + 3 * ST /* [tile] */,
           *s_full = q_full + 4 /* [tile] */, *s_free = q_full + 6 /* [tile] */,
           *p_full = q_full + 8 /* [tile] */, *p_free = q_full + 10 /* [tile] */,
           *o_free = q_full + 14 /* [tile] */, *l_full = q_full + 16 /* [tile] */, *l_free = q_full + 18 /* [tile] */,
           *item_full = q_full + 20 /* [slot] */, *item_empty = q_full + 22 /* [slot] */, *drain = q_full + 24 /* [tile] */;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 26);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* has_bad = abort_flag + 1;      // [slot]
  volatile int* careful = abort_flag + 3;      // 0: nothing found yet, 1: a second pass is due, 2: it runs
  ApItem* items = reinterpret_cast<ApItem*>(sm + Sh::OFF_ITEM);
  uint32_t* bad = reinterpret_cast<uint32_t*>(sm + Sh::OFF_BAD);      // [slot][D]
  float* inv = reinterpret_cast<float*>(sm + Sh::OFF_INV);            // [tile][query vector]: 1 / sum of the weights
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 3);      // either tile, warp 15
      mbar_init(smem_u32(looked + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(q_full + i), 1);
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(s_free + i), 4);
      mbar_init(smem_u32(p_full + i), 4);
      mbar_init(smem_u32(p_free + i), 1);
      mbar_init(smem_u32(o_free + i), 4);
      mbar_init(smem_u32(l_full + i), 4);
      mbar_init(smem_u32(l_free + i), 4);
      mbar_init(smem_u32(item_full + i), 1);
      mbar_init(smem_u32(item_empty + i), AP_SOFT + 4 + 3);
      mbar_init(smem_u32(drain + i), 1);
      has_bad[i] = 0;
    }
    *abort_flag = 0;
    *careful = 0;
    fence_mbar_init();
  }
  if (warp == AP_MMA) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PDL_ENTRY();

  // Phases: a waiter passes every phase of a barrier that it waits on, in order, and no phase can end twice before its waiters
  // have passed it: what ends it next comes behind something that they do after. (Waits that depend on the case, `looked`,
  // come behind one that vouches for the phase before.)
  if (warp < AP_SOFT) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::R_SOFT));
    const int mt = warp >> 2, qv = threadIdx.x & 127;
    const int pos = qv / a.G, low = ((warp & 3) * 32) / a.G;      // this thread's position in the tile, its warp's first
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + Sh::T_S + mt * Sh::T_STEP + lane_off, tP = tS + KT, tO = tmem + mt * D + lane_off;
    uint32_t s_phase = 0, p_phase = 1, l_phase = 1;      // (1: a barrier's first wait passes, nobody holds what it guards)
    // A tile's first warp brings its Q: the next item's as soon as the last S of this one is there, which no product reads Q
    // for any more. (By the warp of the other copies these wait for it: 4096 tokens of 40 heads 157 us instead of 148.)
    const bool brings = (warp & 3) == 0;
    int q_next = 0, q_loads = 0;      // the first item whose Q is not under way yet; loads so far
    // It gives the ring's stages back too: keys when their S is there, values when the product is done (an item's last ones: the
    // warps that write the results).
    int ring = 0;                     // stages before this item
    auto bring = [&](const ApItem& x) {
      if (x.n[mt] <= 0) return;
      ++q_loads;
      if (elect_one()) {
        mbar_expect_tx(smem_u32(q_full + mt), (uint32_t)(Sh::HALVES * a.RB * a.G * 128));
#pragma unroll
        for (int y = 0; y < Sh::HALVES; ++y)
          tma_load_3d(smem_u32(sm + mt * Sh::QB + y * Sh::QHALF), &tmQ, y * 64, x.h * a.G, x.row0 + mt * a.RB, smem_u32(q_full + mt));
      }
      __syncwarp();
    };
    bool ok = true;
    for (int n = 0; ok; ++n) {
      ok = ap_wait(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a);
      if (!ok) break;
      const ApItem& it = items[n & 1];
      if (it.h < 0) break;
      const bool late = brings && q_next <= n;
      const int nt = it.n[mt], both = max(it.n[0], it.n[1]), first = it.lim0 + mt * a.RB;      // the last key that the tile's first row sees
      float m2 = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = late ? -1 : 0; j < nt; ++j) {
        // this item's Q if it was not known in time, the next one's behind the last S
        if (j >= 0) {
          ok = ap_wait(smem_u32(s_full + mt), s_phase, abort_flag, a);
          if (!ok) break;
          s_phase ^= 1;
          tc_fence_after();
          if (brings && elect_one()) mbar_arrive(smem_u32(empty + (ring + (j ? 2 * j - 1 : 0)) % ST));
        }
        if (brings && (j < 0 || j + 1 == nt)) {
          const int x = j < 0 ? n : n + 1;
          if (j < 0 || __all_sync(0xffffffffu, mbar_test(smem_u32(item_full + (x & 1)), (uint32_t)((x >> 1) & 1)))) {
            const ApItem& next = items[x & 1];
            if (next.h >= 0) bring(next);
            q_next = x + 1;
          }
        }
        if (j < 0) continue;
        float s[KT];
#pragma unroll
        for (int c = 0; c < KT / 32 * 32; c += 32) tmem_ld32_async(tS + c, s + c);
        if constexpr (KT % 32) tmem_ld16_async(tS + KT - 16, s + KT - 16);
        tmem_wait_ld_n<KT>(s);
        tc_fence_before();
        warp_arrive(smem_u32(s_free + mt));      // S of the next keys may come
        const int last = first + pos - j * KT, all = first + low - j * KT;      // last keys seen by this row, by all of the warp's
        // (one branch: tested 16 keys at a time, a pair's 128 keys took 1.67 us instead of 1.43)
        if (KT - 1 > all)
#pragma unroll
          for (int c = 0; c < KT; ++c) s[c] = c <= last ? s[c] : -INFINITY;
        float x0 = fmaxf(s[0], s[1]), x1 = fmaxf(s[2], s[3]), x2 = fmaxf(s[4], s[5]), x3 = fmaxf(s[6], s[7]);
#pragma unroll
        for (int c = 8; c < KT; c += 8) {
          x0 = max3(x0, s[c], s[c + 1]);
          x1 = max3(x1, s[c + 2], s[c + 3]);
          x2 = max3(x2, s[c + 4], s[c + 5]);
          x3 = max3(x3, s[c + 6], s[c + 7]);
        }
        const float mx = fmaxf(max3(x0, x1, x2), x3) * a.sl2;
        const bool raise = mx > m2 + AP_LAZY;
        float corr = 1.f;
        if (raise) {
          corr = pf_ex2(m2 - mx);
          m2 = mx;
          l *= corr;
        }
        // the product into O before this one is done: P may be written, and O rescaled
        ok = ap_wait(smem_u32(p_free + mt), p_phase, abort_flag, a);
        if (!ok) break;
        p_phase ^= 1;
        if (brings && j > 0 && elect_one()) mbar_arrive(smem_u32(empty + (ring + 2 * j) % ST));
        tc_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16(tO + c, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= corr;
            tmem_st16(tO + c, o);
          }
        }
        // One rounding of the reference for the whole row, then one of each difference: near the maximum, where weights
        // count, that is exact whatever the size of the scores.
        const float ref = m2 == -INFINITY ? 0.f : m2;
        const f32x2 nm = two(-ref, -ref), s2 = two(a.sl2, a.sl2);
        f32x2 sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
        for (int c0 = 0; c0 < KT; c0 += 16) {
          uint32_t w[8];
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            float2 x = one_by_one(fma2(two(s[c0 + c], s[c0 + c + 1]), s2, nm));
            x.x = pf_ex2(x.x);
            x.y = pf_ex2(x.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], two(x.x, x.y));
            w[c / 2] = bf16_pair(x.x, x.y);
          }
          tmem_st8u(tP + c0 / 2, w);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(smem_u32(p_full + mt));
        const float2 sums = one_by_one(add2(sum[0], sum[1]));
        l += sums.x + sums.y;
      }
      if (!ok) break;
      if (it.rows[mt] > 0) {
        const bool piece = SPLIT && it.slot >= 0;
        if (piece) {
          float2* ml = reinterpret_cast<float2*>(a.part_ml) + (size_t)(it.slot * 2 + mt) * AT + qv;
          *ml = make_float2(m2, l);
        } else if (pos < it.rows[mt] && a.lse) {      // (so pos < RB: not the vectors behind the last head)
          const float ref = m2 == -INFINITY ? 0.f : m2;
          a.lse[(long long)(it.row0 + mt * a.RB + pos) * a.nq + it.h * a.G + qv - pos * a.G] =
              l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.693147180559945309f;
        }
        if (nt) {
          ok = ap_wait(smem_u32(l_free + mt), l_phase, abort_flag, a);
          if (!ok) break;
          l_phase ^= 1;
          inv[mt * AT + qv] = piece ? 1.f : l == 0.f ? 0.f : 1.f / l;
          warp_arrive(smem_u32(l_full + mt));
        }
      }
      ring += 2 * both;
      warp_arrive(smem_u32(item_empty + (n & 1)));
    }
    // a copy in flight lands before the CTA leaves
    if (!ok && q_loads) ap_wait(smem_u32(q_full + mt), (uint32_t)((q_loads - 1) & 1), abort_flag, a, false);
  } else if (warp < AP_TMA) {
    // ---- results: both tiles' in turn, a quarter of the lanes a warp, while the softmax warps are at the next item ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::R_OUT));
    const int lane = threadIdx.x & 31, quad = lane & 3, lane0 = (warp & 3) * 32;
    // position and head (of the tile, of the group) of the four query vectors of this thread's fragments
    uint32_t at[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int v = lane0 + x * 8 + (lane >> 2);
      at[x] = (uint32_t)(v / a.G) << 16 | (uint32_t)(v % a.G);
    }
    uint32_t phase = 0, units = 0;      // a bit a tile: phase of l_full; whether its products so far are odd
    int ring = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      ok = ap_wait(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a);
      if (!ok) break;
      const ApItem& it = items[n & 1];
      if (it.h < 0) break;
#pragma unroll 1
      for (int mt = 0; mt < 2; ++mt) {
        const int rows = it.rows[mt], nt = it.n[mt];
        if (rows <= 0 || (SPLIT && it.slot >= 0 && !nt)) continue;
        __nv_bfloat16* base = a.out + (long long)(it.row0 + mt * a.RB) * a.ldo + (long long)it.h * a.G * D;
        if (nt) {
          // the last product's phase of p_free: the one before is over, or l_full would not be
          units ^= (uint32_t)(nt & 1) << mt;
          ok = ap_wait(smem_u32(l_full + mt), phase >> mt & 1, abort_flag, a) &&
               ap_wait(smem_u32(p_free + mt), (units >> mt & 1) ^ 1, abort_flag, a);
          if (!ok) break;
          phase ^= 1u << mt;
          tc_fence_after();
          if (warp == AP_SOFT && elect_one())
            mbar_arrive(smem_u32(empty + (ring + (nt == max(it.n[0], it.n[1]) ? 2 * nt - 1 : 2 * nt)) % ST));
        }
        // Fragments of 16 rows, four threads a row, 64 columns at a time: a row's 64 bytes go out together. Rolled, as all
        // that runs once an item: what falls out of the instruction cache comes back at some ten clocks an instruction.
#pragma unroll 1
        for (int fc = 0; fc < 2 * D / 64; ++fc) {
          const int f = fc / (D / 64), c = fc % (D / 64) * 64;
          float o[32], part[2];
          if (nt) {
            frag_ld64(tmem + ((uint32_t)(lane0 + f * 16) << 16) + mt * D + c, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int y = 0; y < 2; ++y) part[y] = inv[mt * AT + lane0 + f * 16 + y * 8 + (lane >> 2)];
            if (fc == 2 * D / 64 - 1) {      // O is read: the next item's products may begin
              tc_fence_before();
              warp_arrive(smem_u32(o_free + mt));
              warp_arrive(smem_u32(l_free + mt));
            }
          } else {      // rows that see no key
            part[0] = part[1] = 0.f;
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0.f;
          }
          if (SPLIT && it.slot >= 0) {
            // two neighbours exchange pairs: 16 bytes a thread, of the first eight rows or of the other
            const int odd = quad & 1;
            float* part = a.part_o + ((size_t)(it.slot * 2 + mt) * AT + lane0 + f * 16 + (lane >> 2) + 8 * odd) * D + c + (quad >> 1) * 4;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float* v = o + 4 * x;
              const float g0 = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[2], 1), g1 = __shfl_xor_sync(0xffffffffu, odd ? v[1] : v[3], 1);
              *reinterpret_cast<float4*>(part + x * 8) = odd ? make_float4(g0, g1, v[2], v[3]) : make_float4(v[0], v[1], g0, g1);
            }
            continue;
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t v = f ? at[2 + y] : at[y];
            const int p = v >> 16;
            __nv_bfloat16* dst = base + (long long)p * a.ldo + (int)(v & 0xffff) * D + c + quad * 8;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = bf16_pair(o[(x * 4 + i) * 4 + 2 * y] * part[y], o[(x * 4 + i) * 4 + 2 * y + 1] * part[y]);
              quad_transpose(w, quad);
              if (p < rows)      // (so p < RB: not the vectors behind the last head)
                *reinterpret_cast<uint4*>(dst + x * 32) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (nt && has_bad[n & 1]) {      // (rare: over what this warp has just written, a row a thread)
          __syncwarp();
          const int p = (lane0 + lane) / a.G, i = mt * a.RB + p;
          if (p < rows) {
            __nv_bfloat16* o = base + (long long)p * a.ldo + (lane0 + lane - p * a.G) * D;
#pragma unroll 1
            for (int c = 0; c < D; ++c) {
              const uint32_t x = bad[(n & 1) * D + c];
              float add = 0.f;
              if (i >= (int)((x >> 10) & 1023)) add += INFINITY;
              if (i >= (int)((x >> 20) & 1023)) add -= INFINITY;      // (both: NaN)
              if (i >= (int)(x & 1023)) add = __int_as_float(0x7fffffff);
              if (add == 0.f) continue;
              if (SPLIT && it.slot >= 0) a.part_o[((size_t)(it.slot * 2 + mt) * AT + lane0 + lane) * D + c] += add;
              else o[c] = __float2bfloat16_rn(__bfloat162float(o[c]) + add);
            }
          }
        }
      }
      ring += 2 * max(it.n[0], it.n[1]);
      if (ok) warp_arrive(smem_u32(item_empty + (n & 1)));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::R_ONE));
    // The ring's order of an item of n key tiles: K 0, then K j + 1 and V j for j = 0 .. n - 1 (no K n).
    if (warp == AP_TMA) {
      // ---- items, TMA ----
      ApList list{};
      ApStart at0{};      // split: where this CTA goes on
      int s = 0;                        // stages of the ring so far
      ApItem it{}, next{};
      bool ok = true;
      // The loads of item n - 1; halfway item n is found and its Q brought into L2, behind them it is published.
#pragma unroll 1
      for (int n = 0, m = 0;; ++n, ++m) {      // slots, items of this pass
        if (m == 0) {
          if constexpr (SPLIT) {
            at0 = a.starts[blockIdx.x];
          } else {
            list = ap_begin(a, n == 0 && blockIdx.x == 0);
          }
        }
        const int nt = max(it.n[0], it.n[1]);
#pragma unroll 1
        for (int x = 0; ok && x < max(1, 2 * nt); ++x) {
          if (x == nt) {
            if constexpr (SPLIT) {
              next.h = -1;
              if (at0.units > 0) {
                bool bad_;
                ApSeq q = ap_seq(a, at0.b, bad_);
#pragma unroll 1
                while (at0.t >= ap_pairs(a, q.lq)) {      // (ends: there are units left)
                  q = ap_seq(a, ++at0.b, bad_);
                  at0.t = 0;
                }
                const int tiles = ap_tiles<KT>(a, q, at0.t), j0 = at0.j, j1 = min(tiles, j0 + at0.units);
                next.h = at0.h;
                next.row0 = q.r0 + at0.t * 2 * a.RB;
                ap_rows(a, q, at0.t, next.rows);
                // slot 0 for a piece at the start of the CTA's range, 1 for one at its end
                next.slot = j0 == 0 && j1 == tiles ? -1 : 2 * blockIdx.x + (m == 0 ? 0 : 1);
                next.k0 = q.k0 + j0 * KT;
                const int lim = q.lk - q.lq + at0.t * 2 * a.RB;
                next.lim0 = lim - j0 * KT;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int last = lim + y * a.RB + next.rows[y] - 1, all = next.rows[y] > 0 && last >= 0 ? last / KT + 1 : 0;
                  next.n[y] = max(0, min(all, j1) - j0);
                }
                at0.units -= j1 - j0;
                at0.j = 0;
                if (++at0.h == a.nkv) {
                  at0.h = 0;
                  ++at0.t;
                }
              }
            } else {
              // to and fro over the CTAs: who takes the largest of one round takes the smallest of the next
              const int at = m & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
              next = ap_item<KT>(a, list, at + (long long)m * gridDim.x);
              next.slot = -1;
            }
            if (next.h >= 0 && elect_one())
#pragma unroll 1
              for (int y = 0; y < 2 * Sh::HALVES; ++y)
                if (y & 1 ? next.n[1] : next.n[0]) tma_prefetch_3d(&tmQ, (y >> 1) * 64, next.h * a.G, next.row0 + (y & 1) * a.RB);
            __syncwarp();
          }
          if (nt == 0) break;
          const int st = s % ST;
          const bool is_v = x && (!(x & 1) || x + 1 == 2 * nt);
          if (s >= ST) ok = ap_wait(smem_u32(empty + st), (uint32_t)((s / ST - 1) & 1), abort_flag, a);
          if (!ok) break;
          if (elect_one()) {
            mbar_expect_tx(smem_u32(full + st), Sh::KB);
            for (int y = 0; y < Sh::HALVES; ++y)
              tma_load_3d(smem_u32(sm + Sh::OFF_RING + st * Sh::KB + y * Sh::KHALF), is_v ? &tmV : &tmK, y * 64, it.h,
                          it.k0 + (x ? is_v ? (x - 1) >> 1 : (x + 1) >> 1 : 0) * KT, smem_u32(full + st));
          }
          __syncwarp();
          ++s;
        }
        if (ok && n >= 2) ok = ap_wait(smem_u32(item_empty + (n & 1)), (uint32_t)(((n >> 1) - 1) & 1), abort_flag, a);
        if (ok && next.h < 0 && n) {      // the end, unless warp 15 found something
          ok = ap_wait(smem_u32(item_empty + (n - 1 & 1)), (uint32_t)((n - 1 >> 1) & 1), abort_flag, a);
          if (ok && *careful == 1) {
            __syncwarp();
            *careful = 2;
            it = ApItem{};
            --n;
            m = -1;
            continue;
          }
        }
        if (!ok) break;
        if (elect_one()) {
          items[n & 1] = next;
          has_bad[n & 1] = 0;
          mbar_arrive(smem_u32(item_full + (n & 1)));
        }
        __syncwarp();
        if (next.h < 0) break;
        it = next;
      }
      if (*abort_flag) {      // copies in flight land before the CTA leaves: the last ones of the ring
#pragma unroll 1
        for (int x = max(0, s - ST); x < s; ++x) ap_wait(smem_u32(full + x % ST), (uint32_t)((x / ST) & 1), abort_flag, a, false);
      }
    } else if (warp < AP_LOOK) {
      // ---- MMA: one warp a query tile ----
      constexpr uint32_t IS = pf_idesc(KT, false), IO = pf_idesc(D, true);
      // What the products are issued with goes through a warp reduction, whose result is in a uniform register: from there
      // descriptors are one addition each (held in the threads' registers, each product waits for several moves).
      const int mt = (int)__reduce_max_sync(0xffffffffu, (uint32_t)(warp - AP_MMA));
      const uint32_t base = __reduce_max_sync(0xffffffffu, tmem);
      const uint32_t tS = base + Sh::T_S + mt * Sh::T_STEP, tP = tS + KT, tO = base + mt * D;
      // low halves of the operand descriptors; an offset of n bytes adds n >> 4
      const uint32_t dq = (uint32_t)sdesc_sw128(smem_u32(sm + mt * Sh::QB)), dk = (uint32_t)sdesc_sw128(smem_u32(sm + Sh::OFF_RING)),
                     dv = (uint32_t)pf_desc_mn(smem_u32(sm + Sh::OFF_RING), Sh::KHALF);
      int s = 0, used = 0, units = 0;      // stages, items and key tiles with products of this tile so far
      uint32_t p_phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int n = 0; ok; ++n) {
        ok = ap_wait(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a);
        if (!ok) break;
        const ApItem it = items[n & 1];
        if (it.h < 0) break;
        const int mine = mt ? it.n[1] : it.n[0], nt = max(it.n[0], it.n[1]);
        // Stage by stage: S of the keys in it, or O of the values in it; those of the other tile alone are given back. One commit
        // each, which costs the issuing warp some 150 clocks: that a stage is free and O complete follows from the same.
#pragma unroll 1
        for (int x = 0; ok && x < 2 * nt; ++x, ++s) {
          const int st = s % ST;
          const bool is_v = x && (!(x & 1) || x + 1 == 2 * nt);
          const int j = x ? is_v ? (x - 1) >> 1 : (x + 1) >> 1 : 0;
          const uint32_t turn = (uint32_t)((s / ST) & 1);
          ok = ap_wait(smem_u32(full + st), turn, abort_flag, a);
          if (!ok) break;
          if (j >= mine) {
            if (elect_one()) mbar_arrive(smem_u32(empty + st));
            __syncwarp();
          } else if (!is_v) {
            if (x == 0) ok = ap_wait(smem_u32(q_full + mt), (uint32_t)(used & 1), abort_flag, a);
            // the softmax warps hold the S before
            if (ok && units) ok = ap_wait(smem_u32(s_free + mt), (uint32_t)((units - 1) & 1), abort_flag, a);
            if (!ok) break;
            ++units;
            tc_fence_after();
            const uint32_t k = __reduce_max_sync(0xffffffffu, dk + ((uint32_t)(st * Sh::KB) >> 4));
            if (elect_one()) {
#pragma unroll
              for (int y = 0; y < D / 16; ++y)
                ap_mma_ss(tS, dq + (((y >> 2) * Sh::QHALF + (y & 3) * 32) >> 4), k + (((y >> 2) * Sh::KHALF + (y & 3) * 32) >> 4),
                          IS, y ? 1u : 0u);
              tc_commit(smem_u32(s_full + mt));
            }
            __syncwarp();
          } else {
            int seen;
            if (*careful == 2 && ap_partial<KT>(it, a.RB, j, seen))      // (behind the wait for the stage: warp 15 has passed its use before)
              ok = ap_wait(smem_u32(looked + st), turn, abort_flag, a);
            if (ok && j == 0 && used) ok = ap_wait(smem_u32(o_free + mt), (uint32_t)((used - 1) & 1), abort_flag, a);
            ok = ok && ap_wait(smem_u32(p_full + mt), p_phase, abort_flag, a);
            if (!ok) break;
            p_phase ^= 1;
            tc_fence_after();
            const uint32_t v = __reduce_max_sync(0xffffffffu, dv + ((uint32_t)(st * Sh::KB) >> 4));
            const uint32_t more = __reduce_max_sync(0xffffffffu, (uint32_t)j);
            if (elect_one()) {
#pragma unroll
              for (int y = 0; y < KT / 16; ++y)      // 16 keys a product
                ap_mma_ts(tO, tP + y * 8, v + (y * 2048 >> 4), IO, y ? 1u : more);
              tc_commit(smem_u32(p_free + mt));
            }
            __syncwarp();
          }
        }
        if (mine) ++used;
        if (ok && elect_one()) mbar_arrive(smem_u32(item_empty + (n & 1)));
        __syncwarp();
      }
      if (!ok) {      // products in flight end before the CTA frees its TMEM
        if (elect_one()) tc_commit(smem_u32(drain + mt));
        __syncwarp();
        ap_wait(smem_u32(drain + mt), 0, abort_flag, a, false);
      }
    } else {
      // ---- value tiles that some rows see only in part ----
      int s = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        ok = ap_wait(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a);
        if (!ok) break;
        const ApItem it = items[n & 1];
        if (it.h < 0) break;
        const int nt = max(it.n[0], it.n[1]);
        bool found = false;
        // every stage is waited for and given back, so that this warp is never a turn of the ring behind
#pragma unroll 1
        for (int x = 0; ok && x < 2 * nt; ++x, ++s) {
          ok = ap_wait(smem_u32(full + s % ST), (uint32_t)((s / ST) & 1), abort_flag, a);
          const bool is_v = x && (!(x & 1) || x + 1 == 2 * nt);
          const int j = (x - 1) >> 1;
          int seen;
          if (ok && is_v && ap_partial<KT>(it, a.RB, j, seen)) {
            const bool mend = *careful == 2;
            if (ap_clean<D>(sm + Sh::OFF_RING + (s % ST) * Sh::KB, max(0, seen + 1 - j * KT), j * KT, it.lim0, bad + (n & 1) * D,
                            !found, mend)) {
              if (mend) {
                found = true;
                if (elect_one()) has_bad[n & 1] = 1;
                fence_async_shared();
              } else if (elect_one()) {
                *careful = 1;
              }
            }
            __syncwarp();
          }
          if (ok && elect_one()) {
            mbar_arrive(smem_u32(looked + s % ST));
            mbar_arrive(smem_u32(empty + s % ST));
          }
          __syncwarp();
        }
        if (ok && elect_one()) mbar_arrive(smem_u32(item_empty + (n & 1)));
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == AP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The pieces of the item that starts in CTA x's range and ends behind it: 16 of its 256 query vectors a block, a warp for
// each, D / 32 columns a lane. The weights of up to 32 pieces come first, a piece a lane, so that the sums' loads wait for
// nothing.
constexpr int AP_JOIN = 16;      // blocks an item
template <int D>
__global__ void __launch_bounds__(256) prompt_join_k(const ApArgs a) {
  constexpr int C = D / 32;
  PDL_ENTRY();
  const int x = blockIdx.x / AP_JOIN, lane = threadIdx.x & 31;
  const ApJoin r = a.joins[x];
  if (r.h < 0) return;
#pragma unroll 1
  for (int i = 0; i < 256 / AP_JOIN; i += 8) {
    const int v = blockIdx.x % AP_JOIN * (256 / AP_JOIN) + i + (threadIdx.x >> 5), mt = v / AT, qv = v % AT;
    const int pos = qv / a.G;
    if (pos >= r.rows[mt]) continue;
    const int pieces = r.last - x + 1;
    auto place = [&](int y) { return (size_t)((y ? 2 * (x + y) : r.first) * 2 + mt) * AT + qv; };
    // (a piece with no key that this row sees has no sum, and its columns are not written)
    float m = -INFINITY, l = 0.f, o[C];
#pragma unroll 1
    for (int y = lane; y < pieces; y += 32) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + place(y));
      if (ml.y != 0.f) m = fmaxf(m, ml.x);
    }
    m = warp_max(m);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll 1
    for (int y0 = 0; y0 < pieces; y0 += 32) {
      float2 ml = make_float2(0.f, 0.f);
      if (y0 + lane < pieces) ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + place(y0 + lane));
      const float w = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;
      l += warp_sum(ml.y != 0.f ? ml.y * w : 0.f);
      const unsigned there = __ballot_sync(0xffffffffu, ml.y != 0.f);
      const int n = min(32, pieces - y0);
#pragma unroll 8
      for (int y = 0; y < n; ++y) {
        const float f = __shfl_sync(0xffffffffu, w, y);
        const float* at = a.part_o + place(y0 + y) * D;
        float p[C];
#pragma unroll
        for (int c = 0; c < C; ++c) p[c] = 0.f;
        if (there >> y & 1) {
          if constexpr (C == 4) {
            const float4 q = __ldcg(reinterpret_cast<const float4*>(at) + lane);
            p[0] = q.x; p[1] = q.y; p[2] = q.z; p[3] = q.w;
          } else {
            const float2 q = __ldcg(reinterpret_cast<const float2*>(at) + lane);
            p[0] = q.x; p[1] = q.y;
          }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] += p[c] * f;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int row = r.row0 + mt * a.RB + pos, head = r.h * a.G + qv - pos * a.G;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (long long)row * a.ldo + (long long)head * D + lane * C);
    if constexpr (C == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(o[0] * inv, o[1] * inv), bf16_pair(o[2] * inv, o[3] * inv));
    else
      *dst = bf16_pair(o[0] * inv, o[1] * inv);
    if (a.lse && lane == 0)
      a.lse[(long long)row * a.nq + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
  }
}

// bf16 rows of `heads` vectors of d, ld elements from a row to the next, as boxes of 64 x b1 heads x b2 rows.
bool ap_map(CUtensorMap* m, const void* p, int d, int heads, long long rows, long long ld, int b1, int b2) {
  const auto fn = pf_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool SPLIT>
cudaError_t launch_prompt(cudaStream_t st, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const ApArgs& p, int grid) {
  static_assert(ApShape<D>::BYTES <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(prompt_k<D, SPLIT>), ApShape<D>::BYTES);
  if (e != cudaSuccess) return e;
  if (SPLIT) e = launch_k(prompt_plan_k<ApShape<D>::KT>, dim3(1), dim3(AP_PLAN), 0, st, p, grid);
  if (e != cudaSuccess) return e;
  e = launch_k(prompt_k<D, SPLIT>, dim3(grid), dim3(AP_THREADS), ApShape<D>::BYTES, st, q, k, v, p);
  if (e == cudaSuccess && SPLIT) e = launch_k(prompt_join_k<D>, dim3(grid * AP_JOIN), dim3(256), 0, st, p);
  return e;
}

}  // namespace

// Whether to split, from what the host knows, the rows and keys in all. A whole item takes its key tiles (1 us each), a range
// its share of all items' and some AP_EXTRA more: the plan, the pieces' sums (up to 40 MB through L2) and the join. Measured with
// every case split, whole / split in us, behind the tiles that the rule compares with AP_EXTRA:
//   heads of 128, 32 over 8 unless said: 1 row behind 4096 keys (48) 50 / 20, 61 rows (49) 56 / 27, 512 rows behind 3584 (30) 56 / 47,
//   of 40 heads over 40 (24) 57 / 55, 8 x 1 row behind 2048 (14.8) 29 / 28, 1 row behind 1200 (14.2) 20 / 16, 700 rows behind 700 of 8 over
//   1 (15.0) 24.6 / 25.4; below it 256 rows behind 1024
//   (12.6) 23 / 25, 4 x 200 rows behind 1800 (8) 33 / 48, a whole prompt of 1024 (2) 21 / 42;
//   heads of 64: 1 row behind 4096 (30) 38 / 18, 512 rows behind 3584 of 12 over 12 (27) 49 / 27, 1024 rows behind 2048 of 8 over 1 (19)
//   40 / 29; below it 2 x 64 rows behind 1500 of 10 over 5 (11.4) 19 / 22, 1 row behind 1500 (11.3) 17.6 / 16.1, 8 x 1 row behind 2048 of
//   32 over 8 (9) 23 / 24, a whole prompt of 1024 (1) 18 / 29, of 4096 of 12 over 12 (-8) 50 / 73.
// The longest item is taken for the mean: one long sequence among short ones is not split.
constexpr int AP_EXTRA = 14;
static bool prompt_split(int R, int Rk, int G, int nkv, int d, int B, int sms) {
  const int RB = AT / G, KT = d == 128 ? ApShape<128>::KT : ApShape<64>::KT;
  const long long most = (long long)R / (2 * RB) + B;      // pairs
  if (most > AP_PLAN || sms > AP_PLAN || most * nkv > 8 * sms) return false;
  const double items = (double)std::max((long long)B, ((long long)R + 2 * RB - 1) / (2 * RB)) * nkv, tiles = (double)Rk / B / KT;
  return most * nkv * ((double)Rk / KT + 1) < 1 << 30 && tiles - items * tiles / sms > AP_EXTRA;
}

size_t prompt_attention_scratch(int R, int Rk, int nq, int nkv, int d, int B) {
  const int sms = device_sm_count();
  if (sms < 1 || !prompt_split(R, Rk, nq / nkv, nkv, d, B, sms)) return 0;
  return (size_t)2 * sms * 2 * AT * (d + 2) * sizeof(float) + (size_t)sms * (sizeof(ApStart) + sizeof(ApJoin));
}

int prompt_attention(cudaStream_t st, const PromptArgs& a) {
  ApArgs p{};
  p.R = a.R; p.Rk = a.Rk; p.nq = a.nq; p.nkv = a.nkv; p.G = a.nq / a.nkv; p.RB = AT / p.G; p.B = a.B;
  p.start = a.start; p.kstart = a.kstart;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(a.out); p.ldo = a.ldo; p.lse = a.lse; p.err = a.err;
  // at most this many items: each sequence ends a pair of tiles early
  const long long most = ((long long)a.R / (2 * p.RB) + a.B) * a.nkv;
  const int sms = device_sm_count();
  if (sms < 1) return -4;
  const size_t need = prompt_attention_scratch(a.R, a.Rk, a.nq, a.nkv, a.d, a.B);
  const bool split = need && a.scratch && a.scratch_bytes >= need;
  if (split) {
    p.part_o = static_cast<float*>(a.scratch);
    p.part_ml = p.part_o + (size_t)2 * sms * 2 * AT * a.d;
    p.starts = reinterpret_cast<ApStart*>(p.part_ml + (size_t)2 * sms * 2 * AT * 2);
    p.joins = reinterpret_cast<ApJoin*>(p.starts + sms);
  }
  const int grid = split ? sms : (int)(most < sms ? most : sms);
  const int KT = a.d == 128 ? ApShape<128>::KT : ApShape<64>::KT;
  p.wait_ns = EAGLE_WAIT_LIMIT_NS + (unsigned long long)AP_TILE_NS * (a.Rk / KT + 1);
  CUtensorMap q, k, v;
  // without keys K and V are not read; their maps still need memory
  const bool none = a.Rk == 0;
  if (!ap_map(&q, a.q, a.d, a.nq, a.R, a.ldq, p.G, p.RB) ||
      !ap_map(&k, none ? a.q : a.k, a.d, none ? a.nq : a.nkv, none ? a.R : a.Rk, none ? a.ldq : a.ldk, 1, KT) ||
      !ap_map(&v, none ? a.q : a.v, a.d, none ? a.nq : a.nkv, none ? a.R : a.Rk, none ? a.ldq : a.ldv, 1, KT))
    return -4;
  const cudaError_t e = a.d == 128 ? (split ? launch_prompt<128, true>(st, q, k, v, p, grid) : launch_prompt<128, false>(st, q, k, v, p, grid))
                                   : (split ? launch_prompt<64, true>(st, q, k, v, p, grid) : launch_prompt<64, false>(st, q, k, v, p, grid));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return -4;
  }
  return 0;
}

}  // namespace eagle
