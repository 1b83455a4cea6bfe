// Attention over the 8-bit KV cache, behind an optional bf16 prefix that all rows share: up to 16 query vectors a block
// of rows (all of head_dim 64), the join of what range ends cut, and the host side.
//
//   o = sum_s p_s v_s / sum_s p_s,  p_s = 2^(x_s - m),  x_s = log2(e) scale q.k_s,  m near the maximum,
// over the prefix and the slots that the row sees: one softmax, in one pass over the keys.
//
// Own slots (kv8_attn_k). A decoding step or a small verify pass has few query vectors (rows x query heads of a KV
// head) and many keys, so the keys are the long side of both products, on mma.sync m16n8k16 (fp16, fp32 sums):
//   S^T [16 keys x 8 query vectors] = K Q^T,   O^T [16 dims x 8 query vectors] += V^T P^T.
// With the query vectors on the 8-wide side four of them cost half an instruction, where a 128-row tcgen05 tile
// would be 3% full; and both operands that come from the cache are A fragments, which a warp converts from e4m3
// right after ldmatrix (fp16 holds every code exactly; cvt runs at 128 codes a clock and SM against the 23 bytes a
// clock that HBM delivers).
//   - A key's factor multiplies its score, a value's exponent is added to it: the codes are never scaled.
//   - q is scaled by a power of two into fp16's range (entries down to 2^-30 of its largest exactly, others to 2^-38 of it).
//   - Weights times their values' factors enter the value product as fp16 (2^-11), against a reference of each query
//     vector that is raised only when a product passes it by 2^15: most tiles then need no reduction across lanes and no
//     rescaling of O. Each column decides for itself.
// A producer warp streams the tiles (TMA, 128- or 64-byte swizzle) through a ring that runs on across items, row warps
// prepare the next item's query vectors, and the key groups' sums meet in shared memory, side by side where it lasts.
// Bound by HBM once a range is long: one sequence of 32768 slots (8 KV heads of 128, 4 query heads each) 22 us, of them
// some 12 us of loads at 5.6 TB/s, 4 us until the first tile is there and 5 us for the join's launch; 64 ragged sequences
// of up to 2048 slots 41 us (21 us of bytes at the copy rate).
#include "kv8_split.cuh"
#include "kernels.h"

#include <algorithm>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

namespace eagle {
namespace {

constexpr int TK = 32;            // keys a tile
// head_dim 128 with more query vectors a block goes to tcgen05 (128-key tiles), on either side of which (mma.sync, tcgen05):
// 64 ragged sequences of up to 2048 slots, 8 KV heads, T rows of 4 query heads each: T = 1 41, 70 us; 2 41, 70; 4 49, 71; 6 -,
// 72; 8 -, 72 (when mma.sync still had forms for these it took 14% more than tcgen05 there). One sequence of 32768 slots:
// T = 1 23, 36 us; 4 27, 36; 6 -, 37. 64 sequences of up to 1024, 32 KV heads of one query head: T = 1 81, 152 us; 8 85, 154;
// 16 104, 158; 17 -, 159.
constexpr int TC_ABOVE = 16;

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Partial k of the prefix for query vector `at` of all (row, query head).
template <int D>
__device__ __forceinline__ Part prefix_part(const Kv8Attn& a, const Plan& p, int k, size_t at) {
  const size_t q = (size_t)k * a.R * a.nq + at;
  return Part{p.pp_ml + 2 * q, p.pp_o + q * D};
}
// Shared memory of one configuration: D dims; NT query tiles (of 8) a warp, WN warps side by side over the query
// tiles, WK groups of them over the keys; NS tiles in the ring.
template <int D, int NT, int WN, int WK, int NS, int CTAS>
struct Shape {
  static_assert(NS < 32, "a producer lane has at most one tile in flight");
  static constexpr int QV = 8 * NT * WN, NW = WN * WK;
  // Eight consumer warps that hold wide accumulators: the other warpgroup (one producer, three row warps) gives
  // registers to them (168 a thread at launch; 2 x 128 x 216 + 128 x 72 = 384 x 168; the row warps spill some 250 bytes a
  // thread with 40, 10 with 72).
  static constexpr bool SPLIT_REGS = NW == 8;
  static constexpr int ROWS_W = SPLIT_REGS ? 3 : 1;       // warps that prepare the rows of the next item
  static constexpr int THREADS = (NW + 1 + ROWS_W) * 32;
  static constexpr int TILE = 2 * TK * D;                 // K codes, V codes
  static constexpr int Q_LD = 2 * D + 32;                 // bytes a query row: 8-byte reads without bank conflicts
  static constexpr int O_LD = D + 4;
  static constexpr int OFF_EXP = NS * TILE;               // [NS][2][TK] exponent bytes
  static constexpr int OFF_Q = OFF_EXP + NS * 2 * TK;
  static constexpr int Q_BUF = QV * (Q_LD + 8 + 32);      // query rows, (factor, slot limit) of each, masks
  static constexpr int OFF_O = OFF_Q + 2 * Q_BUF;
  // Key groups that write their O side by side: all of them where shared memory lasts for NS tiles and 512 row blocks
  static constexpr int O_BUF = QV * O_LD * 4, MLE = 2 * WK * QV * 8;   // m, l of each key group, by item parity
  static constexpr int bytes_with(int nr, int groups) {
    return 1024 + OFF_O + nr * O_BUF + MLE + NS * 16 + 192 + (3 * groups + 1) * 4;
  }
  static constexpr int ROOM = (228 / CTAS - 1) * 1024;
  static constexpr int regions(int nr) { return nr == 1 || bytes_with(nr, KV8_MAX_GROUPS) <= ROOM ? nr : regions(nr / 2); }
  static constexpr int NR = regions(WK);
  static_assert(bytes_with(NR, KV8_MAX_GROUPS) <= ROOM, "shared memory");
  static constexpr int OFF_MLE = OFF_O + NR * O_BUF;
  static constexpr int OFF_BAR = OFF_MLE + MLE;
  static constexpr int OFF_GROUP = OFF_BAR + NS * 16 + 192;
  static int bytes(int groups) { return bytes_with(NR, groups); }
};

template <int D, int NT, int WN, int WK, int NS, int CTAS>
__global__ void __launch_bounds__(Shape<D, NT, WN, WK, NS, CTAS>::THREADS, CTAS)
    kv8_attn_k(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Attn a,
               const Plan p) {
  using Sh = Shape<D, NT, WN, WK, NS, CTAS>;
  constexpr int NW = Sh::NW, NC = NW * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + (-smem_u32(smem_raw) & 1023u);   // (not by pointer masks: accesses then lose the shared space)
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + Sh::OFF_BAR);
  uint64_t* empty = full + NS;
  uint64_t *q_full = empty + NS, *q_empty = q_full + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(q_empty + 2);
  int* s_fullvis = reinterpret_cast<int*>(q_empty + 2) + 1;   // [2][16], by warp; [15] the context's length
  int* s_pref = reinterpret_cast<int*>(sm + Sh::OFF_GROUP);
  int* s_lim = s_pref + p.groups + 1;
  int* s_seq = s_lim + p.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkv = a.c.nkv;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(full + s), 33);   // the codes' bytes, and each producer lane's exponent copies
      mbar_init(smem_u32(empty + s), WN);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(q_full + b), Sh::ROWS_W);
      mbar_init(smem_u32(q_empty + b), NW);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  late_entry(p);
  lay_out(a, p, s_pref, s_lim, s_seq);
  const uint32_t tiles = (uint32_t)s_pref[p.groups] * nkv;
  const int pad = pad_of(p, tiles);
  const Share share(p, tiles, pad);
  if (threadIdx.x == 0) cut_none(p, blockIdx.x);
  if (blockIdx.x >= share.ctas) {
    if (threadIdx.x == 0) late_wait(p);
    return;
  }
  const Range range{s_pref, pad, nkv, p.groups, share.start(blockIdx.x), share.start(blockIdx.x + 1)};

  // The query vectors of an item as fp16 of q 2^-e, the factor that gives its scores in log2 units, what each sees. By
  // `warps` warps, of which this is number sw.
  auto prepare = [&](int item, const Walk& k, int sw, int warps) {
    constexpr int LQ = D / 8, PER = 32 / LQ, BATCH = 4;   // lanes a vector, 16 bytes each
    const int sub = lane % LQ;
    const float sl2 = a.scale * 1.4426950408889634f;
    const int gi = k.gi, h = k.h;
    const int buf = item & 1, seq = s_seq[gi];
    const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
    const int r0 = sidx * a.rows_per_seq + rb * p.RB;
    const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
    const int nqv = (r1 - r0) * p.G;
    const int ctx = a.mode == 1 && seq >= 0 ? __ldcg(a.ctx_len + seq) : 0;
    uint8_t* q_rows = sm + Sh::OFF_Q + buf * Sh::Q_BUF;
    float2* q_cols = reinterpret_cast<float2*>(q_rows + Sh::QV * Sh::Q_LD);
    uint64_t* q_mask = reinterpret_cast<uint64_t*>(q_cols + Sh::QV);
    if (item >= 2) kv8_wait(smem_u32(q_empty + buf), (uint32_t)((item / 2 - 1) & 1), abort_flag, a.err);
    if (a.mode == 1)
      for (int x = sw * 32 + lane; x < (r1 - r0) * 4; x += warps * 32) {
        const int r = r0 + x / 4, w = x & 3;
        uint64_t m = 0;
        if (w * 64 < a.tree_T) {
          m = __ldcg(a.mask + (size_t)r * a.mask_words + w);
          if (w == (a.tree_T - 1) >> 6 && (a.tree_T & 63)) m &= (1ull << (a.tree_T & 63)) - 1;
        }
        q_mask[x] = seq >= 0 && __ldcg(a.row_seq + r) == seq ? m : 0ull;
      }
    int fullvis = INT32_MAX;   // keys below this are seen by every row that counts
    for (int x0 = sw * PER; x0 < Sh::QV; x0 += PER * warps * BATCH) {
      uint4 raw[BATCH];
      int rs[BATCH], lim[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int x = x0 + lane / LQ + b * PER * warps;
        raw[b] = make_uint4(0, 0, 0, 0);
        rs[b] = -1;
        lim[b] = 0;
        if (x < nqv) {
          const int in = (int)(x * p.G_inv >> 16), row = r0 + in;
          raw[b] = __ldcg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                                         ((size_t)row * a.nq + h * p.G + x - in * p.G) * D + sub * 8));
          rs[b] = __ldcg(a.row_seq + row);
          lim[b] = a.mode == 1 ? ctx : min(__ldcg(a.row_slot + row), INT32_MAX - 1) + 1;
        }
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int x = x0 + lane / LQ + b * PER * warps;
        const bool live = seq >= 0 && rs[b] == seq;
        const uint32_t r[4] = {live ? raw[b].x : 0u, live ? raw[b].y : 0u, live ? raw[b].z : 0u, live ? raw[b].w : 0u};
        uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(r[k] << 16 & 0x7fffffffu, r[k] & 0x7fff0000u));
#pragma unroll
        for (int d = LQ / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        // largest entry into [2^13, 2^14); a vector with an entry that is not finite gives NaN
        const bool fine = top < 0x7f800000u;
        const int e = top && fine ? max((int)(top >> 23) - 127, -126) - 13 : 0;
        const float up = pow2i(-e / 2), up2 = pow2i(-e - (-e / 2));   // two factors: -e can pass 127
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = fine ? half2_of(__uint_as_float(r[k] << 16) * up * up2, __uint_as_float(r[k] & 0xffff0000u) * up * up2)
                      : 0x7fff7fffu;
        if (x < Sh::QV) {
          const int l = live ? max(0, min(lim[b], a.c.cap)) : -1;   // -1: padding
          *reinterpret_cast<uint4*>(q_rows + x * Sh::Q_LD + sub * 16) = make_uint4(w[0], w[1], w[2], w[3]);
          if (sub == 0) q_cols[x] = make_float2(sl2 * pow2i(e / 2) * pow2i(e - e / 2), __int_as_float(l));
          if (live) fullvis = min(fullvis, l);
        }
      }
    }
    fullvis = __reduce_min_sync(0xffffffffu, fullvis);
    if (lane == 0) s_fullvis[buf * 16 + sw] = fullvis;
    if (sw == 0 && lane == 0) s_fullvis[buf * 16 + 15] = ctx;
    __syncwarp();
  };
  constexpr int FIRST = (NW + Sh::ROWS_W) * 32;   // threads that prepare the first item

  if (warp >= NW) {
    if constexpr (Sh::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp > NW) {
      // row warps: the first item together with the consumers, each later one in the buffer that the consumers are not at
      const int sw = warp - NW - 1;
      Walk k;
      bool more = k.begin(range);
      if (more) prepare(0, k, NW + sw, NW + Sh::ROWS_W);
      asm volatile("bar.arrive 2, %0;" ::"n"(FIRST) : "memory");
      more = more && k.next(range);
      for (int item = 1; more; ++item, more = k.next(range)) {
        prepare(item, k, sw, Sh::ROWS_W);
        if (lane == 0) mbar_arrive(smem_u32(q_full + (item & 1)));
      }
      return;
    }
    // producer: lane j looks up every 32nd tile of an item (block-table reads of 32 tiles overlap); lane 0 issues
    // the codes of all of them, lanes 0-3 copy a tile's exponents, 16 bytes each
    const int box = a.c.table ? min(TK, 1 << a.c.block_log2) : TK;
    const uint64_t pol = l2_policy_evict_first();
    int st = 0, issued = 0;
    uint32_t ph = 1;
    bool ok = true;
    Walk k;
    for (bool more = k.begin(range); more && ok; more = k.next(range)) {
      const int limit = s_lim[k.gi], seq = s_seq[k.gi];
      for (int b = k.t0; ok && b < k.t1; b += 32) {
        int halves = 0, vec0 = 0, vec1 = 0;   // the tile's 16-key halves that hold keys, and where they are
        const int t = b + lane, live = limit - t * TK;
        if (t < k.t1 && live > 0) {
          const long long v = kv8_vec(a.c, seq, k.h, t * TK);
          halves = 1;
          if (box == TK ? (a.c.table || t * TK + 16 < a.c.cap) : live > 16) halves = 2;
          // the second half's vector: of its own block, or 16 on from the first, if that one has a block at all
          // (every start stays a multiple of 16: its exponents are copied 16 bytes at a time)
          const long long u = halves == 2 && box < TK ? kv8_vec(a.c, seq, k.h, t * TK + 16) : v < 0 ? v : v + 16;
          if (v < 0 || (halves == 2 && u < 0)) latch_error(a.err, DEVERR_BOUNDS);   // not assigned: unspecified keys
          vec0 = (int)max(v, 0ll);
          vec1 = (int)max(u, 0ll);
        }
        const int m = min(32, k.t1 - b);
        for (int j = 0; j < m; ++j) {
          const int nh = __shfl_sync(0xffffffffu, halves, j);
          const int v0 = __shfl_sync(0xffffffffu, vec0, j), v1 = __shfl_sync(0xffffffffu, vec1, j);
          if (issued >= NS && !kv8_wait(smem_u32(empty + st), ph, abort_flag, a.err)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t bar = smem_u32(full + st);
          ++issued;
          if (lane < 2 * nh)
            copy16(smem_u32(sm + Sh::OFF_EXP + st * 2 * TK) + (lane & 1) * TK + (lane >> 1) * 16,
                   ((lane & 1) ? a.c.ve : a.c.ke) + (lane < 2 ? v0 : v1));
          copies_arrive(bar);
          if (lane == 0) {
            const int boxes = box == TK ? min(nh, 1) : nh;
            const uint32_t kd = smem_u32(sm + st * Sh::TILE);
            mbar_expect_tx(bar, (uint32_t)(boxes * 2 * box * D));
            if (boxes) {
              tma_load_2d(kd, &tmK, 0, v0, bar, pol);
              tma_load_2d(kd + TK * D, &tmV, 0, v0, bar, pol);
            }
            if (boxes > 1) {
              tma_load_2d(kd + 16 * D, &tmK, 0, v1, bar, pol);
              tma_load_2d(kd + TK * D + 16 * D, &tmV, 0, v1, bar, pol);
            }
          }
          if (++st == NS) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
    // after a timeout the tiles in flight land before the CTA leaves: the last NS that were issued
    if (!ok)
      for (int x = max(0, issued - NS); x < issued; ++x)
        kv8_wait(smem_u32(full + x % NS), (uint32_t)((x / NS) & 1), abort_flag, a.err, false);
  } else {
    if constexpr (Sh::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int kw = warp / WN, nw = warp % WN;
    const int g = lane >> 2, t4 = lane & 3;
    float* s_o = reinterpret_cast<float*>(sm + Sh::OFF_O);
    Walk k;
    bool more = k.begin(range);
    if (more) prepare(0, k, warp, NW + Sh::ROWS_W);
    asm volatile("bar.sync 2, %0;" ::"n"(FIRST) : "memory");
    // this lane's row of the ldmatrix tiles, with its swizzle, 16-byte column 0: column c is at ^ (16 c)
    auto swizzled = [&](int row, int col) { return row * D + (D == 128 ? col ^ (row & 7) : col ^ ((row >> 1) & 3)) * 16; };
    const uint32_t k_at = swizzled(lane, 0), v_at = swizzled(lane & 15, lane >> 4);
    int i = 0;   // tiles of the range that are behind
    for (int item = 0; more; ++item, more = k.next(range)) {
      const int gi = k.gi, h = k.h, t0 = k.t0, t1 = k.t1, nt = k.nt;
      const int limit = s_lim[gi];
      const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
      const int r0 = sidx * a.rows_per_seq + rb * p.RB;
      const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
      const int nqv = (r1 - r0) * p.G;

      const int buf = item & 1;
      const uint8_t* s_q = sm + Sh::OFF_Q + buf * Sh::Q_BUF;
      const float2* s_col = reinterpret_cast<const float2*>(s_q + Sh::QV * Sh::Q_LD);
      const uint64_t* s_mask = reinterpret_cast<const uint64_t*>(s_col + Sh::QV);
      if (item) kv8_wait(smem_u32(q_full + buf), (uint32_t)((item / 2 - (buf == 0)) & 1), abort_flag, a.err);
      const int ctx = s_fullvis[buf * 16 + 15];
      int fullvis = s_fullvis[buf * 16];
      for (int w = 1; w < (item ? Sh::ROWS_W : NW + Sh::ROWS_W); ++w) fullvis = min(fullvis, s_fullvis[buf * 16 + w]);

      float O[D / 16][NT][4], ref[NT][2], l[NT][2], qf[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) O[c][x][0] = O[c][x][1] = O[c][x][2] = O[c][x][3] = 0.f;
        const int col = (nw * NT + x) * 8 + 2 * t4;
        ref[x][0] = ref[x][1] = -INFINITY;
        l[x][0] = l[x][1] = 0.f;
        qf[x][0] = s_col[col].x;
        qf[x][1] = s_col[col + 1].x;
      }

      for (int t = t0; t < t1; ++t, ++i) {
        if (i % WK != kw) continue;
        const int st = i % NS;
        kv8_wait(smem_u32(full + st), (uint32_t)((i / NS) & 1), abort_flag, a.err);
        const int key0 = t * TK;
        if (key0 < limit && !*abort_flag) {
          const uint8_t* s_ke = sm + Sh::OFF_EXP + st * 2 * TK;
          const uint8_t* s_ve = s_ke + TK;
          const uint32_t kb = smem_u32(sm + st * Sh::TILE), vb = kb + TK * D;
          const bool masked = key0 + TK > fullvis;
          // the tile's keys that a query vector sees, one bit a key
          auto sees = [&](int col) -> uint32_t {
            const int below = __float_as_int(s_col[col].y) - key0;
            uint32_t v = below >= TK ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1;
            if (a.mode == 1 && col < nqv) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(s_mask + (col * p.G_inv >> 16) * 4);
              const int tt = key0 - ctx;   // tree slot of the tile's first key
              const uint32_t lo = tt >= 0 && tt < 256 ? w[tt >> 5] : 0u;
              const uint32_t hi = tt >= -31 && tt < 224 ? w[(tt + 32) >> 5] : 0u;
              v |= __funnelshift_r(lo, hi, tt & 31);
            }
            return limit - key0 >= TK ? v : v & ((1u << (limit - key0)) - 1);
          };
          uint32_t seen = 0xffffffffu, vis[NT][2];   // keys that one of this warp's query vectors sees; that each sees
          if (masked) {
            seen = 0;
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                vis[x][e] = sees((nw * NT + x) * 8 + 2 * t4 + e);
                seen |= vis[x][e];
                vis[x][e] >>= g;   // this thread's keys: bits 0, 8, 16, 24
              }
            seen |= __shfl_xor_sync(0xffffffffu, seen, 1);
            seen |= __shfl_xor_sync(0xffffffffu, seen, 2);
          }
          // lane = key: its factor, its value's exponent and the inverse of that one's power
          const float fk = kv8_pow2(s_ke[lane]), ev = kv8_exponent(s_ve[lane]), iv = kv8_inverse(s_ve[lane]);
          float s[2][NT][4];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int x = 0; x < NT; ++x) s[mt][x][0] = s[mt][x][1] = s[mt][x][2] = s[mt][x][3] = 0.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t r[4], a0[4], a1[4];
            ldsm4(kb + (k_at ^ (c * 16)), r);
            e4m3x4_f16(r[0], a0[0], a0[2]);
            e4m3x4_f16(r[1], a0[1], a0[3]);
            e4m3x4_f16(r[2], a1[0], a1[2]);
            e4m3x4_f16(r[3], a1[1], a1[3]);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              const uint2 b = *reinterpret_cast<const uint2*>(s_q + ((nw * NT + x) * 8 + g) * Sh::Q_LD + c * 32 + t4 * 8);
              mma_f16(s[0][x], a0, b.x, b.y);
              mma_f16(s[1][x], a1, b.x, b.y);
            }
          }
          float mx[NT][2];
#pragma unroll
          for (int x = 0; x < NT; ++x) mx[x][0] = mx[x][1] = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const float f0 = __shfl_sync(0xffffffffu, fk, mt * 16 + g), f1 = __shfl_sync(0xffffffffu, fk, mt * 16 + 8 + g);
            const float e0 = __shfl_sync(0xffffffffu, ev, mt * 16 + g), e1 = __shfl_sync(0xffffffffu, ev, mt * 16 + 8 + g);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              // a rounded sum here, and the reference taken off it below: that difference is exact near the reference,
              // where a fused one would leave the rounding of a huge score over, and a weight of 2^(that)
              s[mt][x][0] = s[mt][x][0] * f0 * qf[x][0] + e0; s[mt][x][1] = s[mt][x][1] * f0 * qf[x][1] + e0;
              s[mt][x][2] = s[mt][x][2] * f1 * qf[x][0] + e1; s[mt][x][3] = s[mt][x][3] * f1 * qf[x][1] + e1;
              if (masked)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!((vis[x][e & 1] >> (mt * 16 + (e >> 1) * 8)) & 1u)) s[mt][x][e] = -INFINITY;
              mx[x][0] = fmaxf(mx[x][0], fmaxf(s[mt][x][0], s[mt][x][2]));
              mx[x][1] = fmaxf(mx[x][1], fmaxf(s[mt][x][1], s[mt][x][3]));
            }
          }
          bool raise = false;
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) raise = raise || mx[x][e] - ref[x][e] > KV8_TOP;
          if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v = mx[x][e];
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                if (!(v - ref[x][e] > KV8_TOP)) continue;
                const float corr = ex2(ref[x][e] - (v - KV8_HEAD));
                ref[x][e] = v - KV8_HEAD;
                l[x][e] *= corr;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  O[c][x][e] *= corr;
                  O[c][x][2 + e] *= corr;
                }
              }
          }
          // weights, as the B operand of the value product
          uint32_t pb[2][NT][2];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const float i0 = __shfl_sync(0xffffffffu, iv, mt * 16 + g), i1 = __shfl_sync(0xffffffffu, iv, mt * 16 + 8 + g);
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              float w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float base = ref[x][e & 1] == -INFINITY ? 0.f : ref[x][e & 1];
                w[e] = ex2(s[mt][x][e] - base);
                l[x][e & 1] = fmaf(w[e], e < 2 ? i0 : i1, l[x][e & 1]);
              }
              pb[mt][x][0] = transpose8(half2_of(w[0], w[1]));
              pb[mt][x][1] = transpose8(half2_of(w[2], w[3]));
            }
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            // a pair's bytes (k0 d0, k0 d1, k1 d0, k1 d1) to (k0 d0, k1 d0, k0 d1, k1 d1); zeros for keys that nobody sees
            uint32_t sel0 = 0x3120, sel1 = 0x3120;
            if (masked) {
              const uint32_t k = seen >> (mt * 16 + 2 * t4);
              sel0 = ((k & 1u) ? 0x0100u : 0x0404u) | ((k & 2u) ? 0x3020u : 0x4040u);
              sel1 = ((k & 256u) ? 0x0100u : 0x0404u) | ((k & 512u) ? 0x3020u : 0x4040u);
            }
#pragma unroll
            for (int c = 0; c < D / 16; c += 2) {
              uint32_t r[4], va[4], vc[4];
              ldsm4_t(vb + mt * 16 * D + (v_at ^ (c * 16)), r);
              e4m3x4_f16(__byte_perm(r[0], 0, sel0), va[0], va[1]);
              e4m3x4_f16(__byte_perm(r[1], 0, sel1), va[2], va[3]);
              e4m3x4_f16(__byte_perm(r[2], 0, sel0), vc[0], vc[1]);
              e4m3x4_f16(__byte_perm(r[3], 0, sel1), vc[2], vc[3]);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                mma_f16(O[c][x], va, pb[mt][x][0], pb[mt][x][1]);
                mma_f16(O[c + 1][x], vc, pb[mt][x][0], pb[mt][x][1]);
              }
            }
          }
        }
        warp_arrive(smem_u32(empty + st));
      }

      // join the key groups: sums in the order of the groups
      float* s_m = reinterpret_cast<float*>(sm + Sh::OFF_MLE) + buf * 2 * WK * Sh::QV;
      float* s_l = s_m + WK * Sh::QV;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = l[x][e];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (g == 0) {
            const int at = kw * Sh::QV + (nw * NT + x) * 8 + 2 * t4 + e;
            s_m[at] = ref[x][e];
            s_l[at] = v;
          }
        }
      named_bar_sync(1, NC);   // (and the item before has been read from s_o)
#pragma unroll 1
      for (int r = 0; r < WK; r += Sh::NR) {
        if (r == kw / Sh::NR * Sh::NR) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = (nw * NT + x) * 8 + 2 * t4 + e;
              if (col >= nqv) continue;
              float top = s_m[col];
#pragma unroll
              for (int k = 1; k < WK; ++k) top = fmaxf(top, s_m[k * Sh::QV + col]);
              const float f = ex2(ref[x][e] - (top == -INFINITY ? 0.f : top));
              float* o = s_o + (kw % Sh::NR * Sh::QV + col) * Sh::O_LD + 2 * g;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                float2 v = r ? *reinterpret_cast<float2*>(o + 16 * c) : make_float2(0.f, 0.f);
                v.x = fmaf(O[c][x][e], f, v.x);
                v.y = fmaf(O[c][x][2 + e], f, v.y);
                *reinterpret_cast<float2*>(o + 16 * c) = v;
              }
            }
        }
        named_bar_sync(1, NC);
      }
      const bool whole = t0 == 0 && t1 == nt;
      if (whole) late_wait(p);
      if (threadIdx.x == 0 && t0 == 0) cut_begin(p, blockIdx.x, k, (int)share.cta_of(k.base + pad + nt - 1));
      const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
      for (int x = threadIdx.x; x < nqv * (D / 8); x += NC) {
        const int col = x / (D / 8), c = x % (D / 8) * 8;
        float top = s_m[col];
#pragma unroll
        for (int k = 1; k < WK; ++k) top = fmaxf(top, s_m[k * Sh::QV + col]);
        float L = 0.f, o[8];
#pragma unroll
        for (int k = 0; k < WK; ++k)
          L += s_l[k * Sh::QV + col] * ex2(s_m[k * Sh::QV + col] - (top == -INFINITY ? 0.f : top));
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll
        for (int k = 0; k < Sh::NR; ++k) {
          const float* src = s_o + (k * Sh::QV + col) * Sh::O_LD + c;
          const float4 u = *reinterpret_cast<const float4*>(src), v = *reinterpret_cast<const float4*>(src + 4);
          o[0] += u.x; o[1] += u.y; o[2] += u.z; o[3] += u.w; o[4] += v.x; o[5] += v.y; o[6] += v.z; o[7] += v.w;
        }
        if (whole) {
          const int in = (int)(col * p.G_inv >> 16), row = r0 + in;
          const size_t at = (size_t)row * a.nq + h * p.G + col - in * p.G;
          fold<D, (NT == 1 ? 6 : 2)>(p.n_prefix, [&](int k) { return prefix_part<D>(a, p, k, at); }, c / 8, top, L, o);
          store8(a, at, D, c, __float_as_int(s_col[col].y) >= 0, L, o);
        } else {
          const size_t q = (size_t)slot * p.qv_pad + col;
          *reinterpret_cast<float4*>(p.part_o + q * D + c) = make_float4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<float4*>(p.part_o + q * D + c + 4) = make_float4(o[4], o[5], o[6], o[7]);
          if (c == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * q) = make_float2(top, L);
        }
      }
      warp_arrive(smem_u32(q_empty + buf));
    }
    if (threadIdx.x == 0) late_wait(p);
  }
}

// Joins the pieces of the items that range ends cut, and the prefix's partials with them: CTA (x, y) takes the
// item of p.cut[x], p.join_cols of its query vectors. D / 8 lanes a query vector and p.join_ways such
// teams, which take every join_ways-th partial each and are joined through shared memory, in the order of the teams.
template <int D>
__global__ void __launch_bounds__(256) kv8_join_k(const Kv8Attn a, const Plan p) {
  constexpr int GL = D / 8;
  __shared__ float s_part[256 / GL][D + 4];
  __shared__ float2 s_ml[256 / GL];
  PDL_ENTRY();
  const int4 cut = p.cut[blockIdx.x];
  const int lo = cut.x, h = cut.y, c0 = cut.z, c1 = cut.w;
  if (c1 < 0) return;
  if (lo < 0 || lo >= p.groups || h < 0 || h >= p.nkv || c0 < 0 || c1 < c0 || c1 >= p.grid) return;   // a wait gave up
  const int sidx = (p.g0 + lo) / p.nb, rb = (p.g0 + lo) - sidx * p.nb;
  const int s0 = sidx * a.rows_per_seq, s1 = (int)min((long long)s0 + a.rows_per_seq, (long long)a.R);
  const int r0 = s0 + rb * p.RB, nqv = (min(r0 + p.RB, s1) - r0) * p.G;
  const int team = threadIdx.x / GL, ways = p.join_ways, way = team / p.join_cols;
  const int col = blockIdx.y * p.join_cols + team % p.join_cols, c = threadIdx.x % GL * 8;
  const int col_in = min(col, nqv - 1), in = (int)(col_in * p.G_inv >> 16), row = r0 + in;
  const size_t at = (size_t)row * a.nq + h * p.G + col_in - in * p.G;
  const int lead = __ldcg(a.row_seq + s0), own = __ldcg(a.row_seq + row);
  const int seq = lead >= 0 ? lead : seq_behind_padding(a.row_seq, s0, s1, r0, s1, 32);
  // piece 0 in slot 2 c0 + 1 (it holds the item's start), the others in slot 2 c, then the prefix's
  const int pieces = c1 - c0 + 1, n = pieces + p.n_prefix;
  float top = -INFINITY, L = 0.f, o[8] = {};
  fold<D, 3>((n - way + ways - 1) / ways, [&](int i) {
    const int k = i * ways + way;
    if (k >= pieces) return prefix_part<D>(a, p, k - pieces, at);
    const size_t q = (size_t)(k ? 2 * (c0 + k) : 2 * c0 + 1) * p.qv_pad + col_in;
    return Part{p.part_ml + 2 * q, p.part_o + q * D};
  }, c / 8, top, L, o);
  if (ways > 1) {
    if (way) {
      *reinterpret_cast<float4*>(&s_part[team][c]) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(&s_part[team][c + 4]) = make_float4(o[4], o[5], o[6], o[7]);
      if (c == 0) s_ml[team] = make_float2(top, L);
    }
    __syncthreads();
    if (way) return;
    float mx = top;
    for (int w = 1; w < ways; ++w) mx = fmaxf(mx, s_ml[team + w * p.join_cols].x);
    const float base = mx == -INFINITY ? 0.f : mx, f = ex2(top - base);
    L *= f;
#pragma unroll
    for (int x = 0; x < 8; ++x) o[x] *= f;
    for (int w = 1; w < ways; ++w) {
      const int from = team + w * p.join_cols;
      const float2 ml = s_ml[from];
      const float g = ex2(ml.x - base);
      L = fmaf(ml.y, g, L);
#pragma unroll
      for (int x = 0; x < 8; ++x) o[x] = fmaf(s_part[from][c + x], g, o[x]);
    }
  }
  if (col < nqv) store8(a, at, D, c, seq >= 0 && seq < a.c.max_batch && own == seq, L, o);
}


}  // namespace

// ---- host side ------------------------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Codes as rows of d bytes, boxes of `box` rows, swizzled by the row's width.
bool code_map(CUtensorMap* m, const uint8_t* codes, long long rows, int d, int box) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d};
  const cuuint32_t boxes[2] = {(cuuint32_t)d, (cuuint32_t)box}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, boxes, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// Row blocks: a sequence's rows in one block when their query vectors fit, else in equal blocks.
void cut_rows(const Kv8& c, int nq, int rows_per_seq, Plan& p) {
  p.nkv = c.nkv;
  p.tk = TK;
  p.G = nq / c.nkv;
  const int most = KV8_MAX_QV / p.G;
  p.nb = (rows_per_seq + most - 1) / most;
  p.RB = (rows_per_seq + p.nb - 1) / p.nb;
  p.QV = p.RB * p.G;
  p.qv_pad = (p.QV + 7) / 8 * 8;
  p.G_inv = 65536u / p.G + 1;
  p.width = 1;
  while (p.width < 8 && p.width < p.RB) p.width *= 2;
}

size_t own_scratch(const Kv8& c, const Plan& p) {
  return al256((size_t)2 * KV8_MAX_CTAS * p.qv_pad * c.d * sizeof(float)) +
         al256((size_t)2 * KV8_MAX_CTAS * p.qv_pad * 2 * sizeof(float)) + al256(KV8_MAX_CTAS * sizeof(int4));
}

// A join CTA holds up to 256 / (D / 8) teams: as many on one query vector as leave each about four partials, if the
// grid's ranges are spread evenly over the items, the others on further query vectors; fewer where items that are all cut
// would make more than two CTAs an SM (61 rows of one sequence: 25.4 us with 992 CTAs, 19.5 with 248 at the time).
template <int D>
cudaError_t launch_join(cudaStream_t st, const Kv8Attn& a, Plan& p) {
  constexpr int TEAMS = 256 / (D / 8);
  const int items = p.groups * p.nkv, partials = p.grid / items + 2 + p.n_prefix;
  p.join_ways = 1;
  while (p.join_ways < TEAMS && p.join_ways * 4 < partials) p.join_ways *= 2;
  p.join_cols = 32 / (D / 8);   // whole warps
  while (p.join_cols * p.join_ways < TEAMS && p.join_cols < p.QV) p.join_cols *= 2;
  if (p.join_cols * p.join_ways > TEAMS) p.join_ways = TEAMS / p.join_cols;
  while (p.join_ways > 1 && p.by_item && items * ((p.QV + p.join_cols - 1) / p.join_cols) > 2 * device_sm_count()) {
    p.join_ways /= 2;
    p.join_cols *= 2;
  }
  return launch_k(kv8_join_k<D>, dim3(p.by_item ? items : p.grid, (p.QV + p.join_cols - 1) / p.join_cols),
                  dim3(p.join_cols * p.join_ways * (D / 8)), 0, st, a, p);
}

template <int D, int NT, int WN, int WK, int NS, int CTAS>
cudaError_t launch_own(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& mk, const CUtensorMap& mv) {
  using Sh = Shape<D, NT, WN, WK, NS, CTAS>;
  const auto fn = kv8_attn_k<D, NT, WN, WK, NS, CTAS>;
  p.grid = std::min(KV8_MAX_CTAS, CTAS * device_sm_count());
  p.by_item = p.groups * p.nkv <= p.grid;
  p.min_tiles = WK;
  p.pad = 6 + p.n_prefix / 2;
  const int smem = Sh::bytes(p.groups);
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  e = launch_k(fn, dim3(p.grid), dim3(Sh::THREADS), smem, st, mk, mv, a, p);
  return e != cudaSuccess ? e : launch_join<D>(st, a, p);
}

// A configuration that holds a block's query vectors: up to 64 in two CTAs an SM (one's joins under the other's loads), more
// in one CTA of eight warps. A second query tile goes to other warps, not to the same: they widen
// the codes once more, but nothing spills (16 query vectors of 128: 58 us at the time, 65 with both in a warp). 64 ragged
// sequences of up to 2048 slots, 8 KV heads of 64: 16 query vectors a block 43 us, 32 48 us, 48 76 us (82 in one CTA of three
// query tiles a warp), 64 77 us, 96 102 us (123 in the form for 128), 128 128 us. (The last two spill 8 and 12 bytes a thread.)
template <int D>
cudaError_t launch_mma(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& mk, const CUtensorMap& mv) {
  const int t = p.qv_pad / 8;
  if (t <= 1) return launch_own<D, 1, 1, 4, 10, 2>(st, a, p, mk, mv);
  if (t <= 2) return launch_own<D, 1, 2, 2, 10, 2>(st, a, p, mk, mv);
  if constexpr (D == 64) {
    if (t <= 4) return launch_own<D, 2, 2, 2, 9, 2>(st, a, p, mk, mv);
    if (t <= 8) return launch_own<D, 2, 4, 1, 7, 2>(st, a, p, mk, mv);
    if (t <= 12) return launch_own<D, 3, 4, 2, 11, 1>(st, a, p, mk, mv);
    return launch_own<D, 4, 4, 2, 7, 1>(st, a, p, mk, mv);
  }
  return cudaErrorInvalidValue;   // (head_dim 128 with more goes to launch_tc)
}

cudaError_t launch_tc(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& mk, const CUtensorMap& mv) {
  p.grid = 2 * std::min(KV8_MAX_CTAS / 2, device_sm_count());   // two workers a CTA
  p.by_item = p.groups * p.nkv <= p.grid;
  p.min_tiles = 1;
  p.pad = 2;
  const cudaError_t e = kv8_launch_tc(st, a, p, mk, mv);
  return e != cudaSuccess ? e : launch_join<128>(st, a, p);
}

}  // namespace

size_t kv8_attention_scratch(const Kv8& c, int R, int nq, int rows_per_seq, int P) {
  Plan p{};
  cut_rows(c, nq, rows_per_seq, p);
  const size_t qv = (size_t)R * nq * (P ? kv8_prefix_splits(c.nkv, R, nq, P) : 0);
  return own_scratch(c, p) + al256(qv * c.d * sizeof(float)) + al256(qv * 2 * sizeof(float));
}

int kv8_attention(cudaStream_t st, const Kv8Attn& a) {
  Plan p{};
  cut_rows(a.c, a.nq, a.rows_per_seq, p);
  uint8_t* s = (uint8_t*)a.scratch;
  p.part_o = (float*)s;
  s += al256((size_t)2 * KV8_MAX_CTAS * p.qv_pad * a.c.d * sizeof(float));
  p.part_ml = (float*)s;
  s += al256((size_t)2 * KV8_MAX_CTAS * p.qv_pad * 2 * sizeof(float));
  p.cut = (int4*)s;
  if (a.P) {
    p.n_prefix = kv8_prefix_splits(a.c.nkv, a.R, a.nq, a.P);
    const size_t qv = (size_t)a.R * a.nq * p.n_prefix;
    float* o = (float*)(s + al256(KV8_MAX_CTAS * sizeof(int4)));
    float* ml = (float*)((uint8_t*)o + al256(qv * a.c.d * sizeof(float)));
    p.pp_o = o;
    p.pp_ml = ml;
    const int r = kv8_prefix(st, a, p.n_prefix, o, ml);
    if (r) return r;
  }
  const long long rows = a.c.table ? ((long long)a.c.n_blocks * a.c.nkv) << a.c.block_log2
                                   : (long long)a.c.max_batch * a.c.nkv * a.c.cap;
  const bool tc = a.c.d == 128 && p.qv_pad > TC_ABOVE;
  if (tc) p.tk = 128;
  const int box = a.c.table ? std::min(p.tk, 1 << a.c.block_log2) : p.tk;
  CUtensorMap mk, mv;
  if (!code_map(&mk, a.c.k, rows, a.c.d, box) || !code_map(&mv, a.c.v, rows, a.c.d, box)) return -4;
  // row blocks that hold rows: the last sequence may have fewer
  const long long seqs = ((long long)a.R + a.rows_per_seq - 1) / a.rows_per_seq;
  const long long blocks = (seqs - 1) * p.nb + (a.R - (seqs - 1) * a.rows_per_seq + p.RB - 1) / p.RB;
  // tiles of a launch and their flat numbers stay in 32 bits
  if (blocks > 0x7fffffffll || (double)std::min<long long>(blocks, KV8_MAX_GROUPS) * (a.c.cap / TK + 32) * a.c.nkv > 2e9) return -1;
  for (long long g0 = 0; g0 < blocks; g0 += KV8_MAX_GROUPS) {
    p.g0 = (int)g0;
    p.late = a.P && g0 == 0;
    p.groups = (int)std::min<long long>(KV8_MAX_GROUPS, blocks - g0);
    const cudaError_t e = tc ? launch_tc(st, a, p, mk, mv)
                          : a.c.d == 128 ? launch_mma<128>(st, a, p, mk, mv)
                                         : launch_mma<64>(st, a, p, mk, mv);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return -4;
    }
  }
  return 0;
}

}  // namespace eagle
