// Causal attention over whole prompts: rows and keys of many sequences packed one behind another, on the 5th-generation
// tensor cores.
//
//   o_i = sum_{j <= i + off} p_j v_j / sum p_j,  p_j = 2^(s_j - m),  s_j = q_i k_j scale log2(e),  off = keys - rows.
// 4 d operations for each (row, visible key, query head) against 2 d (2 nq + 2 nkv) bytes a token: bound by the tensor cores
// from a few hundred tokens on, by latency below.
//
// The query heads of a KV head read the same keys, so a tile of 128 query vectors is RB = 128 / G positions times the G
// heads: one TMA box lays them out so, and grouped heads need neither copies nor masks of their own. An item is a pair of such
// tiles (2 RB positions of one KV head) with all the keys that its rows see, 128 at a time. A CTA an SM takes items in
// turn, the ones with the most keys first. 20 warps:
//   warps 0-7, 8-15 softmax of tile 0 / 1, four threads a query vector (16 TMEM lanes a warp): S row -> maximum, weights as bf16
//                   back into TMEM over S, running sum; O is rescaled only when the maximum moves by more than 2^8; results;
//   warp 16         finds the items; TMA: Q of each tile, K and V tiles through one ring;
//   warps 17, 18    tcgen05.mma of tile 0 / 1, in turn: S = Q K^T (operands in shared memory), O += P V (P in TMEM, V read
//                   MN-major);
//   warp 19         looks through value tiles that not all rows see (below).
// TMEM: S0 S1 (128 columns each, P over the first 64), O0 O1 (d each). While one tile is in its softmax warps the tensor cores
// run the other's products. Weights are rounded to bf16 (2^-8 relative at most, as the values that they meet); maxima, sums
// and outputs are fp32, the sum of the unrounded weights.
//
// A weight of zero does not hide a value that is not finite (0 * inf = NaN). In the tiles that some rows see only in part
// warp 19 replaces such values by zero and keeps, for each column, the first key that held a NaN, +inf and -inf: rows that
// see it get that value in their results, the others are left alone.
#include "attn_tc.cuh"
#include "kernels.h"
#include "ops_ext.h"

#include <cuda_bf16.h>

namespace eagle {
namespace {

constexpr int AT = 128;              // keys a tile, query vectors a tile
constexpr int AP_SOFT = 16;          // softmax warps, eight a tile
constexpr int AP_THREADS = (AP_SOFT + 4) * 32;
constexpr float AP_LAZY = 8.f;       // binary orders that a maximum may pass its reference by
constexpr uint32_t AP_NONE = 0x3fffffffu;      // three fields of ten bits, "no key"

template <int D>
struct ApShape {
  static constexpr int HALVES = D / 64, HALF = AT * 128;        // 64 dims of 128 rows
  static constexpr int OP = HALVES * HALF;                      // one operand tile
  static constexpr int STAGES = D == 128 ? 5 : 8;
  static constexpr int OFF_RING = 2 * OP, OFF_BAR = OFF_RING + STAGES * OP;
  static constexpr int OFF_ITEM = OFF_BAR + 400, OFF_BAD = OFF_ITEM + 2 * 48;
  static constexpr int BYTES = 1024 + OFF_BAD + 2 * D * 4;
};

// What a CTA does next. lim0: the last key that the first row sees (negative: none); rows of tile 0 and 1; key tiles of each.
struct ApItem {
  int h, row0, rows[2], n[2], k0, lim0;
};

struct ApArgs {
  int R, Rk, nq, nkv, G, RB, B;
  const int *start, *kstart;
  float sl2;                   // scale * log2(e)
  __nv_bfloat16* out;
  long long ldo;
  float* lse;
  int* err;
};

// One sequence's rows and keys; none where the starts are not in order or out of range.
struct ApSeq { int r0, lq, k0, lk; };
__device__ __forceinline__ ApSeq ap_seq(const ApArgs& a, int b, bool& bad) {
  const int r0 = __ldg(a.start + b), r1 = __ldg(a.start + b + 1), k0 = __ldg(a.kstart + b), k1 = __ldg(a.kstart + b + 1);
  bad = r0 < 0 || r1 < r0 || r1 > a.R || k0 < 0 || k1 < k0 || k1 > a.Rk;
  return bad ? ApSeq{0, 0, 0, 0} : ApSeq{r0, r1 - r0, k0, k1 - k0};
}

// The items' order. Pair t of a sequence has level t + (off >> log2 of a pair's positions): about its number of key tiles.
// Items go by falling level, then sequence, then head: the last ones are the short ones, so the CTAs end together.
struct ApList {
  int level, above, upto;      // pairs of higher levels, of this and higher ones
  int total;
};
__device__ __forceinline__ int ap_pairs(const ApArgs& a, int lq) { return (lq + 2 * a.RB - 1) / (2 * a.RB); }
__device__ __forceinline__ int ap_first(const ApArgs& a, const ApSeq& s) { return s.lk > s.lq ? (s.lk - s.lq) / (2 * a.RB) : 0; }
// pairs of level e and higher (a converged warp)
__device__ __forceinline__ int ap_count(const ApArgs& a, int e) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    bool bad;
    const ApSeq s = ap_seq(a, b, bad);
    const int T = ap_pairs(a, s.lq);
    n += max(0, min(T, ap_first(a, s) + T - e));
  }
  return __reduce_add_sync(0xffffffffu, n);
}
__device__ __forceinline__ ApList ap_begin(const ApArgs& a, bool latch) {
  int total = 0, top = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    bool bad;
    const ApSeq s = ap_seq(a, b, bad);
    if (bad && latch) latch_error(a.err, DEVERR_BOUNDS);
    const int T = ap_pairs(a, s.lq);
    total += T;
    if (T) top = max(top, ap_first(a, s) + T - 1);
  }
  ApList l;
  l.total = __reduce_add_sync(0xffffffffu, total);
  l.level = __reduce_max_sync(0xffffffffu, top);
  l.above = 0;
  l.upto = ap_count(a, l.level);
  return l;
}
// Item i; h = -1 behind the last one. i rises from call to call.
__device__ __forceinline__ ApItem ap_item(const ApArgs& a, ApList& l, long long i) {
  ApItem it{};
  it.h = -1;
  const long long rank = i / a.nkv;
  if (rank >= l.total) return it;
  while (rank >= l.upto) {      // (ends: all pairs are of level zero or higher)
    l.above = l.upto;
    l.upto = ap_count(a, --l.level);
  }
  int k = (int)rank - l.above;
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    ApSeq s{0, 0, 0, 0};
    bool bad;
    if (b < a.B) s = ap_seq(a, b, bad);
    const int first = ap_first(a, s), t = l.level - first;
    const unsigned who = __ballot_sync(0xffffffffu, t >= 0 && t < ap_pairs(a, s.lq));
    const int n = __popc(who);
    if (k >= n) {
      k -= n;
      continue;
    }
    const int src = __fns(who, 0, k + 1);
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
      x.n[y] = x.rows[y] > 0 && last >= 0 ? last / AT + 1 : 0;
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

// Whether key tile j holds keys that a row of the tiles that use it does not see, and the last one that all of them see.
__device__ __forceinline__ bool ap_partial(const ApItem& it, int RB, int j, int& seen) {
  seen = j < it.n[0] ? it.lim0 : it.lim0 + RB;
  return j * AT + AT - 1 > seen;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
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
// 64 bf16 a row as 32 columns of pairs: w[2 i] of the first row, w[2 i + 1] of the second, in frag_ld64's order.
__device__ __forceinline__ void frag_st_pairs(uint32_t t, const uint32_t* w) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}
// The maximum over the four threads that share a row.
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
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

// Values that are not finite in rows [r0, 128) of a value tile (16-byte pieces, 128-byte swizzle): replaced by zero, the
// first key (of those after the first row's last, 0: seen by all) kept for each column. By a converged warp.
template <int D>
__device__ __forceinline__ bool ap_clean(uint8_t* v, int r0, int key0, int lim0, uint32_t* bad, bool fresh) {
  using Sh = ApShape<D>;
  const int lane = threadIdx.x & 31;
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 acc = zero;
  r0 &= ~3;      // (rows before the first that is hidden from some: seen by all, and looked at for nothing)
#pragma unroll 1
  for (int x = 0; x < Sh::HALVES; ++x)
#pragma unroll 4
    for (int i = r0 * 8 + lane; i < AT * 8; i += 32) {
      const uint4 w = *reinterpret_cast<const uint4*>(v + x * Sh::HALF + i * 16);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u[y]), zero, acc);   // inf * 0 = NaN
    }
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&acc);
  if (!__any_sync(0xffffffffu, (bits & 0x7fff7fffu) != 0)) return false;
  if (fresh) {
    for (int c = lane; c < D; c += 32) bad[c] = AP_NONE;
    __syncwarp();
  }
#pragma unroll 1
  for (int x = 0; x < Sh::HALVES; ++x)
#pragma unroll 1
    for (int i = r0 * 8 + lane; i < AT * 8; i += 32) {
      const int row = i >> 3, piece = (i & 7) ^ (row & 7);
      __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(v + x * Sh::HALF + i * 16);
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

template <int D>
__global__ void __launch_bounds__(AP_THREADS, 1)
    prompt_k(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const ApArgs a) {
  using Sh = ApShape<D>;
  constexpr int ST = Sh::STAGES;
  extern __shared__ uint8_t ap_smem[];
  uint8_t* sm = ap_smem + (-smem_u32(ap_smem) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::OFF_BAR);
  uint64_t *full = bars, *empty = bars + ST /* ring */, *q_full = bars + 2 * ST /* [tile] */, *q_empty = q_full + 2,
           *s_full = q_full + 4 /* [tile] */, *p_full = q_full + 6 /* [tile][half] */, *o_done = q_full + 10 /* [tile] */,
           *o_free = q_full + 12 /* [tile] */, *item_full = q_full + 14 /* [slot] */, *item_empty = q_full + 16 /* [slot] */,
           *drain = q_full + 18 /* [tile] */, *turn = q_full + 20 /* [tile] */, *looked = q_full + 22 /* ring */;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(looked + ST);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* has_bad = abort_flag + 1;      // [slot]
  ApItem* items = reinterpret_cast<ApItem*>(sm + Sh::OFF_ITEM);
  uint32_t* bad = reinterpret_cast<uint32_t*>(sm + Sh::OFF_BAD);      // [slot][D]
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 3);
      mbar_init(smem_u32(looked + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(q_full + i), 1);
      mbar_init(smem_u32(q_empty + i), 1);
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(p_full + 2 * i), AP_SOFT / 2);
      mbar_init(smem_u32(p_full + 2 * i + 1), AP_SOFT / 2);
      mbar_init(smem_u32(o_done + i), 1);
      mbar_init(smem_u32(o_free + i), AP_SOFT / 2);
      mbar_init(smem_u32(turn + i), 1);
      mbar_init(smem_u32(item_full + i), 1);
      mbar_init(smem_u32(item_empty + i), AP_SOFT + 3);
      mbar_init(smem_u32(drain + i), 1);
      has_bad[i] = 0;
    }
    *abort_flag = 0;
    fence_mbar_init();
    mbar_arrive(smem_u32(turn));      // tile 0 begins
  }
  if (warp == AP_SOFT + 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PDL_ENTRY();

  if (warp < AP_SOFT) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // a warp has 16 rows of its tile, of its own quarter of the TMEM lanes: threads 4 r .. 4 r + 3 rows r and r + 8
    const int mt = warp >> 3, quad = threadIdx.x & 3, lane0 = (warp & 3) * 32 + (warp >> 2 & 1) * 16;
    const int qv = lane0 + ((threadIdx.x & 31) >> 2);
    const uint32_t tS = tmem + mt * AT + ((uint32_t)lane0 << 16), tO = tmem + 2 * AT + mt * D + ((uint32_t)lane0 << 16);
    int pos[2], g[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      pos[y] = (qv + 8 * y) / a.G;
      g[y] = qv + 8 * y - pos[y] * a.G;
    }
    uint32_t s_phase = 0, o_phase = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      ok = kv8_wait(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a.err);
      if (!ok) break;
      const ApItem& it = items[n & 1];
      if (it.h < 0) break;
      const int nt = it.n[mt], first = it.lim0 + mt * a.RB;      // the last key that the tile's first row sees
      float m2[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};      // l: this thread's part
      for (int j = 0; j < nt; ++j) {
        ok = kv8_wait(smem_u32(s_full + mt), s_phase, abort_flag, a.err);
        if (!ok) break;
        s_phase ^= 1;
        tc_fence_after();
        float s[64];
        frag_ld64(tS, s);
        tmem_wait_ld(s);
        frag_ld64(tS + 64, s + 32);
        const bool partial = j * AT + AT - 1 > first;      // some row of the tile does not see all of these keys
        float mx[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {      // (the second half arrives under the first one's maximum)
          if (hf) tmem_wait_ld(s + 32);
          if (partial) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int last = first + pos[y] - j * AT - hf * 64 - 2 * quad;
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                s[hf * 32 + 4 * c + 2 * y] = 8 * c <= last ? s[hf * 32 + 4 * c + 2 * y] : -INFINITY;
                s[hf * 32 + 4 * c + 2 * y + 1] = 8 * c + 1 <= last ? s[hf * 32 + 4 * c + 2 * y + 1] : -INFINITY;
              }
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float* x = s + hf * 32 + 2 * y;
            float x0 = hf ? max3(mx[y], x[0], x[1]) : fmaxf(x[0], x[1]), x1 = fmaxf(x[4], x[5]);
#pragma unroll
            for (int c = 2; c < 8; c += 2) {
              x0 = max3(x0, x[4 * c], x[4 * c + 1]);
              x1 = max3(x1, x[4 * c + 4], x[4 * c + 5]);
            }
            mx[y] = fmaxf(x0, x1);
          }
        }
        float corr[2] = {1.f, 1.f};
        bool raise = false;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          mx[y] = quad_max(mx[y]) * a.sl2;
          if (mx[y] > m2[y] + AP_LAZY) {
            corr[y] = pf_ex2(m2[y] - mx[y]);
            m2[y] = mx[y];
            l[y] *= corr[y];
            raise = true;
          }
        }
        // (this S came behind the product into O before it, so O is there)
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[8];
            asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=f"(o[0]), "=f"(o[1]), "=f"(o[2]), "=f"(o[3]), "=f"(o[4]), "=f"(o[5]), "=f"(o[6]), "=f"(o[7])
                         : "r"(tO + c));
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              asm volatile("" : "+f"(o[x]));
              o[x] *= corr[x >> 1 & 1];
            }
            asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(tO + c), "f"(o[0]),
                         "f"(o[1]), "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7])
                         : "memory");
          }
        }
        // One rounding of the reference for the whole row, then one of each difference: near the maximum, where weights
        // count, that is exact whatever the size of the scores.
        f32x2 nm[2], sum[2];
        const f32x2 s2 = two(a.sl2, a.sl2);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float ref = m2[y] == -INFINITY ? 0.f : m2[y];
          nm[y] = two(-ref, -ref);
          sum[y] = two(0.f, 0.f);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {      // 2 c': first row, 2 c' + 1: second row
            const float* x = s + hf * 32 + 2 * c;
            float2 e = one_by_one(fma2(two(x[0], x[1]), s2, nm[c & 1]));
            e.x = pf_ex2(e.x);
            e.y = pf_ex2(e.y);
            sum[c & 1] = add2(sum[c & 1], two(e.x, e.y));
            w[c] = bf16_pair(e.x, e.y);
          }
          frag_st_pairs(tS + hf * 32, w);
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(smem_u32(p_full + 2 * mt + hf));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float2 sums = one_by_one(sum[y]);
          l[y] += sums.x + sums.y;
        }
      }
      if (!ok) break;
      if (it.rows[mt] > 0) {
        float inv[2];
        __nv_bfloat16* dst[2];
        bool write[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
          l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
          const int row = it.row0 + mt * a.RB + pos[y], head = it.h * a.G + g[y];
          write[y] = pos[y] < it.rows[mt];      // (so pos < RB: not the vectors behind the last head)
          dst[y] = a.out + (long long)row * a.ldo + (long long)head * D;
          inv[y] = l[y] == 0.f ? 0.f : 1.f / l[y];
          if (write[y] && a.lse && quad == 0) {
            const float ref = m2[y] == -INFINITY ? 0.f : m2[y];
            a.lse[(long long)row * a.nq + head] = l[y] == 0.f ? -INFINITY : (ref + log2f(l[y])) * 0.693147180559945309f;
          }
        }
        if (nt == 0) {      // rows that see no key
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (write[y])
              for (int c = quad * 8; c < D; c += 32) *reinterpret_cast<uint4*>(dst[y] + c) = make_uint4(0, 0, 0, 0);
        } else {
          ok = kv8_wait(smem_u32(o_done + mt), o_phase, abort_flag, a.err);
          if (!ok) break;
          o_phase ^= 1;
          tc_fence_after();
          const bool poisoned = has_bad[n & 1] != 0;
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            float o[32];
            frag_ld64(tO + c, o);
            tmem_wait_ld(o);
            if (c + 64 == D) {      // O is read: the next item's products may begin
              tc_fence_before();
              warp_arrive(smem_u32(o_free + mt));
            }
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= inv[x >> 1 & 1];
            if (poisoned) {
              const uint32_t* from = bad + (n & 1) * D + c + 2 * quad;
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const uint32_t w = from[(x >> 2) * 8 + (x & 1)];
                const int i = mt * a.RB + pos[x >> 1 & 1];
                const bool nan = i >= (int)(w & 1023), up = i >= (int)((w >> 10) & 1023), down = i >= (int)((w >> 20) & 1023);
                if (nan || up || down) o[x] = nan || (up && down) ? __int_as_float(0x7fffffff) : up ? o[x] + INFINITY : o[x] - INFINITY;
              }
            }
            // a thread gets whole 16-byte pieces: the four of a row write 64 bytes in one go
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) w[z] = bf16_pair(o[(x * 4 + z) * 4 + 2 * y], o[(x * 4 + z) * 4 + 2 * y + 1]);
                quad_transpose(w, quad);
                if (write[y]) *reinterpret_cast<uint4*>(dst[y] + c + x * 32 + quad * 8) = make_uint4(w[0], w[1], w[2], w[3]);
              }
          }
        }
      }
      warp_arrive(smem_u32(item_empty + (n & 1)));
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == AP_SOFT) {
      // ---- items, TMA ----
      ApList list = ap_begin(a, blockIdx.x == 0);
      const uint32_t qbytes = (uint32_t)(a.RB * a.G * 128);
      int used[2] = {0, 0}, s = 0;      // tiles of Q and stages of the ring so far
      bool ok = true;
      // K or V tile j into the ring's next stage
      auto load = [&](const CUtensorMap* map, const ApItem& it, int j) {
        const int st = s % ST;
        if (s >= ST && !kv8_wait_all(smem_u32(empty + st), (uint32_t)((s / ST - 1) & 1), abort_flag, a.err)) return false;
        if (elect_one()) {
          mbar_expect_tx(smem_u32(full + st), Sh::OP);
          for (int x = 0; x < Sh::HALVES; ++x)
            tma_load_3d(smem_u32(sm + Sh::OFF_RING + st * Sh::OP + x * Sh::HALF), map, x * 64, it.h, it.k0 + j * AT,
                        smem_u32(full + st));
        }
        __syncwarp();
        ++s;
        return true;
      };
      auto load_q = [&](const ApItem& it, int t) {
        if (used[t] && !kv8_wait_all(smem_u32(q_empty + t), (uint32_t)((used[t] - 1) & 1), abort_flag, a.err)) return false;
        if (elect_one()) {
          mbar_expect_tx(smem_u32(q_full + t), Sh::HALVES * qbytes);
          for (int x = 0; x < Sh::HALVES; ++x)
            tma_load_3d(smem_u32(sm + t * Sh::OP + x * Sh::HALF), &tmQ, x * 64, it.h * a.G, it.row0 + t * a.RB,
                        smem_u32(q_full + t));
        }
        __syncwarp();
        ++used[t];
        return true;
      };
      for (int n = 0; ok; ++n) {
        // to and fro over the CTAs: who takes the largest of one round takes the smallest of the next
        const int turn = n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
        const ApItem it = ap_item(a, list, turn + (long long)n * gridDim.x);
        if (n >= 2) ok = kv8_wait_all(smem_u32(item_empty + (n & 1)), (uint32_t)(((n >> 1) - 1) & 1), abort_flag, a.err);
        if (!ok) break;
        if (elect_one()) {
          items[n & 1] = it;
          has_bad[n & 1] = 0;
          mbar_arrive(smem_u32(item_full + (n & 1)));
        }
        __syncwarp();
        if (it.h < 0) break;
        const int nt = max(it.n[0], it.n[1]);
        if (nt == 0) continue;
        if (it.n[0]) ok = load_q(it, 0);
        ok = ok && load(&tmK, it, 0);
        if (it.n[1]) ok = ok && load_q(it, 1);
        for (int j = 0; ok && j < nt; ++j) {
          ok = load(&tmV, it, j);
          if (j + 1 < nt) ok = ok && load(&tmK, it, j + 1);
        }
      }
      if (*abort_flag) {      // copies in flight land before the CTA leaves: the last ones of the ring and of Q
        for (int t = 0; t < 2; ++t)
          if (used[t]) kv8_wait_all(smem_u32(q_full + t), (uint32_t)((used[t] - 1) & 1), abort_flag, a.err, false);
        for (int x = max(0, s - ST); x < s; ++x)
          kv8_wait_all(smem_u32(full + x % ST), (uint32_t)((x / ST) & 1), abort_flag, a.err, false);
      }
    } else if (warp < AP_SOFT + 3) {
      // ---- MMA: one warp a query tile ----
      constexpr uint32_t IS = pf_idesc(AT, false), IO = pf_idesc(D, true);
      const int mt = warp - AP_SOFT - 1;
      const uint32_t tS = tmem + mt * AT, tO = tmem + 2 * AT + mt * D;
      // operand descriptors; an offset of n bytes adds n >> 4
      const uint64_t dq = sdesc_sw128(smem_u32(sm + mt * Sh::OP)), dk = sdesc_sw128(smem_u32(sm + Sh::OFF_RING)),
                     dv = pf_desc_mn(smem_u32(sm + Sh::OFF_RING), Sh::HALF);
      int s = 0, used = 0;
      uint32_t p_phase = 0, t_phase = 0;
      bool ok = true;
      auto wait_stage = [&](int x) { return kv8_wait_all(smem_u32(full + x % ST), (uint32_t)((x / ST) & 1), abort_flag, a.err); };
      // (behind wait_stage: warp 19 has then passed the stage's use before, so this phase is the current one)
      auto wait_looked = [&](int x) { return kv8_wait_all(smem_u32(looked + x % ST), (uint32_t)((x / ST) & 1), abort_flag, a.err); };
      auto issue_s = [&](int x, bool last) {      // by one lane
        const uint64_t k = dk + ((uint64_t)(x % ST) * Sh::OP >> 4);
#pragma unroll
        for (int y = 0; y < D / 16; ++y) {
          const int at = ((y >> 2) * Sh::HALF + (y & 3) * 32) >> 4;
          tc_mma_bf16(tS, dq + at, k + at, IS, y ? 1u : 0u);
        }
        tc_commit(smem_u32(s_full + mt));
        tc_commit(smem_u32(empty + x % ST));
        if (last) tc_commit(smem_u32(q_empty + mt));
      };
      auto issue_o = [&](int x, int half, bool first) {      // by one lane
        const uint64_t v = dv + ((uint64_t)(x % ST) * Sh::OP >> 4);
#pragma unroll
        for (int y = 0; y < 4; ++y)
          mma_ts(tO, tS + (half * 4 + y) * 8, v + ((half * 4 + y) * 2048 >> 4), IO, first && !half && !y ? 0u : 1u);
      };
      for (int n = 0; ok; ++n) {
        ok = kv8_wait_all(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a.err);
        if (!ok) break;
        const ApItem it = items[n & 1];
        if (it.h < 0) break;
        const int mine = it.n[mt], nt = max(it.n[0], it.n[1]);
        if (mine) {
          ok = kv8_wait_all(smem_u32(q_full + mt), (uint32_t)(used & 1), abort_flag, a.err) && wait_stage(s);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) issue_s(s, mine == 1);
          __syncwarp();
        }
        for (int j = 0; ok && j < nt; ++j, s += 2) {      // stages s: K of this tile, s + 1: V
          int seen;
          const bool partial = ap_partial(it, a.RB, j, seen);
          if (j >= mine) {      // the other tile's keys alone
            ok = wait_stage(s) && wait_stage(s + 1) && kv8_wait_all(smem_u32(turn + mt), t_phase, abort_flag, a.err);
            t_phase ^= 1;
            if (!ok) break;
            if (elect_one()) {
              mbar_arrive(smem_u32(turn + (mt ^ 1)));
              mbar_arrive(smem_u32(empty + s % ST));
              mbar_arrive(smem_u32(empty + (s + 1) % ST));
            }
            __syncwarp();
            continue;
          }
          const bool next = j + 1 < mine;
          ok = wait_stage(s + 1);
          if (ok && partial) ok = wait_looked(s + 1);
          if (ok && next) ok = wait_stage(s + 2);
          if (ok && j == 0 && used) ok = kv8_wait_all(smem_u32(o_free + mt), (uint32_t)((used - 1) & 1), abort_flag, a.err);
          ok = ok && kv8_wait_all(smem_u32(p_full + 2 * mt), p_phase, abort_flag, a.err) &&
               kv8_wait_all(smem_u32(turn + mt), t_phase, abort_flag, a.err);
          t_phase ^= 1;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) issue_o(s + 1, 0, j == 0);
          __syncwarp();
          ok = kv8_wait_all(smem_u32(p_full + 2 * mt + 1), p_phase, abort_flag, a.err);
          p_phase ^= 1;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_o(s + 1, 1, false);
            tc_commit(smem_u32(empty + (s + 1) % ST));
            if (next) issue_s(s + 2, j + 2 == mine);
            else tc_commit(smem_u32(o_done + mt));
            mbar_arrive(smem_u32(turn + (mt ^ 1)));
          }
          __syncwarp();
        }
        if (mine) ++used;
        if (ok && elect_one()) mbar_arrive(smem_u32(item_empty + (n & 1)));
        __syncwarp();
      }
      if (!ok) {      // products in flight end before the CTA frees its TMEM
        if (elect_one()) tc_commit(smem_u32(drain + mt));
        __syncwarp();
        kv8_wait_all(smem_u32(drain + mt), 0, abort_flag, a.err, false);
      }
    } else {
      // ---- value tiles that some rows see only in part ----
      int s = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        ok = kv8_wait_all(smem_u32(item_full + (n & 1)), (uint32_t)((n >> 1) & 1), abort_flag, a.err);
        if (!ok) break;
        const ApItem it = items[n & 1];
        if (it.h < 0) break;
        const int nt = max(it.n[0], it.n[1]);
        bool found = false;
        for (int j = 0; ok && j < nt; ++j) {
          // every stage is waited for and given back, so that this warp is never a turn of the ring behind
          for (int y = 0; ok && y < 2; ++y, ++s) {
            ok = kv8_wait_all(smem_u32(full + s % ST), (uint32_t)((s / ST) & 1), abort_flag, a.err);
            int seen;
            if (ok && y == 1 && ap_partial(it, a.RB, j, seen)) {
              const bool here = ap_clean<D>(sm + Sh::OFF_RING + (s % ST) * Sh::OP, max(0, seen + 1 - j * AT), j * AT, it.lim0,
                                            bad + (n & 1) * D, !found);
              found |= here;
              if (here) {
                if (elect_one()) has_bad[n & 1] = 1;
                fence_async_shared();
              }
              __syncwarp();
            }
            if (ok && elect_one()) {
              mbar_arrive(smem_u32(looked + s % ST));
              mbar_arrive(smem_u32(empty + s % ST));
            }
            __syncwarp();
          }
        }
        if (ok && elect_one()) mbar_arrive(smem_u32(item_empty + (n & 1)));
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == AP_SOFT + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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

template <int D>
cudaError_t launch_prompt(cudaStream_t st, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const ApArgs& p, int grid) {
  static_assert(ApShape<D>::BYTES <= 227 * 1024, "shared memory of a CTA");
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(prompt_k<D>), ApShape<D>::BYTES);
  if (e != cudaSuccess) return e;
  return launch_k(prompt_k<D>, dim3(grid), dim3(AP_THREADS), ApShape<D>::BYTES, st, q, k, v, p);
}

}  // namespace

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
  const int grid = (int)(most < sms ? most : sms);
  CUtensorMap q, k, v;
  // without keys K and V are not read; their maps still need memory
  const bool none = a.Rk == 0;
  if (!ap_map(&q, a.q, a.d, a.nq, a.R, a.ldq, p.G, p.RB) ||
      !ap_map(&k, none ? a.q : a.k, a.d, none ? a.nq : a.nkv, none ? a.R : a.Rk, none ? a.ldq : a.ldk, 1, AT) ||
      !ap_map(&v, none ? a.q : a.v, a.d, none ? a.nq : a.nkv, none ? a.R : a.Rk, none ? a.ldq : a.ldv, 1, AT))
    return -4;
  const cudaError_t e = a.d == 128 ? launch_prompt<128>(st, q, k, v, p, grid) : launch_prompt<64>(st, q, k, v, p, grid);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return -4;
  }
  return 0;
}

}  // namespace eagle
