// Attention over the 8-bit KV cache, behind an optional bf16 prefix that all rows share.
//
//   o = sum_s p_s v_s / sum_s p_s,  p_s = 2^(x_s - m),  x_s = log2(e) scale q.k_s,  m near the maximum,
// over the prefix and the slots that the row sees: one softmax, in one pass over the keys.
//
// Own slots (kv8_attn_k). A decoding step or a verify pass has few query vectors (rows x query heads of a KV
// head) and many keys, so the keys are the long side of both products, on mma.sync m16n8k16 (fp16, fp32 sums):
//   S^T [16 keys x 8 query vectors] = K Q^T,   O^T [16 dims x 8 query vectors] += V^T P^T.
// With the query vectors on the 8-wide side four of them cost half an instruction, where a 128-row tcgen05 tile
// would be 3% full; and both operands that come from the cache are A fragments, which a warp converts from e4m3
// right after ldmatrix (fp16 holds every code exactly; cvt runs at 128 codes a clock and SM against the 23 bytes a
// clock that HBM delivers). tcgen05 would need the fp16 tiles back in shared memory: 64 KB written and
// read again for each 32 KB of codes, as much time as the load itself.
//   - A key's exponent multiplies its score, a value's exponent its weight: the codes are never scaled.
//   - q is scaled by a power of two into fp16's range (exact down to 2^-38 of its largest entry).
//   - Weights enter the value product as fp16 (2^-11), scaled by 2^(e_s - E), E the warp's running
//     reference exponent; a tile whose exponents span more than fp16 bears is taken in several passes.
//   - The maximum is raised only when a score passes it by 2^8: fp16 holds weights up to 2^16, and most tiles
//     then need no reduction across lanes and no rescaling of O. Each column decides for itself.
// Work is split over CTAs by tiles of 32 keys: CTA c takes tiles [c W / G, (c + 1) W / G) of all (sequence, head)
// items laid end to end, lengths read on the device, so ragged batches and one long sequence balance alike. An
// item inside one CTA's range is finished there; the pieces of an item cut by range ends (at most two a
// CTA) go to scratch as (o, m, l) and a second launch joins them in order. A producer warp streams the tiles (TMA,
// 128- or 64-byte swizzle) through a ring that runs on across items.
#include "kv8.cuh"
#include "kernels.h"

#include <algorithm>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

namespace eagle {
namespace {

constexpr int TK = 32;            // keys a tile
constexpr int MAX_QV = 128;       // query vectors a block of rows
constexpr int MAX_GROUPS = 512;   // row blocks a launch (more: several launches)
constexpr int MAX_CTAS = 384;     // grid limit that the scratch is sized for
constexpr float LAZY = 8.f;       // how far (log2) a score may pass the reference maximum
constexpr int E_UP = 4, E_DOWN = 12;   // exponents a tile may have around the reference, E_SPAN within one pass
constexpr int E_SPAN = 14;

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
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^n, 0 below the normal range.
__device__ __forceinline__ float pow2i(int n) { return n < -126 ? 0.f : __int_as_float((min(n, 127) + 127) << 23); }

// How a call's rows are cut and its tiles shared out: the same numbers in both kernels and the scratch size.
struct Plan {
  int G, RB, nb, QV;      // query heads a KV head; rows a block; blocks a sequence; query vectors a block
  int groups;             // row blocks of this launch, from block g0 on
  int g0;
  int grid, min_tiles;    // CTAs at most; tiles a CTA at least
  int qv_pad;             // query vectors of a partial
  float* part_o;          // [2 grid][qv_pad][D]
  float* part_ml;         // [2 grid][qv_pad][2]
  int* pref;              // [groups + 1] tiles a head before each row block (written by CTA 0)
  const float *pp_o, *pp_ml;   // prefix partials [n_prefix][R * nq][D], [..][2]
  int n_prefix;
};

__device__ __forceinline__ int active_ctas(const Plan& p, long long W) {
  return (int)max(1ll, min((long long)p.grid, W / p.min_tiles));
}
__device__ __forceinline__ long long range_start(long long c, long long W, int G) { return c * W / G; }
__device__ __forceinline__ int cta_of(long long u, long long W, int G) { return (int)(((u + 1) * G - 1) / W); }

// Rows of a block, its sequence (that of the first row that is not padding among the sequence's rows) and the
// first slot past everything that its rows see. Run by one warp; every lane gets the values.
struct Group {
  int r0, r1, seq, limit;
};
__device__ __forceinline__ Group group_of(const Kv8Attn& a, const Plan& p, int gi, bool latch) {
  const int lane = threadIdx.x & 31;
  Group o;
  const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) % p.nb;
  const int s0 = sidx * a.rows_per_seq, s1 = min(s0 + a.rows_per_seq, a.R);
  o.r0 = s0 + rb * p.RB;
  o.r1 = min(o.r0 + p.RB, s1);
  o.seq = -1;
  o.limit = 0;
  if (o.r0 >= o.r1) return o;
  for (int r = s0; r < s1 && o.seq < 0; r += 32) {
    const int s = r + lane < s1 ? a.row_seq[r + lane] : -1;
    const unsigned any = __ballot_sync(0xffffffffu, s >= 0);
    if (any) o.seq = __shfl_sync(0xffffffffu, s, __ffs(any) - 1);
  }
  if (o.seq < 0) return o;
  bool bad = o.seq >= a.c.max_batch;
  if (bad) {
    o.seq = -1;
  } else {
    int lim = 0;
    const int ctx = a.mode == 1 ? a.ctx_len[o.seq] : 0;
    for (int r = o.r0 + lane; r < o.r1; r += 32) {
      if (a.row_seq[r] != o.seq) {
        bad = bad || a.row_seq[r] >= 0;
        continue;
      }
      if (a.mode == 0) {
        lim = max(lim, min(a.row_slot[r], INT32_MAX - 1) + 1);
      } else {
        int top = ctx;
        for (int w = (a.tree_T - 1) >> 6; w >= 0; --w) {
          uint64_t m = a.mask[(size_t)r * a.mask_words + w];
          if (w == (a.tree_T - 1) >> 6 && (a.tree_T & 63)) m &= (1ull << (a.tree_T & 63)) - 1;
          if (m) {
            top = (int)min((long long)INT32_MAX, (long long)ctx + w * 64 + 64 - __clzll((long long)m));
            break;
          }
        }
        lim = max(lim, top);
        bad = bad || ctx < 0;
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) lim = max(lim, __shfl_xor_sync(0xffffffffu, lim, d));
    bad = bad || lim > a.c.cap;
    o.limit = min(lim, a.c.cap);
  }
  if (latch && __any_sync(0xffffffffu, bad) && lane == 0) latch_error(a.err, DEVERR_BOUNDS);
  return o;
}

// out (or partial) values of 8 dims: joined with the prefix's partials.
__device__ __forceinline__ void join_prefix(const Plan& p, size_t at, size_t stride, int D, int c, float& M, float& L, float* o) {
  float top = M;
  for (int s = 0; s < p.n_prefix; ++s) top = fmaxf(top, p.pp_ml[(s * stride + at) * 2]);
  const float base = top == -INFINITY ? 0.f : top;
  const float f = ex2(M - base);
  L *= f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] *= f;
  for (int s = 0; s < p.n_prefix; ++s) {
    const float w = ex2(p.pp_ml[(s * stride + at) * 2] - base);
    L = fmaf(p.pp_ml[(s * stride + at) * 2 + 1], w, L);
    const float4* x = reinterpret_cast<const float4*>(p.pp_o + (s * stride + at) * D + c);
    const float4 a = x[0], b = x[1];
    o[0] = fmaf(a.x, w, o[0]); o[1] = fmaf(a.y, w, o[1]); o[2] = fmaf(a.z, w, o[2]); o[3] = fmaf(a.w, w, o[3]);
    o[4] = fmaf(b.x, w, o[4]); o[5] = fmaf(b.y, w, o[5]); o[6] = fmaf(b.z, w, o[6]); o[7] = fmaf(b.w, w, o[7]);
  }
  M = top;
}

// 8 finished values of one query vector; nothing seen, or a row that is padding or invalid: zeros.
__device__ __forceinline__ void store8(const Kv8Attn& a, size_t at, int D, int c, bool live, float L, const float* o) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool none = !live || L == 0.f;
    const __nv_bfloat162 h = __floats2bfloat162_rn(none ? 0.f : o[2 * i] / L, none ? 0.f : o[2 * i + 1] / L);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + at * D + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Shared memory of one configuration: D dims; NT query tiles (of 8) a warp, WN warps side by side over the query
// tiles, WK groups of them over the keys; NS tiles in the ring.
template <int D, int NT, int WN, int WK, int NS>
struct Shape {
  static_assert(NS < 32, "a producer lane has at most one tile in flight");
  static constexpr int QV = 8 * NT * WN, NW = WN * WK;
  // Eight consumer warps that hold wide accumulators: a producer warpgroup of its own gives its registers to them
  // (168 a thread at launch; 2 x 128 x 232 + 128 x 40 = 384 x 168).
  static constexpr bool SPLIT_REGS = NW == 8;
  static constexpr int THREADS = (NW + (SPLIT_REGS ? 4 : 1)) * 32;
  static constexpr int TILE = 2 * TK * D;                 // K codes, V codes
  static constexpr int Q_LD = 2 * D + 32;                 // bytes a query row: 8-byte reads without bank conflicts
  static constexpr int O_LD = D + 4;
  static constexpr int OFF_EXP = NS * TILE;               // [NS][2][TK] exponent bytes
  static constexpr int OFF_Q = OFF_EXP + NS * 2 * TK;
  static constexpr int OFF_O = OFF_Q + QV * Q_LD;
  static constexpr int OFF_COL = OFF_O + QV * O_LD * 4;   // qf, slot limit of each query vector
  static constexpr int OFF_MLE = OFF_COL + QV * 8;        // m, l of each key group
  static constexpr int OFF_MASK = OFF_MLE + WK * QV * 8;
  static constexpr int OFF_BAR = OFF_MASK + MAX_QV * 32;
  static constexpr int OFF_GROUP = OFF_BAR + NS * 16 + 64;
  static int bytes(int groups) { return 1024 + OFF_GROUP + (3 * groups + 1) * 4; }
};

template <int D, int NT, int WN, int WK, int NS, int CTAS>
__global__ void __launch_bounds__(Shape<D, NT, WN, WK, NS>::THREADS, CTAS)
    kv8_attn_k(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Attn a,
               const Plan p) {
  using Sh = Shape<D, NT, WN, WK, NS>;
  constexpr int NW = Sh::NW, NC = NW * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + Sh::OFF_BAR);
  uint64_t* empty = full + NS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + NS);
  int* s_fullvis = reinterpret_cast<int*>(empty + NS) + 1;
  int* s_pref = reinterpret_cast<int*>(sm + Sh::OFF_GROUP);
  int* s_lim = s_pref + p.groups + 1;
  int* s_seq = s_lim + p.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkv = a.c.nkv;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), WN);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  PDL_ENTRY();
  for (int gi = warp; gi < p.groups; gi += Sh::THREADS / 32) {
    const Group gr = group_of(a, p, gi, blockIdx.x == 0);
    if (lane == 0) {
      s_lim[gi] = gr.limit;
      s_seq[gi] = gr.seq;
      s_pref[gi + 1] = gr.r0 < gr.r1 ? max(1, (gr.limit + TK - 1) / TK) : 0;
    }
  }
  __syncthreads();
  if (warp == 0) {   // inclusive sums
    int run = 0;
    for (int b = 0; b < p.groups; b += 32) {
      int v = b + lane < p.groups ? s_pref[b + lane + 1] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
      }
      if (b + lane < p.groups) s_pref[b + lane + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) s_pref[0] = 0;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.groups; i += blockDim.x) p.pref[i] = s_pref[i];
  const long long W = (long long)s_pref[p.groups] * nkv;
  const int Gd = active_ctas(p, W);
  if ((int)blockIdx.x >= Gd) return;
  const long long w0 = range_start(blockIdx.x, W, Gd), w1 = range_start(blockIdx.x + 1, W, Gd);
  const int n = (int)(w1 - w0);

  // the item (row block, head) that holds flat tile w
  auto find = [&](long long w, int& gi, int& h, int& t) {
    int lo = 0, hi = p.groups;   // the last group with pref * nkv <= w
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)s_pref[mid] * nkv <= w) lo = mid;
      else hi = mid;
    }
    gi = lo;
    const int nt = s_pref[lo + 1] - s_pref[lo], rem = (int)(w - (long long)s_pref[lo] * nkv);
    h = rem / nt;
    t = rem - h * nt;
  };

  if (warp >= NW) {
    if constexpr (Sh::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp > NW) return;
    // producer: lane j looks after tiles j, j + 32, ... of the range, so that block-table reads of 32 tiles overlap
    const int box = a.c.table ? min(TK, 1 << a.c.block_log2) : TK, nbox = TK / box;
    const uint64_t pol = l2_policy_evict_first();
    int last = -1;
    for (int b = 0; b < n; b += 32) {
      const int i = b + lane;
      int live = 0, t = 0;
      long long vec[2] = {0, 0};
      if (i < n) {
        int gi, h;
        find(w0 + i, gi, h, t);
        live = s_lim[gi] - t * TK;
        const int seq = s_seq[gi];
        for (int x = 0; x < nbox && x * box < live; ++x) {
          vec[x] = kv8_vec(a.c, seq, h, t * TK + x * box);
          if (vec[x] < 0) {   // not assigned: what is read instead is unspecified
            latch_error(a.err, DEVERR_BOUNDS);
            vec[x] = 0;
          }
        }
      }
      for (int j = 0; j < 32 && b + j < n; ++j) {
        if (lane == j) {
          const int st = i % NS;
          const uint32_t bar = smem_u32(full + st);
          bool ok = *abort_flag == 0;
          if (ok && i >= NS) ok = mbar_wait(smem_u32(empty + st), (uint32_t)((i / NS - 1) & 1), abort_flag, a.err);
          if (ok) {
            last = i;
            if (live <= 0) {
              mbar_arrive(bar);
            } else {
              const int ne = a.c.table ? box : min(TK, a.c.cap - t * TK);   // exponent bytes a box (16 or 32)
              int boxes = 0;
              for (int x = 0; x < nbox; ++x) boxes += x * box < live;
              mbar_expect_tx(bar, (uint32_t)(boxes * 2 * (box * D + ne)));
              for (int x = 0; x < boxes; ++x) {
                const uint32_t k = smem_u32(sm + st * Sh::TILE + x * box * D), v = k + TK * D;
                const uint32_t ke = smem_u32(sm + Sh::OFF_EXP + st * 2 * TK + x * box), ve = ke + TK;
                tma_load_2d(k, &tmK, 0, (int)vec[x], bar, pol);
                tma_load_2d(v, &tmV, 0, (int)vec[x], bar, pol);
                bulk_load(ke, a.c.ke + vec[x], (uint32_t)ne, bar);
                bulk_load(ve, a.c.ve + vec[x], (uint32_t)ne, bar);
              }
            }
          }
        }
        __syncwarp();
      }
    }
    // after a timeout the tiles in flight land before the CTA leaves: a tile in flight is the last one of its lane (the
    // ring has fewer than 32 tiles)
    if (*abort_flag && last >= 0) mbar_wait(smem_u32(full + last % NS), (uint32_t)((last / NS) & 1), abort_flag, a.err, false);
  } else {
    if constexpr (Sh::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int kw = warp / WN, nw = warp % WN;
    const int g = lane >> 2, t4 = lane & 3;
    float* s_qf = reinterpret_cast<float*>(sm + Sh::OFF_COL);
    int* s_klim = reinterpret_cast<int*>(s_qf + Sh::QV);
    float* s_m = reinterpret_cast<float*>(sm + Sh::OFF_MLE);
    float* s_l = s_m + WK * Sh::QV;
    float* s_o = reinterpret_cast<float*>(sm + Sh::OFF_O);
    uint64_t* s_mask = reinterpret_cast<uint64_t*>(sm + Sh::OFF_MASK);
    const float sl2 = a.scale * 1.4426950408889634f;
    int i = 0;   // tiles of the range that are behind
    while (i < n) {
      int gi, h, t0;
      find(w0 + i, gi, h, t0);
      const int nt = s_pref[gi + 1] - s_pref[gi];
      const int t1 = min(nt, t0 + n - i);
      const int seq = s_seq[gi], limit = s_lim[gi];
      const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) % p.nb;
      const int r0 = sidx * a.rows_per_seq + rb * p.RB;
      const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
      const int nqv = (r1 - r0) * p.G;
      const int ctx = a.mode == 1 && seq >= 0 ? a.ctx_len[seq] : 0;

      // the rows: query vectors as fp16 of q 2^-e, what they see
      if (threadIdx.x == 0) *s_fullvis = INT32_MAX;
      if (a.mode == 1)
        for (int x = threadIdx.x; x < (r1 - r0) * 4; x += NC) {
          const int r = r0 + x / 4, w = x & 3;
          uint64_t m = 0;
          if (seq >= 0 && a.row_seq[r] == seq && w * 64 < a.tree_T) {
            m = a.mask[(size_t)r * a.mask_words + w];
            if (w == (a.tree_T - 1) >> 6 && (a.tree_T & 63)) m &= (1ull << (a.tree_T & 63)) - 1;
          }
          s_mask[x] = m;
        }
      for (int x = warp; x < Sh::QV; x += NW) {
        const int row = r0 + x / p.G, head = h * p.G + x % p.G;
        const bool live = x < nqv && seq >= 0 && a.row_seq[row] == seq;
        constexpr int E = D / 32;
        float f[E];
        float top = 0.f;
        bool fine = true;
        if (live) {
          const __nv_bfloat16* q = (const __nv_bfloat16*)a.q + ((size_t)row * a.nq + head) * D + lane * E;
#pragma unroll
          for (int k = 0; k < E; k += 2) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(q + k));
            f[k] = v.x;
            f[k + 1] = v.y;
          }
        } else {
#pragma unroll
          for (int k = 0; k < E; ++k) f[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
          top = fmaxf(top, fabsf(f[k]));
          fine = fine && isfinite(f[k]);
        }
        top = warp_max(top);
        fine = __all_sync(0xffffffffu, fine);
        // largest entry into [2^13, 2^14); a vector with an entry that is not finite gives NaN
        int e = top > 0.f && fine ? max((int)(__float_as_uint(top) >> 23) - 127, -126) - 13 : 0;
        const float up = pow2i(-e / 2), up2 = pow2i(-e - (-e / 2));   // two factors: -e can pass 127
        uint32_t w[E / 2];
#pragma unroll
        for (int k = 0; k < E / 2; ++k)
          w[k] = fine ? half2_of(f[2 * k] * up * up2, f[2 * k + 1] * up * up2) : 0x7fff7fffu;
        uint8_t* dst = sm + Sh::OFF_Q + x * Sh::Q_LD + lane * E * 2;
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(dst) = w[0];
        if (lane == 0) {
          s_qf[x] = sl2 * pow2i(e / 2) * pow2i(e - e / 2);
          int lim = 0;
          if (live) lim = a.mode == 1 ? ctx : min(a.row_slot[row], INT32_MAX - 1) + 1;
          s_klim[x] = max(0, min(lim, a.c.cap));
        }
      }
      named_bar_sync(1, NC);
      // keys below this are seen by every row that counts
      for (int x = threadIdx.x; x < nqv; x += NC)
        if (seq >= 0 && a.row_seq[r0 + x / p.G] == seq) atomicMin(s_fullvis, s_klim[x]);
      named_bar_sync(1, NC);
      const int fullvis = *s_fullvis;

      float O[D / 16][NT][4], m[NT][2], l[NT][2], qf[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) O[c][x][0] = O[c][x][1] = O[c][x][2] = O[c][x][3] = 0.f;
        const int col = (nw * NT + x) * 8 + 2 * t4;
        m[x][0] = m[x][1] = -INFINITY;
        l[x][0] = l[x][1] = 0.f;
        qf[x][0] = s_qf[col];
        qf[x][1] = s_qf[col + 1];
      }
      int E_run = 0;

      for (int t = t0; t < t1; ++t, ++i) {
        if (i % WK != kw) continue;
        const int st = i % NS;
        mbar_wait(smem_u32(full + st), (uint32_t)((i / NS) & 1), abort_flag, a.err);
        const int key0 = t * TK;
        if (key0 < limit && !*abort_flag) {
          const uint8_t* s_ke = sm + Sh::OFF_EXP + st * 2 * TK;
          const uint8_t* s_ve = s_ke + TK;
          const uint32_t kb = smem_u32(sm + st * Sh::TILE), vb = kb + TK * D;
          const bool masked = key0 + TK > fullvis;
          auto visible = [&](int key, int col) -> bool {
            if (key < s_klim[col]) return true;
            const int tt = key - ctx;
            if (a.mode != 1 || tt < 0 || tt >= 256 || col >= nqv || key >= limit) return false;
            return (s_mask[col / p.G * 4 + (tt >> 6)] >> (tt & 63)) & 1;
          };
          // keys that one of this warp's query vectors sees: bit = key in tile
          uint32_t seen = 0xffffffffu;
          uint32_t vis[2] = {0xffffffffu, 0xffffffffu};   // [key half of 16][..]: bits of this thread's scores
          if (masked) {
            seen = 0;
            vis[0] = vis[1] = 0;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                bool any = false;
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const bool v = visible(key0 + mt * 16 + hf * 8 + g, (nw * NT + x) * 8 + 2 * t4 + e);
                    vis[mt] |= (uint32_t)v << (x * 4 + hf * 2 + e);
                    any = any || v;
                  }
                const uint32_t bal = __ballot_sync(0xffffffffu, any);
#pragma unroll
                for (int r = 0; r < 8; ++r) seen |= (((bal >> (4 * r)) & 15u) ? 1u : 0u) << (mt * 16 + hf * 8 + r);
              }
          }
          // exponents of the values: the largest and smallest of the seen ones
          const int vbyte = s_ve[lane];
          const bool counts = ((seen >> lane) & 1u) && vbyte != KV8_BAD;
          int hi = (int)__reduce_max_sync(0xffffffffu, counts ? (uint32_t)vbyte : 0u);
          const int lo_all = (int)__reduce_min_sync(0xffffffffu, counts ? (uint32_t)vbyte : 255u);
          bool first = true;
          while (true) {
            const bool one = hi - lo_all <= E_SPAN;
            const int lo = one ? 0 : hi - E_SPAN;
            if (hi > E_run + E_UP || (one ? lo_all : lo) < E_run - E_DOWN) {
              const float f = pow2i(E_run - hi);   // O is zero before the first tile
              if (E_run)
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
#pragma unroll
                  for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[c][x][e] *= f;
              E_run = hi;
            }
            float s[2][NT][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int x = 0; x < NT; ++x) s[mt][x][0] = s[mt][x][1] = s[mt][x][2] = s[mt][x][3] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t r[4], a0[4], a1[4];
              const int row = (lane >> 3) * 8 + (lane & 7);
              const int ch = D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
              ldsm4(kb + row * D + ch * 16, r);
              a0[0] = e4m3x2_f16x2(r[0]); a0[1] = e4m3x2_f16x2(r[1]);
              a0[2] = e4m3x2_f16x2(r[0] >> 16); a0[3] = e4m3x2_f16x2(r[1] >> 16);
              a1[0] = e4m3x2_f16x2(r[2]); a1[1] = e4m3x2_f16x2(r[3]);
              a1[2] = e4m3x2_f16x2(r[2] >> 16); a1[3] = e4m3x2_f16x2(r[3] >> 16);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                const uint2 b = *reinterpret_cast<const uint2*>(sm + Sh::OFF_Q + ((nw * NT + x) * 8 + g) * Sh::Q_LD +
                                                                c * 32 + t4 * 8);
                mma_f16(s[0][x], a0, b.x, b.y);
                mma_f16(s[1][x], a1, b.x, b.y);
              }
            }
            float mx[NT][2];
#pragma unroll
            for (int x = 0; x < NT; ++x) mx[x][0] = mx[x][1] = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const float f0 = kv8_pow2(s_ke[mt * 16 + g]), f1 = kv8_pow2(s_ke[mt * 16 + 8 + g]);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                // to log2 units here, not inside the subtraction below: a fused x - m would leave the rounding of a
                // huge m over, and a weight of 2^(that)
                s[mt][x][0] = s[mt][x][0] * f0 * qf[x][0]; s[mt][x][1] = s[mt][x][1] * f0 * qf[x][1];
                s[mt][x][2] = s[mt][x][2] * f1 * qf[x][0]; s[mt][x][3] = s[mt][x][3] * f1 * qf[x][1];
                if (masked)
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    if (!((vis[mt] >> (x * 4 + e)) & 1u)) s[mt][x][e] = -INFINITY;
                mx[x][0] = fmaxf(mx[x][0], fmaxf(s[mt][x][0], s[mt][x][2]));
                mx[x][1] = fmaxf(mx[x][1], fmaxf(s[mt][x][1], s[mt][x][3]));
              }
            }
            bool raise = false;
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) raise = raise || mx[x][e] > m[x][e] + LAZY;
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
              for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float v = mx[x][e];
                  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                  if (v > m[x][e] + LAZY) {
                    const float corr = ex2(m[x][e] - v);
                    m[x][e] = v;
                    l[x][e] *= corr;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                      O[c][x][e] *= corr;
                      O[c][x][2 + e] *= corr;
                    }
                  }
                }
            }
            // weights, then weights times 2^(exponent - E_run) as the B operand of the value product
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const int b0 = s_ve[mt * 16 + g], b1 = s_ve[mt * 16 + 8 + g];
              // not finite: NaN where seen; outside this pass's exponents, or seen by nobody: 0
              const float v0 = b0 == KV8_BAD ? kv8_pow2(b0) : (b0 >= lo && b0 <= hi ? pow2i(b0 - E_run) : 0.f);
              const float v1 = b1 == KV8_BAD ? kv8_pow2(b1) : (b1 >= lo && b1 <= hi ? pow2i(b1 - E_run) : 0.f);
#pragma unroll
              for (int x = 0; x < NT; ++x) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float base = m[x][e & 1] == -INFINITY ? 0.f : m[x][e & 1];
                  const float pr = ex2(s[mt][x][e] - base);
                  if (first) l[x][e & 1] += pr;
                  w[e] = pr * (e < 2 ? v0 : v1);
                  if (masked && !((vis[mt] >> (x * 4 + e)) & 1u)) w[e] = 0.f;
                }
                pb[mt][x][0] = transpose8(half2_of(w[0], w[1]));
                pb[mt][x][1] = transpose8(half2_of(w[2], w[3]));
              }
            }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;   // codes of keys that nobody sees are left out
              if (masked) {
                const uint32_t k = seen >> (mt * 16 + 2 * t4);
                z0 = ((k & 1u) ? 0xffffu : 0u) | ((k & 2u) ? 0xffff0000u : 0u);
                z1 = ((k & 256u) ? 0xffffu : 0u) | ((k & 512u) ? 0xffff0000u : 0u);
              }
#pragma unroll
              for (int c = 0; c < D / 16; c += 2) {
                uint32_t r[4], va[4], vc[4];
                const int row = mt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), cc = c + (lane >> 4);
                const int ch = D == 128 ? cc ^ (row & 7) : cc ^ ((row >> 1) & 3);
                ldsm4_t(vb + row * D + ch * 16, r);
                r[0] = __byte_perm(r[0] & z0, 0, 0x3120); r[1] = __byte_perm(r[1] & z1, 0, 0x3120);
                r[2] = __byte_perm(r[2] & z0, 0, 0x3120); r[3] = __byte_perm(r[3] & z1, 0, 0x3120);
                va[0] = e4m3x2_f16x2(r[0]); va[1] = e4m3x2_f16x2(r[0] >> 16);
                va[2] = e4m3x2_f16x2(r[1]); va[3] = e4m3x2_f16x2(r[1] >> 16);
                vc[0] = e4m3x2_f16x2(r[2]); vc[1] = e4m3x2_f16x2(r[2] >> 16);
                vc[2] = e4m3x2_f16x2(r[3]); vc[3] = e4m3x2_f16x2(r[3] >> 16);
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                  mma_f16(O[c][x], va, pb[mt][x][0], pb[mt][x][1]);
                  mma_f16(O[c + 1][x], vc, pb[mt][x][0], pb[mt][x][1]);
                }
              }
            }
            if (one) break;
            hi = (int)__reduce_max_sync(0xffffffffu, counts && vbyte < lo ? (uint32_t)vbyte : 0u);
            if (hi == 0) break;
            first = false;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(empty + st));
      }

      // join the key groups: sums in the order of the groups
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
            s_m[at] = m[x][e];
            s_l[at] = v;
          }
        }
      named_bar_sync(1, NC);
      const float unit = E_run ? pow2i(E_run - KV8_BIAS) : 1.f;
#pragma unroll 1
      for (int r = 0; r < WK; ++r) {
        if (r == kw) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int col = (nw * NT + x) * 8 + 2 * t4 + e;
              float top = s_m[col];
#pragma unroll
              for (int k = 1; k < WK; ++k) top = fmaxf(top, s_m[k * Sh::QV + col]);
              const float f = ex2(m[x][e] - (top == -INFINITY ? 0.f : top)) * unit;
              float* o = s_o + col * Sh::O_LD + 2 * g;
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
        const float4 u = *reinterpret_cast<const float4*>(s_o + col * Sh::O_LD + c);
        const float4 v = *reinterpret_cast<const float4*>(s_o + col * Sh::O_LD + c + 4);
        o[0] = u.x; o[1] = u.y; o[2] = u.z; o[3] = u.w; o[4] = v.x; o[5] = v.y; o[6] = v.z; o[7] = v.w;
        if (whole) {
          const int row = r0 + col / p.G;
          const size_t at = (size_t)row * a.nq + h * p.G + col % p.G;
          join_prefix(p, at, (size_t)a.R * a.nq, D, c, top, L, o);
          store8(a, at, D, c, seq >= 0 && a.row_seq[row] == seq, L, o);
        } else {
          const size_t q = (size_t)slot * p.qv_pad + col;
          *reinterpret_cast<float4*>(p.part_o + q * D + c) = u;
          *reinterpret_cast<float4*>(p.part_o + q * D + c + 4) = v;
          if (c == 0) {
            p.part_ml[2 * q] = top;
            p.part_ml[2 * q + 1] = L;
          }
        }
      }
    }
  }
}

// Joins the pieces of the items that range ends cut: CTA (c, y) takes the item that CTA c's range begins and does
// not finish, its query vectors from 32 y on; D / 8 threads a query vector, the pieces in order.
template <int D>
__global__ void __launch_bounds__(256) kv8_join_k(const Kv8Attn a, const Plan p) {
  PDL_ENTRY();
  const int nkv = a.c.nkv;
  const long long W = (long long)p.pref[p.groups] * nkv;
  const int Gd = active_ctas(p, W), c0 = blockIdx.x;
  if (c0 + 1 >= Gd) return;
  const long long w0 = range_start(c0, W, Gd), w1 = range_start(c0 + 1, W, Gd);
  int lo = 0, hi = p.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((long long)p.pref[mid] * nkv <= w1 - 1) lo = mid;
    else hi = mid;
  }
  const int nt = p.pref[lo + 1] - p.pref[lo];
  const int h = (int)((w1 - 1 - (long long)p.pref[lo] * nkv) / nt);
  const long long ts = (long long)p.pref[lo] * nkv + (long long)h * nt;
  if (ts < w0 || ts + nt <= w1) return;   // begun by an earlier CTA, or finished by this one
  const int c1 = cta_of(ts + nt - 1, W, Gd);
  const int sidx = (p.g0 + lo) / p.nb, rb = (p.g0 + lo) % p.nb;
  const int s0 = sidx * a.rows_per_seq, s1 = min(s0 + a.rows_per_seq, a.R);
  const int r0 = s0 + rb * p.RB, nqv = (min(r0 + p.RB, s1) - r0) * p.G;
  const int col = blockIdx.y * (256 / (D / 8)) + threadIdx.x / (D / 8), c = threadIdx.x % (D / 8) * 8;
  if (col >= nqv) return;
  int seq = -1;
  for (int r = s0; r < s1 && seq < 0; ++r) seq = a.row_seq[r];
  // piece 0 in slot 2 c0 + 1 (it holds the item's start), the others in slot 2 c
  auto at_of = [&](int k) { return (size_t)(k == c0 ? 2 * k + 1 : 2 * k) * p.qv_pad + col; };
  float top = -INFINITY, L = 0.f, o[8] = {};
  for (int k = c0; k <= c1; ++k) top = fmaxf(top, p.part_ml[2 * at_of(k)]);
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll 4
  for (int k = c0; k <= c1; ++k) {
    const size_t q = at_of(k);
    const float f = ex2(p.part_ml[2 * q] - base);
    L = fmaf(p.part_ml[2 * q + 1], f, L);
    const float4 u = *reinterpret_cast<const float4*>(p.part_o + q * D + c);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + q * D + c + 4);
    o[0] = fmaf(u.x, f, o[0]); o[1] = fmaf(u.y, f, o[1]); o[2] = fmaf(u.z, f, o[2]); o[3] = fmaf(u.w, f, o[3]);
    o[4] = fmaf(v.x, f, o[4]); o[5] = fmaf(v.y, f, o[5]); o[6] = fmaf(v.z, f, o[6]); o[7] = fmaf(v.w, f, o[7]);
  }
  const int row = r0 + col / p.G;
  const size_t at = (size_t)row * a.nq + h * p.G + col % p.G;
  join_prefix(p, at, (size_t)a.R * a.nq, D, c, top, L, o);
  store8(a, at, D, c, seq >= 0 && seq < a.c.max_batch && a.row_seq[row] == seq, L, o);
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
  p.G = nq / c.nkv;
  const int most = MAX_QV / p.G;
  p.nb = (rows_per_seq + most - 1) / most;
  p.RB = (rows_per_seq + p.nb - 1) / p.nb;
  p.QV = p.RB * p.G;
  p.qv_pad = (p.QV + 7) / 8 * 8;
}

size_t own_scratch(const Kv8& c, const Plan& p) {
  return al256((size_t)2 * MAX_CTAS * p.qv_pad * c.d * sizeof(float)) +
         al256((size_t)2 * MAX_CTAS * p.qv_pad * 2 * sizeof(float)) + al256((MAX_GROUPS + 1) * sizeof(int));
}

template <int D, int NT, int WN, int WK, int NS, int CTAS>
cudaError_t launch_own(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& mk, const CUtensorMap& mv) {
  using Sh = Shape<D, NT, WN, WK, NS>;
  const auto fn = kv8_attn_k<D, NT, WN, WK, NS, CTAS>;
  p.grid = std::min(MAX_CTAS, CTAS * device_sm_count());
  p.min_tiles = WK;
  const int smem = Sh::bytes(p.groups);
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  e = launch_k(fn, dim3(p.grid), dim3(Sh::THREADS), smem, st, mk, mv, a, p);
  if (e != cudaSuccess) return e;
  return launch_k(kv8_join_k<D>, dim3(p.grid, (p.QV + 256 / (D / 8) - 1) / (256 / (D / 8))), dim3(256), 0, st, a, p);
}

// The narrowest configuration that holds a block's query vectors: up to 16 in two small CTAs an SM (one's joins
// under the other's loads), more in one CTA whose warps share the query tiles.
template <int D>
cudaError_t launch_d(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& mk, const CUtensorMap& mv) {
  const int t = p.qv_pad / 8;
  if (t <= 1) return launch_own<D, 1, 1, 4, 11, 2>(st, a, p, mk, mv);
  if (t <= 2) return launch_own<D, 2, 1, 4, 10, 2>(st, a, p, mk, mv);
  if (t <= 4) return launch_own<D, 4, 1, 8, 20, 1>(st, a, p, mk, mv);
  if (t <= 6) return launch_own<D, 3, 2, 4, 18, 1>(st, a, p, mk, mv);
  if (t <= 8) return launch_own<D, 4, 2, 4, 16, 1>(st, a, p, mk, mv);
  if (t <= 12) return launch_own<D, 3, 4, 2, 12, 1>(st, a, p, mk, mv);
  return launch_own<D, 4, 4, 2, 10, 1>(st, a, p, mk, mv);
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
  s += al256((size_t)2 * MAX_CTAS * p.qv_pad * a.c.d * sizeof(float));
  p.part_ml = (float*)s;
  s += al256((size_t)2 * MAX_CTAS * p.qv_pad * 2 * sizeof(float));
  p.pref = (int*)s;
  if (a.P) {
    p.n_prefix = kv8_prefix_splits(a.c.nkv, a.R, a.nq, a.P);
    const size_t qv = (size_t)a.R * a.nq * p.n_prefix;
    float* o = (float*)(s + al256((MAX_GROUPS + 1) * sizeof(int)));
    float* ml = (float*)((uint8_t*)o + al256(qv * a.c.d * sizeof(float)));
    p.pp_o = o;
    p.pp_ml = ml;
    const int r = kv8_prefix(st, a, p.n_prefix, o, ml);
    if (r) return r;
  }
  const long long rows = a.c.table ? ((long long)a.c.n_blocks * a.c.nkv) << a.c.block_log2
                                   : (long long)a.c.max_batch * a.c.nkv * a.c.cap;
  const int box = a.c.table ? std::min(TK, 1 << a.c.block_log2) : TK;
  CUtensorMap mk, mv;
  if (!code_map(&mk, a.c.k, rows, a.c.d, box) || !code_map(&mv, a.c.v, rows, a.c.d, box)) return -4;
  const long long blocks = (((long long)a.R + a.rows_per_seq - 1) / a.rows_per_seq) * p.nb;
  if (blocks > 0x7fffffffll) return -1;
  for (long long g0 = 0; g0 < blocks; g0 += MAX_GROUPS) {
    p.g0 = (int)g0;
    p.groups = (int)std::min<long long>(MAX_GROUPS, blocks - g0);
    const cudaError_t e = a.c.d == 128 ? launch_d<128>(st, a, p, mk, mv) : launch_d<64>(st, a, p, mk, mv);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return -4;
    }
  }
  return 0;
}

}  // namespace eagle
