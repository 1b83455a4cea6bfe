// Attention of many query vectors over the 8-bit KV cache on the 5th-generation tensor cores (head_dim 128).
//
// A verify pass has tens of query vectors a KV head: per 128-key tile two products of a 128-row tile, which
// tcgen05 takes with the cache's e4m3 codes as they lie - one TMA copy from HBM to the operand, no conversion. The other
// operands are brought to 8 bits in parts that add up:
//   S = (Q_hi + Q_lo) K^T     q scaled by a power of two, each part e4m3: together 8 significant bits, as many as bf16
//                             has, down to 2^-11 of the vector's largest entry (below, a step of 2^-19 of it);
//   O += (P_1 + P_2 + P_3) V  the weight times its value's exponent in fp16, cut into e5m2 parts (its upper byte, the
//                             remainder's, the second remainder rounded): 9 significant bits, down to 2^-20 of the
//                             largest weight; 5 exponent bits, so that the long tail of a row with one strong key keeps
//                             its weight (e4m3 parts would flush it).
// kind::f8f6f4 runs at twice the fp16 rate, so the five products cost 8 x 66 + 12 x 76 clocks a tile (measured), as much as
// HBM takes to deliver its 33 KB; mma.sync took 3000 clocks for a quarter of the keys.
//
// One CTA an SM, 16 warps: two softmax warpgroups that take alternate key tiles of an item, each with S and O of its own in
// TMEM (one thread a query vector; S is overwritten by P), joined at the item's end; K and V producer warps (TMA); an MMA
// warp, which issues the next tile's S before it waits for this tile's P; five warps that prepare the next item's query
// vectors. Exponents: a key's multiplies its scores, a value's its weights, against a running reference E; a tile whose
// values' exponents span more than fp16 bears goes through the value product in several passes.
#include "kv8_split.cuh"
#include "kernels.h"
#include "tc_common.cuh"

#include <algorithm>
#include <cuda_fp16.h>

namespace eagle {
namespace {

constexpr int TT = 128;                 // keys a tile, query vectors a block, dims
constexpr int NSTAGE = 4;
constexpr int OPB = TT * TT;            // bytes of an 8-bit operand tile
constexpr int T_THREADS = 512, T_ROWS_W = 5, T_FIRST_W = 8 + T_ROWS_W;
constexpr float T_LAZY = 2.f;           // how far (log2) a score may pass the reference maximum
constexpr int T_SHIFT = 12;             // weights are held times 2^12: at most 2^(12 + 2 + 1), in fp16's and e5m2's range
constexpr int TE_UP = 1, TE_DOWN = 8, TE_SPAN = 9;   // exponents around the reference; within one pass

constexpr int TO_K = 0, TO_V = TO_K + NSTAGE * OPB, TO_Q = TO_V + NSTAGE * OPB;   // Q: [2 buffers][hi, lo]
constexpr int TO_EXP = TO_Q + 4 * OPB;                    // [stage][K, V][128] exponent bytes
constexpr int TO_KF = TO_EXP + NSTAGE * 256;              // [warpgroup][tile parity][128] key factors
constexpr int TO_VF = TO_KF + 2 * 2 * 512;                // [warpgroup][128] value factors
constexpr int TO_COL = TO_VF + 2 * 512;                   // [2 buffers][128] (score factor, slot limit)
constexpr int TO_MASK = TO_COL + 2 * TT * 8;              // [2 buffers][128 rows][4] tree masks
constexpr int TO_ML = TO_MASK + 2 * TT * 32;              // [item parity][warpgroup][128] (m, l)
constexpr int TO_RED = TO_ML + 2 * 2 * TT * 8;            // small tables, below
constexpr int TO_BAR = TO_RED + 1024;
constexpr int TO_GROUP = TO_BAR + 256;
constexpr int tc_smem(int groups) { return 1024 + TO_GROUP + (3 * groups + 1) * 4; }

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// kind::f8f6f4: A e4m3 (0) or e5m2 (1), B e4m3, fp32 sums, M = N = 128, B K-major or MN-major.
constexpr uint32_t f8_idesc(int a_fmt, bool b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | (b_mn ? (1u << 16) : 0u) | ((uint32_t)(TT >> 3) << 17) | ((uint32_t)(TT >> 4) << 24);
}
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void ld32_async(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t));
}
// Waits for this thread's TMEM loads; the values pass through, so that nothing of them is used before.
__device__ __forceinline__ void wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void st8(uint32_t t, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 two(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 each(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two fp16 -> two e5m2, rounded, in the low 16 bits (first in the low byte).
__device__ __forceinline__ uint32_t h2_e5m2(uint32_t h) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e5m2x2.f16x2 t, %1;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t f32x2_f16x2(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t two_codes) {
  uint32_t lo, hi;
  e4m3x4_f16(two_codes, lo, hi);
  return __half22float2(*reinterpret_cast<const __half2*>(&lo));
}
// A bounded wait taken by lane 0 for its warp: tcgen05.ld / st are collective, so every lane takes the same branch.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = kv8_wait(bar, parity, abort_flag, err) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

__global__ void __launch_bounds__(T_THREADS, 1)
    kv8_attn_tc_k(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Attn a,
                  const Plan p) {
  extern __shared__ uint8_t tc_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + TO_BAR);
  uint64_t *kv_full = bars, *kv_empty = bars + 4, *q_full = bars + 8, *q_empty = bars + 10, *s_full = bars + 12, *p_full = bars + 14,
           *o_done = bars + 16, *o_free = bars + 18, *q_first = bars + 19, *drain = bars + 20;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 21);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* red = reinterpret_cast<int*>(sm + TO_RED);
  int* r_hi = red;                       // [warpgroup][tile parity][4 warps] largest exponent
  int* r_lo = red + 16;                  // smallest
  uint32_t* r_seen = reinterpret_cast<uint32_t*>(red + 32);   // [warpgroup][4 warps][4] keys seen
  volatile int* s_more = red + 64;       // [warpgroup] another pass of the same tile follows
  int* s_fullvis = red + 66;             // [2 buffers][16 warps]
  int* s_e = red + 98;                   // [item parity][warpgroup] reference exponent (-1: no tile)
  int* s_pref = reinterpret_cast<int*>(sm + TO_GROUP);
  int* s_lim = s_pref + p.groups + 1;
  int* s_seq = s_lim + p.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NSTAGE; ++i) {
      mbar_init(smem_u32(kv_full + i), 2 * 33);   // K's and V's bytes, and their producers' exponent copies
      mbar_init(smem_u32(kv_empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(q_full + i), T_ROWS_W);
      mbar_init(smem_u32(q_empty + i), 9);        // eight softmax warps and the last S product
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(p_full + i), TT);
      mbar_init(smem_u32(o_done + i), 1);
    }
    mbar_init(smem_u32(o_free), 2 * TT);
    mbar_init(smem_u32(q_first), T_FIRST_W);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 10) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;     // S0, S1, O0, O1: 128 columns each
  PDL_ENTRY();
  lay_out(a, p, s_pref, s_lim, s_seq);
  const uint32_t tiles = (uint32_t)s_pref[p.groups] * a.c.nkv;
  const int pad = pad_of(p, tiles);
  const Share share(p, tiles, pad);
  if (threadIdx.x == 0) p.cut[blockIdx.x] = make_int4(0, 0, -1, 0);
  const bool work = blockIdx.x < share.ctas;
  const Range range{s_pref, pad, a.c.nkv, p.groups, share.start(blockIdx.x), share.start(blockIdx.x + 1)};
  Walk k;
  bool more = work && k.begin(range);

  // The query vectors of an item, e4m3 in two parts, and what each sees. By `warps` warps, this being number sw.
  auto prepare = [&](int item, int sw, int warps) {
    const int gi = k.gi, h = k.h, buf = item & 1, seq = s_seq[gi];
    const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
    const int r0 = sidx * a.rows_per_seq + rb * p.RB;
    const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
    const int nqv = (r1 - r0) * p.G;
    const int ctx = a.mode == 1 && seq >= 0 ? a.ctx_len[seq] : 0;
    uint8_t* q_hi = sm + TO_Q + buf * 2 * OPB;
    float2* cols = reinterpret_cast<float2*>(sm + TO_COL) + buf * TT;
    uint64_t* masks = reinterpret_cast<uint64_t*>(sm + TO_MASK) + buf * TT * 4;
    if (item >= 2) kv8_wait(smem_u32(q_empty + buf), (uint32_t)((item / 2 - 1) & 1), abort_flag, a.err);
    if (a.mode == 1)
      for (int x = sw * 32 + lane; x < (r1 - r0) * 4; x += warps * 32) {
        const int r = r0 + x / 4, w = x & 3;
        uint64_t m = 0;
        if (w * 64 < a.tree_T) {
          m = a.mask[(size_t)r * a.mask_words + w];
          if (w == (a.tree_T - 1) >> 6 && (a.tree_T & 63)) m &= (1ull << (a.tree_T & 63)) - 1;
        }
        masks[x] = seq >= 0 && a.row_seq[r] == seq ? m : 0ull;
      }
    int fullvis = INT32_MAX;   // keys below this are seen by every row that counts
    const float sl2 = a.scale * 1.4426950408889634f;
    const int sub = lane & 7;  // eight lanes a vector, 16 entries each
    for (int x0 = sw * 4; x0 < TT; x0 += warps * 8) {
      uint4 raw[2][2];
      int rs[2], lim[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int x = x0 + b * warps * 4 + (lane >> 3);
        raw[b][0] = raw[b][1] = make_uint4(0, 0, 0, 0);
        rs[b] = -1;
        lim[b] = 0;
        if (x < nqv) {
          const int in = (int)(x * p.G_inv >> 16), row = r0 + in;
          const uint4* q = reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.q +
                                                          ((size_t)row * a.nq + h * p.G + x - in * p.G) * TT + sub * 16);
          raw[b][0] = q[0];
          raw[b][1] = q[1];
          rs[b] = a.row_seq[row];
          lim[b] = a.mode == 1 ? ctx : min(a.row_slot[row], INT32_MAX - 1) + 1;
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int x = x0 + b * warps * 4 + (lane >> 3);
        const bool live = seq >= 0 && rs[b] == seq;
        uint32_t r[8] = {raw[b][0].x, raw[b][0].y, raw[b][0].z, raw[b][0].w, raw[b][1].x, raw[b][1].y, raw[b][1].z, raw[b][1].w};
        uint32_t top = 0;   // the largest magnitude's bits
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[i] = live ? r[i] : 0u;
          top = max(top, max(r[i] << 16 & 0x7fffffffu, r[i] & 0x7fff0000u));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
        // largest entry into [2^7, 2^8); a vector with an entry that is not finite gives NaN
        const bool fine = top < 0x7f800000u;
        const int e = top && fine ? max((int)(top >> 23) - 127, -126) - 7 : 0;
        const float up = pow2i(-e / 2), up2 = pow2i(-e - (-e / 2));   // two factors: -e can pass 127
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = lo[i] = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f0 = __uint_as_float(r[2 * i + j] << 16) * up * up2, f1 = __uint_as_float(r[2 * i + j] & 0xffff0000u) * up * up2;
            const uint32_t c = fine ? e4m3x2(f0, f1) : 0x7f7fu;
            const float2 back = e4m3x2_f32(c);
            hi[i] |= c << (16 * j);
            lo[i] |= (fine ? e4m3x2(f0 - back.x, f1 - back.y) : 0u) << (16 * j);
          }
        }
        if (x < TT) {
          const int at = x * TT + ((sub ^ (x & 7)) << 4);   // 128-byte swizzle
          *reinterpret_cast<uint4*>(q_hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(q_hi + OPB + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          const int l = live ? max(0, min(lim[b], a.c.cap)) : 0;
          if (sub == 0) cols[x] = make_float2(fmaxf(sl2 * pow2i(e / 2) * pow2i(e - e / 2), 1.17549435e-38f), __int_as_float(l));
          if (live) fullvis = min(fullvis, l);
        }
      }
    }
    fullvis = __reduce_min_sync(0xffffffffu, fullvis);
    if (lane == 0) s_fullvis[buf * 16 + sw] = fullvis;
    fence_proxy_async_all();
    __syncwarp();
  };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (more) prepare(0, warp, T_FIRST_W);
    if (lane == 0) mbar_arrive(smem_u32(q_first));
    const int wg = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + wg * TT + lane_off, tO = tmem + 2 * TT + wg * TT + lane_off;
    float* s_vf = reinterpret_cast<float*>(sm + TO_VF) + wg * TT;
    int i = 0, passes = 0;       // tiles of the range; value passes of this warpgroup
    for (int item = 0; more; ++item, more = k.next(range)) {
      const int gi = k.gi, h = k.h, buf = item & 1, par = item & 1;
      const int seq = s_seq[gi], limit = s_lim[gi];
      const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
      const int r0 = sidx * a.rows_per_seq + rb * p.RB;
      const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
      const int nqv = (r1 - r0) * p.G;
      const int ctx = a.mode == 1 && seq >= 0 ? a.ctx_len[seq] : 0;
      if (item) kv8_wait(smem_u32(q_full + buf), (uint32_t)((item / 2 - (buf == 0)) & 1), abort_flag, a.err);
      else kv8_wait(smem_u32(q_first), 0, abort_flag, a.err);
      int fullvis = s_fullvis[buf * 16];
      for (int w = 1; w < (item ? T_ROWS_W : T_FIRST_W); ++w) fullvis = min(fullvis, s_fullvis[buf * 16 + w]);
      const float2 col = reinterpret_cast<const float2*>(sm + TO_COL)[buf * TT + r];
      const float qf = col.x;
      const int klim = __float_as_int(col.y);
      const uint32_t* my_mask = reinterpret_cast<const uint32_t*>(sm + TO_MASK) + (buf * TT + (r < nqv ? (r * p.G_inv >> 16) : 0)) * 8;
      float m = -INFINITY, l = 0.f;
      int E = 0, mine = 0;       // reference exponent byte; tiles of this item that were this warpgroup's
      for (int t = k.t0; t < k.t1; ++t, ++i) {
        if ((i & 1) != wg) continue;
        const int st = i % NSTAGE, key0 = t * TT, tp = (i >> 1) & 1;
        kv8_wait(smem_u32(kv_full + st), (uint32_t)((i / NSTAGE) & 1), abort_flag, a.err);
        const int kbyte = sm[TO_EXP + st * 256 + r], vbyte = sm[TO_EXP + st * 256 + TT + r];   // of key r of the tile
        const bool masked = key0 + TT > fullvis || limit <= key0;
        uint32_t vis[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};   // keys that this row sees
        bool seen = true;                                                        // key r of the tile, by any row
        if (masked) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int kb = key0 + w * 32, below = klim - kb;
            uint32_t v = below >= 32 ? 0xffffffffu : below <= 0 ? 0u : (1u << below) - 1;
            if (a.mode == 1 && r < nqv) {
              const int tt = kb - ctx;   // tree slot of the word's first key
              const uint32_t lo = tt >= 0 && tt < 256 ? my_mask[tt >> 5] : 0u;
              const uint32_t hi = tt >= -31 && tt < 224 ? my_mask[(tt + 32) >> 5] : 0u;
              v |= __funnelshift_r(lo, hi, tt & 31);
            }
            const int room = limit - kb;
            vis[w] = room >= 32 ? v : room <= 0 ? 0u : v & ((1u << room) - 1);
            const uint32_t any = __reduce_or_sync(0xffffffffu, r < nqv ? vis[w] : 0u);
            if (lane == 0) r_seen[(wg * 4 + (warp & 3)) * 4 + w] = any;
          }
          named_bar_sync(2 + wg, TT);
          const int w = r >> 5;
          const uint32_t any = r_seen[wg * 16 + w] | r_seen[wg * 16 + 4 + w] | r_seen[wg * 16 + 8 + w] | r_seen[wg * 16 + 12 + w];
          seen = (any >> (r & 31)) & 1u;
          if (!seen) {   // a slot that no row sees may hold anything: 0 * NaN must not come of it
            uint4* z = reinterpret_cast<uint4*>(sm + TO_V + st * OPB + r * TT);
#pragma unroll
            for (int x = 0; x < 8; ++x) z[x] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_all();
        }
        const bool counts = seen && vbyte != KV8_BAD;
        const uint32_t whi = __reduce_max_sync(0xffffffffu, counts ? (uint32_t)vbyte : 0u);
        const uint32_t wlo = __reduce_min_sync(0xffffffffu, counts ? (uint32_t)vbyte : 255u);
        if (lane == 0) {
          r_hi[(wg * 2 + tp) * 4 + (warp & 3)] = (int)whi;
          r_lo[(wg * 2 + tp) * 4 + (warp & 3)] = (int)wlo;
        }
        float* s_kf = reinterpret_cast<float*>(sm + TO_KF) + (wg * 2 + tp) * TT;
        s_kf[r] = kv8_pow2(kbyte);
        named_bar_sync(2 + wg, TT);
        const int* rh = r_hi + (wg * 2 + tp) * 4;
        const int* rl = r_lo + (wg * 2 + tp) * 4;
        int hi = max(max(rh[0], rh[1]), max(rh[2], rh[3]));
        const int lo_all = min(min(rl[0], rl[1]), min(rl[2], rl[3]));

        warp_wait(smem_u32(s_full + wg), (uint32_t)((i >> 1) & 1), abort_flag, a.err);
        tc_fence_after();
        float s[TT];
#pragma unroll
        for (int c = 0; c < TT; c += 32) ld32_async(tS + c, s + c);
#pragma unroll
        for (int c = 0; c < TT; c += 32) wait_ld(s + c);
#pragma unroll
        for (int c = 0; c < TT; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s_kf + c);
          const float2 u = each(mul2(two(s[c], s[c + 1]), two(f.x, f.y))), v = each(mul2(two(s[c + 2], s[c + 3]), two(f.z, f.w)));
          s[c] = u.x; s[c + 1] = u.y; s[c + 2] = v.x; s[c + 3] = v.y;
        }
        if (masked)
#pragma unroll
          for (int c = 0; c < TT; ++c) s[c] = (vis[c >> 5] >> (c & 31)) & 1u ? s[c] : -INFINITY;
        float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
        for (int c = 4; c + 7 < TT; c += 8) {
          x0 = max3(x0, s[c], s[c + 1]);
          x1 = max3(x1, s[c + 2], s[c + 3]);
          x2 = max3(x2, s[c + 4], s[c + 5]);
          x3 = max3(x3, s[c + 6], s[c + 7]);
        }
        const float mx = fmaxf(max3(x0, x1, fmaxf(s[TT - 4], s[TT - 3])), max3(x2, x3, fmaxf(s[TT - 2], s[TT - 1])));
        float corr = 1.f;
        if ((mx - m) * qf > T_LAZY) {
          corr = ex2((m - mx) * qf);
          m = mx;
          l *= corr;
        }
        // weights; the difference comes first: it is exact where it matters, whatever the size of the scores
        {
          const float base = m == -INFINITY ? 0.f : -m;
          const f32x2 nm = two(base, base), q2 = two(qf, qf);
          f32x2 sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < TT; c += 2) {
            float2 x = each(mul2(add2(two(s[c], s[c + 1]), nm), q2));
            s[c] = ex2(x.x);
            s[c + 1] = ex2(x.y);
            sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], two(s[c], s[c + 1]));
          }
          const float2 u = each(add2(sum[0], sum[1]));
          l += u.x + u.y;
        }
        bool first = true;
        while (true) {
          const bool one = hi - lo_all <= TE_SPAN;
          const int lo = one ? 0 : hi - TE_SPAN;
          float unit = 1.f;    // O from the old reference exponent to the new one
          if (hi > E + TE_UP || (one ? lo_all : lo) < E - TE_DOWN) {
            if (E) unit = pow2i(E - hi);
            E = hi;
          }
          // not finite: NaN where seen; outside this pass's exponents, or seen by nobody: 0
          s_vf[r] = !seen ? 0.f : vbyte == KV8_BAD ? (first ? kv8_pow2(vbyte) : 0.f)
                                                   : vbyte >= lo && vbyte <= hi ? pow2i(vbyte - E + T_SHIFT) : 0.f;
          named_bar_sync(2 + wg, TT);
          const float scale_o = first ? corr * unit : unit;
          const bool begun = mine > 0 || !first;      // O holds something
          // a pass before this one must be out of P, and O complete before it is rescaled
          if (!first || (begun && __any_sync(0xffffffffu, scale_o != 1.f))) {
            warp_wait(smem_u32(o_done + wg), (uint32_t)((passes - 1) & 1), abort_flag, a.err);
            tc_fence_after();
            if (__any_sync(0xffffffffu, scale_o != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < TT; c += 16) {
                float o[16];
                tmem_ld16(tO + c, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= scale_o;
                tmem_st16(tO + c, o);
              }
            }
          }
#pragma unroll
          for (int c0 = 0; c0 < TT; c0 += 32) {
            uint32_t p1[8], p2[8], p3[8];
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 f = *reinterpret_cast<const float4*>(s_vf + c0 + c);
              const uint32_t u = f32x2_f16x2(each(mul2(two(s[c0 + c], s[c0 + c + 1]), two(f.x, f.y))));
              const uint32_t v = f32x2_f16x2(each(mul2(two(s[c0 + c + 2], s[c0 + c + 3]), two(f.z, f.w))));
              const uint32_t u2 = h2_sub(u, u & 0xff00ff00u), v2 = h2_sub(v, v & 0xff00ff00u);
              p1[c / 4] = __byte_perm(u, v, 0x7531);          // upper bytes: the fp16 cut to e5m2
              p2[c / 4] = __byte_perm(u2, v2, 0x7531);
              p3[c / 4] = __byte_perm(h2_e5m2(h2_sub(u2, u2 & 0xff00ff00u)), h2_e5m2(h2_sub(v2, v2 & 0xff00ff00u)), 0x5410);
            }
            st8(tS + c0 / 4, p1);
            st8(tS + 32 + c0 / 4, p2);
            st8(tS + 64 + c0 / 4, p3);
          }
          tmem_wait_st();
          if (r == 0) s_more[wg] = !one;
          int next_hi = 0;
          if (!one) {   // the next pass's exponents
            const uint32_t below = __reduce_max_sync(0xffffffffu, counts && vbyte < lo ? (uint32_t)vbyte : 0u);
            if (lane == 0) r_hi[(wg * 2 + tp) * 4 + (warp & 3)] = (int)below;
            named_bar_sync(2 + wg, TT);
            next_hi = max(max(rh[0], rh[1]), max(rh[2], rh[3]));
          }
          tc_fence_before();
          mbar_arrive(smem_u32(p_full + wg));
          ++passes;
          if (one) break;
          hi = next_hi;      // > 0: lo_all itself is still to come
          first = false;
        }
        ++mine;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(q_empty + buf));

      // both warpgroups' sums of the item, each thread 64 dims of its query vector
      if (mine) warp_wait(smem_u32(o_done + wg), (uint32_t)((passes - 1) & 1), abort_flag, a.err);
      float2* s_ml = reinterpret_cast<float2*>(sm + TO_ML) + par * 2 * TT;
      s_ml[wg * TT + r] = make_float2(m, l);
      if (r == 0) s_e[par * 2 + wg] = mine ? E : -1;
      tc_fence_before();
      named_bar_sync(1, 2 * TT);
      tc_fence_after();
      const float2 ml0 = s_ml[r], ml1 = s_ml[TT + r];
      const int e0 = s_e[par * 2], e1 = s_e[par * 2 + 1];
      const float mt = fmaxf(ml0.x, ml1.x), mb = mt == -INFINITY ? 0.f : mt;
      const float f0 = ex2((ml0.x - mb) * qf), f1 = ex2((ml1.x - mb) * qf);
      float L = ml0.y * f0 + ml1.y * f1, top = mt * qf;
      // (E = 0: no value counted, O is zero or NaN)
      const float u0 = f0 * pow2i(e0 > 0 ? e0 - KV8_BIAS - T_SHIFT : 0), u1 = f1 * pow2i(e1 > 0 ? e1 - KV8_BIAS - T_SHIFT : 0);
      float o[64];
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        float x[32], y[32];
        ld32_async(tmem + 2 * TT + lane_off + wg * 64 + c, x);
        ld32_async(tmem + 3 * TT + lane_off + wg * 64 + c, y);
        wait_ld(x);
        wait_ld(y);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[c + j] = (e0 >= 0 ? x[j] * u0 : 0.f) + (e1 >= 0 ? y[j] * u1 : 0.f);
      }
      tc_fence_before();
      mbar_arrive(smem_u32(o_free));
      const bool whole = k.t0 == 0 && k.t1 == k.nt;
      if (threadIdx.x == 0 && k.t0 == 0 && k.t1 < k.nt)
        p.cut[blockIdx.x] = make_int4(gi, h, (int)share.cta_of(k.base + pad + k.nt - 1), 0);
      if (r < nqv) {
        if (whole) {
          const int in = (int)(r * p.G_inv >> 16), row = r0 + in;
          const size_t at = (size_t)row * a.nq + h * p.G + r - in * p.G, stride = (size_t)a.R * a.nq;
          for (int s = 0; s < p.n_prefix; ++s) {
            const float2 v = *reinterpret_cast<const float2*>(p.pp_ml + 2 * (s * stride + at));
            const float4* x = reinterpret_cast<const float4*>(p.pp_o + (s * stride + at) * TT + wg * 64);
            const float nt = fmaxf(top, v.x), b = nt == -INFINITY ? 0.f : nt, f = ex2(top - b), g = ex2(v.x - b);
            top = nt;
            L = L * f + v.y * g;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float4 y = x[c];
              o[4 * c] = o[4 * c] * f + y.x * g; o[4 * c + 1] = o[4 * c + 1] * f + y.y * g;
              o[4 * c + 2] = o[4 * c + 2] * f + y.z * g; o[4 * c + 3] = o[4 * c + 3] * f + y.w * g;
            }
          }
          const bool live = seq >= 0 && a.row_seq[row] == seq;
#pragma unroll
          for (int c = 0; c < 64; c += 8) store8(a, at, TT, wg * 64 + c, live, L, o + c);
        } else {
          const size_t q = (size_t)(2 * blockIdx.x + (k.t0 == 0 ? 1 : 0)) * p.qv_pad + r;
          float4* x = reinterpret_cast<float4*>(p.part_o + q * TT + wg * 64);
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          if (wg == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * q) = make_float2(top, L);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp < 10) {
      // ---- producers: 8 the keys, 9 the values. Lanes 0-7 look after a tile's eight 16-slot parts ----
      const bool is_v = warp == 9;
      const int box = a.c.table ? min(TT, 1 << a.c.block_log2) : TT;
      const uint8_t* exps = is_v ? a.c.ve : a.c.ke;
      const uint64_t pol = l2_policy_evict_first();
      int i = 0;
      bool ok = true;
      auto where = [&](const Walk& w, int t) -> long long {   // this lane's part of a tile; -1: none, or not assigned
        const int slot = t * TT + lane * 16;
        if (lane >= 8 || slot >= s_lim[w.gi]) return -1;
        return kv8_vec(a.c, s_seq[w.gi], w.h, slot);
      };
      for (; more && ok; more = k.next(range)) {
        const int limit = s_lim[k.gi];
        long long vec = where(k, k.t0);
        for (int t = k.t0; ok && t < k.t1; ++t, ++i) {
          const long long ahead = t + 1 < k.t1 ? where(k, t + 1) : -1;   // the next tile's table entries, a tile early
          const int st = i % NSTAGE, parts = max(0, min(8, (limit - t * TT + 15) / 16));
          if (lane < parts && vec < 0) latch_error(a.err, DEVERR_BOUNDS);   // not assigned: unspecified keys
          const int at = (int)max(vec, 0ll);
          if (i >= NSTAGE && !kv8_wait(smem_u32(kv_empty + st), (uint32_t)((i / NSTAGE - 1) & 1), abort_flag, a.err)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t bar = smem_u32(kv_full + st), dst = smem_u32(sm + (is_v ? TO_V : TO_K) + st * OPB);
          if (lane < parts) copy16(smem_u32(sm + TO_EXP + st * 256) + (is_v ? TT : 0) + lane * 16, exps + at);
          copies_arrive(bar);
          const int per = box / 16, boxes = (parts + per - 1) / per;
          if (lane == 0) mbar_expect_tx(bar, (uint32_t)(boxes * box * TT));
          for (int x = 0; x < boxes; ++x) {
            const int row = __shfl_sync(0xffffffffu, at, x * per);
            if (lane == 0) tma_load_2d(dst + x * box * TT, is_v ? &tmV : &tmK, 0, row, bar, pol);
          }
          vec = ahead;
        }
      }
      if (!ok)   // the tiles in flight land before the CTA leaves
        for (int x = max(0, i - NSTAGE); x < i; ++x)
          kv8_wait(smem_u32(kv_full + x % NSTAGE), (uint32_t)((x / NSTAGE) & 1), abort_flag, a.err, false);
    } else if (warp == 10) {
      // ---- MMA: S of the tile ahead, then the value product of this one ----
      constexpr uint32_t IS = f8_idesc(0, false), IO = f8_idesc(1, true);
      const uint64_t dq = sdesc_sw128(smem_u32(sm + TO_Q)), dk = sdesc_sw128(smem_u32(sm + TO_K)), dv = sdesc_sw128(smem_u32(sm + TO_V));
      Walk a_head = k;                 // the tile whose S comes next
      bool s_left = more;
      int s_item = 0, s_tile = s_left ? k.t0 : 0, si = 0, passes[2] = {0, 0};
      bool ok = true;
      auto issue_s = [&]() {
        if (!s_left) return;
        const int buf = s_item & 1, st = si % NSTAGE;
        if (s_tile == a_head.t0)
          ok = ok && (s_item ? kv8_wait(smem_u32(q_full + buf), (uint32_t)((s_item / 2 - (buf == 0)) & 1), abort_flag, a.err)
                             : kv8_wait(smem_u32(q_first), 0, abort_flag, a.err));
        ok = ok && kv8_wait(smem_u32(kv_full + st), (uint32_t)((si / NSTAGE) & 1), abort_flag, a.err);
        if (ok) {
          tc_fence_after();
          if (elect_one()) {
            // rolled loops: unrolled, their operands are hoisted out of the tile loop and spilled (2500 clocks an S)
            uint64_t q = dq + buf * (2 * OPB >> 4);
            uint32_t acc = 0;
#pragma unroll 1
            for (int part = 0; part < 2; ++part, q += (OPB >> 4) - 8) {   // high part, low part
              uint64_t kd = dk + st * (OPB >> 4);
#pragma unroll 1
              for (int x = 0; x < 4; ++x, q += 2, kd += 2, acc = 1) mma8_ss(tmem + (si & 1) * TT, q, kd, IS, acc);
            }
            tc_commit(smem_u32(s_full + (si & 1)));
            if (s_tile + 1 == a_head.t1) tc_commit(smem_u32(q_empty + buf));
          }
          __syncwarp();
        }
        ++si;
        if (++s_tile == a_head.t1) {
          s_left = a_head.next(range);
          ++s_item;
          if (s_left) s_tile = a_head.t0;
        }
      };
      issue_s();
      int i = 0;
      for (int item = 0; more && ok; ++item, more = k.next(range)) {
        for (int t = k.t0; ok && t < k.t1; ++t, ++i) {
          issue_s();
          const int wg = i & 1, st = i % NSTAGE, j = t - k.t0;
          if (j == 0 && item) ok = ok && kv8_wait(smem_u32(o_free), (uint32_t)((item - 1) & 1), abort_flag, a.err);
          bool again = true;
          for (int pass = 0; ok && again; ++pass) {
            ok = kv8_wait(smem_u32(p_full + wg), (uint32_t)(passes[wg] & 1), abort_flag, a.err);
            if (!ok) break;
            again = s_more[wg] != 0;
            tc_fence_after();
            if (elect_one()) {
              uint32_t acc = j < 2 && pass == 0 ? 0u : 1u;   // the warpgroup's first tile of the item begins O
              uint32_t pa = tmem + wg * TT;
#pragma unroll 1
              for (int part = 0; part < 3; ++part) {
                uint64_t v = dv + st * (OPB >> 4);
#pragma unroll 1
                for (int x = 0; x < 4; ++x, pa += 8, v += 32 * TT >> 4, acc = 1) mma8_ts(tmem + 2 * TT + wg * TT, pa, v, IO, acc);
              }
              tc_commit(smem_u32(o_done + wg));
              if (!again) tc_commit(smem_u32(kv_empty + st));
            }
            __syncwarp();
            ++passes[wg];
          }
        }
      }
      if (!ok) {   // products in flight end before the CTA frees its TMEM
        if (elect_one()) tc_commit(smem_u32(drain));
        kv8_wait(smem_u32(drain), 0, abort_flag, a.err, false);
      }
    } else {
      // ---- row warps: the first item together with the softmax warps, each later one ahead of them ----
      const int sw = warp - 11;
      if (more) prepare(0, 8 + sw, T_FIRST_W);
      if (lane == 0) mbar_arrive(smem_u32(q_first));
      more = more && k.next(range);
      for (int item = 1; more; ++item, more = k.next(range)) {
        prepare(item, sw, T_ROWS_W);
        if (lane == 0) mbar_arrive(smem_u32(q_full + (item & 1)));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t kv8_launch_tc(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& k, const CUtensorMap& v) {
  const int smem = tc_smem(p.groups);
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kv8_attn_tc_k), smem);
  if (e != cudaSuccess) return e;
  return launch_k(kv8_attn_tc_k, dim3(p.grid), dim3(T_THREADS), smem, st, k, v, a, p);
}

}  // namespace eagle
