// Attention of many query vectors over the 8-bit KV cache on the 5th-generation tensor cores (head_dim 128).
//
// A verify pass has tens of query vectors a KV head: per 128-key tile two products of a 128-row tile.
//   S = (Q_hi + Q_lo) K^T   kind::f8f6f4 on the cache's e4m3 codes as they lie: one TMA copy from HBM to the operand. q is
//                           scaled by a power of two and cut into two e4m3 parts, together 8 significant bits, as many as
//                           bf16 has, down to 2^-9 of the vector's largest entry (below, a step of 2^-17 of it).
//   O += P V                kind::f16: the weights times their values' exponents as fp16 (2^-11) in TMEM; the codes are
//                           widened to fp16 (exact) in shared memory by the softmax threads while they wait for S. (Weights
//                           in 8-bit parts, e5m2 for their range, need three products of the codes as they lie, but cutting
//                           them took twice the arithmetic of the whole softmax: 5000 clocks a tile against HBM's 1500.)
// A key's factor multiplies its scores; a value's exponent is added to them and taken out again of the weights' sum.
//
// One CTA an SM, 20 warps, two workers with a range of items each, so that one's softmax and epilogue run under the other's
// products (one worker: 151 us instead of 118 at the time). A worker has eight softmax warps (two threads a query vector, 64
// keys of a tile each: four warps a scheduler hide each other's latencies, and prepare the next item's query vectors; S is
// read twice from TMEM, for the maximum, which leaves scores plus exponents there, and for the weights, which keeps a thread
// below 96 registers, and each 32 columns of S are overwritten by the weights of their keys), an MMA warp and a producer
// warp (TMA: the next tile's keys under this one's softmax, its values as soon as these are widened). TMEM: S and O, 128
// columns each, of either worker.
// 64 ragged sequences of up to 2048 slots, 17 tree rows of 32 heads over 8 KV heads: 83 us (24 us of bytes at the copy rate),
// 180 us on mma.sync at the time. Bound by the softmax warps: of a tile's some 5700 clocks the weights take 1400, the maximum
// 1400, widening the values 1000, the two products, the barriers and their hand-overs the rest.
#include "kv8_split.cuh"
#include "kernels.h"
#include "tc_common.cuh"

#include <algorithm>
#include <cuda_fp16.h>

namespace eagle {
namespace {

constexpr int TT = 128;                 // keys a tile, query vectors a block, dims
constexpr int OPB = TT * TT;            // bytes of an 8-bit operand tile
constexpr int SOFT = 256;               // softmax threads of a worker
constexpr int SOFT_W = SOFT / 32;
constexpr int T_THREADS = 2 * SOFT + 128;

// a worker's shared memory, [2]
constexpr int TO_K = 0, TO_V8 = TO_K + 2 * OPB, TO_V = TO_V8 + 2 * OPB, TO_Q = TO_V + 4 * OPB;   // keys; values: codes, fp16
                                                          // [half of the dims]; query vectors [part]
constexpr int TO_EXP = TO_Q + 4 * OPB;                    // [worker][tile parity][K, V][128] exponent bytes
constexpr int TO_KF = TO_EXP + 2 * 2 * 256;               // [worker][tile parity][128] key factors
constexpr int TO_VF = TO_KF + 2 * 2 * 512;                // [worker][tile parity][2][128] value exponents, inverses of their powers
constexpr int TO_COL = TO_VF + 2 * 2 * 1024;              // [worker][item parity][128] (score factor, slot limit)
constexpr int TO_MASK = TO_COL + 4 * TT * 8;              // [worker][128 rows][4] tree masks: the last tile's barrier on its
                                                          // exponents comes after their last use in an item
constexpr int TO_X = TO_MASK + 2 * TT * 32;               // [worker][tile parity][half][128] maxima; then sums
constexpr int TO_RED = TO_X + 2 * 2 * 2 * TT * 4;         // [worker] small tables, below
constexpr int TO_BAR = TO_RED + 2 * 512;
constexpr int TO_GROUP = TO_BAR + 2 * 128 + 64;
constexpr int tc_smem(int groups) { return 1024 + TO_GROUP + (3 * groups + 1) * 4; }
static_assert(tc_smem(KV8_MAX_GROUPS) <= 227 * 1024, "shared memory");

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// M = N = 128, fp32 sums, A K-major. kind::f8f6f4 with e4m3 operands, B K-major; kind::f16 with fp16 operands, B MN-major.
constexpr uint32_t S_IDESC = (1u << 4) | ((uint32_t)(TT >> 3) << 17) | ((uint32_t)(TT >> 4) << 24);
constexpr uint32_t O_IDESC = (1u << 4) | (1u << 16) | ((uint32_t)(TT >> 3) << 17) | ((uint32_t)(TT >> 4) << 24);
// MN-major operand, 128-byte swizzle: 64 fp16 a row, one row per k, the next 64 dims OPB on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)(OPB >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma8_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void st8(uint32_t t, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
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
__global__ void __launch_bounds__(T_THREADS, 1)
    kv8_attn_tc_k(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Attn a,
                  const Plan p) {
  extern __shared__ uint8_t tc_smem_raw[];
  uint8_t* sm = tc_smem_raw + (-smem_u32(tc_smem_raw) & 1023u);   // (not by pointer masks: accesses then lose the shared space)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wk = warp < 16 ? warp >> 3 : warp & 1;   // this warp's worker (16, 17: MMA; 18, 19: producers)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + TO_BAR + 256);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + TO_BAR + wk * 128);
  uint64_t *k_full = bars, *k_empty = bars + 1, *v_full = bars + 2, *v_empty = bars + 3, *q_full = bars + 4, *s_full = bars + 5,
           *p_full = bars + 6, *o_done = bars + 7, *o_free = bars + 8, *drain = bars + 9;
  int* red = reinterpret_cast<int*>(sm + TO_RED + wk * 512);
  uint32_t* r_seen = reinterpret_cast<uint32_t*>(red);        // [8 warps][2] keys seen
  int* s_fullvis = red + 16;                                  // [item parity][16 warps]
  int* s_pref = reinterpret_cast<int*>(sm + TO_GROUP);
  int* s_lim = s_pref + p.groups + 1;
  int* s_seq = s_lim + p.groups;
  if (warp == 16 || warp == 17) {
    if (lane == 0) {
      mbar_init(smem_u32(k_full), 33);   // the codes' bytes, and each producer lane's exponent copies
      mbar_init(smem_u32(k_empty), 1 + SOFT_W);   // S of the tile, and its exponents read by each softmax warp
      mbar_init(smem_u32(v_full), 1);
      mbar_init(smem_u32(v_empty), SOFT_W);
      mbar_init(smem_u32(q_full), SOFT_W);
      mbar_init(smem_u32(s_full), 1);
      mbar_init(smem_u32(p_full), SOFT_W);
      mbar_init(smem_u32(o_done), 1);
      mbar_init(smem_u32(o_free), SOFT_W);
      mbar_init(smem_u32(drain), 1);
      if (warp == 16) *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
  }
  if (warp == 18) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS0 = *tmem_slot + wk * TT, tO0 = *tmem_slot + 2 * TT + wk * TT;
  late_entry(p);
  lay_out(a, p, s_pref, s_lim, s_seq);
  const uint32_t tiles = (uint32_t)s_pref[p.groups] * a.c.nkv;
  const int pad = pad_of(p, tiles);
  const Share share(p, tiles, pad);                          // over the workers: all first ones, then all second ones
  const uint32_t me = wk * gridDim.x + blockIdx.x;
  if (threadIdx.x < 2) cut_none(p, threadIdx.x * gridDim.x + blockIdx.x);
  __syncthreads();
  const Range range{s_pref, pad, a.c.nkv, p.groups, share.start(me), share.start(me + 1)};
  Walk k;
  bool more = me < share.ctas && k.begin(range);

  // The query vectors of an item, e4m3 in two parts, and what each sees. By a worker's softmax warps; the last S of the
  // item before is done.
  auto prepare = [&](const Walk& k, int item) {
    constexpr int warps = SOFT_W;
    const int sw = warp & 7;
    const int gi = k.gi, h = k.h, buf = item & 1, seq = s_seq[gi];
    const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
    const int r0 = sidx * a.rows_per_seq + rb * p.RB;
    const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
    const int nqv = (r1 - r0) * p.G;
    const int ctx = a.mode == 1 && seq >= 0 ? __ldcg(a.ctx_len + seq) : 0;
    uint8_t* q_hi = sm + TO_Q + wk * 2 * OPB;
    float2* cols = reinterpret_cast<float2*>(sm + TO_COL) + (wk * 2 + buf) * TT;
    uint64_t* masks = reinterpret_cast<uint64_t*>(sm + TO_MASK) + wk * TT * 4;
    if (a.mode == 1)
      for (int x = sw * 32 + lane; x < (r1 - r0) * 4; x += warps * 32) {
        const int r = r0 + x / 4, w = x & 3;
        uint64_t m = 0;
        if (w * 64 < a.tree_T) {
          m = __ldcg(a.mask + (size_t)r * a.mask_words + w);
          if (w == (a.tree_T - 1) >> 6 && (a.tree_T & 63)) m &= (1ull << (a.tree_T & 63)) - 1;
        }
        masks[x] = seq >= 0 && __ldcg(a.row_seq + r) == seq ? m : 0ull;
      }
    int fullvis = INT32_MAX;   // keys below this are seen by every row that counts
    const float sl2 = a.scale * 1.4426950408889634f;
    const int sub = lane & 7;  // eight lanes a vector, 16 entries each
    for (int x0 = sw * 4; x0 < nqv; x0 += warps * 8) {
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
          raw[b][0] = __ldcg(q);
          raw[b][1] = __ldcg(q + 1);
          rs[b] = __ldcg(a.row_seq + row);
          lim[b] = a.mode == 1 ? ctx : min(__ldcg(a.row_slot + row), INT32_MAX - 1) + 1;
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
        if (x < nqv) {   // rows past the block's keep what they held: their results go nowhere
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
    fence_async_shared();
    warp_arrive(smem_u32(q_full));
  };

  if (warp < 16) {
    if (more) prepare(k, 0);
    const int hf = (warp >> 2) & 1, r = threadIdx.x & 127, c0 = hf * 64;   // half of a tile's keys and of O's columns; row
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tS0 + lane_off + c0, tO = tO0 + lane_off + c0;
    int i = 0;                   // tiles of the range
    for (int item = 0; more; ++item) {
      const int gi = k.gi, h = k.h, buf = item & 1;
      const int seq = s_seq[gi], limit = s_lim[gi];
      const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
      const int r0 = sidx * a.rows_per_seq + rb * p.RB;
      const int r1 = min(min(r0 + p.RB, (sidx + 1) * a.rows_per_seq), a.R);
      const int nqv = (r1 - r0) * p.G;
      const int ctx = a.mode == 1 && seq >= 0 ? __ldcg(a.ctx_len + seq) : 0;
      kv8_wait(smem_u32(q_full), (uint32_t)(item & 1), abort_flag, a.err);
      int fullvis = s_fullvis[buf * 16];
#pragma unroll 1
      for (int w = 1; w < SOFT_W; ++w) fullvis = min(fullvis, s_fullvis[buf * 16 + w]);
      const float2 col = reinterpret_cast<const float2*>(sm + TO_COL)[(wk * 2 + buf) * TT + r];
      const float qf = r < nqv ? col.x : 0.f;   // a row past the block's never raises its maximum
      const int klim = __float_as_int(col.y);
      const uint32_t* my_mask =
          reinterpret_cast<const uint32_t*>(sm + TO_MASK) + (wk * TT + (r < nqv ? (r * p.G_inv >> 16) : 0)) * 8;
      float ref = -INFINITY, l = 0.f;
      for (int t = k.t0; t < k.t1; ++t, ++i) {
        const int key0 = t * TT, tp = i & 1;
        kv8_wait(smem_u32(k_full), (uint32_t)(i & 1), abort_flag, a.err);
        const uint8_t* s_exp = sm + TO_EXP + (wk * 2 + tp) * 256;
        const bool masked = key0 + TT > fullvis || limit <= key0;
        uint32_t vis[2] = {0xffffffffu, 0xffffffffu};   // this thread's keys that its row sees
        bool seen = true;                               // key r of the tile, by any row
        if (masked) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int kb = key0 + c0 + w * 32, below = klim - kb;
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
            if (lane == 0) r_seen[(warp & 7) * 2 + w] = any;
          }
          named_bar_sync(1 + wk, SOFT);
          // a slot that no row sees may hold anything: its codes become zeros, 0 * NaN must not come of it
          const uint32_t* any = r_seen + (r >> 6) * 8 + ((r >> 5) & 1);
          seen = ((any[0] | any[2] | any[4] | any[6]) >> (r & 31)) & 1u;
        }
        // the tile's keys: the first half's threads take their factors, the second's their values'
        float* s_kf = reinterpret_cast<float*>(sm + TO_KF) + (wk * 2 + tp) * TT;
        float* s_va = reinterpret_cast<float*>(sm + TO_VF) + (wk * 2 + tp) * 2 * TT;   // exponents
        float* s_vi = s_va + TT;                                                      // the inverses of their powers
        if (!hf) {
          s_kf[r] = kv8_pow2(s_exp[r]);
        } else {
          s_va[r] = kv8_exponent(s_exp[TT + r]);
          s_vi[r] = kv8_inverse(s_exp[TT + r]);
        }
        // (without this arrival the next tile's keys could be there before a warp still at the item's end has seen this
        // phase of k_full end, and it would wait for the phase after)
        warp_arrive(smem_u32(k_empty));
        named_bar_sync(1 + wk, SOFT);
        // value r's codes to fp16, this thread's half of the dims, under S: the product of the tile before must be done
        if (i) kv8_wait(smem_u32(o_done), (uint32_t)((i - 1) & 1), abort_flag, a.err);
        kv8_wait(smem_u32(v_full), (uint32_t)(i & 1), abort_flag, a.err);
        {
          const uint8_t* from = sm + TO_V8 + wk * OPB + r * TT;
          uint8_t* to = sm + TO_V + (wk * 2 + hf) * OPB + r * TT;
          uint4 codes[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) codes[c] = *reinterpret_cast<const uint4*>(from + (((hf * 4 + c) ^ (r & 7)) << 4));
#pragma unroll
          for (int c = 0; c < 4; ++c) {   // 16 codes to two 16-byte parts of fp16
            const uint32_t w[4] = {codes[c].x, codes[c].y, codes[c].z, codes[c].w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint4 f;
              e4m3x4_f16(seen ? w[2 * j] : 0u, f.x, f.y);
              e4m3x4_f16(seen ? w[2 * j + 1] : 0u, f.z, f.w);
              *reinterpret_cast<uint4*>(to + (((2 * c + j) ^ (r & 7)) << 4)) = f;
            }
          }
          fence_async_shared();
          warp_arrive(smem_u32(v_empty));
        }
        kv8_wait(smem_u32(s_full), (uint32_t)(i & 1), abort_flag, a.err);
        tc_fence_after();
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          float s[16];
          tmem_ld16(tS + c, s);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {   // (a key's factor is a power of two: that product is exact)
            const float4 f = *reinterpret_cast<const float4*>(s_kf + c0 + c + j);
            const float4 v = *reinterpret_cast<const float4*>(s_va + c0 + c + j);
            s[j] = fmaf(s[j] * f.x, qf, v.x);
            s[j + 1] = fmaf(s[j + 1] * f.y, qf, v.y);
            s[j + 2] = fmaf(s[j + 2] * f.z, qf, v.z);
            s[j + 3] = fmaf(s[j + 3] * f.w, qf, v.w);
          }
          if (masked)
#pragma unroll
            for (int j = 0; j < 16; ++j)   // last: a hidden key may hold NaN
              s[j] = (vis[c >> 5] >> ((c & 16) + j)) & 1u ? s[j] : -INFINITY;
#pragma unroll
          for (int j = 0; j < 16; j += 8)
            mx = max3(mx, max3(s[j], s[j + 1], s[j + 2]), max3(max3(s[j + 3], s[j + 4], s[j + 5]), s[j + 6], s[j + 7]));
          tmem_st16(tS + c, s);
        }
        tmem_wait_st();
        float* x_max = reinterpret_cast<float*>(sm + TO_X) + (wk * 2 + tp) * 2 * TT;
        x_max[hf * TT + r] = mx;
        named_bar_sync(1 + wk, SOFT);
        mx = fmaxf(x_max[r], x_max[TT + r]);
        float corr = 1.f;
        if (r < nqv && mx - ref > KV8_TOP) {
          corr = ex2(ref - (mx - KV8_HEAD));
          ref = mx - KV8_HEAD;
          l *= corr;
        }
        if (t > k.t0 && __any_sync(0xffffffffu, corr != 1.f)) {   // (the product of the tile before is done)
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            float o[16];
            tmem_ld16(tO + c, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] *= corr;
            tmem_st16(tO + c, o);
          }
        }
        // weights: a difference of two rounded numbers, exact near the reference, whatever the size of the scores
        const float base = ref == -INFINITY ? 0.f : ref;
        // (scalar arithmetic: pairs of fp32 cost as many moves into aligned registers as they save)
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          float s[16];
          tmem_ld16(tS + c, s);
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 u = *reinterpret_cast<const float4*>(s_vi + c0 + c + j);
            s[j] = ex2(s[j] - base);
            s[j + 1] = ex2(s[j + 1] - base);
            s[j + 2] = ex2(s[j + 2] - base);
            s[j + 3] = ex2(s[j + 3] - base);
            sum[0] = fmaf(s[j], u.x, sum[0]);
            sum[1] = fmaf(s[j + 1], u.y, sum[1]);
            sum[2] = fmaf(s[j + 2], u.z, sum[2]);
            sum[3] = fmaf(s[j + 3], u.w, sum[3]);
            w[j / 2] = half2_of(s[j], s[j + 1]);
            w[j / 2 + 1] = half2_of(s[j + 2], s[j + 3]);
          }
          st8(tS + (c & 32) + (c & 16) / 2, w);   // the weights of 32 keys over the first 16 of their 32 score columns
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(smem_u32(p_full));
      }

      // the next item's query vectors, so that its first S runs under this item's end
      const Walk done = k;
      more = k.next(range);
      if (more) prepare(k, item + 1);
      // the item's sum: l of both halves; this thread's 64 dims of its query vector
      float* x_l = reinterpret_cast<float*>(sm + TO_X) + (wk * 2 + (i & 1)) * 2 * TT;   // the parity that the last tile did not use
      x_l[hf * TT + r] = l;
      kv8_wait(smem_u32(o_done), (uint32_t)((i - 1) & 1), abort_flag, a.err);
      tc_fence_after();
      named_bar_sync(1 + wk, SOFT);
      float L = x_l[r] + x_l[TT + r], top = ref;
      const bool whole = done.t0 == 0 && done.t1 == done.nt;
      if (threadIdx.x % SOFT == 0 && done.t0 == 0) cut_begin(p, me, done, (int)share.cta_of(done.base + pad + done.nt - 1));
      const int in = r < nqv ? (int)(r * p.G_inv >> 16) : 0, row = r0 + in;
      const size_t at = (size_t)row * a.nq + h * p.G + (r < nqv ? r - in * p.G : 0), stride = (size_t)a.R * a.nq;
      const size_t slot = (size_t)(2 * me + (done.t0 == 0 ? 1 : 0)) * p.qv_pad + r;
      const int n_prefix = whole ? p.n_prefix : 0;
      if (whole) late_wait(p);
      const float own_top = top;
      for (int s = 0; s < n_prefix; ++s) top = fmaxf(top, p.pp_ml[2 * (s * stride + at)]);
      const float tb = top == -INFINITY ? 0.f : top, own = ex2(own_top - tb);
      L *= own;
      for (int s = 0; s < n_prefix; ++s) {
        const float2 v = *reinterpret_cast<const float2*>(p.pp_ml + 2 * (s * stride + at));
        L = fmaf(v.y, ex2(v.x - tb), L);
      }
      const bool live = whole && r < nqv && seq >= 0 && __ldcg(a.row_seq + row) == seq;
      const float inv = whole ? (live && L != 0.f ? 1.f / L : 0.f) : 1.f;
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        __syncwarp();
        float o[16];
        tmem_ld16(tO + c, o);
        if (c == 48) {
          tc_fence_before();
          warp_arrive(smem_u32(o_free));
        }
        if (r >= nqv) continue;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] *= own;
        for (int s = 0; s < n_prefix; ++s) {
          const float g = ex2(p.pp_ml[2 * (s * stride + at)] - tb);
          const float4* x = reinterpret_cast<const float4*>(p.pp_o + (s * stride + at) * TT + c0 + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 y = x[j];
            o[4 * j] = fmaf(y.x, g, o[4 * j]); o[4 * j + 1] = fmaf(y.y, g, o[4 * j + 1]);
            o[4 * j + 2] = fmaf(y.z, g, o[4 * j + 2]); o[4 * j + 3] = fmaf(y.w, g, o[4 * j + 3]);
          }
        }
        if (whole) {
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 b = inv == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          uint4* dst = reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + at * TT + c0 + c);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + slot * TT + c0 + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          if (hf == 0 && c == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * slot) = make_float2(top, L);
        }
      }
    }
  } else if (warp < 18) {
    // ---- MMA: S of a tile, then its value product ----
    const uint64_t dq = sdesc_sw128(smem_u32(sm + TO_Q + wk * 2 * OPB)), dk = sdesc_sw128(smem_u32(sm + TO_K + wk * OPB)),
                   dv = desc_mn(smem_u32(sm + TO_V + wk * 2 * OPB));
    int i = 0;
    bool ok = true;
    for (int item = 0; more && ok; ++item, more = k.next(range)) {
      ok = kv8_wait_all(smem_u32(q_full), (uint32_t)(item & 1), abort_flag, a.err);
      for (int t = k.t0; ok && t < k.t1; ++t, ++i) {
        ok = kv8_wait_all(smem_u32(k_full), (uint32_t)(i & 1), abort_flag, a.err);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < 8; ++x)   // high part, low part
            mma8_ss(tS0, dq + (((x >> 2) * OPB + (x & 3) * 32) >> 4), dk + (((x & 3) * 32) >> 4), S_IDESC, x ? 1u : 0u);
          tc_commit(smem_u32(s_full));
          tc_commit(smem_u32(k_empty));
        }
        __syncwarp();
        if (t == k.t0 && item) ok = kv8_wait_all(smem_u32(o_free), (uint32_t)((item - 1) & 1), abort_flag, a.err);
        ok = ok && kv8_wait_all(smem_u32(p_full), (uint32_t)(i & 1), abort_flag, a.err);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t fresh = t == k.t0 ? 0u : 1u;   // the first product of an item begins O
#pragma unroll
          for (int x = 0; x < 8; ++x)
            mma16_ts(tO0, tS0 + (x >> 1) * 32 + (x & 1) * 8, dv + ((x * 16 * TT) >> 4), O_IDESC, x ? 1u : fresh);
          tc_commit(smem_u32(o_done));
        }
        __syncwarp();
      }
    }
    if (!ok) {   // products in flight end before the CTA frees its TMEM
      if (elect_one()) tc_commit(smem_u32(drain));
      kv8_wait_all(smem_u32(drain), 0, abort_flag, a.err, false);
    }
  } else if (warp == 18 || warp == 19) {
    // ---- producer. Lanes 0-7 look after the eight 16-slot parts of a tile's keys, lanes 8-15 of its values ----
    const int box = a.c.table ? min(TT, 1 << a.c.block_log2) : TT, per = box / 16, part = lane & 7;
    const uint8_t* exps = (lane & 8) ? a.c.ve : a.c.ke;
    const uint64_t pol = l2_policy_evict_first();
    int i = 0, nk = 0, nv = 0;
    bool ok = true;
    auto where = [&](const Walk& w, int t) -> long long {   // this lane's part of a tile; -1: none, or not assigned
      const int slot = t * TT + part * 16;
      if (lane >= 16 || slot >= s_lim[w.gi]) return -1;
      return kv8_vec(a.c, s_seq[w.gi], w.h, slot);
    };
    for (; more && ok; more = k.next(range)) {
      const int limit = s_lim[k.gi];
      long long vec = where(k, k.t0);
      for (int t = k.t0; ok && t < k.t1; ++t, ++i) {
        const long long ahead = t + 1 < k.t1 ? where(k, t + 1) : -1;   // the next tile's table entries, a tile early
        const int parts = max(0, min(8, (limit - t * TT + 15) / 16));
        if (lane < parts && vec < 0) latch_error(a.err, DEVERR_BOUNDS);   // not assigned: unspecified keys
        const int at = (int)max(vec, 0ll);
        const int boxes = (parts + per - 1) / per;
        auto load = [&](const CUtensorMap* map, uint32_t dst, uint32_t bar) {
          if (lane == 0) mbar_expect_tx(bar, (uint32_t)(boxes * box * TT));
          for (int x = 0; x < boxes; ++x) {
            const int row = __shfl_sync(0xffffffffu, at, x * per);
            if (lane == 0) tma_load_2d(dst + x * box * TT, map, 0, row, bar, pol);
          }
        };
        // the keys' buffer is free when S of the tile before is done, the values' when they are widened
        if (i) ok = kv8_wait_all(smem_u32(k_empty), (uint32_t)((i - 1) & 1), abort_flag, a.err);
        if (!ok) break;
        if (lane < 16 && part < parts)
          copy16(smem_u32(sm + TO_EXP + (wk * 2 + (i & 1)) * 256) + (lane & 8) * 16 + part * 16, exps + at);
        copies_arrive(smem_u32(k_full));
        load(&tmK, smem_u32(sm + TO_K + wk * OPB), smem_u32(k_full));
        ++nk;
        if (i) ok = kv8_wait_all(smem_u32(v_empty), (uint32_t)((i - 1) & 1), abort_flag, a.err);
        if (!ok) break;
        load(&tmV, smem_u32(sm + TO_V8 + wk * OPB), smem_u32(v_full));
        ++nv;
        vec = ahead;
      }
    }
    if (!ok) {   // the tiles in flight land before the CTA leaves
      if (nk) kv8_wait_all(smem_u32(k_full), (uint32_t)((nk - 1) & 1), abort_flag, a.err, false);
      if (nv) kv8_wait_all(smem_u32(v_full), (uint32_t)((nv - 1) & 1), abort_flag, a.err, false);
    }
  }
  if (threadIdx.x == 0) late_wait(p);
  tc_fence_before();
  __syncthreads();
  if (warp == 18) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
}

}  // namespace

cudaError_t kv8_launch_tc(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& k, const CUtensorMap& v) {
  const int smem = tc_smem(p.groups);
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kv8_attn_tc_k), smem);
  if (e != cudaSuccess) return e;
  return launch_k(kv8_attn_tc_k, dim3(p.grid / 2), dim3(T_THREADS), smem, st, k, v, a, p);
}

}  // namespace eagle
