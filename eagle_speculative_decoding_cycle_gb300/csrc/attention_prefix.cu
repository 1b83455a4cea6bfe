// Attention of all rows of a batch over one shared bf16 prefix, on the 5th-generation tensor cores.
//
// Every row sees every prefix key, so the rows of all sequences are one long side: per KV head two dense products,
// S = Q K^T and O = P V, with M = rows x query heads (hundreds to tens of thousands), N = P keys, and no
// mask but the prefix's end. 4 M P d flops a head against 4 P d + 6 M d bytes: bound by the tensor cores from
// some 150 query vectors a head on, and below by reading the prefix once.
//
// One CTA takes two tiles of 128 query vectors of one KV head and a range of 128-key tiles, 12 warps:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one thread a query vector (TMEM lane): S row -> maximum, weights as bf16 back
//                   into TMEM over S, running sum; O is rescaled only when the maximum moves by more than 2^8;
//   warp 8          TMA: Q once, K and V tiles through two-stage rings (128-byte swizzle);
//   warps 9, 10     tcgen05.mma of tile 0 / 1: S = Q K^T (operands in shared memory), O += P V (P in TMEM, V read MN-major).
// S comes in halves of 64 keys, each with its own barriers: while one half is in its softmax warps the tensor cores run the
// other half's value product and next S, and the other tile's. (S of 128 keys at once leaves a chain of product, softmax,
// product: 121 us in all for 4096 shared tokens under 64 x 17 rows of 32 heads, against 106 (103 since); with two threads a
// query vector 118; halves with one issuing warp for both tiles 135, each of its waits taking some 250 clocks.)
// TMEM: S0 S1 (128 columns each, P over the first half of each 64), O0 O1 (d each). That prefix alone: 62 us, of them 38 us
// of products at the rate of a large GEMM; tensor pipe 46% active. 128 keys of a pair of tiles take some 3300 clocks where
// their products take 2048: bound by the way of a half through its warps and back (softmax 900 clocks, hand-overs and issue
// some 1500, two halves under way a tile; with an eighth of the products 8 us less, without the ex2 2 us less).
// Weights are rounded to bf16 (2^-8 relative at most, as the bf16 V that they meet; their sum is kept in fp32 of the
// unrounded weights). A second part, as the attention over the bf16 cache has it, takes half of the products again: 120 us
// instead of 103 for that case and 46 instead of 42 for 8192 shared tokens under 64 rows, for 0.0016 relative off the 64-bit
// results instead of 0.0021 (0.0015 of it the weights', 0.0016 the rounding of the results to bf16). Results leave as fp32
// partials (o, m, l) of each key range, which the attention over the rows' own slots joins in its epilogue.
#include "attn_tc.cuh"
#include "kernels.h"

#include <algorithm>

namespace eagle {
namespace {

constexpr int PT = 128;            // keys a tile, query vectors a tile
constexpr int PH = PT / 2;         // keys of one S: half a tile
constexpr int PF_THREADS = 384;
constexpr float PF_LAZY = 8.f;
// CTAs that run at once, one an SM. A number, not the current device's count: the scratch size is asked for without a
// device in hand, and both must cut alike. With another count the results are the same, the cut is only a worse guess.
constexpr int PF_SMS = 152;

template <int D>
struct PfShape {
  static constexpr int HALVES = D / 64, HALF = PT * 128;        // 64 dims of 128 rows
  static constexpr int OP = HALVES * HALF;                      // one operand tile
  static constexpr int OFF_Q = 0, OFF_K = 2 * OP, OFF_V = OFF_K + 2 * OP, OFF_BAR = OFF_V + 2 * OP;
  static constexpr int BYTES = 1024 + OFF_BAR + 256;
};

struct PfArgs {
  int R, nq, G, RB, P;         // rows, query heads, query heads a KV head, rows a tile
  int splits, tiles, pairs;    // key ranges, key tiles, pairs of query tiles
  float sl2;                   // scale * log2(e)
  float *o, *ml;               // [splits][R * nq][D], [splits][R * nq][2]
  int* err;
};

template <int D>
__global__ void __launch_bounds__(PF_THREADS, 1)
    prefix_k(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const PfArgs a) {
  using Sh = PfShape<D>;
  extern __shared__ uint8_t pf_smem[];
  uint8_t* sm = pf_smem + (-smem_u32(pf_smem) & 1023u);   // (not by pointer masks: accesses then lose the shared space)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::OFF_BAR);
  uint64_t *q_full = bars, *k_full = bars + 1, *k_empty = bars + 3, *v_full = bars + 5, *v_empty = bars + 7,
           *s_full = bars + 9 /* [tile][half] */, *p_full = bars + 13 /* [tile][half] */, *o_done = bars + 17 /* [tile][half] */, *drain = bars + 21 /* [tile] */;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 23);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int split = blockIdx.x % a.splits, pair = blockIdx.x / a.splits % a.pairs, h = blockIdx.x / (a.splits * a.pairs);
  const int r0 = pair * 2 * a.RB;
  const int nmt = r0 + a.RB < a.R ? 2 : 1;     // query tiles of this CTA
  const int t0 = (int)((long long)a.tiles * split / a.splits), t1 = (int)((long long)a.tiles * (split + 1) / a.splits);
  const int nt = t1 - t0;                      // >= 1: splits <= tiles
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(q_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(k_full + i), 1);
      mbar_init(smem_u32(k_empty + i), nmt);
      mbar_init(smem_u32(v_full + i), 1);
      mbar_init(smem_u32(v_empty + i), nmt);
      mbar_init(smem_u32(drain + i), 1);
      for (int hf = 0; hf < 2; ++hf) {
        mbar_init(smem_u32(s_full + 2 * i + hf), 1);
        mbar_init(smem_u32(p_full + 2 * i + hf), 4);
        mbar_init(smem_u32(o_done + 2 * i + hf), 1);
      }
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PDL_ENTRY();

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int mt = warp >> 2, qv = threadIdx.x & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + mt * PT + lane_off, tO = tmem + 2 * PT + mt * D + lane_off;
    float m = -INFINITY, l = 0.f;
    bool ok = mt < nmt;
    for (int j = 0; ok && j < 2 * nt; ++j) {   // halves of the key tiles
      const int i = j >> 1, hf = j & 1;
      const uint32_t tP = tS + hf * PH;
      ok = kv8_wait(smem_u32(s_full + 2 * mt + hf), (uint32_t)(i & 1), abort_flag, a.err);
      if (!ok) break;
      tc_fence_after();
      float s[PH];
#pragma unroll
      for (int c = 0; c < PH; c += 32) tmem_ld32_async(tP + c, s + c);
#pragma unroll
      for (int c = 0; c < PH; c += 32) tmem_wait_ld(s + c);
      const int last = a.P - (t0 + i) * PT - hf * PH;    // keys of this half, 64 but at the prefix's end
      if (last < PH)
#pragma unroll
        for (int c = 0; c < PH; ++c) s[c] = c < last ? s[c] : -INFINITY;
      float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
      for (int c = 4; c + 7 < PH; c += 8) {
        x0 = max3(x0, s[c], s[c + 1]);
        x1 = max3(x1, s[c + 2], s[c + 3]);
        x2 = max3(x2, s[c + 4], s[c + 5]);
        x3 = max3(x3, s[c + 6], s[c + 7]);
      }
      const float mx = fmaxf(max3(x0, x1, fmaxf(s[PH - 4], s[PH - 3])), max3(x2, x3, fmaxf(s[PH - 2], s[PH - 1])));
      const bool raise = (mx - m) * a.sl2 > PF_LAZY;
      float corr = 1.f;
      if (raise) {
        corr = pf_ex2((m - mx) * a.sl2);
        m = mx;
        l *= corr;
      }
      if (j > 0 && __any_sync(0xffffffffu, raise)) {
        // the last product into O must be there before O is rescaled (the one before it is: this S came behind it)
        ok = kv8_wait(smem_u32(o_done + 2 * mt + (hf ^ 1)), (uint32_t)(((j - 1) >> 1) & 1), abort_flag, a.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tmem_ld16(tO + c, o);
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] *= corr;
          tmem_st16(tO + c, o);
        }
      }
      // the difference comes first: it is exact where it matters, near the maximum, whatever the size of the scores
      const f32x2 nm = two(-m, -m), s2 = two(a.sl2, a.sl2);
      f32x2 sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
      for (int qt = 0; qt < PH / 32; ++qt) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float2 x = one_by_one(mul2(add2(two(s[qt * 32 + c], s[qt * 32 + c + 1]), nm), s2));
          x.x = pf_ex2(x.x);
          x.y = pf_ex2(x.y);
          sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], two(x.x, x.y));
          const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
          w[c / 2] = *reinterpret_cast<const uint32_t*>(&b);
        }
        tmem_st16u(tP + qt * 16, w);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(smem_u32(p_full + 2 * mt + hf));
      const float2 sums = one_by_one(add2(sum[0], sum[1]));
      l += sums.x + sums.y;
    }
    if (mt < nmt) {
      const int row = r0 + mt * a.RB + qv / a.G;
      const bool write = qv < a.RB * a.G && row < a.R;
      const size_t q = (size_t)split * a.R * a.nq + (size_t)row * a.nq + h * a.G + qv % a.G;
      if (ok && kv8_wait(smem_u32(o_done + 2 * mt + 1), (uint32_t)((nt - 1) & 1), abort_flag, a.err)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(tO + c, o);
          if (write)
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(a.o + q * D + c + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
        if (write) {
          a.ml[2 * q] = m * a.sl2;
          a.ml[2 * q + 1] = l;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 8) {
      // ---- TMA ----
      const int qbytes = a.RB * a.G * 128;
      if (elect_one()) {
        mbar_expect_tx(smem_u32(q_full), (uint32_t)(nmt * Sh::HALVES * qbytes));
        for (int mt = 0; mt < nmt; ++mt)
          for (int x = 0; x < Sh::HALVES; ++x)
            tma_load_3d(smem_u32(sm + Sh::OFF_Q + mt * Sh::OP + x * Sh::HALF), &tmQ, x * 64, h * a.G, r0 + mt * a.RB,
                        smem_u32(q_full));
      }
      int nk = 0, nv = 0;
      for (int i = 0; i < nt; ++i) {
        const int st = i & 1;
        const uint32_t ph = (uint32_t)((i / 2 - 1) & 1);
        if (i >= 2 && !kv8_wait_all(smem_u32(k_empty + st), ph, abort_flag, a.err)) break;
        if (elect_one()) {
          mbar_expect_tx(smem_u32(k_full + st), Sh::OP);
          for (int x = 0; x < Sh::HALVES; ++x)
            tma_load_3d(smem_u32(sm + Sh::OFF_K + st * Sh::OP + x * Sh::HALF), &tmK, x * 64, (t0 + i) * PT, h,
                        smem_u32(k_full + st));
        }
        ++nk;
        if (i >= 2 && !kv8_wait_all(smem_u32(v_empty + st), ph, abort_flag, a.err)) break;
        if (elect_one()) {
          mbar_expect_tx(smem_u32(v_full + st), Sh::OP);
          for (int x = 0; x < Sh::HALVES; ++x)
            tma_load_3d(smem_u32(sm + Sh::OFF_V + st * Sh::OP + x * Sh::HALF), &tmV, x * 64, (t0 + i) * PT, h,
                        smem_u32(v_full + st));
        }
        ++nv;
      }
      if (*abort_flag) {   // copies in flight land before the CTA leaves: the last two of each ring
        kv8_wait_all(smem_u32(q_full), 0, abort_flag, a.err, false);
        for (int j = max(0, nk - 2); j < nk; ++j) kv8_wait_all(smem_u32(k_full + (j & 1)), (uint32_t)((j / 2) & 1), abort_flag, a.err, false);
        for (int j = max(0, nv - 2); j < nv; ++j) kv8_wait_all(smem_u32(v_full + (j & 1)), (uint32_t)((j / 2) & 1), abort_flag, a.err, false);
      }
    } else if (warp <= 8 + nmt) {
      // ---- MMA: one warp a query tile (both by one warp: 4 waits a tile, some 250 clocks each though what they wait for is
      // there, held the tensor cores up) ----
      constexpr uint32_t IS = pf_idesc(PH, false), IO = pf_idesc(D, true);
      const int mt = warp - 9;
      const uint32_t tS = tmem + mt * PT, tO = tmem + 2 * PT + mt * D;
      // operand descriptors; an offset of n bytes adds n >> 4
      const uint64_t dq = sdesc_sw128(smem_u32(sm + Sh::OFF_Q + mt * Sh::OP)), dk = sdesc_sw128(smem_u32(sm + Sh::OFF_K)),
                     dv = pf_desc_mn(smem_u32(sm + Sh::OFF_V), Sh::HALF);
      auto issue_s = [&](int i, int hf) {   // by one lane
        const uint64_t k = dk + (((i & 1) * Sh::OP + hf * PH * 128) >> 4);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int at = ((x >> 2) * Sh::HALF + (x & 3) * 32) >> 4;
          tc_mma_bf16(tS + hf * PH, dq + at, k + at, IS, x ? 1u : 0u);
        }
        tc_commit(smem_u32(s_full + 2 * mt + hf));
        if (hf) tc_commit(smem_u32(k_empty + (i & 1)));
      };
      bool ok = kv8_wait_all(smem_u32(q_full), 0, abort_flag, a.err) && kv8_wait_all(smem_u32(k_full), 0, abort_flag, a.err);
      if (ok) {
        tc_fence_after();
        if (elect_one()) {
          issue_s(0, 0);
          issue_s(0, 1);
        }
        __syncwarp();
      }
      for (int i = 0; ok && i < nt; ++i) {
        // P V of a half, then the next tile's S over the same columns: the tensor cores take them in this order. The operands
        // are waited for before the weights, so that nothing stands between these and the products.
        const bool next = i + 1 < nt;
        ok = kv8_wait_all(smem_u32(v_full + (i & 1)), (uint32_t)((i / 2) & 1), abort_flag, a.err);
        if (ok && next) ok = kv8_wait_all(smem_u32(k_full + ((i + 1) & 1)), (uint32_t)(((i + 1) / 2) & 1), abort_flag, a.err);
        const uint64_t v = dv + (i & 1) * (Sh::OP >> 4);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          ok = ok && kv8_wait_all(smem_u32(p_full + 2 * mt + hf), (uint32_t)(i & 1), abort_flag, a.err);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma_ts(tO, tS + hf * PH + x * 8, v + ((hf * 4 + x) * 2048 >> 4), IO, i || hf || x ? 1u : 0u);
            tc_commit(smem_u32(o_done + 2 * mt + hf));
            if (hf) tc_commit(smem_u32(v_empty + (i & 1)));
            if (next) issue_s(i + 1, hf);
          }
          __syncwarp();
        }
      }
      if (!ok) {   // products in flight end before the CTA frees its TMEM
        if (elect_one()) tc_commit(smem_u32(drain + mt));
        kv8_wait_all(smem_u32(drain + mt), 0, abort_flag, a.err, false);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// bf16 [n2][n1][d] as boxes of 64 x b1 x b2.
bool map3(CUtensorMap* m, const void* p, int d, int n1, int n2, int b1, int b2) {
  const auto fn = pf_encode();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)n1 * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_prefix(cudaStream_t st, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const PfArgs& p, int grid) {
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(prefix_k<D>), PfShape<D>::BYTES);
  if (e != cudaSuccess) return e;
  return launch_k(prefix_k<D>, dim3(grid), dim3(PF_THREADS), PfShape<D>::BYTES, st, q, k, v, p);
}

}  // namespace

// Key ranges: the count that ends first on 152 SMs, a range costing its tiles plus about one and a half for filling the
// pipeline and writing its partials, which the joining side reads again (a third of a tile each).
int kv8_prefix_splits(int nkv, int R, int nq, int P) {
  const int RB = PT / (nq / nkv), tiles = (P + PT - 1) / PT;
  const long long items = (long long)nkv * ((R + 2 * RB - 1) / (2 * RB));
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= std::min(tiles, 32); ++s) {
    const double t = (double)((items * s + PF_SMS - 1) / PF_SMS) * ((tiles + s - 1) / s + 1.5) + s / 3.0;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

int kv8_prefix(cudaStream_t st, const Kv8Attn& a, int splits, float* o, float* ml) {
  PfArgs p{};
  const int nkv = a.c.nkv, d = a.c.d;
  p.R = a.R; p.nq = a.nq; p.G = a.nq / nkv; p.RB = PT / p.G; p.P = a.P;
  p.splits = splits; p.tiles = (a.P + PT - 1) / PT; p.pairs = (a.R + 2 * p.RB - 1) / (2 * p.RB);
  p.sl2 = a.scale * 1.4426950408889634f;
  p.o = o; p.ml = ml; p.err = a.err;
  const long long grid = (long long)nkv * p.pairs * splits;
  if (grid > 0x7fffffffll) return -1;
  CUtensorMap q, k, v;
  if (!map3(&q, a.q, d, a.nq, a.R, p.G, p.RB) || !map3(&k, a.pk, d, a.P, nkv, PT, 1) || !map3(&v, a.pv, d, a.P, nkv, PT, 1))
    return -4;
  const cudaError_t e = d == 128 ? launch_prefix<128>(st, q, k, v, p, (int)grid) : launch_prefix<64>(st, q, k, v, p, (int)grid);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return -4;
  }
  return 0;
}

}  // namespace eagle
