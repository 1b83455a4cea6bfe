// How an 8-bit cache attention call is cut into work and put together again: shared by its kernels.
//
// A call is a list of items (row block, KV head), each with the tiles of the slots that its rows see; lengths are
// read on the device. Laid end to end the tiles are shared out over the CTAs in equal contiguous ranges, so that
// ragged batches and one long sequence balance alike. An item inside one CTA's range is finished there; the pieces of
// an item cut by range ends (at most two a CTA) go to scratch as (o, m, l) and a second launch joins them in order.
// An item also costs its start and its end, counted as `pad` tiles (with 0, 2, 4, 6, 8 of them: 64 ragged sequences, one row
// each, 44.8, 39.9, 40.2, 40.9, 41.4 us; one of 32768 slots 23.8, 23.0, 22.2, 22.3, 22.3; 64 behind 8192 shared slots 43.9,
// 43.3, 43.2, 42.9, 43.7).
#pragma once

#include "kv8.cuh"

#include <cuda.h>

namespace eagle {

constexpr int KV8_MAX_QV = 128;       // query vectors a block of rows
constexpr int KV8_MAX_GROUPS = 512;   // row blocks a launch (more: several launches)
constexpr int KV8_MAX_CTAS = 384;     // grid limit that the scratch is sized for

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 16 bytes into shared memory; this thread's earlier copies arrive on `bar` once they are there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Weights of own slots. With x a score (log2 units) and 2^e its value's factor, the B operand of the value product is
// w = 2^(x + e - ref) of each query vector, fp16, and the sum takes w 2^-e in fp32. ref is set KV8_HEAD below the largest
// x + e and moved once one passes it by more than KV8_TOP: w is at most 2^15, the largest at least 2^7 (fp16 holds 2^-24 to
// 2^16), so that what a weight loses to fp16's smallest step, 2^-25, is 2^-32 of the largest product of a weight and its
// value's size, whatever the sizes of values that the query vector gives no weight. (One reference exponent for all values of
// a tile lost small weights beside them: 6000 keys, most of weight 2^-16 beside values 2^12 times theirs, 7% off.)
constexpr float KV8_HEAD = 7.f, KV8_TOP = 15.f;

// A value's e and 2^-e from its byte. A vector that held something not finite makes NaN of the weight.
__device__ __forceinline__ float kv8_exponent(int byte) {
  return byte == KV8_BAD ? __int_as_float(0x7fffffff) : (float)(max(byte, KV8_LOWEST) - KV8_BIAS);
}
// 2^n, 0 below the normal range.
__device__ __forceinline__ float pow2i(int n) { return n < -126 ? 0.f : __int_as_float((min(n, 127) + 127) << 23); }
__device__ __forceinline__ float kv8_inverse(int byte) { return pow2i(KV8_BIAS - max(byte, KV8_LOWEST)); }

// How a call's rows are cut and its tiles shared out: the same numbers in both kernels and the scratch size.
struct Plan {
  int G, RB, nb, QV;      // query heads a KV head; rows a block; blocks a sequence; query vectors a block
  uint32_t G_inv;         // x / G = x * G_inv >> 16 for x < 128
  int width;              // lanes that look at one row block
  int nkv;
  int tk;                 // keys a tile
  int groups;             // row blocks of this launch, from block g0 on
  int g0;
  int grid, min_tiles;    // CTAs at most; tiles a CTA at least
  int join_cols, join_ways;   // a join CTA: query vectors, threads' teams that share one's pieces (powers of two)
  int pad;                // what starting and joining an item costs, in tiles: an item of nt tiles spans pad + nt units
  int qv_pad;             // query vectors of a partial
  float* part_o;          // [2 grid][qv_pad][D]
  float* part_ml;         // [2 grid][qv_pad][2]
  int4* cut;              // items that range ends cut: row block, head, first CTA, last CTA (-1: not cut)
  int by_item;            // cut is indexed by item (no more items than CTAs), else by the item's first CTA
  const float *pp_o, *pp_ml;   // prefix partials [n_prefix][R * nq][D], [..][2]
  int n_prefix;
  int late;               // the launch just before this one makes the prefix's partials: wait for it where they are read
};

// Behind the prefix kernel the own slots' kernel starts as soon as that one's last CTAs have started (they trigger it
// after their own wait, so all that came before the call is complete), and waits for its partials where it reads them.
// One thread of each CTA waits before it ends, so that the join finds both kernels complete.
// What it reads before that (rows, lengths, masks, tables, q) comes from L2 by __ldcg, cp.async.cg or TMA: no line that an
// earlier kernel left in an SM's L1.
__device__ __forceinline__ void late_entry(const Plan& p) {
  if (!p.late) pdl_wait();
  pdl_trigger();
}
__device__ __forceinline__ void late_wait(const Plan& p) {
  if (p.late) pdl_wait();
}

// The units W of a launch over its CTAs: the first `more` CTAs take `per` + 1, the others `per`. An item's tiles are its
// last units, so a range that ends inside its first `pad` units has none of it.
struct Share {
  uint32_t ctas, per, more;
  __device__ __forceinline__ Share(const Plan& p, uint32_t tiles, int pad) {
    // a CTA takes p.min_tiles tiles at least (one for each key group), or a whole average item where those are shorter
    const uint32_t items = (uint32_t)p.groups * p.nkv, W = tiles + items * pad;
    ctas = max(1u, min((uint32_t)p.grid, tiles / max(1u, min((uint32_t)p.min_tiles, tiles / items))));
    per = W / ctas;
    more = W - per * ctas;
  }
  __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * per + min(c, more); }
  __device__ __forceinline__ uint32_t cta_of(uint32_t u) const {
    const uint32_t wide = more * (per + 1);
    return u < wide ? u / (per + 1) : more + (u - wide) / per;
  }
};
// The pad of a launch: p.pad, but not more than a CTA's even share of the tiles (few long items: ranges would lie in pads).
__device__ __forceinline__ int pad_of(const Plan& p, uint32_t tiles) { return (int)min((uint32_t)p.pad, tiles / (uint32_t)p.grid); }

// A row block's rows, its sequence (that of the first row that is not padding among the sequence's rows) and the
// first slot past everything that its rows see.
struct Group {
  int r0, r1, seq, limit;
};
// For a sequence whose first row is padding: that of its first row in [s0, s1) that is not, -1 if [r0, r1) is all padding. By
// `width` neighbouring lanes (a power of two), eight rows a lane in flight (one after another they cost a load's latency a row:
// two chunks of 4096 rows, one of them all padding, 1912 us; now 346, and 560 with none padding). Not inline: its rare call
// then costs the others nothing.
static __device__ __noinline__ int seq_behind_padding(const int* row_seq, int s0, int s1, int r0, int r1, int width) {
  const int lane = threadIdx.x & 31, sub = lane & (width - 1);
  const unsigned group = (width == 32 ? 0xffffffffu : (1u << width) - 1u) << (lane - sub);
  bool any = false;
  for (int r = r0 + sub; r < r1 && !any; r += width) any = __ldcg(row_seq + r) >= 0;
  if (!__any_sync(group, any)) return -1;
  for (int b = s0; b < s1; b += 8 * width) {
    int v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = b + j * width + sub < s1 ? __ldcg(row_seq + b + j * width + sub) : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const unsigned live = __ballot_sync(group, v[j] >= 0);
      if (live) return __shfl_sync(group, v[j], __ffs(live) - 1);
    }
  }
  return -1;
}
// By `width` neighbouring lanes (a power of two up to 8); gi out of range gives an empty block. All lanes of a warp call.
__device__ __forceinline__ Group group_of(const Kv8Attn& a, const Plan& p, int gi, int width, bool latch) {
  const int sub = threadIdx.x & (width - 1);
  Group o;
  const int sidx = (p.g0 + gi) / p.nb, rb = (p.g0 + gi) - sidx * p.nb;
  const int s0 = sidx * a.rows_per_seq, s1 = (int)min((long long)s0 + a.rows_per_seq, (long long)a.R);
  o.r0 = s0 + rb * p.RB;
  o.r1 = gi < p.groups ? min(o.r0 + p.RB, s1) : o.r0;   // a block that exists has rows
  // (the first rows' numbers are on their way while the sequence's is)
  const int first = o.r0 + sub;
  const int first_rs = first < o.r1 ? __ldcg(a.row_seq + first) : -1, first_slot = first < o.r1 && a.mode == 0 ? __ldcg(a.row_slot + first) : 0;
  o.seq = o.r0 < o.r1 ? __ldcg(a.row_seq + s0) : -1;
  if (o.r0 < o.r1 && o.seq < 0) o.seq = seq_behind_padding(a.row_seq, s0, s1, o.r0, o.r1, width);
  bool bad = o.seq >= a.c.max_batch;
  if (bad) o.seq = -1;
  const int ctx = a.mode == 1 && o.seq >= 0 ? __ldcg(a.ctx_len + o.seq) : 0;
  int lim = 0;
  if (o.seq >= 0) {
    bad = bad || ctx < 0;
    const int words = (a.tree_T + 63) >> 6;
    for (int r = o.r0 + sub; r < o.r1; r += width) {
      const int rs = r == first ? first_rs : __ldcg(a.row_seq + r);
      int end = a.mode == 0 ? min(r == first ? first_slot : __ldcg(a.row_slot + r), INT32_MAX - 1) + 1 : ctx;
      if (a.mode == 1)
        for (int w = 0; w < words; ++w) {
          uint64_t m = __ldcg(a.mask + (size_t)r * a.mask_words + w);
          if (w == words - 1 && (a.tree_T & 63)) m &= (1ull << (a.tree_T & 63)) - 1;
          if (m) end = (int)min((long long)INT32_MAX, (long long)ctx + w * 64 + 64 - __clzll((long long)m));
        }
      if (rs == o.seq) lim = max(lim, end);
      else bad = bad || rs >= 0;
    }
  }
  for (int d = width >> 1; d > 0; d >>= 1) lim = max(lim, __shfl_xor_sync(0xffffffffu, lim, d));
  bad = bad || lim > a.c.cap;
  o.limit = ctx < 0 ? 0 : max(0, min(lim, a.c.cap));
  if (latch && bad) latch_error(a.err, DEVERR_BOUNDS);
  return o;
}

// A partial of one query vector: its maximum and sum (ml), its D values (o).
struct Part {
  const float *ml, *o;
};
// Adds n partials to (top, L, o), o 8 values of a query vector whose D values are spread over D / 8 neighbouring
// lanes (sub: this lane's place among them): the lanes share the (m, l) pairs, the sums run in the order of the partials,
// the values of FB partials are in flight at a time.
__device__ __forceinline__ void load8(const float* p, float4* x) {
  x[0] = reinterpret_cast<const float4*>(p)[0];
  x[1] = reinterpret_cast<const float4*>(p)[1];
}
template <int D, int FB, typename At>
__device__ __forceinline__ void fold(int n, At at, int sub, float& top, float& L, float* o) {
  constexpr int GL = D / 8;
  const unsigned group = ((1u << GL) - 1u) << ((threadIdx.x & 31) / GL * GL);
  for (int i0 = 0; i0 < n; i0 += GL) {   // GL partials at a time
    float2 ml = make_float2(-INFINITY, 0.f);
    if (i0 + sub < n) ml = *reinterpret_cast<const float2*>(at(i0 + sub).ml);
    const int cnt = min(GL, n - i0);
    float4 x[FB][2];   // the first partials' values come under the maximum's way through the lanes
#pragma unroll
    for (int j = 0; j < FB; ++j)
      if (j < cnt) load8(at(i0 + j).o + sub * 8, x[j]);
    float mx = fmaxf(top, ml.x);
#pragma unroll
    for (int d = GL / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(group, mx, d));
    const float base = mx == -INFINITY ? 0.f : mx, f = ex2(top - base), w = ex2(ml.x - base), lw = ml.y * w;
    top = mx;
    L *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= f;
    for (int j0 = 0; j0 < cnt; j0 += FB) {
#pragma unroll
      for (int j = 0; j < FB; ++j)
        if (j0 && j0 + j < cnt) load8(at(i0 + j0 + j).o + sub * 8, x[j]);
#pragma unroll
      for (int j = 0; j < FB; ++j)
        if (j0 + j < cnt) {
          const float4 a = x[j][0], b = x[j][1];
          const float wj = __shfl_sync(group, w, j0 + j, GL);
          L += __shfl_sync(group, lw, j0 + j, GL);
          o[0] = fmaf(a.x, wj, o[0]); o[1] = fmaf(a.y, wj, o[1]); o[2] = fmaf(a.z, wj, o[2]); o[3] = fmaf(a.w, wj, o[3]);
          o[4] = fmaf(b.x, wj, o[4]); o[5] = fmaf(b.y, wj, o[5]); o[6] = fmaf(b.z, wj, o[6]); o[7] = fmaf(b.w, wj, o[7]);
        }
    }
  }
}

// 8 finished values of one query vector; nothing seen, or a row that is padding or invalid: zeros.
__device__ __forceinline__ void store8(const Kv8Attn& a, size_t at, int D, int c, bool live, float L, const float* o) {
  uint32_t w[4];
  const bool none = !live || L == 0.f;
  const float inv = 1.f / L;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(none ? 0.f : o[2 * i] * inv, none ? 0.f : o[2 * i + 1] * inv);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>((__nv_bfloat16*)a.out + at * D + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA's range as a walk over its items, in order.
struct Range {
  const int* pref;           // [groups + 1] tiles a head before each row block
  int pad, nkv, groups;
  uint32_t w0, w1;
  __device__ __forceinline__ uint32_t units(int g) const { return (uint32_t)(pref[g] + g * pad) * nkv; }
};
struct Walk {
  int gi, h, t0, t1, nt;     // row block, head, its tiles [t0, t1) of nt
  uint32_t base;             // the item's first unit
  __device__ __forceinline__ void enter(const Range& r, uint32_t from) {   // from unit `from` of the item on
    nt = r.pref[gi + 1] - r.pref[gi];
    t0 = max(0, (int)from - r.pad);
    t1 = min(nt, (int)(r.w1 - base) - r.pad);
  }
  __device__ __forceinline__ bool begin(const Range& r) {   // false: no tiles in the whole range
    int lo = 0, hi = r.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (r.units(mid) <= r.w0) lo = mid;
      else hi = mid;
    }
    gi = lo;
    const uint32_t first = r.units(lo), span = r.pref[lo + 1] - r.pref[lo] + r.pad;
    h = (int)((r.w0 - first) / span);
    base = first + h * span;
    enter(r, r.w0 - base);
    return t0 < t1;
  }
  __device__ __forceinline__ bool next(const Range& r) {    // false: the range ends
    base += nt + r.pad;
    if (base + r.pad >= r.w1) return false;
    if (++h == r.nkv) {
      h = 0;
      ++gi;
    }
    enter(r, 0);
    return true;
  }
};

// Who writes p.cut: by CTA, each CTA at its start (none) and for the item that it begins and does not finish; by item,
// the CTA that begins the item.
__device__ __forceinline__ void cut_none(const Plan& p, int cta) {
  if (!p.by_item) p.cut[cta] = make_int4(0, 0, 0, -1);
}
__device__ __forceinline__ void cut_begin(const Plan& p, int cta, const Walk& k, int last) {   // of an item with t0 = 0
  if (k.t1 < k.nt) p.cut[p.by_item ? k.gi * p.nkv + k.h : cta] = make_int4(k.gi, k.h, cta, last);
  else if (p.by_item) p.cut[k.gi * p.nkv + k.h] = make_int4(0, 0, 0, -1);
}

// The launch's items as every CTA sees them: s_pref [groups + 1] (tiles a head before each row block), s_lim and s_seq
// [groups]. By all threads of the CTA; ends with a barrier.
__device__ __forceinline__ void lay_out(const Kv8Attn& a, const Plan& p, int* s_pref, int* s_lim, int* s_seq) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g0 = 0; g0 < p.groups; g0 += blockDim.x / p.width) {
    const int gi = g0 + threadIdx.x / p.width;
    const Group gr = group_of(a, p, gi, p.width, blockIdx.x == 0);
    if (gi < p.groups && (threadIdx.x & (p.width - 1)) == 0) {
      s_lim[gi] = gr.limit;
      s_seq[gi] = gr.seq;
      s_pref[gi + 1] = max(1, (gr.limit + p.tk - 1) / p.tk);
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
}

// Host side: the kernel for up to 128 query vectors a block on tcgen05 (head_dim 128).
cudaError_t kv8_launch_tc(cudaStream_t st, const Kv8Attn& a, Plan& p, const CUtensorMap& k, const CUtensorMap& v);

}  // namespace eagle
