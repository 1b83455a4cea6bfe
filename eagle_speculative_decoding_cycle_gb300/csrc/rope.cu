// Rotary positions for the rows of a projection, outside the engine: any part of the head, both layouts of the pairs,
// frequencies of the caller's choice.
//
// A row at position p turns pair i of each head by the angle p f[i]:
//   (a, b) -> m (a cos - b sin, b cos + a sin),   inverse: the angle's sign changed.
// The angle is kept in turns, as a 64-bit fraction: f[i] / 2 pi = turns[i] 2^-64, and p * turns[i] modulo 2^64 is the angle's
// fraction of a turn without any rounding, for every 32-bit position. What is lost is turns[i]'s own rounding (a double's 2^-53, and
// 2^-64 of a turn), 2^-33 of a turn at position 2^20 at most. fp32 takes over where the fraction, in (-1/2, 1/2], meets
// sincospi. (An fp32 angle is off by 2^-24 p f: at position 100000 by 0.006 of a radian.) Sums and products are fp32, rounded once
// to the output's type.
//
// Bound by HBM for a prompt, by the launch for a step: every entry is read and written once, and a warp takes the
// cosines and sines of a row once for all of its heads (two a lane for heads of 128, handed on through shared memory). 4096 rows of
// 80 heads of 128 from fp32 columns to bf16: 40.8 us, 6.2 TB/s; 64 rows of 40 heads: 2.3 us, the time of a launch.
#include "kernels.h"
#include "ops_ext.h"

#include "common.cuh"

namespace eagle {
namespace {

constexpr int ROPE_WARPS = 8;
constexpr int ROPE_PAIRS = 128;        // most pairs a head (heads of 256 turned throughout)

// 8 entries of a row: 16 bytes of bf16, 32 of fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 r = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = r.x; x[4 * i + 1] = r.y; x[4 * i + 2] = r.z; x[4 * i + 3] = r.w;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}

// A warp takes part `slice` of the heads of a row. Its lanes take units of 16 entries: eight pairs, or 16 entries behind the
// turned part, which are copied.
template <typename TI, typename TO, bool NEIGHBOURS>
__global__ void __launch_bounds__(ROPE_WARPS * 32)
    rope_k(const RopeArgs a) {
  __shared__ __align__(16) float cs[ROPE_WARPS][ROPE_PAIRS], sn[ROPE_WARPS][ROPE_PAIRS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long job = (long long)blockIdx.x * ROPE_WARPS + warp;
  const int row = (int)(job / a.slices), slice = (int)(job - (long long)row * a.slices);
  PDL_ENTRY();
  if (row >= a.R) return;
  const long long pos = a.pos[row];
  for (int i = lane; i < a.rot / 2; i += 32) {
    const float turn = __ll2float_rn((long long)((unsigned long long)pos * a.turns[i])) * 0x1p-63f;   // half turns
    float s, c;
    sincospif(turn, &s, &c);
    cs[warp][i] = c * a.factor;
    sn[warp][i] = (a.inverse ? -s : s) * a.factor;
  }
  __syncwarp();
  const int units = a.d / 16, heads = a.nq + a.nkv;
  const int h0 = (int)((long long)heads * slice / a.slices), h1 = (int)((long long)heads * (slice + 1) / a.slices);
  const int step = 32 / units * units;      // lanes in use: each keeps its unit of the head
  if (lane >= step) return;
  const int u = lane % units, turned = a.rot / 16;
  const bool turn = u < turned;
  // the entries of this lane: 8 at e0 and 8 at e1
  const int e0 = !turn || NEIGHBOURS ? u * 16 : u * 8, e1 = !turn || NEIGHBOURS ? e0 + 8 : e0 + a.rot / 2;
  float c[8], s[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = cs[warp][u * 8 + i];
      s[i] = sn[warp][u * 8 + i];
    }
  }
#pragma unroll 2
  for (int h = h0 + lane / units; h < h1; h += step / units) {
    const bool is_k = h >= a.nq;
    const int hh = is_k ? h - a.nq : h;
    const TI* src = reinterpret_cast<const TI*>(is_k ? a.k : a.q) + row * (is_k ? a.ldk : a.ldq) + (long long)hh * a.d;
    TO* dst = reinterpret_cast<TO*>(is_k ? a.ko : a.qo) + row * (is_k ? a.ldko : a.ldqo) + (long long)hh * a.d;
    float x[8], y[8];
    load8(src + e0, x);
    load8(src + e1, y);
    if (turn) {
      if (NEIGHBOURS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rope_pair(x[2 * i], x[2 * i + 1], c[i], s[i], x[2 * i], x[2 * i + 1]);
          rope_pair(y[2 * i], y[2 * i + 1], c[4 + i], s[4 + i], y[2 * i], y[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_pair(x[i], y[i], c[i], s[i], x[i], y[i]);
      }
    }
    store8(dst + e0, x);
    store8(dst + e1, y);
  }
}

template <typename TI, typename TO>
cudaError_t launch_rope(cudaStream_t st, const RopeArgs& a, bool neighbours, unsigned grid) {
  return neighbours ? launch_k(rope_k<TI, TO, true>, dim3(grid), dim3(ROPE_WARPS * 32), 0, st, a)
                    : launch_k(rope_k<TI, TO, false>, dim3(grid), dim3(ROPE_WARPS * 32), 0, st, a);
}

}  // namespace

int rope_rows(cudaStream_t st, RopeArgs a, bool in_f32, bool out_f32, bool neighbours) {
  // few rows: their heads shared out until there is a warp for each 2 KB or some 16 warps an SM
  const int heads = a.nq + a.nkv, per_pass = 32 / (a.d / 16);
  const int most = (heads + per_pass - 1) / per_pass;
  const long long want = (152ll * 16 + a.R - 1) / a.R;
  a.slices = (int)(want < most ? want : most);
  if (a.slices < 1) a.slices = 1;
  const long long jobs = (long long)a.R * a.slices, grid = (jobs + ROPE_WARPS - 1) / ROPE_WARPS;
  if (grid > 0x7fffffffll) return -1;
  const cudaError_t e = in_f32 ? (out_f32 ? launch_rope<float, float>(st, a, neighbours, (unsigned)grid)
                                          : launch_rope<float, __nv_bfloat16>(st, a, neighbours, (unsigned)grid))
                               : (out_f32 ? launch_rope<__nv_bfloat16, float>(st, a, neighbours, (unsigned)grid)
                                          : launch_rope<__nv_bfloat16, __nv_bfloat16>(st, a, neighbours, (unsigned)grid));
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace eagle
