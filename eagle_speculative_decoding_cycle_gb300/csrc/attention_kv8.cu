// Attention over the 8-bit KV cache, behind an optional bf16 prefix that all rows share.
//
//   o = sum_s p_s v_s / sum_s p_s,  p_s = exp(scale q.k_s - m),  m the running maximum,
// over the prefix and the slots that the row sees: one softmax, in one pass over the keys.
#include "kv8.cuh"
#include "kernels.h"

#include <cuda_fp16.h>

namespace eagle {
namespace {

// One warp a (row, query head): the lanes share the head dimension, the keys come one by one.
template <int D>
__global__ void __launch_bounds__(128) kv8_attn_simple_k(Kv8Attn a) {
  constexpr int E = D / 32;   // entries a lane
  PDL_ENTRY();
  const Kv8& c = a.c;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (long long)a.R * a.nq) return;
  const int lane = threadIdx.x & 31, row = (int)(item / a.nq), head = (int)(item % a.nq), h = head / (a.nq / c.nkv);
  __nv_bfloat16* out = (__nv_bfloat16*)a.out + item * D + lane * E;
  int seq = a.row_seq[row], first = -1;
  for (int r = row / a.rows_per_seq * a.rows_per_seq; first < 0 && r <= row; ++r) first = a.row_seq[r];
  const bool live = seq >= 0 && seq == first && seq < c.max_batch;
  if (seq >= 0 && !live && lane == 0) latch_error(a.err, DEVERR_BOUNDS);
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(((const __nv_bfloat16*)a.q)[item * D + lane * E + i]);
    o[i] = 0.f;
  }
  auto key = [&](const float* k, const float* v) {
    float s = 0.f;
    for (int i = 0; i < E; ++i) s = fmaf(q[i], k[i], s);
    s = warp_sum(s) * a.scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float p = expf(s - base), corr = expf(m - base);
    m = mn;
    l = l * corr + p;
    for (int i = 0; i < E; ++i) o[i] = o[i] * corr + p * v[i];
  };
  if (live) {
    float k[E], v[E];
    for (int s = 0; s < a.P; ++s) {
      const size_t at = ((size_t)h * a.P + s) * D + lane * E;
      for (int i = 0; i < E; ++i) {
        k[i] = __bfloat162float(((const __nv_bfloat16*)a.pk)[at + i]);
        v[i] = __bfloat162float(((const __nv_bfloat16*)a.pv)[at + i]);
      }
      key(k, v);
    }
    const int ctx = a.mode == 1 ? a.ctx_len[seq] : 0;
    const int end = a.mode == 1 ? ctx + a.tree_T : a.row_slot[row] + 1;
    for (int s = 0; s < end; ++s) {
      const int t = s - ctx;
      if (a.mode == 1 && t >= 0 && !((a.mask[(size_t)row * a.mask_words + (t >> 6)] >> (t & 63)) & 1)) continue;
      const long long vec = s < c.cap ? kv8_vec(c, seq, h, s) : -1;
      if (vec < 0) {
        if (lane == 0) latch_error(a.err, DEVERR_BOUNDS);
        continue;
      }
      const float fk = kv8_pow2(c.ke[vec]), fv = kv8_pow2(c.ve[vec]);
      for (int i = 0; i < E; i += 2) {
        const uint32_t hk = e4m3x2_f16x2(*(const uint16_t*)(c.k + vec * D + lane * E + i));
        const uint32_t hv = e4m3x2_f16x2(*(const uint16_t*)(c.v + vec * D + lane * E + i));
        const float2 x = __half22float2(*(const __half2*)&hk), y = __half22float2(*(const __half2*)&hv);
        k[i] = x.x * fk; k[i + 1] = x.y * fk;
        v[i] = y.x * fv; v[i + 1] = y.y * fv;
      }
      key(k, v);
    }
  }
  for (int i = 0; i < E; ++i) out[i] = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
}

}  // namespace

size_t kv8_attention_scratch(const Kv8&, int, int, int, int) { return 256; }

int kv8_attention(cudaStream_t st, const Kv8Attn& a) {
  const long long blocks = ((long long)a.R * a.nq + 3) / 4;
  if (blocks > 0x7fffffffll) return -1;
  if (a.c.d == 128) launch_k(kv8_attn_simple_k<128>, dim3((unsigned)blocks), 128, 0, st, a);
  else launch_k(kv8_attn_simple_k<64>, dim3((unsigned)blocks), 128, 0, st, a);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace eagle
