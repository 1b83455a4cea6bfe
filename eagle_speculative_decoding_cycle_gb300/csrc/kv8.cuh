// The 8-bit KV cache as the kernels see it: e4m3 codes, one exponent byte per (slot, head)
// vector, contiguous or paged, and the internal launchers of its operators.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/eagle_ops.h"
#include "common.cuh"

namespace eagle {

constexpr int KV8_E_LO = -40, KV8_E_HI = 40;   // exponents that a written vector can get
constexpr int KV8_BIAS = 127;
constexpr int KV8_LOWEST = KV8_E_LO + KV8_BIAS;   // the lowest byte that is written; attention takes the byte 0 of cleared
                                               // memory (zero codes) for it, so that 0 can mean "none" beside the bytes
constexpr int KV8_BAD = 255;                   // exponent byte of a vector with an entry that is not finite

struct Kv8 {
  uint8_t *k, *v, *ke, *ve;
  const int* table;     // nullptr: contiguous
  int nkv, d, max_batch, cap;
  int block_log2, tab_w, n_blocks;
};

// Vector index (in units of d codes, of one exponent byte) of head h of sequence seq at slot; -1 when the
// slot's block is not assigned or outside the pool. seq and slot are in range. 64-bit: codes of a
// long cache pass 2^32 bytes.
__device__ __forceinline__ long long kv8_vec(const Kv8& c, int seq, int h, int slot) {
  if (!c.table) return ((long long)seq * c.nkv + h) * c.cap + slot;
  const int blk = __ldcg(c.table + (size_t)seq * c.tab_w + (slot >> c.block_log2));
  if (blk < 0 || blk >= c.n_blocks) return -1;
  return (((long long)blk * c.nkv + h) << c.block_log2) + (slot & ((1 << c.block_log2) - 1));
}

// 2^(byte - 127), NaN for a vector that held something not finite. Bytes of written vectors are
// 87 .. 167, so the power is a normal fp32 put together from its exponent bits.
__device__ __forceinline__ float kv8_pow2(int byte) {
  return byte == KV8_BAD ? __int_as_float(0x7fffffff) : __int_as_float(byte << 23);
}

// Four e4m3 codes (low byte first) as two pairs of fp16: exact.
__device__ __forceinline__ void e4m3x4_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// Bounded wait of a converged warp for an mbarrier phase: lane 0 tries (a try by 32 lanes is 32 accesses to the barrier:
// waiting warps then took half of the shared-memory pipe), looking at the abort flag and the clock every 64th time. Gives
// up as mbar_wait does. Every lane gets the same answer: whether the CTA goes on.
__device__ __forceinline__ bool kv8_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                         bool honor_abort = true) {
  if ((threadIdx.x & 31) == 0) {
    uint64_t t0 = 0;
    for (uint32_t tries = 1; !mbar_try(bar, parity); ++tries) {
      if (tries & 63u) continue;
      if (honor_abort && *abort_flag) break;
      const uint64_t now = globaltimer();
      if (!t0) t0 = now;
      if (now - t0 > EAGLE_WAIT_LIMIT_NS) {
        *abort_flag = 1;
        latch_error(err, DEVERR_MBAR_TIMEOUT);
        break;
      }
    }
  }
  __syncwarp();
  return *abort_flag == 0;
}
// The same, every lane trying: for the single warps that issue copies and products, which go on some hundred clocks earlier
// without the divergence (4096 shared tokens, 64 x 17 rows: 147 -> 134 us).
__device__ __forceinline__ bool kv8_wait_all(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                             bool honor_abort = true) {
  uint64_t t0 = 0;
  for (uint32_t tries = 1; !mbar_try(bar, parity); ++tries) {
    if (tries & 63u) continue;
    if (honor_abort && *abort_flag) break;
    const uint64_t now = globaltimer();
    if (!t0) t0 = now;
    if (now - t0 > EAGLE_WAIT_LIMIT_NS) {
      *abort_flag = 1;
      latch_error(err, DEVERR_MBAR_TIMEOUT);
      break;
    }
  }
  __syncwarp();
  return *abort_flag == 0;
}
// Orders this thread's shared-memory accesses before later ones of the tensor cores and bulk copies. (The fence over all
// state spaces waits for global accesses too: some 700 clocks more.)
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// One arrival for the warp, after what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

struct Kv8Attn {
  Kv8 c;
  const void* q;          // bf16 [R][nq][d]
  void* out;
  const void *pk, *pv;    // bf16 [nkv][P][d], P == 0: none
  int P;
  int R, nq, rows_per_seq, mode, tree_T, mask_words;
  const int *row_seq, *row_slot, *ctx_len;
  const uint64_t* mask;
  float scale;
  void* scratch;
  int* err;
};

int kv8_write(cudaStream_t st, const Kv8& c, bool f32, const void* k, long long ldk, const void* v, long long ldv, int R,
              const int* row_seq, const int* row_slot, int* err);
int kv8_read(cudaStream_t st, const Kv8& c, bool f32, void* k, long long ldk, void* v, long long ldv, int R,
             const int* row_seq, const int* row_slot, int* err);
size_t kv8_attention_scratch(const Kv8& c, int R, int nq, int rows_per_seq, int P);
int kv8_attention(cudaStream_t st, const Kv8Attn& a);
// Partials of all rows over the shared prefix, in `splits` key ranges: o [splits][R * nq][d], ml [splits][R * nq][2]
// (maximum in log2 units, sum).
int kv8_prefix_splits(int nkv, int R, int nq, int P);
int kv8_prefix(cudaStream_t st, const Kv8Attn& a, int splits, float* o, float* ml);

}  // namespace eagle
