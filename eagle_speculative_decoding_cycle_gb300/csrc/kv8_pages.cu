// Blocks of a paged 8-bit cache: assigned, released, shared by forks; and accepted paths moved to their committed slots,
// in all layers at once.
//
// All state is the block table that attention reads and a count for each block of the table entries that hold it; a block is
// free when its count is zero. There is no free list to keep: the lowest-numbered free blocks are found by a pass over the
// counts, so the result of a call depends on the table and counts alone, not on the order of earlier calls.
//
// kv8_plan_k, one CTA, phases with a barrier between them:
//   rows      a warp a sequence: which take part (a fork's parent keeps its entries during the call and has all that are
//             shared); entries past the last block, and all that a fork held, released; a fork's taken from its parent's;
//             counts down and up (integer atomics: any order). Entries that are missing, or lie outside the pool, are counted;
//   last      a thread a sequence: its last block, if that is partly filled and others hold it too, is to be replaced: the
//             sequence would write where they read. Exclusive sums of the entries wanted over the sequences;
//   find      that many free blocks in rising order, 16 counts a thread at a time;
//   assign    the n-th missing entry, in the order of sequences and slots, gets the n-th free block.
// Up to 2048 sequences and 4096 new blocks what the phases hand on is in shared memory. A call for 64 sequences over 8400 blocks
// takes 8 us with the copies' launch behind it (11 with a phase for each step, all through L2); fifteen forks of a prompt of
// 1000 tokens, its last block copied in 32 layers, 13 us (8 MB written).
// kv8_copy_k then copies the filled slots of the blocks that were replaced, in all layers and heads, a warp for each
// (copy, layer, K or V, head): the slots of a head are next to each other in a block.
//
// A call of a batch's size is bound by latency: tens of kilobytes behind a chain of loads. The copies are bound by HBM.
#include "kernels.h"
#include "ops_ext.h"

namespace eagle {
namespace {

constexpr int PLAN_THREADS = 1024, PLAN_WARPS = PLAN_THREADS / 32;
constexpr int MAX_LAYERS = 64;      // layers a launch (their pointers are kernel arguments)
constexpr int COPY_THREADS = 256;

struct LayerSet { Kv8Layer l[MAX_LAYERS]; };

constexpr int PLAN_SEQS = 2048, PLAN_FOUND = 4096, PLAN_COUNTS = 16;

struct PlanArgs {
  int* table;
  int* refs;
  const int *parent, *length;
  int B, max_batch, tab_w, n_blocks, block_log2, cap;
  int* err;
  // scratch, for what does not fit into shared memory
  int* state;      // [B]: blocks wanted, -1: takes no part; bit 30: the last one is to be replaced
  int* need;       // [B]: missing entries, then the sum of those of earlier sequences
  int* tail;       // [B]: the block that ends the sequence, if it is partly filled; -1: none
  int* copies;     // [0]: their number, then (from, to, slots) each
  int* found;      // free blocks, rising
};
constexpr int PLAN_LAST = 1 << 30;

// Sum over the threads before this one, and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int w = warp_sums[lane];      // (32 warps)
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  total = __reduce_add_sync(0xffffffffu, w);
  __syncthreads();      // warp_sums may be written again
  return before + x - v;
}

__device__ __forceinline__ void release(const PlanArgs& a, int e) {
  if (e >= a.n_blocks) {
    latch_error(a.err, DEVERR_BOUNDS);
  } else if (atomicSub(a.refs + e, 1) <= 0) {      // a count that did not match the table
    atomicAdd(a.refs + e, 1);
    latch_error(a.err, DEVERR_BOUNDS);
  }
}

__global__ void __launch_bounds__(PLAN_THREADS, 1) kv8_plan_k(const PlanArgs a) {
  __shared__ int warp_sums[PLAN_WARPS], sh_state[PLAN_SEQS], sh_need[PLAN_SEQS], sh_tail[PLAN_SEQS], sh_found[PLAN_FOUND];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = 1 << a.block_log2;
  volatile int* state = a.B <= PLAN_SEQS ? sh_state : a.state;
  volatile int* need = a.B <= PLAN_SEQS ? sh_need : a.need;
  volatile int* tail = a.B <= PLAN_SEQS ? sh_tail : a.tail;
  PDL_ENTRY();
  // ---- rows ----
  if (threadIdx.x == 0) a.copies[0] = 0;
  for (int b = warp; b < a.B; b += PLAN_WARPS) {
    const int n = __ldcg(a.length + b), p = a.parent ? __ldcg(a.parent + b) : -1;
    const int nb = n > 0 ? (int)(((long long)n + block - 1) >> a.block_log2) : 0;
    const int end = n & (block - 1) ? nb - 1 : -1;      // the entry of a partly filled last block
    int missing = 0, last = -1;
    bool ok = n >= 0, bad = n > a.cap;
    if (ok && !bad && p >= 0) {
      bad = p >= a.max_batch || p == b || (p < a.B && __ldcg(a.length + p) >= 0);      // the parent takes no part itself
      if (!bad) {
        bool holes = false;
#pragma unroll 4
        for (int j = lane; j < nb; j += 32) {
          const int e = __ldcg(a.table + (size_t)p * a.tab_w + j);
          holes |= e < 0 || e >= a.n_blocks;
        }
        bad = __any_sync(0xffffffffu, holes);
      }
    }
    if (ok && bad) {
      if (lane == 0) latch_error(a.err, DEVERR_BOUNDS);
      ok = false;
    }
    if (ok) {
      int* row = a.table + (size_t)b * a.tab_w;
      if (p >= 0) {
        const int* from = a.table + (size_t)p * a.tab_w;
#pragma unroll 4
        for (int j = lane; j < a.tab_w; j += 32) {
          const int e = __ldcg(row + j), x = j < nb ? __ldcg(from + j) : -1;
          row[j] = x;
          last = j == end ? x : last;
          if (x >= 0) atomicAdd(a.refs + x, 1);
          if (e >= 0) release(a, e);
        }
      } else {
#pragma unroll 8
        for (int j = lane; j < a.tab_w; j += 32) {
          const int e = __ldcg(row + j);
          if (j < nb) {
            if (e >= a.n_blocks) {      // no block: a missing entry
              latch_error(a.err, DEVERR_BOUNDS);
              row[j] = -1;
            }
            const bool there = e >= 0 && e < a.n_blocks;
            missing += !there;
            last = j == end && there ? e : last;
          } else if (e >= 0) {
            row[j] = -1;
            release(a, e);
          }
        }
        missing = __reduce_add_sync(0xffffffffu, missing);
      }
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
      state[b] = ok ? nb : -1;
      need[b] = missing;
      tail[b] = last;
    }
  }
  __syncthreads();
  // ---- last; the first counts are on their way meanwhile ----
  int counts[PLAN_COUNTS];
  auto load_counts = [&](int b0) {
    const int at = b0 + PLAN_COUNTS * threadIdx.x;
#pragma unroll
    for (int i = 0; i < PLAN_COUNTS; i += 4) {
      int4 v = make_int4(1, 1, 1, 1);
      if (at + i + 3 < a.n_blocks && !(reinterpret_cast<uintptr_t>(a.refs) & 15)) {
        v = __ldcg(reinterpret_cast<const int4*>(a.refs + at + i));
      } else {
        if (at + i < a.n_blocks) v.x = __ldcg(a.refs + at + i);
        if (at + i + 1 < a.n_blocks) v.y = __ldcg(a.refs + at + i + 1);
        if (at + i + 2 < a.n_blocks) v.z = __ldcg(a.refs + at + i + 2);
        if (at + i + 3 < a.n_blocks) v.w = __ldcg(a.refs + at + i + 3);
      }
      counts[i] = v.x; counts[i + 1] = v.y; counts[i + 2] = v.z; counts[i + 3] = v.w;
    }
  };
  load_counts(0);
  int wanted = 0;
  for (int b0 = 0; b0 < a.B; b0 += PLAN_THREADS) {
    const int b = b0 + threadIdx.x;
    int v = 0;
    if (b < a.B) {
      const int e = tail[b];
      v = need[b];
      if (e >= 0 && __ldcg(a.refs + e) > 1) {
        state[b] = state[b] | PLAN_LAST;
        ++v;
      }
    }
    int total;
    const int before = block_scan(v, warp_sums, total);
    if (b < a.B) need[b] = wanted + before;
    wanted += total;
  }
  if (wanted == 0) return;      // (the same in all threads)
  // ---- find ----
  volatile int* found_at = wanted <= PLAN_FOUND ? sh_found : a.found;
  int found = 0;
  for (int b0 = 0; b0 < a.n_blocks && found < wanted; b0 += PLAN_COUNTS * PLAN_THREADS) {
    if (b0) load_counts(b0);
    int n = 0;
#pragma unroll
    for (int i = 0; i < PLAN_COUNTS; ++i) n += counts[i] == 0;
    int total;
    int rank = found + block_scan(n, warp_sums, total);
#pragma unroll
    for (int i = 0; i < PLAN_COUNTS; ++i)
      if (counts[i] == 0) {
        if (rank < wanted) found_at[rank] = b0 + PLAN_COUNTS * threadIdx.x + i;
        ++rank;
      }
    found += total;
  }
  if (found < wanted && threadIdx.x == 0) latch_error(a.err, DEVERR_CAPACITY);
  __syncthreads();
  // ---- assign ----
  for (int b = warp; b < a.B; b += PLAN_WARPS) {
    const int st = state[b], rank0 = need[b];
    if (st <= 0 || (b + 1 < a.B ? need[b + 1] == rank0 : wanted == rank0)) continue;
    const int nb = st & (PLAN_LAST - 1);
    const bool last = st & PLAN_LAST;
    int* row = a.table + (size_t)b * a.tab_w;
    int rank = rank0;
#pragma unroll 4
    for (int j0 = 0; j0 < nb; j0 += 32) {
      const int j = j0 + lane;
      const int e = j < nb ? __ldcg(row + j) : 0;
      const bool replace = last && j == nb - 1, take = j < nb && (e < 0 || replace);
      const unsigned who = __ballot_sync(0xffffffffu, take);
      const int mine = rank + __popc(who & ((1u << lane) - 1));
      rank += __popc(who);
      if (!take || mine >= found) continue;
      const int blk = found_at[mine];
      row[j] = blk;
      a.refs[blk] = 1;
      if (replace) {
        atomicSub(a.refs + e, 1);
        const int c = atomicAdd(a.copies, 1);
        a.copies[1 + 3 * c] = e;
        a.copies[2 + 3 * c] = blk;
        a.copies[3 + 3 * c] = __ldcg(a.length + b) & (block - 1);
      }
    }
  }
}

__global__ void __launch_bounds__(COPY_THREADS)
    kv8_copy_k(const __grid_constant__ LayerSet set, int layers, int nkv, int d, int block_log2, const int* copies) {
  PDL_ENTRY();
  const int n = __ldcg(copies);
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (COPY_THREADS / 32), items = (long long)n * layers * 2 * nkv;
  for (long long it = (long long)blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const int head = (int)(it % nkv);
    long long r = it / nkv;
    const int y = (int)(r & 1);
    r >>= 1;
    const int layer = (int)(r % layers), c = (int)(r / layers);
    const int from = __ldcg(copies + 1 + 3 * c), to = __ldcg(copies + 2 + 3 * c), slots = __ldcg(copies + 3 + 3 * c);
    const long long fv = ((long long)from * nkv + head) << block_log2, tv = ((long long)to * nkv + head) << block_log2;
    const uint4* src = reinterpret_cast<const uint4*>(set.l[layer].p[y] + fv * d);
    uint4* dst = reinterpret_cast<uint4*>(set.l[layer].p[y] + tv * d);
    const int chunks = slots * (d / 16);
#pragma unroll 4
    for (int i = lane; i < chunks; i += 32) dst[i] = src[i];
    const uint8_t* es = set.l[layer].p[2 + y] + fv;
    uint8_t* ed = set.l[layer].p[2 + y] + tv;
    for (int i = lane; i < slots; i += 32) ed[i] = es[i];
  }
}

// ---- accepted paths --------------------------------------------------------------------------------
// Slot n + j <- slot n + path[j - 1], j = 1 .. len, for all layers and heads of a sequence. A thread takes one 16-byte piece
// of a head (or its exponent bytes) along the whole path: all reads, then all writes, so paths of any order are moved
// as if at once. The slots' places are looked up once a CTA. 64 paths of up to 5 in 32 layers of 8 heads of 128: 7.6 us for 25 MB, a
// chain of four loads and a launch; one path in 40 layers of 40 heads: 3.3 us.
template <int MOST>
__global__ void __launch_bounds__(COPY_THREADS)
    kv8_compact_k(const __grid_constant__ LayerSet set, Kv8 c, int layers, int parts, const int* n_old, const int* acc_len,
                  const int* acc_path, int Dmax, int* err) {
  __shared__ long long from[MOST], to[MOST];      // vector of head 0, -1: none
  __shared__ int n_moves;
  PDL_ENTRY();
  const int b = blockIdx.x / parts, part = blockIdx.x % parts;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int took = acc_len[b], n = n_old[b], node = lane < Dmax ? acc_path[(size_t)b * Dmax + lane] : 0;
    const int len = min(took, min(Dmax, MOST));
    bool bad = took > Dmax;
    if (lane < len) {
      const long long f = (long long)n + node, t = (long long)n + lane + 1;
      const bool in = n >= 0 && f >= 0 && f < c.cap && t < c.cap;
      const long long fv = in ? kv8_vec(c, b, 0, (int)f) : -1, tv = in ? kv8_vec(c, b, 0, (int)t) : -1;
      const bool ok = fv >= 0 && tv >= 0;
      bad |= !ok;
      from[lane] = ok ? fv : -1;
      to[lane] = tv;
    }
    if (lane == 0) n_moves = len;
    if (bad && part == 0) latch_error(err, DEVERR_BOUNDS);
  }
  __syncthreads();
  const int len = n_moves;
  if (len <= 0) return;
  const long long hs = c.table ? 1ll << c.block_log2 : c.cap;      // vectors from a head to the next
  const int pieces = c.d / 16 + 1;
  const long long items = (long long)layers * 2 * c.nkv * pieces, it = (long long)part * COPY_THREADS + threadIdx.x;
  if (it >= items) return;
  const int piece = (int)(it % pieces);
  long long r = it / pieces;
  const int head = (int)(r % c.nkv);
  r /= c.nkv;
  const int y = (int)(r & 1), layer = (int)(r >> 1);
  const long long at = head * hs;
  if (piece == pieces - 1) {
    uint8_t* e = set.l[layer].p[2 + y];
    uint8_t x[MOST];
#pragma unroll
    for (int j = 0; j < MOST; ++j)
      if (j < len && from[j] >= 0) x[j] = e[from[j] + at];
#pragma unroll
    for (int j = 0; j < MOST; ++j)
      if (j < len && from[j] >= 0) e[to[j] + at] = x[j];
  } else {
    uint8_t* p = set.l[layer].p[y] + piece * 16;
    uint4 x[MOST];
#pragma unroll
    for (int j = 0; j < MOST; ++j)
      if (j < len && from[j] >= 0) x[j] = *reinterpret_cast<const uint4*>(p + (from[j] + at) * c.d);
#pragma unroll
    for (int j = 0; j < MOST; ++j)
      if (j < len && from[j] >= 0) *reinterpret_cast<uint4*>(p + (to[j] + at) * c.d) = x[j];
  }
}

}  // namespace

static LayerSet layer_set(const Kv8Layer* layers, int from, int n) {
  LayerSet s{};
  for (int i = 0; i < n; ++i) s.l[i] = layers[from + i];
  return s;
}

int kv8_compact(cudaStream_t st, const Kv8& c, const Kv8Layer* layers, int n_layers, int B, const int* n_old,
                const int* acc_len, const int* acc_path, int Dmax, int* err) {
  for (int l0 = 0; l0 < n_layers; l0 += MAX_LAYERS) {
    const int n = n_layers - l0 < MAX_LAYERS ? n_layers - l0 : MAX_LAYERS;
    const LayerSet s = layer_set(layers, l0, n);
    const long long items = (long long)n * 2 * c.nkv * (c.d / 16 + 1), parts = (items + COPY_THREADS - 1) / COPY_THREADS;
    if (parts * B > 0x7fffffffll) return -1;
    const dim3 grid((unsigned)(parts * B));
    const cudaError_t e = Dmax <= 8 ? launch_k(kv8_compact_k<8>, grid, dim3(COPY_THREADS), 0, st, s, c, n, (int)parts,
                                               n_old, acc_len, acc_path, Dmax, err)
                                    : launch_k(kv8_compact_k<16>, grid, dim3(COPY_THREADS), 0, st, s, c, n, (int)parts,
                                               n_old, acc_len, acc_path, Dmax, err);
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return -4;
  }
  return 0;
}

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

size_t kv8_resize_scratch(const Kv8& c) {
  return align256((size_t)c.max_batch * 6 * 4 + 4) + align256((size_t)c.n_blocks * 4);
}

int kv8_resize(cudaStream_t st, const Kv8& c, const Kv8Layer* layers, int n_layers, int B, int* refs, const int* parent,
               const int* length, void* scratch, int* err) {
  PlanArgs a{};
  a.table = const_cast<int*>(c.table);
  a.refs = refs; a.parent = parent; a.length = length;
  a.B = B; a.max_batch = c.max_batch; a.tab_w = c.tab_w; a.n_blocks = c.n_blocks; a.block_log2 = c.block_log2; a.cap = c.cap; a.err = err;
  int* s = static_cast<int*>(scratch);
  a.state = s;
  a.need = s + c.max_batch;
  a.tail = s + 2 * (size_t)c.max_batch;
  a.copies = s + 3 * (size_t)c.max_batch;
  a.found = reinterpret_cast<int*>(static_cast<char*>(scratch) + align256((size_t)c.max_batch * 6 * 4 + 4));
  cudaError_t e = launch_k(kv8_plan_k, dim3(1), dim3(PLAN_THREADS), 0, st, a);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return -4;
  for (int l0 = 0; l0 < n_layers; l0 += MAX_LAYERS) {
    const int n = n_layers - l0 < MAX_LAYERS ? n_layers - l0 : MAX_LAYERS;
    const LayerSet set = layer_set(layers, l0, n);
    // at most one copy a sequence; CTAs past the copies that there are end at once
    const long long most = ((long long)B * n * 2 * c.nkv + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32);
    const unsigned grid = (unsigned)(most < 152 * 8 ? most : 152 * 8);
    e = launch_k(kv8_copy_k, dim3(grid), dim3(COPY_THREADS), 0, st, set, n, c.nkv, c.d, c.block_log2, (const int*)a.copies);
    if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return -4;
  }
  return 0;
}

}  // namespace eagle
