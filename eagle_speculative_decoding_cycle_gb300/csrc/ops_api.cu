// Kernel-level C ABI (eagle_ops.h): each entry point runs one of the cycle's kernels on
// caller-provided device buffers.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/eagle.h"
#include "../../include/eagle_ops.h"
#include "common.cuh"
#include "cycle.h"
#include "kernels.h"
#include "kv8.cuh"
#include "lmhead.cuh"
#include "ops_ext.h"

using namespace eagle;

namespace {
size_t al(size_t x) { return (x + 255) / 256 * 256; }
int tiles_for(int M, int N) {
  const int BN = gemm_bn_for(M);
  return ((N + 127) / 128) * ((M + BN - 1) / BN);
}
}  // namespace

extern "C" {

size_t eagle_op_gemm_scratch_bytes(int M, int N) {
  if (M <= 0 || N <= 0) return 0;
  return al(gemm_bf16_scratch_bytes(M)) + al((size_t)tiles_for(M, N) * sizeof(int));
}

int eagle_op_gemm(int dtype, void* stream, const void* W, int N, int K, const void* X, int M, int epi, void* out,
                  int ldo, void* scratch, size_t scratch_bytes) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!W || !X || !out || M <= 0 || N <= 0 || K <= 0 || ldo < N) return EAGLE_EINVAL;
  if (dtype == EAGLE_DTYPE_F32) {
    if (epi != EPI_F32 && epi != EPI_ADD_F32) return EAGLE_EINVAL;
    return gemm_f32(st, (const float*)W, N, K, (const float*)X, M, epi, (float*)out, ldo) == 0 ? EAGLE_OK : EAGLE_ECUDA;
  }
  if (dtype != EAGLE_DTYPE_BF16 || epi < 0 || epi == EPI_HEAD || epi > EPI_SWIGLU || K % 8) return EAGLE_EINVAL;
  const int tiles_N = epi == EPI_SWIGLU ? 2 * N : N;   // SwiGLU: W has 2N rows, tiles of 64 + 64
  if (!scratch || scratch_bytes < eagle_op_gemm_scratch_bytes(M, tiles_N)) return EAGLE_ECAPACITY;
  float* part = reinterpret_cast<float*>(scratch);
  int* cnt = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(scratch) + al(gemm_bf16_scratch_bytes(M)));
  const int r = gemm_bf16(st, W, N, K, X, M, epi, out, ldo, part, gemm_bf16_scratch_bytes(M) / sizeof(float), cnt,
                          tiles_for(M, tiles_N), nullptr, nullptr);
  return r == 0 ? EAGLE_OK : (r == -4 ? EAGLE_ECUDA : EAGLE_EINVAL);
}

size_t eagle_op_lm_head_scratch_bytes(int dtype, int V, int M, int K) {
  if (V <= 0 || M <= 0 || K < 1 || K > 16) return 0;
  size_t s = al(head_part_bytes(V, M, K));
  if (dtype == EAGLE_DTYPE_F32) s += al((size_t)M * V * sizeof(float));
  else s += eagle_op_gemm_scratch_bytes(M, V);
  return s;
}

int eagle_op_lm_head(int dtype, void* stream, const void* W_lm, int V, int H, const void* X, int M, int K, float inv_t,
                     int gumbel, int lse_excl, const int32_t* specials, int S, float* spec_logit,
                     const int32_t* row_seq, const int32_t* row_key, uint32_t cycle, uint64_t seed, int stream_id,
                     int32_t* top_id, float* top_val, float* lse, void* scratch, size_t scratch_bytes) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!W_lm || !X || !top_id || !top_val || !lse || V <= 0 || H <= 0 || M <= 0 || K < 1 || K > 16) return EAGLE_EINVAL;
  if (specials && (S < 1 || !spec_logit)) return EAGLE_EINVAL;
  if (!scratch || scratch_bytes < eagle_op_lm_head_scratch_bytes(dtype, V, M, K)) return EAGLE_ECAPACITY;
  HeadParams p{};
  p.vocab = V; p.n_rows = M; p.K = K; p.inv_t = inv_t; p.gumbel = gumbel; p.lse_excl = lse_excl;
  p.specials = specials; p.S = specials ? S : 0; p.spec_logit = spec_logit;
  p.row_seq = row_seq; p.row_key = row_key; p.cycle_const = cycle; p.stream = (uint32_t)stream_id; p.seed = seed;
  uint8_t* s = reinterpret_cast<uint8_t*>(scratch);
  p.part = reinterpret_cast<float*>(s);
  s += al(head_part_bytes(V, M, K));
  p.n_tiles = (V + 127) / 128;
  p.top_id = top_id; p.top_val = top_val; p.lse = lse;
  if (dtype == EAGLE_DTYPE_F32) {
    float* logits = reinterpret_cast<float*>(s);
    if (gemm_f32(st, (const float*)W_lm, V, H, (const float*)X, M, EPI_F32, logits, V)) return EAGLE_ECUDA;
    if (head_partials_from_logits(st, logits, V, p)) return EAGLE_ECUDA;
  } else if (dtype == EAGLE_DTYPE_BF16) {
    if (H % 8) return EAGLE_EINVAL;
    float* part = reinterpret_cast<float*>(s);
    int* cnt = reinterpret_cast<int*>(s + al(gemm_bf16_scratch_bytes(M)));
    const int r = gemm_bf16(st, W_lm, V, H, X, M, EPI_HEAD, nullptr, 0, part, gemm_bf16_scratch_bytes(M) / sizeof(float),
                            cnt, tiles_for(M, V), nullptr, &p);
    if (r) return r == -4 ? EAGLE_ECUDA : EAGLE_EINVAL;
  } else {
    return EAGLE_EINVAL;
  }
  return head_merge(st, p) == 0 ? EAGLE_OK : EAGLE_ECUDA;
}

size_t eagle_op_attention_scratch_bytes(int R, int nq, int d) {
  if (R <= 0 || nq <= 0 || d <= 0) return 0;
  return al(attention_scratch_floats(R, nq, d) * sizeof(float));
}

int eagle_op_attention(int dtype, void* stream, const void* q, const void* kcache, const void* vcache, void* out, int R,
                       int nq, int nkv, int d, int cap, int rows_per_seq, const int32_t* row_seq,
                       const int32_t* row_slot, const int32_t* ctx_len, int mode, int tree_T, const uint64_t* mask,
                       int mask_words, float scale, int max_batch, void* scratch, size_t scratch_bytes) {
  if (!q || !kcache || !vcache || !out || !row_seq || !row_slot || !ctx_len || R <= 0 || nq <= 0 || nkv <= 0 ||
      d <= 0 || d > 128 || nq % nkv || rows_per_seq <= 0 || max_batch < 1 || (mode == 1 && (!mask || mask_words < 1)))
    return EAGLE_EINVAL;
  AttnArgs a{};
  a.q = q; a.kcache = kcache; a.vcache = vcache; a.out = out;
  a.R = R; a.nq = nq; a.nkv = nkv; a.d = d; a.cap = cap; a.rows_per_seq = rows_per_seq;
  a.row_seq = row_seq; a.row_slot = row_slot; a.ctx_len = ctx_len; a.mode = mode; a.tree_T = tree_T;
  a.mask = mask; a.mask_words = mask_words; a.scale = scale > 0.f ? scale : 1.f / sqrtf((float)d);
  if (scratch && scratch_bytes >= eagle_op_attention_scratch_bytes(R, nq, d)) {
    a.part_o = reinterpret_cast<float*>(scratch);
    a.part_floats = attention_scratch_floats(R, nq, d) / (d + 2) * d;
    a.part_ml = a.part_o + a.part_floats;
    a.max_splits = attention_max_splits(cap, max_batch);   // the engine's split policy for this cache
    a.kv_rows = (long long)max_batch * nkv * cap;
    a.max_batch = max_batch;
  } else if (dtype != EAGLE_DTYPE_F32) {
    return EAGLE_ECAPACITY;
  }
  const int r = attention(reinterpret_cast<cudaStream_t>(stream), dtype == EAGLE_DTYPE_F32 ? DT_F32 : DT_BF16, a);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_EINVAL : EAGLE_ECUDA);
}

size_t eagle_op_tree_scratch_bytes(int B, int k, int depth, int m) {
  if (B < 1 || k < 1 || k > 16 || depth < 1 || depth > 8 || m < 1) return 0;
  const size_t NG = k + (size_t)(depth - 1) * k * k;
  const size_t T1 = m + 1;
  const size_t dmw = std::max<size_t>(1, ((depth - 1) * k + 63) / 64);
  size_t s = 0;
  s += al(B * NG * 4);                 // node_rank
  s += al((size_t)B * depth * k * 4);  // exp_node
  s += 7 * al((size_t)B * k * 4);      // drow_* (tok,pos,slot,seq,feat,plant) + head lse
  s += al((size_t)B * k * dmw * 8);    // dmask
  s += 3 * al(B * T1 * 4);             // tree_slot, tree_seq, margin
  s += al(B * T1 * k * 4);             // tree_kids
  s += 8 * al((size_t)B * 4);          // n_old, committed, on_track, cycle, acc_len, bonus, root_plant, spare
  s += 2 * al((size_t)B * k * k * 4);  // injected head rows of one depth (ids, values)
  return s;
}

int eagle_op_tree_build(void* stream, int B, int k, int depth, int m, const int32_t* cand_tok, const float* cand_logc,
                        const int32_t* child_tok, const float* child_logc, const int32_t* ctx_len,
                        const int32_t* root_tok, int32_t* node_tok, int32_t* node_parent, int32_t* node_depth,
                        float* node_logv, int32_t* tree_tok, int32_t* tree_pos, int32_t* tree_parent,
                        int32_t* tree_node, uint64_t* tree_mask, void* scratch, size_t scratch_bytes) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t need = eagle_op_tree_scratch_bytes(B, k, depth, m);
  const int NG = k + (depth - 1) * k * k;
  if (!need || m > NG || !cand_tok || !cand_logc || !ctx_len || !root_tok || !node_tok || !node_parent ||
      !node_depth || !node_logv || !tree_tok || !tree_pos || !tree_parent || !tree_node || !tree_mask ||
      (depth > 1 && (!child_tok || !child_logc)))
    return EAGLE_EINVAL;
  if (!scratch || scratch_bytes < need) return EAGLE_ECAPACITY;
  const int T1 = m + 1;
  const int dmw = std::max(1, ((depth - 1) * k + 63) / 64);
  uint8_t* s = reinterpret_cast<uint8_t*>(scratch);
  auto take = [&](size_t bytes) { uint8_t* p = s; s += al(bytes); return p; };
  CycleDev c{};
  c.B = B; c.k = k; c.D = depth; c.m = m; c.T1 = T1; c.NG = NG; c.V = 0x7fffffff;
  c.dmask_words = dmw; c.tmask_words = (T1 + 63) / 64; c.fsrc_rows = 1 + (depth - 1) * k;
  c.ctx_len = const_cast<int*>(ctx_len);
  c.root_tok = const_cast<int*>(root_tok);
  c.kc = k;
  c.cand_tok = const_cast<int*>(cand_tok);
  c.cand_logc = const_cast<float*>(cand_logc);
  c.node_tok = node_tok; c.node_parent = node_parent; c.node_depth = node_depth; c.node_logv = node_logv;
  c.node_rank = (int*)take((size_t)B * NG * 4);
  c.exp_node = (int*)take((size_t)B * depth * k * 4);
  c.drow_tok = (int*)take((size_t)B * k * 4);
  c.drow_pos = (int*)take((size_t)B * k * 4);
  c.drow_slot = (int*)take((size_t)B * k * 4);
  c.drow_seq = (int*)take((size_t)B * k * 4);
  c.drow_feat = (int*)take((size_t)B * k * 4);
  c.drow_plant = (int*)take((size_t)B * k * 4);
  float* lse0 = (float*)take((size_t)B * k * 4);
  c.dmask = (uint64_t*)take((size_t)B * k * dmw * 8);
  c.tree_tok = tree_tok; c.tree_pos = tree_pos; c.tree_parent = tree_parent; c.tree_node = tree_node;
  c.tmask = tree_mask;
  c.tree_slot = (int*)take((size_t)B * T1 * 4);
  c.tree_seq = (int*)take((size_t)B * T1 * 4);
  c.margin = (float*)take((size_t)B * T1 * 4);
  c.tree_kids = (int*)take((size_t)B * T1 * k * 4);
  uint8_t* small = take(8 * al((size_t)B * 4)) ;
  c.n_old = (int*)small;
  c.committed = (int*)(small + al((size_t)B * 4));
  c.on_track = (int*)(small + 2 * al((size_t)B * 4));
  c.cycle = (uint32_t*)(small + 3 * al((size_t)B * 4));
  c.acc_len = (int*)(small + 4 * al((size_t)B * 4));
  c.bonus = (int*)(small + 5 * al((size_t)B * 4));
  c.root_plant = (int*)(small + 6 * al((size_t)B * 4));
  int* hid = (int*)take((size_t)B * k * k * 4);
  float* hval = (float*)take((size_t)B * k * k * 4);
  c.ref = nullptr;
  c.planted_p = 0.f;
  c.planted_conf = 0.5f;
  c.err = nullptr;
  if (cudaMemsetAsync(small, 0, 8 * al((size_t)B * 4), st) != cudaSuccess) return EAGLE_ECUDA;
  if (cudaMemsetAsync(lse0, 0, (size_t)B * k * 4, st) != cudaSuccess) return EAGLE_ECUDA;
  if (tree_start(st, c)) return EAGLE_ECUDA;
  for (int d = 1; d < depth; ++d) {
    if (tree_select(st, c, d)) return EAGLE_ECUDA;
    const size_t pitch = (size_t)(depth - 1) * k * k * 4;
    const size_t width = (size_t)k * k * 4;
    if (cudaMemcpy2DAsync(hid, width, child_tok + (size_t)(d - 1) * k * k, pitch, width, B, cudaMemcpyDeviceToDevice,
                          st) != cudaSuccess ||
        cudaMemcpy2DAsync(hval, width, child_logc + (size_t)(d - 1) * k * k, pitch, width, B,
                          cudaMemcpyDeviceToDevice, st) != cudaSuccess)
      return EAGLE_ECUDA;
    HeadOut h;
    h.top_id = hid; h.top_val = hval; h.lse = lse0; h.spec_logit = nullptr; h.K = k; h.S = 1;
    if (tree_add(st, c, d, h)) return EAGLE_ECUDA;
  }
  if (tree_finalize(st, c)) return EAGLE_ECUDA;
  return EAGLE_OK;
}

int eagle_op_compact(int dtype, void* stream, void* kcache, void* vcache, int layers, int B, int nkv, int cap, int d,
                     const int32_t* n_old, const int32_t* acc_len, const int32_t* acc_path, int Dmax) {
  if (!kcache || !vcache || !n_old || !acc_len || !acc_path || layers < 1 || B < 1 || nkv < 1 || d < 1 || Dmax < 1 ||
      Dmax > 8)
    return EAGLE_EINVAL;
  const int r = compact_kv(reinterpret_cast<cudaStream_t>(stream), dtype == EAGLE_DTYPE_F32 ? DT_F32 : DT_BF16, kcache,
                           vcache, layers, (size_t)B * nkv * cap * d, B, nkv, cap, d, n_old, acc_len, acc_path,
                           Dmax, KvPage{nullptr, 0, 0});
  return r == 0 ? EAGLE_OK : EAGLE_ECUDA;
}

// ---- 8-bit KV cache ----------------------------------------------------------------------------
static bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The kernels' view of a cache; EAGLE_EINVAL / EAGLE_ECAPACITY when it breaks the header's rules.
// Vectors of a cache, slots of a prefix: their numbers, rounded up to whole tiles, stay in 32 bits.
constexpr double KV8_MOST = 2147483648.0 - 4096;

static int kv8_view(const eagle_kv8* c, Kv8& o) {
  if (!c || !c->k_code || !c->v_code || !c->k_exp || !c->v_exp || c->n_kv_heads < 1 || c->max_batch < 1 || c->cap < 1 ||
      (c->head_dim != 64 && c->head_dim != 128))
    return EAGLE_EINVAL;
  if (!on16(c->k_code) || !on16(c->v_code) || !on16(c->k_exp) || !on16(c->v_exp)) return EAGLE_EINVAL;
  o = Kv8{};
  o.k = (uint8_t*)c->k_code; o.v = (uint8_t*)c->v_code; o.ke = (uint8_t*)c->k_exp; o.ve = (uint8_t*)c->v_exp;
  o.nkv = c->n_kv_heads; o.d = c->head_dim; o.max_batch = c->max_batch; o.cap = c->cap; o.table = c->table;
  double vecs;
  if (c->table) {
    if (c->block < 16 || c->block > 256 || (c->block & (c->block - 1)) || c->n_blocks < 1 || c->cap % c->block)
      return EAGLE_EINVAL;
    while ((1 << o.block_log2) < c->block) ++o.block_log2;
    o.tab_w = c->cap / c->block;
    o.n_blocks = c->n_blocks;
    vecs = (double)c->n_blocks * c->n_kv_heads * c->block;
  } else {
    if (c->cap % 16) return EAGLE_EINVAL;
    vecs = (double)c->max_batch * c->n_kv_heads * c->cap;
  }
  return vecs < KV8_MOST ? EAGLE_OK : EAGLE_ECAPACITY;
}

static int kv8_rows(const Kv8& c, int dtype, const void* k, int64_t ldk, const void* v, int64_t ldv, int R,
                    const int32_t* row_seq, const int32_t* row_slot) {
  if (dtype != EAGLE_DTYPE_F32 && dtype != EAGLE_DTYPE_BF16) return EAGLE_EINVAL;
  if (R < 0) return EAGLE_EINVAL;
  if (R == 0) return EAGLE_OK;
  const int64_t unit = dtype == EAGLE_DTYPE_F32 ? 4 : 8, width = (int64_t)c.nkv * c.d;
  if (!k || !v || !row_seq || !row_slot || !on16(k) || !on16(v) || ldk < width || ldv < width || ldk % unit ||
      ldv % unit)
    return EAGLE_EINVAL;
  return EAGLE_OK;
}

int eagle_op_kv8_write(void* stream, const eagle_kv8* cache, int dtype, const void* k, int64_t ldk, const void* v,
                       int64_t ldv, int R, const int32_t* row_seq, const int32_t* row_slot, int32_t* d_err) {
  Kv8 c;
  int r = kv8_view(cache, c);
  if (r == EAGLE_OK) r = kv8_rows(c, dtype, k, ldk, v, ldv, R, row_seq, row_slot);
  if (r != EAGLE_OK || R == 0) return r;
  r = kv8_write(reinterpret_cast<cudaStream_t>(stream), c, dtype == EAGLE_DTYPE_F32, k, ldk, v, ldv, R, row_seq,
                row_slot, d_err);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_ECAPACITY : EAGLE_ECUDA);
}

int eagle_op_kv8_read(void* stream, const eagle_kv8* cache, int dtype, void* k, int64_t ldk, void* v, int64_t ldv,
                      int R, const int32_t* row_seq, const int32_t* row_slot, int32_t* d_err) {
  Kv8 c;
  int r = kv8_view(cache, c);
  if (r == EAGLE_OK) r = kv8_rows(c, dtype, k, ldk, v, ldv, R, row_seq, row_slot);
  if (r != EAGLE_OK || R == 0) return r;
  r = kv8_read(reinterpret_cast<cudaStream_t>(stream), c, dtype == EAGLE_DTYPE_F32, k, ldk, v, ldv, R, row_seq,
               row_slot, d_err);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_ECAPACITY : EAGLE_ECUDA);
}

// Sizes that both attention entry points and their scratch size accept.
static int kv8_attn_sizes(const Kv8& c, int R, int nq, int rows_per_seq, int prefix_len) {
  if (R < 1 || nq < 1 || nq % c.nkv || nq / c.nkv > 64 || rows_per_seq < 1 || prefix_len < 0) return EAGLE_EINVAL;
  if ((double)R * nq >= 2147483648.0 / c.d || (double)prefix_len * c.nkv >= KV8_MOST) return EAGLE_ECAPACITY;
  return EAGLE_OK;
}

size_t eagle_op_attention_kv8_scratch_bytes(const eagle_kv8* cache, int R, int nq, int rows_per_seq, int prefix_len) {
  Kv8 c;
  if (kv8_view(cache, c) != EAGLE_OK || kv8_attn_sizes(c, R, nq, rows_per_seq, prefix_len) != EAGLE_OK) return 0;
  return al(kv8_attention_scratch(c, R, nq, std::min(rows_per_seq, R), prefix_len));
}

int eagle_op_attention_shared_kv8(void* stream, const eagle_kv8* cache, const void* prefix_k, const void* prefix_v,
                                  int prefix_len, const void* q, void* out, int R, int nq, int rows_per_seq,
                                  const int32_t* row_seq, const int32_t* row_slot, const int32_t* ctx_len, int mode,
                                  int tree_T, const uint64_t* mask, int mask_words, float scale, void* scratch,
                                  size_t scratch_bytes, int32_t* d_err) {
  Kv8Attn a{};
  int r = kv8_view(cache, a.c);
  if (r == EAGLE_OK) r = kv8_attn_sizes(a.c, R, nq, rows_per_seq, prefix_len);
  if (r != EAGLE_OK) return r;
  if (!q || !out || !on16(q) || !on16(out) || !row_seq || (mode != 0 && mode != 1) || (mode == 0 && !row_slot))
    return EAGLE_EINVAL;
  if (mode == 1 && (!ctx_len || !mask || tree_T < 1 || tree_T > 256 || mask_words < (tree_T + 63) / 64)) return EAGLE_EINVAL;
  if (prefix_len && (!prefix_k || !prefix_v || !on16(prefix_k) || !on16(prefix_v))) return EAGLE_EINVAL;
  rows_per_seq = std::min(rows_per_seq, R);
  const size_t need = al(kv8_attention_scratch(a.c, R, nq, rows_per_seq, prefix_len));
  if (!scratch || !on16(scratch) || scratch_bytes < need) return EAGLE_ECAPACITY;
  const uintptr_t q0 = (uintptr_t)q, o0 = (uintptr_t)out, len = (uintptr_t)R * nq * a.c.d * 2;
  if (q0 != o0 && q0 < o0 + len && o0 < q0 + len) return EAGLE_EINVAL;   // (out = q: a block's rows are read before they are written)
  a.q = q; a.out = out; a.pk = prefix_k; a.pv = prefix_v; a.P = prefix_len;
  a.R = R; a.nq = nq; a.rows_per_seq = rows_per_seq; a.mode = mode; a.tree_T = mode == 1 ? tree_T : 0;
  a.mask_words = mask_words; a.row_seq = row_seq; a.row_slot = row_slot; a.ctx_len = ctx_len; a.mask = mask;
  a.scale = scale > 0.f ? scale : 1.f / sqrtf((float)a.c.d);
  a.scratch = scratch; a.err = d_err;
  r = kv8_attention(reinterpret_cast<cudaStream_t>(stream), a);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_ECAPACITY : EAGLE_ECUDA);
}

int eagle_op_attention_kv8(void* stream, const eagle_kv8* cache, const void* q, void* out, int R, int nq,
                           int rows_per_seq, const int32_t* row_seq, const int32_t* row_slot, const int32_t* ctx_len,
                           int mode, int tree_T, const uint64_t* mask, int mask_words, float scale, void* scratch,
                           size_t scratch_bytes, int32_t* d_err) {
  return eagle_op_attention_shared_kv8(stream, cache, nullptr, nullptr, 0, q, out, R, nq, rows_per_seq, row_seq,
                                       row_slot, ctx_len, mode, tree_T, mask, mask_words, scale, scratch, scratch_bytes,
                                       d_err);
}


// ---- blocks and accepted paths of an 8-bit cache's layers -----------------------------------------
// The layers' common shape and their arrays. They must agree in everything but the four arrays.
static int kv8_layers(const eagle_kv8* caches, int layers, Kv8& c, std::vector<Kv8Layer>& l) {
  if (!caches || layers < 1) return EAGLE_EINVAL;
  if (layers > 4096) return EAGLE_ECAPACITY;
  l.resize(layers);
  for (int i = 0; i < layers; ++i) {
    Kv8 x;
    const int r = kv8_view(caches + i, x);
    if (r != EAGLE_OK) return r;
    if (i == 0) c = x;
    if (x.nkv != c.nkv || x.d != c.d || x.max_batch != c.max_batch || x.cap != c.cap || x.table != c.table ||
        x.block_log2 != c.block_log2 || x.n_blocks != c.n_blocks)
      return EAGLE_EINVAL;
    l[i] = Kv8Layer{{x.k, x.v, x.ke, x.ve}};
  }
  return EAGLE_OK;
}

int eagle_op_kv8_compact(void* stream, const eagle_kv8* caches, int layers, int B, const int32_t* n_old,
                         const int32_t* acc_len, const int32_t* acc_path, int Dmax, int32_t* d_err) try {
  Kv8 c;
  std::vector<Kv8Layer> l;
  int r = kv8_layers(caches, layers, c, l);
  if (r != EAGLE_OK) return r;
  if (B < 0 || B > c.max_batch || Dmax < 1 || Dmax > 16) return EAGLE_EINVAL;
  if (B == 0) return EAGLE_OK;
  if (!n_old || !acc_len || !acc_path) return EAGLE_EINVAL;
  r = kv8_compact(reinterpret_cast<cudaStream_t>(stream), c, l.data(), layers, B, n_old, acc_len, acc_path, Dmax, d_err);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_ECAPACITY : EAGLE_ECUDA);
} catch (const std::bad_alloc&) {
  return EAGLE_ECAPACITY;
}

// Entries are counted in 32 bits.
static bool kv8_table_fits(const Kv8& c) { return (int64_t)c.max_batch * c.tab_w <= 0x7fffffff; }

size_t eagle_op_kv8_resize_scratch_bytes(const eagle_kv8* cache) {
  Kv8 c;
  if (kv8_view(cache, c) != EAGLE_OK || !c.table || !kv8_table_fits(c)) return 0;
  return kv8_resize_scratch(c);
}

int eagle_op_kv8_resize(void* stream, const eagle_kv8* caches, int layers, int B, int32_t* refs, const int32_t* parent,
                        const int32_t* length, void* scratch, size_t scratch_bytes, int32_t* d_err) try {
  Kv8 c;
  std::vector<Kv8Layer> l;
  int r = kv8_layers(caches, layers, c, l);
  if (r != EAGLE_OK) return r;
  if (!c.table || B < 0 || B > c.max_batch) return EAGLE_EINVAL;
  if (B == 0) return EAGLE_OK;
  if (!refs || !length) return EAGLE_EINVAL;
  if (!kv8_table_fits(c)) return EAGLE_ECAPACITY;
  if (!scratch || !on16(scratch) || scratch_bytes < kv8_resize_scratch(c)) return EAGLE_ECAPACITY;
  r = kv8_resize(reinterpret_cast<cudaStream_t>(stream), c, l.data(), layers, B, refs, parent, length, scratch, d_err);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_ECAPACITY : EAGLE_ECUDA);
} catch (const std::bad_alloc&) {
  return EAGLE_ECAPACITY;
}

// ---- rotary positions -------------------------------------------------------------------------------
int eagle_rope_frequencies(int rot, double theta, const eagle_rope_scaling* s, double* freq, float* factor) {
  if (!freq || !factor || rot < 2 || rot % 2 || rot > 65536 || !(theta > 1.0) || !std::isfinite(theta)) return EAGLE_EINVAL;
  const double pi2 = 6.283185307179586476925286766559;
  const int kind = s ? s->kind : EAGLE_ROPE_PLAIN;
  if (kind < EAGLE_ROPE_PLAIN || kind > EAGLE_ROPE_YARN) return EAGLE_EINVAL;
  if (kind != EAGLE_ROPE_PLAIN && !(s->factor >= 1.0 && std::isfinite(s->factor))) return EAGLE_EINVAL;
  *factor = 1.f;
  double base = theta, lo = 0, hi = 0;
  if (kind == EAGLE_ROPE_NTK) {
    if (rot < 4) return EAGLE_EINVAL;
    base = theta * std::pow(s->factor, (double)rot / (rot - 2));
  } else if (kind == EAGLE_ROPE_LLAMA3) {
    if (!(s->original > 0 && s->low >= 0 && s->high > s->low && std::isfinite(s->high) && std::isfinite(s->original)))
      return EAGLE_EINVAL;
  } else if (kind == EAGLE_ROPE_YARN) {
    // the pairs (as real numbers) that make `high` and `low` turns over the original context
    if (!(s->original > 0 && s->low > 0 && s->high >= s->low && std::isfinite(s->high) && std::isfinite(s->original)))
      return EAGLE_EINVAL;
    const double unit = rot / (2 * std::log(theta));
    lo = std::max(0.0, std::floor(unit * std::log(s->original / (s->high * pi2))));
    hi = std::min(rot - 1.0, std::ceil(unit * std::log(s->original / (s->low * pi2))));
    *factor = s->attention > 0 ? (float)s->attention : (float)(0.1 * std::log(s->factor) + 1);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (kind == EAGLE_ROPE_LINEAR) {
      f /= s->factor;
    } else if (kind == EAGLE_ROPE_LLAMA3) {
      const double turns = s->original * f / pi2;
      const double keep = std::min(1.0, std::max(0.0, (turns - s->low) / (s->high - s->low)));
      f = keep * f + (1 - keep) * (f / s->factor);
    } else if (kind == EAGLE_ROPE_YARN) {
      const double slow = i <= lo ? 0.0 : i >= hi ? 1.0 : (i - lo) / (hi - lo);
      f = (1 - slow) * f + slow * (f / s->factor);
    }
    freq[i] = f;
  }
  return EAGLE_OK;
}

int eagle_rope_turns(int n, const double* freq, uint64_t* turns) {
  if (n < 1 || !freq || !turns) return EAGLE_EINVAL;
  for (int i = 0; i < n; ++i) {
    const double t = freq[i] / 6.283185307179586476925286766559;
    if (!std::isfinite(t) || std::fabs(t) > 4503599627370496.0) return EAGLE_EINVAL;
    const double part = t - std::floor(t);
    turns[i] = part < 1.0 ? (uint64_t)std::ldexp(part, 64) : 0;      // (a tiny negative angle's part rounds to 1: no turn)
  }
  return EAGLE_OK;
}

// Whether rows of wa bytes, lda bytes apart, and rows of wb bytes, ldb apart, share a byte. With different strides: whether
// the spans that they lie in do.
static bool rows_meet(const void* pa, int64_t lda, int64_t wa, int Ra, const void* pb, int64_t ldb, int64_t wb, int Rb) {
  const intptr_t a = (intptr_t)pa, b = (intptr_t)pb;
  if (a + (Ra - 1) * lda + wa <= b || b + (Rb - 1) * ldb + wb <= a) return false;
  if (lda != ldb) return true;
  int64_t by = (b - a) % lda;      // b's rows from a's, within a row
  if (by < 0) by += lda;
  return by < wa || by + wb > lda;
}

int eagle_op_rope(void* stream, int dtype_in, int dtype_out, const void* q, int64_t ldq, void* q_out, int64_t ldqo, int nq,
                  const void* k, int64_t ldk, void* k_out, int64_t ldko, int nkv, int head_dim, int rot, int interleaved,
                  int R, const int32_t* pos, const uint64_t* turns, float factor, int inverse) {
  if ((dtype_in != EAGLE_DTYPE_F32 && dtype_in != EAGLE_DTYPE_BF16) ||
      (dtype_out != EAGLE_DTYPE_F32 && dtype_out != EAGLE_DTYPE_BF16))
    return EAGLE_EINVAL;
  if (R < 0 || nq < 0 || nkv < 0 || nq + (int64_t)nkv < 1 || head_dim < 16 || head_dim > 256 || head_dim % 16 || rot < 16 ||
      rot > head_dim || rot % 16 || !std::isfinite(factor))
    return EAGLE_EINVAL;
  if (R == 0) return EAGLE_OK;
  if (nq > 65536 || nkv > 65536) return EAGLE_ECAPACITY;
  if (!pos || !turns || (reinterpret_cast<uintptr_t>(turns) & 7)) return EAGLE_EINVAL;
  const int64_t ei = dtype_in == EAGLE_DTYPE_F32 ? 4 : 2, eo = dtype_out == EAGLE_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; int64_t ld, e, w; } rows[4] = {{q, ldq, ei, (int64_t)nq * head_dim}, {k, ldk, ei, (int64_t)nkv * head_dim},
                                                               {q_out, ldqo, eo, (int64_t)nq * head_dim}, {k_out, ldko, eo, (int64_t)nkv * head_dim}};
  for (const auto& r : rows) {
    if (!r.w) continue;
    if (!r.p || !on16(r.p) || r.ld < r.w || r.ld * r.e % 16 || r.ld > ((int64_t)1 << 40)) return EAGLE_EINVAL;
  }
  // an output is the input that it comes from, with the same rows and type, or meets no input and no other output
  for (int o = 2; o < 4; ++o) {
    if (!rows[o].w) continue;
    for (int i = 0; i < o; ++i) {
      if (!rows[i].w || i == o) continue;
      if (i == o - 2 && rows[i].p == rows[o].p && rows[i].e == rows[o].e && rows[i].ld == rows[o].ld) continue;
      if (rows_meet(rows[o].p, rows[o].ld * rows[o].e, rows[o].w * rows[o].e, R, rows[i].p, rows[i].ld * rows[i].e,
                    rows[i].w * rows[i].e, R))
        return EAGLE_EINVAL;
    }
  }
  RopeArgs a{};
  a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  a.ldq = ldq; a.ldk = ldk; a.ldqo = ldqo; a.ldko = ldko;
  a.R = R; a.nq = nq; a.nkv = nkv; a.d = head_dim; a.rot = rot;
  a.pos = pos; a.turns = reinterpret_cast<const unsigned long long*>(turns); a.factor = factor; a.inverse = inverse != 0;
  const int r = rope_rows(reinterpret_cast<cudaStream_t>(stream), a, dtype_in == EAGLE_DTYPE_F32, dtype_out == EAGLE_DTYPE_F32,
                          interleaved != 0);
  return r == 0 ? EAGLE_OK : (r == -1 ? EAGLE_ECAPACITY : EAGLE_ECUDA);
}

// ---- attention over whole prompts ---------------------------------------------------------------------
static int prompt_sizes(int R, int Rk, int nq, int nkv, int head_dim, int B) {
  if (R < 0 || Rk < 0 || nkv < 1 || nq < nkv || nq % nkv || nq / nkv > 64 || (head_dim != 64 && head_dim != 128) || B < 0)
    return EAGLE_EINVAL;
  // (2^27 keys keep a pair of tiles busy for up to 2 s, which the waits' limit allows for)
  if ((double)R * nq >= 2147483648.0 || Rk > (1 << 27) || nq > 65536 || B > (1 << 20)) return EAGLE_ECAPACITY;
  return EAGLE_OK;
}

size_t eagle_op_attention_prompt_scratch_bytes(int R, int Rk, int nq, int nkv, int head_dim, int B) {
  if (prompt_sizes(R, Rk, nq, nkv, head_dim, B) != EAGLE_OK || R == 0 || B == 0) return 0;
  return prompt_attention_scratch(R, Rk, nq, nkv, head_dim, B);
}

int eagle_op_attention_prompt(void* stream, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                              void* out, int64_t ldo, float* lse, int R, int Rk, int nq, int nkv, int head_dim, int B,
                              const int32_t* q_start, const int32_t* k_start, float scale, void* scratch, size_t scratch_bytes,
                              int32_t* d_err) {
  const int sizes = prompt_sizes(R, Rk, nq, nkv, head_dim, B);
  if (sizes == EAGLE_EINVAL) return sizes;
  if (R == 0 || B == 0) return EAGLE_OK;
  if (sizes != EAGLE_OK) return sizes;
  if (scratch && !on16(scratch)) return EAGLE_EINVAL;
  const int64_t wq = (int64_t)nq * head_dim, wk = (int64_t)nkv * head_dim, most = (int64_t)1 << 36;
  if (!q || !out || !q_start || !k_start || (Rk && (!k || !v))) return EAGLE_EINVAL;
  if (!on16(q) || !on16(k) || !on16(v) || !on16(out)) return EAGLE_EINVAL;
  if (ldq < wq || ldo < wq || ldq % 8 || ldo % 8 || ldq > most || ldo > most) return EAGLE_EINVAL;
  if (Rk && (ldk < wk || ldv < wk || ldk % 8 || ldv % 8 || ldk > most || ldv > most)) return EAGLE_EINVAL;
  // results go out while other items still read: none of the inputs may be their place
  if (rows_meet(out, ldo * 2, wq * 2, R, q, ldq * 2, wq * 2, R)) return EAGLE_EINVAL;
  if (Rk && (rows_meet(out, ldo * 2, wq * 2, R, k, ldk * 2, wk * 2, Rk) || rows_meet(out, ldo * 2, wq * 2, R, v, ldv * 2, wk * 2, Rk)))
    return EAGLE_EINVAL;
  // the sums and the scratch memory lie outside all of them
  const struct { const void* p; int64_t w; } own[2] = {{lse, (int64_t)R * nq * 4}, {scratch, scratch ? (int64_t)scratch_bytes : 0}};
  for (const auto& x : own) {
    if (!x.p || x.w <= 0) continue;
    if (rows_meet(x.p, x.w, x.w, 1, q, ldq * 2, wq * 2, R) || rows_meet(x.p, x.w, x.w, 1, out, ldo * 2, wq * 2, R)) return EAGLE_EINVAL;
    if (Rk && (rows_meet(x.p, x.w, x.w, 1, k, ldk * 2, wk * 2, Rk) || rows_meet(x.p, x.w, x.w, 1, v, ldv * 2, wk * 2, Rk)))
      return EAGLE_EINVAL;
  }
  if (lse && scratch && rows_meet(lse, own[0].w, own[0].w, 1, scratch, own[1].w, own[1].w, own[1].w ? 1 : 0)) return EAGLE_EINVAL;
  PromptArgs a{};
  a.q = q; a.k = k; a.v = v; a.out = out; a.lse = lse;
  a.ldq = ldq; a.ldk = ldk; a.ldv = ldv; a.ldo = ldo;
  a.R = R; a.Rk = Rk; a.nq = nq; a.nkv = nkv; a.d = head_dim; a.B = B;
  a.start = q_start; a.kstart = k_start;
  a.scale = scale > 0.f ? scale : 1.f / sqrtf((float)head_dim);
  a.scratch = scratch; a.scratch_bytes = scratch ? scratch_bytes : 0;
  a.err = d_err;
  const int r = prompt_attention(reinterpret_cast<cudaStream_t>(stream), a);
  return r == 0 ? EAGLE_OK : EAGLE_ECUDA;
}

}  // extern "C"
