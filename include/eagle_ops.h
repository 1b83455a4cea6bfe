/*
 * eagle_ops.h -- kernel-level entry points of the EAGLE cycle library.
 *
 * Each call runs one of the cycle's kernels on caller-provided device buffers, so it
 * can be checked on its own against the CPU oracle with injected inputs. All pointers
 * are DEVICE pointers unless stated; `stream` is a cudaStream_t cast to void*; calls
 * are stream-ordered and return an eagle_status (see eagle.h) without waiting.
 * `scratch` is caller-owned device memory of at least the size the matching
 * *_scratch_bytes function returns; the library never allocates device memory.
 */
#ifndef EAGLE_OPS_H
#define EAGLE_OPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Projection GEMM Y[M][N] = X[M][K] * W[N][K]^T (the nn.Linear layout used for every
 * target and drafter projection and the LM head). dtype EAGLE_DTYPE_BF16: tcgen05
 * tensor-core kernel, X and W bf16 row-major with K a multiple of 8 and 16-byte
 * aligned bases; dtype EAGLE_DTYPE_F32: fp32 FFMA kernel. epi: 0 = store fp32 Y,
 * 1 = store bf16 Y (bf16 only), 2 = Y += result (fp32 residual update), 4 = SwiGLU
 * (bf16 only, N % 64 == 0): W holds 2N rows [Wgate; Wup] and out (bf16, [M][N]) receives
 * silu(X Wgate^T) * (X Wup^T); size its scratch with eagle_op_gemm_scratch_bytes(M, 2N).
 * out has row stride ldo elements. Scratch holds split-tile partial sums and per-tile
 * counters; it must be zero-filled before the first call and is left zeroed by every call.
 * The kernel's CTAs hand partial sums to one another, so no other work may hold SMs for
 * the whole of a call (kernels on other streams that finish on their own are fine). */
size_t eagle_op_gemm_scratch_bytes(int M, int N);
int eagle_op_gemm(int dtype, void* stream, const void* W, int N, int K, const void* X, int M, int epi,
                  void* out, int ldo, void* scratch, size_t scratch_bytes);

/* Allocation-free variant of eagle_op_gemm (bf16 only) for callers that cannot
 * allocate device memory where they run a projection, e.g. plugins of a host framework
 * that hands them only input and output buffers, or runtimes that pool all device
 * memory in advance. The paper has no counterpart: this is a deployment convenience.
 * Its split-tile scratch lives in file-scope device arrays of the library (about 6 MiB
 * on every GPU that loads it, held until the process exits), so the call allocates
 * nothing (no cudaMalloc/cudaFree, no allocating library routine).
 * Limits: M <= 32 rows and at most 8192 output tiles (ceil(N/128) tiles for M <= 32);
 * larger requests return EAGLE_ECAPACITY. epi as eagle_op_gemm (0, 1 or 2).
 * The first call on a device looks up the arrays' device addresses (cudaGetSymbolAddress)
 * with that device current; make that first call before any stream capture. All calls
 * share the one scratch area and the last call's contents remain in it: calls that may
 * overlap on the GPU (different streams without ordering) race and must not be issued;
 * graph replays that contain this call must be serialised the same way.
 * A bounded device wait that gives up leaves `out` incomplete and records a timeout in a
 * status word that is also a file-scope device array; read it with
 * eagle_op_gemm_noalloc_status. */
int eagle_op_gemm_noalloc(void* stream, const void* W, int N, int K, const void* X, int M, int epi, void* out,
                          int ldo);

/* Status of the allocation-free GEMM on the current device: waits for `stream`, reads
 * the status word that its calls share and clears it. EAGLE_OK when no call since the
 * last read gave up, EAGLE_ETIMEOUT when one did (its output is incomplete). */
int eagle_op_gemm_noalloc_status(void* stream);

/* Fused LM head: logits = X[M][H] * W_lm[V][H]^T reduced per row without writing the
 * logits (bf16), or through an fp32 logits buffer inside the scratch (f32). Per row it
 * returns the K best entries by ranking value (value desc, token id asc) and the
 * log-sum-exp of logit * inv_t. Ranking value = logit * inv_t, plus Gumbel(0,1) noise
 * when gumbel != 0, drawn from Philox4x32-10 keyed by (seed; counter = (id >> 2,
 * row_key[row], cycle, row_seq[row] << 8 | stream_id)), word id & 3. specials
 * [M][S] (nullable, -1 = unused): ids left out of the ranking (and out of the
 * log-sum-exp when lse_excl != 0) whose raw logits go to spec_logit [M][S].
 * Outputs: top_id [M][K] int32, top_val [M][K] float, lse [M] float. K in 1..16. */
size_t eagle_op_lm_head_scratch_bytes(int dtype, int V, int M, int K);
int eagle_op_lm_head(int dtype, void* stream, const void* W_lm, int V, int H, const void* X, int M, int K,
                     float inv_t, int gumbel, int lse_excl, const int32_t* specials, int S, float* spec_logit,
                     const int32_t* row_seq, const int32_t* row_key, uint32_t cycle, uint64_t seed,
                     int stream_id, int32_t* top_id, float* top_val, float* lse, void* scratch,
                     size_t scratch_bytes);

/* Tree-masked attention of R query rows over a KV cache laid out
 * [seq][kv_head][slot][d] with `cap` slots and max_batch sequences (storage type dtype;
 * row_seq < max_batch). q, out: [R][nq][d].
 * Rows of one sequence are contiguous, rows_per_seq each; row r belongs to sequence
 * row_seq[r] and its own key sits at slot row_slot[r]. mode 0 (causal): row r sees
 * slots <= row_slot[r]. mode 1 (tree): row r sees slots < ctx_len[seq] and slot
 * ctx_len[seq] + t for t < tree_T where bit t of mask[r][t / 64] is set.
 * Scale = 1/sqrt(d) when scale <= 0. fp32: d <= 128, scratch unused (nullable); bf16
 * (tensor cores): d in {32, 64, 128}, 64 divisible by nq/nkv, tree_T <= 256, scratch of
 * eagle_op_attention_scratch_bytes required (EAGLE_ECAPACITY without it). The bf16 path
 * gives each row a result that does not depend on the other rows of the call: a row at
 * logical position P (its own slot in causal mode, ctx_len + its mask's popcount - 1 in
 * tree mode, whose ancestors must have increasing slots by depth) has its keys up to
 * position P - 16 summed in fixed key splits on the tensor cores, its last 16 positions in
 * position order on the FMA units, and the two merged in a fixed order; so a tree row and
 * a causal row at the same position over the same keys give bit-identical outputs. The
 * split length is that of an engine serving up to max_batch sequences (>= 1): three
 * 64-key tiles below eight sequences, eight from eight on; calls with the same cap and
 * max_batch share it. With d = 128 and EAGLE_ATTN_TC=1 in the environment the splits run on
 * tcgen05 (TMA tiles of the cache, S and O in TMEM; a different summation order, fixed for the
 * process). */
size_t eagle_op_attention_scratch_bytes(int R, int nq, int d);
int eagle_op_attention(int dtype, void* stream, const void* q, const void* kcache, const void* vcache,
                       void* out, int R, int nq, int nkv, int d, int cap, int rows_per_seq,
                       const int32_t* row_seq, const int32_t* row_slot, const int32_t* ctx_len, int mode,
                       int tree_T, const uint64_t* mask, int mask_words, float scale, int max_batch,
                       void* scratch, size_t scratch_bytes);

/* ---- 8-bit KV cache ---------------------------------------------------------------------------
 * One layer's keys and values in e4m3 with one power-of-two exponent byte per (slot, head)
 * vector: value = code * 2^(byte - 127). A written vector x gets the smallest exponent e in
 * [-40, 40] with max|x| <= 448 * 2^e (byte e + 127) and codes rounded to nearest even
 * (magnitudes above 448 * 2^40 saturate); a vector with an entry that is not finite gets byte
 * 255 and zero codes, and reads back as NaN throughout. Reading is exact in bf16 and fp32, and
 * writing what was read stores the same values, so entries move (compaction of an accepted path,
 * a sequence handed to another cache) by eagle_op_kv8_read and eagle_op_kv8_write. Cleared memory
 * (codes and bytes zero) counts as zero vectors. A slot that is read or that an attention row sees
 * holds what was written, or cleared memory; other bytes give unspecified values there.
 *
 * table == NULL: contiguous, codes [max_batch][n_kv_heads][cap][head_dim] and exponents
 * [max_batch][n_kv_heads][cap]; cap a multiple of 16. Otherwise paged: pools
 * [n_blocks][n_kv_heads][block][head_dim] and [n_blocks][n_kv_heads][block], block a power of
 * two from 16 to 256, and the device block table [max_batch][cap / block] (int32, pool block
 * of each sequence's slots [j * block, (j + 1) * block), -1 = unassigned); cap a multiple of
 * block. head_dim 64 or 128. All four arrays start on 16-byte boundaries and hold fewer than
 * 2^31 vectors each. The struct itself is host memory, read during the call. */
typedef struct {
  void *k_code, *v_code; /* e4m3 */
  void *k_exp, *v_exp;   /* uint8 */
  const int32_t* table;
  int n_kv_heads, head_dim, max_batch, cap, block, n_blocks;
} eagle_kv8;

/* Quantise rows into the cache: k and v hold R rows of [n_kv_heads][head_dim] (dtype
 * EAGLE_DTYPE_BF16 or EAGLE_DTYPE_F32, 16-byte aligned) with row strides ldk and ldv elements
 * (multiples of 16 bytes, >= n_kv_heads * head_dim), e.g. the k and v columns of a fused
 * projection. Row r goes to slot row_slot[r] of sequence row_seq[r]; a row with row_seq[r] < 0 is
 * padding and is skipped. The rows of one call name different (sequence, slot) pairs. A sequence,
 * slot or table entry out of range is latched into *d_err (nullable device int32: 2) and its row
 * skipped; nothing else of the cache changes. R = 0 does nothing. */
int eagle_op_kv8_write(void* stream, const eagle_kv8* cache, int dtype, const void* k, int64_t ldk, const void* v,
                       int64_t ldv, int R, const int32_t* row_seq, const int32_t* row_slot, int32_t* d_err);

/* Read cache entries back: row r of k and v (layout, types and strides as above) receives slot
 * row_slot[r] of sequence row_seq[r], any number of times the same. Padding rows and rows out of
 * range (latched into *d_err) receive zeros; the gap between row strides is left as it was. */
int eagle_op_kv8_read(void* stream, const eagle_kv8* cache, int dtype, void* k, int64_t ldk, void* v, int64_t ldv,
                      int R, const int32_t* row_seq, const int32_t* row_slot, int32_t* d_err);

/* Attention of R query rows over an 8-bit cache, with the row model of eagle_op_attention: q and
 * out bf16 [R][nq][head_dim] (16-byte aligned), nq a multiple of n_kv_heads with at most 64
 * query heads per KV head, rows of one sequence contiguous (rows_per_seq each; the last may have
 * fewer). mode 0 (causal): row r sees slots <= row_slot[r]. mode 1 (tree): row r sees slots <
 * ctx_len[seq] and slot ctx_len[seq] + t for t < tree_T (1..256) where bit t of
 * mask[r][t / 64] is set (mask_words >= ceil(tree_T / 64); row_slot is not read). ctx_len is
 * indexed by sequence ([max_batch]; not read in mode 0). A row that sees nothing, and a padding
 * row (row_seq[r] < 0), gets zeros. A row whose sequence differs from that of the first
 * not-padding row among its rows_per_seq, a sequence outside the cache, a negative ctx_len, a
 * visible slot at or past cap and a table entry out of range are latched into *d_err (nullable):
 * such a row gets zeros, a negative ctx_len hides all slots of its sequence, slots past cap are
 * left out, and a bad table entry makes its slots unspecified (every entry up to the last slot that
 * a sequence's rows see is looked up, those of slots in between that no row sees too). Slots
 * that no row sees may hold anything. Scale = 1/sqrt(head_dim) when scale <= 0.
 * out may be q itself; otherwise the two do not overlap (refused).
 * Sums, maxima and softmax weights' sums are fp32. A weight times its value's power of two enters
 * the value product as fp16: to 2^-11 of itself, and to 2^-32 of the query vector's largest such
 * product at least. q is used as fp16 times a power of two (entries down to 2^-30 of its largest
 * exactly, smaller ones to within 2^-38 of the largest), but with head_dim 128 and more than 16 query
 * vectors a block (rows x query heads of a KV head, up to 128 together) it is held in two e4m3 parts:
 * entries down to 2^-9 of the vector's largest exactly, others to within 2^-17 of it.
 * A row's result does not depend on the values of other rows or sequences; their lengths move
 * the points where its sum over slots is split, so it can change in the last bits of fp32. Nor do
 * a decoding step's rows and a verify pass's agree bit for bit, as eagle_op_attention's do: the
 * number of rows chooses the kernel.
 * scratch: eagle_op_attention_kv8_scratch_bytes of the same sizes, no initial value needed; two
 * calls that may overlap on the GPU (graph replays included) need their own. */
size_t eagle_op_attention_kv8_scratch_bytes(const eagle_kv8* cache, int R, int nq, int rows_per_seq, int prefix_len);
int eagle_op_attention_kv8(void* stream, const eagle_kv8* cache, const void* q, void* out, int R, int nq,
                           int rows_per_seq, const int32_t* row_seq, const int32_t* row_slot, const int32_t* ctx_len,
                           int mode, int tree_T, const uint64_t* mask, int mask_words, float scale, void* scratch,
                           size_t scratch_bytes, int32_t* d_err);

/* The same for sequences that share a prefix: every row first sees all prefix_len entries of
 * prefix_k / prefix_v (bf16 [n_kv_heads][prefix_len][head_dim], 16-byte aligned; kept at full
 * precision, being stored once for the whole batch) and then its own slots as above, in one
 * softmax. The prefix is one matrix product over all rows of a head, read once per 256 query
 * vectors rather than once per sequence; its weights enter the value product as bf16 (2^-8), the
 * type of the values that they meet, in one part (eagle_op_attention takes two). Padding rows get zeros. prefix_len = 0 is
 * eagle_op_attention_kv8. */
int eagle_op_attention_shared_kv8(void* stream, const eagle_kv8* cache, const void* prefix_k, const void* prefix_v,
                                  int prefix_len, const void* q, void* out, int R, int nq, int rows_per_seq,
                                  const int32_t* row_seq, const int32_t* row_slot, const int32_t* ctx_len, int mode,
                                  int tree_T, const uint64_t* mask, int mask_words, float scale, void* scratch,
                                  size_t scratch_bytes, int32_t* d_err);

/* ---- blocks and accepted paths of an 8-bit cache's layers -----------------------------------------
 * caches: HOST array of one eagle_kv8 a layer, read during the call; all layers have one shape and
 * one table, and each has arrays of its own (a layer given twice would be moved twice, in any
 * order). Calls on one table (and writes of the cache) change it and are ordered by the caller.
 *
 * Accepted paths to their committed slots, in all layers and heads: slot n_old[b] + j receives what
 * slot n_old[b] + acc_path[b][j - 1] held, j = 1..acc_len[b], for sequences b < B (n_old, acc_len [B],
 * acc_path [B][Dmax], Dmax <= 16; codes and exponents are copied, so values stay exactly). A sequence's
 * moves take effect at once, whatever their order. acc_len <= 0: nothing to do. A length above Dmax
 * is taken for Dmax; it, a slot outside the cache and a block that is not assigned are latched
 * into *d_err (2), such a slot's move is left out. Paged or contiguous. The slots that are written
 * must be the sequence's own (eagle_op_kv8_resize sees to that). */
int eagle_op_kv8_compact(void* stream, const eagle_kv8* caches, int layers, int B, const int32_t* n_old,
                         const int32_t* acc_len, const int32_t* acc_path, int Dmax, int32_t* d_err);

/* Block bookkeeping of a paged cache. State: the table and refs [n_blocks], for each pool block the number of
 * table entries that hold it (zero: free). After the call sequence b < B has blocks for slots
 * [0, length[b]) and no others; length[b] < 0 leaves it as it is. (a) Surplus entries are
 * released: -1 in the table, one off the count. (b) A fork, a sequence with parent[b] >= 0 (parent
 * nullable: no forks), releases all its entries and takes those of its parent's first length[b] slots: the
 * blocks are shared. Any number of sequences may fork one parent; the parent has length < 0 in
 * this call and blocks for all those slots. (c) Missing entries get free blocks, the lowest-numbered
 * first, in the order of sequences and slots. (d) A last block that is partly filled and that other entries
 * hold too is replaced by a free one (counted in the same order) and its filled slots are copied
 * in all layers: what a sequence writes at length[b] and behind is never seen by another. A block
 * that loses its last holder by (d) is free from the next call on.
 * length[b] past cap, and a parent that is out of range, is b itself, takes part in the call or lacks a
 * block, are latched into *d_err (2) and leave b as it was. An entry outside the pool in a sequence that takes part is
 * latched (2) and cleared, so a slot that is to have a block gets one by (c); so is an entry that is released while its
 * block's count is zero already (counts of entries that stay are not looked at). Too few free blocks: latched (3); the entries that come
 * first in the order have theirs, the others stay -1, and a block that should have been copied
 * stays shared. scratch: no initial value, not shared with a call that may overlap on the GPU. A table of 2^31 entries and
 * more is refused (EAGLE_ECAPACITY, scratch bytes 0). */
size_t eagle_op_kv8_resize_scratch_bytes(const eagle_kv8* cache);
int eagle_op_kv8_resize(void* stream, const eagle_kv8* caches, int layers, int B, int32_t* refs, const int32_t* parent,
                        const int32_t* length, void* scratch, size_t scratch_bytes, int32_t* d_err);

/* ---- rotary positions ------------------------------------------------------------------------------
 * Frequencies on the host: freq[i], i < rot / 2, the angle that pair i turns by from one position to the next,
 * theta^(-2i / rot) under one of these rules for contexts beyond the trained one (scaling nullable: plain):
 * LINEAR: divided by factor. NTK: base theta * factor^(rot / (rot - 2)). LLAMA3: pairs of at most
 * `low` turns in the original context divided by factor, of `high` and more unchanged, between them a
 * blend, linear in the turns. YARN: unchanged up to the pair of `high` turns, divided by factor from the pair of
 * `low` turns on (both rounded outwards to whole pairs), a ramp over the pairs between; *factor
 * receives `attention`, or 0.1 ln(factor) + 1 when that is not positive, by which the op scales turned
 * entries; it is 1 otherwise. */
enum { EAGLE_ROPE_PLAIN = 0, EAGLE_ROPE_LINEAR = 1, EAGLE_ROPE_NTK = 2, EAGLE_ROPE_LLAMA3 = 3, EAGLE_ROPE_YARN = 4 };
typedef struct {
  int kind;
  double factor;       /* >= 1 */
  double original;     /* trained context (LLAMA3, YARN) */
  double low, high;    /* turns (LLAMA3, YARN) */
  double attention;    /* YARN */
} eagle_rope_scaling;
int eagle_rope_frequencies(int rot, double theta, const eagle_rope_scaling* scaling, double* freq, float* factor);

/* The op's table from angles per position (radians, of any rule): turns[i] = freq[i] / 2 pi modulo 1, in
 * 2^-64. Host memory; copy it to the device. */
int eagle_rope_turns(int n, const double* freq, uint64_t* turns);

/* Turn the first `rot` entries of each head of R rows of q ([nq][head_dim]) and k ([nkv][head_dim]; either count may be
 * 0), row r by pos[r] * freq: pairs (x[i], x[i + rot / 2]), or (x[2i], x[2i + 1]) when interleaved, become
 * factor * (a cos - b sin, b cos + a sin), with `inverse` the same by the negative angle: so a gradient with respect to
 * turned rows becomes that with respect to the rows. Entries behind `rot` are copied. head_dim 16..256 and rot
 * 16..head_dim, multiples of 16. Types EAGLE_DTYPE_F32 or _BF16, in and out independently; 16-byte aligned rows of free stride (elements, whole 16 bytes), so q
 * and k may be columns of a fused projection. An output may be the input it comes from (same type, rows
 * and stride); otherwise outputs meet neither an input nor each other (refused). turns: device [rot / 2].
 * Positions are any int32: the angle is taken modulo a turn without rounding, then rounded to fp32 (2^-24
 * relative), arithmetic is fp32 and the result is rounded once. */
int eagle_op_rope(void* stream, int dtype_in, int dtype_out, const void* q, int64_t ldq, void* q_out, int64_t ldqo, int nq,
                  const void* k, int64_t ldk, void* k_out, int64_t ldko, int nkv, int head_dim, int rot, int interleaved,
                  int R, const int32_t* pos, const uint64_t* turns, float factor, int inverse);

/* Causal attention over whole prompts, packed: sequence b < B has rows q[q_start[b] .. q_start[b + 1]) and keys and values
 * k, v[k_start[b] .. k_start[b + 1]). Its last row sees all its keys, each row before it one fewer: with as many rows as
 * keys a whole prompt, with fewer the last chunk of one, with more the first rows see nothing (zeros, lse
 * -inf). q, out bf16 [R][nq][head_dim], k, v bf16 [Rk][nkv][head_dim], 16-byte aligned with free row strides (elements,
 * multiples of 8), head_dim 64 or 128, at most 64 query heads a KV head. lse (nullable): fp32 [R][nq], the natural
 * logarithm of each row's sum of exp(score), by which results over different keys can be joined. Scale =
 * 1/sqrt(head_dim) when scale <= 0. q_start, k_start: device [B + 1], read by the kernel, so that a captured call serves
 * any lengths; a sequence whose starts fall, or lie outside [0, R] or [0, Rk], is latched into *d_err (nullable) and
 * skipped (where starts fall back so often that sequences overlap, others may be skipped too). Rows of no
 * sequence are left as they were. out meets none of q, k, v, and lse and scratch none of the others (refused). R * nq < 2^31, Rk <=
 * 2^27, B <= 2^20 (EAGLE_ECAPACITY). A wait inside the kernel that gives up (after 2 s and 4 us for every 80 keys of the call, 128
 * for heads of 64) latches 1 into *d_err and leaves rows unwritten; without d_err nothing tells.
 * Products are bf16 with fp32 sums; weights enter the value product as bf16 (2^-8 relative, the type of the values);
 * maxima, sums and lse are fp32. Keys and values that a row does not see, of its own sequence too, may be anything,
 * NaN and infinities among it: its result is the same bits.
 * scratch (nullable, 16-byte aligned, no initial value, not shared with a call that may overlap on the GPU): with the bytes that
 * eagle_op_attention_prompt_scratch_bytes gives for these sizes (0 where there is no use for it) calls of few rows over many
 * keys have their keys shared out over the GPU, at points that all sequences' lengths move; a row's result can then change in
 * the last bits of fp32 with the batch. With less, or where 0 is given, it does not depend on the batch. */
size_t eagle_op_attention_prompt_scratch_bytes(int R, int Rk, int nq, int nkv, int head_dim, int B);
int eagle_op_attention_prompt(void* stream, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                              void* out, int64_t ldo, float* lse, int R, int Rk, int nq, int nkv, int head_dim, int B,
                              const int32_t* q_start, const int32_t* k_start, float scale, void* scratch, size_t scratch_bytes,
                              int32_t* d_err);

/* EAGLE-2 tree growth and rerank with injected draft confidences, for B sequences:
 * cand_tok/cand_logc [B][k]: the root's children (token, log confidence) in rank order;
 * child_tok/child_logc [B][depth-1][k][k]: children of the r-th node selected at depth
 * d (entry [b][d-1][r][i], rank order). ctx_len [B], root_tok [B].
 * Outputs: node tables [B][NG] (tok, parent, depth int32; logv float), flattened tree
 * [B][m+1] (tok, pos, parent, node int32) and ancestry bitmask [B][m+1][W] uint64 with
 * W = ceil((m+1)/64). */
size_t eagle_op_tree_scratch_bytes(int B, int k, int depth, int m);
int eagle_op_tree_build(void* stream, int B, int k, int depth, int m, const int32_t* cand_tok,
                        const float* cand_logc, const int32_t* child_tok, const float* child_logc,
                        const int32_t* ctx_len, const int32_t* root_tok, int32_t* node_tok, int32_t* node_parent,
                        int32_t* node_depth, float* node_logv, int32_t* tree_tok, int32_t* tree_pos,
                        int32_t* tree_parent, int32_t* tree_node, uint64_t* tree_mask, void* scratch,
                        size_t scratch_bytes);

/* KV compaction: in every layer, slot n_old[b] + j <- slot n_old[b] + acc_path[b][j-1]
 * for j = 1..acc_len[b] (acc_path rows are flattened-tree rows, Dmax per sequence,
 * Dmax <= 8). Cache layout [layer][seq][kv_head][slot][d], cap slots per sequence. */
int eagle_op_compact(int dtype, void* stream, void* kcache, void* vcache, int layers, int B, int nkv, int cap,
                     int d, const int32_t* n_old, const int32_t* acc_len, const int32_t* acc_path, int Dmax);

/* Batch-aware draft budget (host arithmetic only, no device work). For each candidate k
 * (k_values[j], n_k of them) the caller supplies draft_us[j], the measured drafter cost of a
 * cycle, and exp_tokens[off_j + m - 1] for m = 1..m_max[j] (off_j = sum of the earlier
 * m_max), the expected committed tokens per sequence of a tree of m nodes: 1 + the sum of
 * the m largest path values, averaged over real cycles (a node's path value estimates its
 * acceptance: "EAGLE-2: Context-Aware Dynamic Draft Trees", "Path Value Ranks Prefixes").
 * rows_pts / verify_us (n_points, rows strictly increasing) are measured verify-pass times
 * against verify rows; between points the time is interpolated linearly, beyond the last
 * it grows with the last slope (flat before the first; a single point is flat up to it and
 * proportional past it). Returns in best_k / best_m the choice maximising
 * batch * exp_tokens / (draft_us + verify(batch * (m + 1))) and that rate (tokens per
 * microsecond, nullable). Ties keep the earlier k and the smaller m. EAGLE_EINVAL on bad
 * arguments. */
int eagle_plan_budget(int n_k, const int32_t* k_values, const float* draft_us, const int32_t* m_max,
                      const float* exp_tokens, int n_points, const int32_t* rows_pts, const float* verify_us,
                      int batch, int32_t* best_k, int32_t* best_m, float* tokens_per_us);

/* Failure-detection probe. Runs one of the library's bounded device waits on a condition
 * that nothing satisfies and returns once it gives up: kind 0 waits on a shared-memory
 * mbarrier phase that nobody completes (the wait of the TMA / tensor-core pipelines),
 * kind 1 waits until the device word *d_counter (caller-owned, zero, nullable for kind 0)
 * reaches 1 (the wait of the split-tile owner). Each wait stops after
 * the library's limit of 2 s of %globaltimer and atomically latches 1 (timeout) into *d_err
 * if it is still 0; *d_result receives 1 if the wait was satisfied, 0 if it gave up. Launches
 * one CTA on `stream` and returns without synchronising; EAGLE_EINVAL on a bad kind or a
 * null pointer. */
int eagle_op_wait_probe(void* stream, int kind, const unsigned* d_counter, int* d_err, int* d_result);

#ifdef __cplusplus
}
#endif
#endif /* EAGLE_OPS_H */
