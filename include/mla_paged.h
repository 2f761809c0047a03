/*
 * mla_paged.h — paged-cache operators of the B200 (sm_100a) library next to the
 * latent decode and prefill of mla_decode.h: the writers of the caches, and
 * attention over the grouped-head (GQA) cache, the form from which MLA models
 * are converted and against which they are compared.
 *
 *   mla_gqa_append      keys and values into the grouped-head cache, keys (and
 *                       queries) rotated by their positions on the way
 *   mla_latent_append   latent rows into the MLA caches that mla_decode_run and
 *                       mla_decode_run_fp8 read, RoPE keys (and queries)
 *                       rotated on the way
 *   mla_gqa_decode_run  attention of a sequence's newest tokens over its pages,
 *                       split over the cache's length and joined
 *   mla_gqa_prefill_run causal attention of packed prompts over their pages
 *
 * Caches (row-major, pages of 64 tokens):
 *   k_pool, v_pool [num_blocks, Hk, 64, d]   one page of one head is contiguous
 *   latent pools   as in mla_decode.h
 *   block_table int32 [B, block_table_stride], seq_lens int32 [B]: entry (b, i)
 *   is the block of tokens [64 i, 64 i + 64) of sequence b; L_b counts the new
 *   tokens of the call, which are the newest of the cache.
 * Packed tokens: cu_seqlens int32 [B + 1] (device), sequence b owns rows
 * [cu[b], cu[b+1]) of the packed tensors; n_b = cu[b+1] - cu[b] of its L_b
 * tokens are new. Rows at or behind cu[B] belong to no sequence: nothing is made
 * of them and their outputs are left as they were.
 *
 * Slots of a page past L_b are never used, whatever they hold (NaN included).
 * Keys and values of a sequence's own tokens must be finite.
 *
 * Ownership, streams, graph capture and errors are those of mla_decode.h: the
 * caller owns every device buffer, nothing allocates or synchronises, and what
 * is wrong on the device (a block id outside [0, num_blocks), a length outside
 * [0, 64 block_table_stride] or above 2^31 - 4096, rows of cu_seqlens outside the packed tensors, a
 * position outside the rotation table, an append of more packed tokens than L_b) is recorded as MLA_ERR_BOUNDS in the
 * workspace's status word (mla_decode_read_status), while the work it concerns
 * is skipped. Calls run on the current device, which must be the stream's. A
 * workspace belongs to one call in flight at a time (two streams or two graphs
 * that may overlap need one each: the results of calls that share one are not
 * defined, though both end and write nothing but their own outputs); it is
 * initialised once with mla_workspace_init.
 */
#ifndef MLA_PAGED_H
#define MLA_PAGED_H

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which elements of a head form the pairs that a position rotates, for a
 * rotation of D elements: (i, i + D/2), or (2i, 2i + 1). The pair i turns by
 * the table's angle i: (a, b) -> (a cos - b sin, b cos + a sin). */
typedef enum { MLA_ROPE_HALF = 0, MLA_ROPE_INTERLEAVED = 1 } mla_rope_style_t;

typedef struct {
  int32_t num_q_heads;    /* Hq, a multiple of num_kv_heads */
  int32_t num_kv_heads;   /* Hk; query head h reads key head h / (Hq / Hk) */
  int32_t head_dim;       /* d: 64 or 128 */
  int32_t q_len;          /* Lq: new tokens per sequence where no cu_seqlens is given */
  int32_t page_size;      /* tokens per cache block; 64 */
  int32_t rope_dim;       /* D: leading elements of a head that append rotates; 0 (none) or a multiple of 16 up to d */
  int32_t rope_style;     /* mla_rope_style_t */
  int32_t dtype;          /* MLA_BF16 or MLA_FP16: activations, caches and outputs. Attention rounds the softmax
                             weights to it once, before the product with the values; scores, maxima, sums and
                             accumulators are fp32 */
  float softmax_scale;    /* multiplies q.k; usually 1/sqrt(d) */
} mla_gqa_dims_t;

/* ---- Appending ------------------------------------------------------------
 * Token t of a sequence b (i = t - cu[b], or t mod Lq without cu_seqlens) has
 * the position L_b - n_b + i, which gives its page, its slot and its row of the
 * rotation table: fp32 [rope_positions, D], cos of the D/2 angles in the first
 * half of the columns, sin in the second (any base or scaling). Without
 * cu_seqlens a slot of L_b < Lq tokens (0: an idle slot) has only the last L_b
 * of its Lq rows, as in the grouped-head decode; its other rows are like rows
 * that belong to no sequence. Rotation in fp32, one rounding to the stored
 * type. Sources may be views: strides count elements, the last dimension is
 * contiguous. An output may be its own source (q_out = q with the same strides
 * as a contiguous [T, H, D]); otherwise outputs and caches may not overlap the
 * sources. */
typedef struct {
  const void* k;                 /* [T, Hk, d] */
  int64_t k_token_stride, k_head_stride;
  const void* v;                 /* [T, Hk, d] */
  int64_t v_token_stride, v_head_stride;
  const void* q;                 /* [T, Hq, d], or NULL: keys and values only */
  int64_t q_token_stride, q_head_stride;
  void* q_out;                   /* [T, Hq, d] contiguous (with q) */
  void* k_pool;
  void* v_pool;
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t block_table_stride;
  int32_t batch;                 /* B */
  const int32_t* seq_lens;
  const int32_t* cu_seqlens;     /* NULL: Lq tokens of every sequence, T = B Lq */
  int64_t num_tokens;            /* T: rows of the packed tensors (0: nothing to do) */
  const float* rope_table;       /* 16-byte aligned; may be NULL when D = 0 */
  int64_t rope_positions;
} mla_gqa_append_args_t;

/* One kernel on `stream`. Sources, q_out and pools must be 16-byte aligned and
 * the strides multiples of 8 elements (else MLA_ERR_INVALID_ARG). workspace:
 * at least 1 KB, for the status word. */
mla_status_t mla_gqa_append(const mla_gqa_dims_t* dims, const mla_gqa_append_args_t* args,
                            void* workspace, size_t workspace_bytes, void* stream);

typedef struct {
  const void* ckv;               /* [T, r] */
  int64_t ckv_token_stride;
  const void* k_rope;            /* [T, D] before rotation, D = d_rope (NULL when D = 0) */
  int64_t k_rope_token_stride;
  const void* q_rope;            /* [T, H, D] before rotation, or NULL */
  int64_t q_rope_token_stride, q_rope_head_stride;
  void* q_rope_out;              /* [T, H, D] contiguous (with q_rope) */
  void* kv_pool;                 /* [num_blocks, 64, r + D]; FP8 cache: the codes [num_blocks, 64, r] */
  void* kv_rope;                 /* FP8 cache: bf16 [num_blocks, 64, D] (else NULL) */
  float* kv_scale;               /* FP8 cache: fp32 [num_blocks, 64] (else NULL) */
  void* kv_rows;                 /* [T, r + D] contiguous: the rows mla_prefill_run reads (bf16 for an FP8
                                    cache), or NULL */
  int64_t num_blocks;
  const int32_t* block_table;
  int32_t block_table_stride;
  int32_t batch;
  const int32_t* seq_lens;
  const int32_t* cu_seqlens;     /* NULL: dims->q_len tokens of every sequence */
  int64_t num_tokens;
  const float* rope_table;       /* [rope_positions, D], 16-byte aligned; may be NULL when D = 0 */
  int64_t rope_positions;
} mla_latent_append_args_t;

/* Appends to the latent cache of a decode plan with the same dims (num_heads,
 * latent_rank, rope_dim, q_len and dtype are used): bf16, fp32, or the FP8
 * cache (r and D multiples of 16, D <= 256), where a token's scale is
 *   s = max(max_i |cKV_i| / 448, 2^-64),
 * its codes are e4m3(cKV / s) (round to nearest even) and its RoPE key is
 * stored as bf16(k_rope / s). Only the tokens' own slots are written: clear a
 * fresh pool once, since the latent decode weights unused slots of a page by 0
 * and needs them finite. d_rope must be even. Any alignment; 16-byte
 * aligned pointers and strides (and r, D multiples of 16) take the wide path,
 * and the FP8 cache needs them. One kernel on `stream`. */
mla_status_t mla_latent_append(const mla_dims_t* dims, int32_t rope_style,
                               const mla_latent_append_args_t* args,
                               void* workspace, size_t workspace_bytes, void* stream);

/* ---- Decode over the grouped-head cache ------------------------------------
 *   out[b,t,h,:] = sum_j p_j V[b, h', j, :],  p = softmax_j(scale q[b,t,h] . K[b, h', j]),
 *   j <= L_b - Lq + t,  h' = h / (Hq / Hk)
 * q, out [B, Lq, Hq, d]. A query that sees no key (L_b = 0: an idle slot; or
 * t < Lq - L_b) gives zeros. Lq Hq / Hk <= 64 (else MLA_ERR_UNSUPPORTED: use
 * the prefill). A length out of range counts as 0 and is recorded. */
typedef struct mla_gqa_decode_plan* mla_gqa_decode_plan_t;

/* seq_lens_host gives the lengths that the plan balances for and chooses the
 * kernel's layout by; the device lengths of a run may differ (results then
 * agree within rounding with those of a plan for them). opts (may be NULL):
 * num_sms and num_workers. */
mla_status_t mla_gqa_decode_plan(const mla_gqa_dims_t* dims, int32_t batch, const int32_t* seq_lens_host,
                                 const mla_plan_options_t* opts, mla_gqa_decode_plan_t* plan_out,
                                 size_t* workspace_bytes);

mla_status_t mla_gqa_decode_run(mla_gqa_decode_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                                int64_t num_blocks, const int32_t* block_table, int32_t block_table_stride,
                                const int32_t* seq_lens_dev, void* out, void* workspace, size_t workspace_bytes,
                                void* stream);

void mla_gqa_decode_plan_destroy(mla_gqa_decode_plan_t plan);

/* Self-test of the timeout path (diagnostics, as mla_decode_selftest_timeout): a
 * run whose ring slots are never given back, with every wait bounded by
 * wait_limit_ns (1000 to 2e9). Where a worker has more pages than its ring holds
 * (3 at d = 128, 6 at d = 64) the waits run out: the kernel returns,
 * MLA_ERR_DEVICE_TIMEOUT is recorded and `out` is not defined. The plan and the
 * workspace stay usable. */
mla_status_t mla_gqa_decode_selftest_timeout(mla_gqa_decode_plan_t plan, const void* q, const void* k_pool,
                                             const void* v_pool, int64_t num_blocks, const int32_t* block_table,
                                             int32_t block_table_stride, const int32_t* seq_lens_dev, void* out,
                                             void* workspace, size_t workspace_bytes, uint64_t wait_limit_ns,
                                             void* stream);

/* ---- Prefill over the grouped-head cache -----------------------------------
 * Causal attention of the n_b new tokens of each sequence over all its L_b
 * tokens, whose keys and values are in the cache already (appended before this
 * call on the same stream, earlier chunks of the prompt among them):
 *   out[t,h,:] = softmax_{j <= L_b - n_b + i}(scale q[t,h] . K[b, h', j]) V[b, h', :],  t = cu[b] + i
 * q, out [T, Hq, d] packed, T = the sum of the plan's counts. A query that sees
 * no key gives zeros; a length out of range counts as 0 and is recorded. n_b may
 * be 0. Hq / Hk <= 128 (else MLA_ERR_UNSUPPORTED). The device's cu_seqlens
 * must keep every n_b within the largest count of the plan and cu[B] <= T. */
typedef struct mla_gqa_prefill_plan* mla_gqa_prefill_plan_t;

mla_status_t mla_gqa_prefill_plan(const mla_gqa_dims_t* dims, int32_t batch, const int32_t* new_tokens_host,
                                  mla_gqa_prefill_plan_t* plan_out, size_t* workspace_bytes);

mla_status_t mla_gqa_prefill_run(mla_gqa_prefill_plan_t plan, const void* q, const void* k_pool, const void* v_pool,
                                 int64_t num_blocks, const int32_t* block_table, int32_t block_table_stride,
                                 const int32_t* cu_seqlens_dev, const int32_t* seq_lens_dev, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream);

void mla_gqa_prefill_plan_destroy(mla_gqa_prefill_plan_t plan);

/* Self-test of the timeout path: as mla_gqa_decode_selftest_timeout, with the
 * softmax weights of a step never handed over to the second product. */
mla_status_t mla_gqa_prefill_selftest_timeout(mla_gqa_prefill_plan_t plan, const void* q, const void* k_pool,
                                              const void* v_pool, int64_t num_blocks, const int32_t* block_table,
                                              int32_t block_table_stride, const int32_t* cu_seqlens_dev,
                                              const int32_t* seq_lens_dev, void* out, void* workspace,
                                              size_t workspace_bytes, uint64_t wait_limit_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PAGED_H */
