/*
 * mixattn_latent.h -- attention over one shared latent vector a token, for GB300 (sm_103a).
 *
 * A model of this kind caches, per token and for all heads together, a latent vector c
 * (512 elements) and one position key r (64 elements, rotated by the token's position).  Head h's
 * keys and values are linear in c, so attention has two forms:
 *
 *   absorbed   the key projection is taken into the query and the value projection into what
 *              follows: every head's query [512 + 64] meets the cached rows [c | r] themselves,
 *              and the output is a weighted mean of the c.  Reads 1152 bytes a token whatever
 *              the number of heads: for decode rows and for the few tokens of a verify pass.
 *   expanded   the caller makes per-head keys [128] and values [128] of the latent vectors; a
 *              query [128 + 64] meets [key | r].  3.4 times fewer products a pair: for prompts.
 *
 * Conventions (streams, ownership, status codes, device checks, captured graphs) are those of
 * mixattn.h, whose device error word these calls share.  Outputs are rounded to the nearest fp16,
 * saturating at +-65504.  Scores, sums and softmax statistics are fp32, whatever the scores' size; the
 * softmax weights that meet the values are rounded to fp16, 2^-11 of each (those below 2^-20 of their
 * row's largest, 2^-31 of that).  A query with a NaN answers NaN.
 */
#ifndef MIXATTN_LATENT_H
#define MIXATTN_LATENT_H

#include "mixattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The paged latent cache: fp16 [num_pages][page_size][latent_dim + rope_dim], one row a token,
 * the latent vector first.  Plain data; the caller owns `data` (256-byte aligned).
 */
typedef struct {
  int32_t num_pages;  /* > 0, num_pages * page_size <= INT32_MAX */
  int32_t page_size;  /* must be 32  */
  int32_t latent_dim; /* must be 512 */
  int32_t rope_dim;   /* must be 64  */
  void* data;         /* device      */
} mixattn_latent_cache;

/* Bytes of a cache with these dimensions (`data` ignored), or 0 if they are not valid. */
size_t mixattn_latent_cache_bytes(const mixattn_latent_cache* cache);

/* fp16 vectors in device memory: token t's head h at x + t * token_stride + h * head_stride (elements),
 * each contiguous.  16-byte aligned, strides multiples of 8.  The heads of a token do not overlap
 * one another, nor a token's the next one's (token_stride >= heads * head_stride >= 0, or the
 * other way round, heads outermost). */
typedef struct {
  const void* x;
  int64_t token_stride;
  int64_t head_stride;
} mixattn_heads;

/*
 * A step's new tokens into the cache, in one launch: the latent vectors as they are, the position
 * keys rotated by their positions, and the position parts of the queries rotated into q_out.
 *   rope         a table with rot_dim 64
 *   num_heads    query heads, <= 65536; 0 (q and q_out then ignored) appends only
 *   q, q_out     64 elements a head, for instance the ends of the heads of a query projection and
 *                of the absorbed queries [n][heads][576]; q_out may be q itself (same strides) and
 *                must not overlap it otherwise (from its first element to its last), nor c_new or k_rope
 *   c_new        fp16 [n_new], 512 elements every c_stride;  k_rope  64 elements every k_stride
 *                (16-byte aligned, strides multiples of 8 and >= 512 and 64)
 *   positions, slot_mapping   device int32 [n_new]; slots as for mixattn_kv_append_quant (a skipped
 *                token's queries are still rotated).  Two tokens of one slot race.
 * Latent elements that are not finite stay what they are.  Both elements of a rotated pair are sums of products of
 * both: one that is not finite makes them NaN or (an infinity) +-65504, and touches no other pair.
 */
int mixattn_latent_append(const mixattn_latent_cache* cache, const mixattn_rope* rope, int32_t num_heads,
                          const mixattn_heads* q, const mixattn_heads* q_out, const void* c_new, int64_t c_stride,
                          const void* k_rope, int64_t k_stride, const int32_t* positions, const int32_t* slot_mapping,
                          int32_t n_new, mixattn_stream stream);

/* Rows of the cache, gathered: out fp16 [n][576] (16-byte aligned) of device int32 slots [n]; a
 * slot outside the cache sets MIXATTN_DEVERR_SLOT and its row is left as it was.  For the expanded
 * form of a chunk whose history is in the cache, and for persistence. */
int mixattn_latent_export(const mixattn_latent_cache* cache, const int32_t* slots, int32_t n, void* out,
                          mixattn_stream stream);

/*
 * Absorbed attention: a plan as mixattn_plan (the host-side tiling of one batch, reused for every
 * layer), its rows packed in order, of any mixattn_row_kind:
 *   o[t][h] = sum_j softmax_j(softmax_scale q[t][h] . [c_j | r_j]) c_j
 * over the keys that the query sees.  The cache's rows are read once for up to 64 (query, head)
 * pairs of a row.  Work is cut over the SMs for the whole batch (a row's cuts, and so the last
 * bits of its output, depend on the batch it runs in; the same plan gives the same bits every time).
 *   num_heads      1 .. 128
 *   softmax_scale  1e-20 .. 1e6 (usually 1 / sqrt(128 + 64), times the squared rotary multiplier)
 */
typedef struct mixattn_latent_plan mixattn_latent_plan;

int mixattn_latent_plan_create(mixattn_latent_plan** plan_out, const mixattn_latent_cache* cache, int32_t num_heads,
                               double softmax_scale, int32_t n_rows, const int32_t* row_kinds, const int32_t* seq_lens,
                               const int32_t* q_offsets, int32_t max_pages, size_t* workspace_bytes);

/* As mixattn_plan_update. */
int mixattn_latent_plan_update(mixattn_latent_plan* plan, int32_t n_rows, const int32_t* row_kinds,
                               const int32_t* seq_lens, const int32_t* q_offsets, int32_t max_pages,
                               size_t* workspace_bytes);

/*
 *   q           device fp16 [total_q][num_heads][576], 16-byte aligned
 *   page_table  device int32 [n_rows][max_pages]
 *   tree_mask, mask_words   as for mixattn_run_tree; NULL and 0 for a plan without tree rows
 *   o           device fp16 [total_q][num_heads][512], 16-byte aligned
 *   workspace   device, >= workspace_bytes, 256-byte aligned, contents of no account
 * A page id outside the cache sets MIXATTN_DEVERR_PAGE_ID and its keys are left out; a query that
 * sees no key gets zeros.  Keys that no query of a row sees (unused nodes of a tree) need not have
 * been appended; one that some see and that is not finite may reach the row's other outputs.  May be
 * captured into a graph, with mixattn_run's conditions.
 */
int mixattn_latent_run(const mixattn_latent_plan* plan, const void* q, const int32_t* page_table,
                       const uint32_t* tree_mask, int32_t mask_words, void* o, void* workspace,
                       size_t workspace_bytes, mixattn_stream stream);

void mixattn_latent_plan_destroy(mixattn_latent_plan* plan);

/*
 * Expanded attention of prompts and chunks.  Row r's keys are tokens 0 .. seq_len - 1 of its own
 * sequence, packed in row order (those of row r start at the sum of the seq_lens before it); its
 * queries are the last seq_len - q_offset of them, packed likewise, and see keys up to their own.
 *   o[t][h] = sum_j softmax_j(softmax_scale (q[t][h][:128] . k[j][h] + q[t][h][128:] . r[j])) v[j][h]
 * A value that is not finite may reach the outputs of its row's earlier queries too, which do not see it
 * (a weight of 0 times it); those of other rows it does not reach.
 *   num_heads      1 .. 65536
 * Work is cut over the SMs for the whole batch, as that of an absorbed plan.
 */
typedef struct mixattn_expanded_plan mixattn_expanded_plan;

int mixattn_expanded_plan_create(mixattn_expanded_plan** plan_out, int32_t num_heads, double softmax_scale,
                                 int32_t n_rows, const int32_t* seq_lens, const int32_t* q_offsets,
                                 size_t* workspace_bytes);

int mixattn_expanded_plan_update(mixattn_expanded_plan* plan, int32_t n_rows, const int32_t* seq_lens,
                                 const int32_t* q_offsets, size_t* workspace_bytes);

/*
 *   q       192 elements a head, the position part last;  k, v  128 elements a head (for instance
 *           the two halves of one projection's heads);  strides as mixattn_heads says, at least
 *           that many elements, < 2^31 and, of tokens and heads, both > 0
 *   k_rope  device fp16, 64 elements every k_rope_stride (>= 64, a multiple of 8, < 2^31)
 *   o       device fp16 [total_q][num_heads][128], 16-byte aligned
 */
int mixattn_expanded_run(const mixattn_expanded_plan* plan, const mixattn_heads* q, const mixattn_heads* k,
                         const void* k_rope, int64_t k_rope_stride, const mixattn_heads* v, void* o, void* workspace,
                         size_t workspace_bytes, mixattn_stream stream);

void mixattn_expanded_plan_destroy(mixattn_expanded_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* MIXATTN_LATENT_H */
