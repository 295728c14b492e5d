/*
 * exact_topk_cache.h -- C ABI of the operators around the exact Top-K in a
 * sparse-attention step: a paged key/value cache held in 8 bits, the page
 * scores that the selection reads, and the attention over the pages that it
 * selected (or over the whole cache).
 *
 *   exact_topk_cache_write     new keys and values -> codes, scales, key bounds
 *   exact_topk_cache_read      codes and scales -> rows of the cache's type
 *   exact_topk_block_scores    queries x key bounds -> score rows and lengths,
 *                              in the layout exact_topk reads
 *   exact_topk_attention_run   queries x cache (all pages, or the pages listed
 *                              for each token and key head) -> outputs
 *
 * The same four over a cache held in 4 bits (exact_topk_cache4_*), and what comes
 * before them in a step:
 *
 *   exact_topk_update_tables   sequences grow and shrink: lengths, row ranges,
 *                              pages from a ring of free ones and back to it
 *   exact_topk_rotary          queries and keys turned by their positions
 *
 * Conventions are those of exact_topk.h: every entry point returns 0 or a
 * negative exact_topk_status and launches nothing on error, allocates nothing,
 * never synchronizes, enqueues on the given stream only and can be captured in
 * a CUDA graph (after one call outside a capture on each device). Pointers
 * named "device" are memory of the current device. No exception leaves an
 * entry point.
 *
 * Device-side inputs are clamped or ignored, never trusted: a length outside
 * [0, table_width * page_size] is clamped, a row range outside [0, num_tokens]
 * is clamped, a page id outside [0, num_pages) is an absent page (nothing is
 * written to it, it reads as zeros, scores as -inf and is not attended to).
 */
#ifndef EXACT_TOPK_CACHE_H_
#define EXACT_TOPK_CACHE_H_

#include "exact_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define EXACT_TOPK_TYPE_BF16 0
#define EXACT_TOPK_TYPE_FP16 1

/* Limits checked on the host (EXACT_TOPK_ERR_BAD_BATCH beyond them). */
#define EXACT_TOPK_MAX_SEQS 4096
#define EXACT_TOPK_MAX_LISTED_WIDTH 65536 /* table_width of a call with a page list */

/* Exponents that a written scale may have: scale = 2^e, e in [MIN, MAX]. */
#define EXACT_TOPK_SCALE_MIN_EXP (-40)
#define EXACT_TOPK_SCALE_MAX_EXP 40

/* A paged cache. A page holds page_size consecutive tokens of one sequence.
 * For each page and key head: the tokens' codes, one scale for the keys and one
 * for the values (a stored number is code * scale), and the largest and the
 * smallest key of each channel.
 *   k, v        device e4m3 codes [num_pages][kv_heads][page_size][head_dim], 16-byte aligned
 *   k_scale, v_scale  device float32 [num_pages][kv_heads]; positive, between
 *               2^EXACT_TOPK_SCALE_MIN_EXP and 2^EXACT_TOPK_SCALE_MAX_EXP
 *   key_bounds  device `type` [num_pages][kv_heads][2][head_dim]: largest, then
 *               smallest; 16-byte aligned. May be NULL where no bounds are kept:
 *               exact_topk_block_scores then refuses the cache.
 *   page_size   16, 32, 64 or 128;  head_dim 64 or 128;  num_pages * kv_heads below 2^31
 *   type        EXACT_TOPK_TYPE_BF16 or _FP16: of the bounds and of every row array */
typedef struct exact_topk_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  void* key_bounds;
  int32_t num_pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t type;
  int32_t reserved;
} exact_topk_cache;

/* The sequences of a call. Sequence b has kv_len[b] tokens, the call's own rows
 * among them: its rows q_start[b] .. q_start[b+1]-1 are its LAST tokens, row i of
 * n at position kv_len[b] - n + i (a row whose position is negative has no token).
 * Rows at and beyond q_start[num_seqs] belong to no sequence: nothing of them is
 * read, and nothing written for them.
 *   page_table  device int32 [num_seqs][table_pitch]: page of tokens
 *               [j * page_size, (j+1) * page_size) of the sequence at j < table_width
 *   kv_len      device int32 [num_seqs]
 *   q_start     device int32 [num_seqs + 1], ascending; NULL: one row for each
 *               sequence, row b of sequence b (num_tokens must equal num_seqs) */
typedef struct exact_topk_batch {
  const int32_t* page_table;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t num_seqs;
  int32_t table_width;
  int64_t table_pitch;
} exact_topk_batch;

/* Rows [num_tokens][heads][head_dim] of the cache's type, channels contiguous;
 * strides in elements, multiples of 8; data 16-byte aligned (device). */
typedef struct exact_topk_rows {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} exact_topk_rows;

/* Quantises the call's key and value rows into the pages of their positions.
 * A page's scale is 2^e with the smallest e in [MIN, MAX] that brings its largest
 * finite magnitude within 448 (e4m3's largest); larger numbers saturate. A page
 * first written at offset 0 starts anew, whatever it held. One that is continued
 * (first written at offset o > 0) keeps the larger of its scale and the one the
 * new rows need; where that is larger, its codes [0, o) are brought to it. Codes
 * at offsets behind the last written one are left as they were. Codes are
 * rounded to nearest even (where a kept scale is no power of two, of the row times
 * the scale's rounded reciprocal); infinities and NaN become NaN. The bounds
 * are exact: the extremes of the rows as given, NaN taken as 0 and infinities
 * as the type's largest number. No page may be written by two sequences of a
 * call (its contents are undefined then; nothing else is touched).
 * Errors: NULL_POINTER, BAD_CACHE, BAD_BATCH, MISALIGNED, CUDA. */
int exact_topk_cache_write(const exact_topk_cache* cache, const exact_topk_batch* batch,
                           int64_t num_tokens, const exact_topk_rows* k, const exact_topk_rows* v,
                           struct CUstream_st* stream);

/* Writes code * scale, rounded to the cache's type, of the call's tokens (each
 * sequence's last n) into rows. Rows without a token or with an absent page get zeros.
 * Errors: as exact_topk_cache_write. */
int exact_topk_cache_read(const exact_topk_cache* cache, const exact_topk_batch* batch,
                          int64_t num_tokens, const exact_topk_rows* k, const exact_topk_rows* v,
                          struct CUstream_st* stream);

/* Page scores: row r = token * kv_heads + head of `scores` gets, for each page j
 * that the token sees (j * page_size <= position),
 *   max over the q_heads / kv_heads query heads g of the key head of
 *   sum_d max(q[g][d] * hi[j][d], q[g][d] * lo[j][d]),
 * the upper bound of q . k over the page's keys as they were written, in FP32 (products
 * exact); a stored key is off by e4m3's rounding, 2^-4 of itself, and may lie beyond them. Its
 * first keep_first pages and its newest keep_last ones get +inf instead, so that a
 * selection of at least as many always takes them.
 *   scores      device float32 [num_tokens * kv_heads][row_pitch], row_pitch >= table_width;
 *               entries at and beyond a row's length are left as they were
 *   ke          device int32 [num_tokens * kv_heads]: pages seen, 0 for a row without a token
 *   num_valid_rows  NULL, or device int32 [1]: gets q_start[num_seqs] * kv_heads,
 *               the live-row count exact_topk takes
 * Errors: NULL_POINTER, BAD_CACHE, BAD_BATCH, BAD_HEADS, BAD_SHAPE, MISALIGNED, CUDA. */
int exact_topk_block_scores(const exact_topk_cache* cache, const exact_topk_batch* batch,
                            int64_t num_tokens, int q_heads, const exact_topk_rows* q,
                            int keep_first, int keep_last, float* scores, int64_t row_pitch,
                            int32_t* ke, int32_t* num_valid_rows, struct CUstream_st* stream);

/* Launch plan of the attention, fixed before a capture; lengths and row ranges
 * stay device inputs. */
typedef struct exact_topk_attention_plan {
  int64_t num_tokens;
  int32_t num_seqs;
  int32_t q_heads;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t table_width;
  int32_t num_blocks;   /* list slots of each row; 0: the whole cache */
  int32_t columns;      /* query columns (tokens x heads) of a tile: 8, 16 or 32 */
  int32_t tile_tokens;  /* tokens of a tile, at most 8 */
  int32_t tile_heads;   /* heads of a tile (of one key head) */
  int32_t workers;      /* CTAs that share the work */
  int32_t min_units;    /* least pages a CTA takes at a time */
  int32_t prompt_tokens; /* tokens and heads of the tiles of the prompt's kernel, which */
  int32_t prompt_heads;  /* runs first where there are enough rows; 0: it does not run */
  uint64_t counter_bytes;
  uint64_t workspace_bytes;
} exact_topk_attention_plan;

/* Pure host logic. single_rows: nonzero for batches without q_start. prompt: whether the
 * prompt's kernel runs, -1 the planner's choice, 0 no, 1 yes (BAD_PLAN where it cannot: lists
 * over a table of more than 24576 pages).
 * num_tokens * q_heads must stay below 2^31.
 * Errors: NULL_POINTER, BAD_CACHE (page_size, head_dim), BAD_BATCH, BAD_HEADS, BAD_K, BAD_PLAN. */
int exact_topk_make_attention_plan(int64_t num_tokens, int num_seqs, int single_rows, int q_heads,
                                   int kv_heads, int head_dim, int page_size, int table_width,
                                   int num_blocks, int prompt,
                                   const exact_topk_device_info* info,
                                   exact_topk_attention_plan* plan);

/* out[t][head] = sum_p softmax_p(scale * q[t][head] . k[p]) v[p] over the tokens p at
 * positions up to t's own: all of them, or those of the pages listed for the row.
 * A row that sees nothing gets zeros, another one with an infinity or a NaN in its query
 * NaN. Scores, sums and outputs are FP32, rounded once to the cache's type; the
 * probabilities enter the second product in FP16, off by 2^-11 of themselves and, below
 * 2^-20 of the row's largest, by at most 2^-31 of that.
 *   q, out      [num_tokens][q_heads][head_dim]; they must not overlap
 *   scale       finite, as is scale * log2(e) (else BAD_PLAN); the scores of finite queries must be
 *               finite in FP32
 *   blocks      NULL when plan->num_blocks is 0, else device int32
 *               [num_tokens * kv_heads][num_blocks]: pages by their place in the
 *               sequence, as exact_topk selects them. A list is a set: order does not
 *               matter, an entry given twice counts once, one outside the pages
 *               that the token sees (-1 among them) is ignored.
 *   counters    device, >= counter_bytes, 16-byte aligned, all-zero on entry and on return
 *   workspace   device, >= workspace_bytes, 16-byte aligned, contents ignored
 * Results do not depend on the order in which CTAs run. Calls that share counters
 * or workspace must not overlap on the GPU: captured graphs that may run at the same
 * time each take their own.
 * Errors: any exact_topk_status. */
int exact_topk_attention_run(const exact_topk_attention_plan* plan, const exact_topk_cache* cache,
                             const exact_topk_batch* batch, const exact_topk_rows* q,
                             const exact_topk_rows* out, const int32_t* blocks, float scale,
                             void* counters, size_t counter_bytes, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream);

/* A paged cache in 4 bits. 16 neighbouring channels of one token and head share a
 * scale: a stored number is code * scale * unit, exact in FP16 but for the unit (code *
 * scale has at most 6 significant bits and lies between 2^-10 and 2688).
 *   k, v        device e2m1 codes [num_pages][kv_heads][page_size][head_dim / 2], two a byte,
 *               the channel of even number in the lower four bits; 16-byte aligned
 *   k_scale, v_scale  device e4m3 scales [num_pages][kv_heads][page_size][head_dim / 16], not
 *               negative; 16-byte aligned
 *   key_bounds  as of exact_topk_cache
 *   k_unit, v_unit  powers of two between 2^EXACT_TOPK_SCALE_MIN_EXP and
 *               2^EXACT_TOPK_SCALE_MAX_EXP. Groups whose largest magnitude lies between 0.1 and
 *               2688 units keep the codes' precision; smaller ones lose it, larger ones saturate.
 *   the rest as of exact_topk_cache */
typedef struct exact_topk_cache4 {
  void* k;
  void* v;
  void* k_scale;
  void* v_scale;
  void* key_bounds;
  int32_t num_pages;
  int32_t kv_heads;
  int32_t page_size;
  int32_t head_dim;
  int32_t type;
  float k_unit;
  float v_unit;
} exact_topk_cache4;

/* As exact_topk_cache_write. Each group of 16 channels is quantised by itself: its scale
 * is the e4m3 number nearest to max |x| / (6 unit), at least 2^-9 and at most 448, its codes
 * the e2m1 numbers nearest to x / (scale * unit), both to nearest even, saturating. A group
 * with an infinity or a NaN gets the scale NaN: all 16 numbers are NaN. Nothing of earlier tokens
 * changes but their page's bounds. Errors: as exact_topk_cache_write. */
int exact_topk_cache4_write(const exact_topk_cache4* cache, const exact_topk_batch* batch,
                            int64_t num_tokens, const exact_topk_rows* k,
                            const exact_topk_rows* v, struct CUstream_st* stream);

/* As exact_topk_cache_read: code * scale * unit, rounded to the cache's type. */
int exact_topk_cache4_read(const exact_topk_cache4* cache, const exact_topk_batch* batch,
                           int64_t num_tokens, const exact_topk_rows* k, const exact_topk_rows* v,
                           struct CUstream_st* stream);

/* As exact_topk_block_scores. A stored key is off by up to 0.18 of its group's largest magnitude
 * (by more where that is below 0.1 units or beyond 2688), and may lie beyond the bounds, which are
 * of the keys as they were written. */
int exact_topk_cache4_block_scores(const exact_topk_cache4* cache, const exact_topk_batch* batch,
                                   int64_t num_tokens, int q_heads, const exact_topk_rows* q,
                                   int keep_first, int keep_last, float* scores,
                                   int64_t row_pitch, int32_t* ke, int32_t* num_valid_rows,
                                   struct CUstream_st* stream);

/* As exact_topk_make_attention_plan, for exact_topk_cache4_attention_run: the prompt's kernel runs from
 * more rows on. */
int exact_topk_cache4_make_attention_plan(int64_t num_tokens, int num_seqs, int single_rows,
                                          int q_heads, int kv_heads, int head_dim, int page_size,
                                          int table_width, int num_blocks, int prompt,
                                          const exact_topk_device_info* info,
                                          exact_topk_attention_plan* plan);

/* As exact_topk_attention_run; either function's plans will do. scale * k_unit must be finite as
 * scale must. */
int exact_topk_cache4_attention_run(const exact_topk_attention_plan* plan,
                                    const exact_topk_cache4* cache, const exact_topk_batch* batch,
                                    const exact_topk_rows* q, const exact_topk_rows* out,
                                    const int32_t* blocks, float scale, void* counters,
                                    size_t counter_bytes, void* workspace, size_t workspace_bytes,
                                    struct CUstream_st* stream);

#define EXACT_TOPK_MAX_ROTARY_DIM 512

/* Rotary positions. Of each head's head_dim channels the first rotary_dim turn, in pairs
 * (i, i + rotary_dim / 2), or (2 i, 2 i + 1) where neighbours is nonzero; pair i at position
 * p by p * turns[i] / 2^64 turns, modulo one (exact for every position), times amplitude.
 *   turns       device [rotary_dim / 2]
 *   head_dim    a multiple of 8 up to 1024;  rotary_dim even, 2 to head_dim and at most 512
 *   type        of all rows
 *   page_size   16, 32, 64 or 128: of the batch's tables, to whose table_width * page_size tokens lengths
 *               are clamped then, as by the cache's operators; 0: there is no table, lengths are taken
 *               as they are, up to 2^30 */
typedef struct exact_topk_rotary_spec {
  const uint64_t* turns;
  float amplitude;
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t neighbours;
  int32_t type;
  int32_t page_size;
} exact_topk_rotary_spec;

/* Turns q [num_tokens][q_heads][head_dim] into q_out and k [num_tokens][k_heads][head_dim] into
 * k_out; cosines, sines and sums are FP32, rounded once. Each may be its own output (the same data
 * and strides), in no other way may they overlap. k_heads may be 0 (k and k_out are ignored).
 *   batch       the rows' positions are those of their tokens (the page table's entries are not looked
 *               at); rows of no sequence or without a token are left as they were
 *   positions   device int32 [num_tokens] instead of the batch (one of the two is NULL): any
 *               numbers, negative ones turn back
 *   inverse     nonzero: by the negative angles, with the same amplitude. That is the gradient of q and
 *               k by what comes back for q_out and k_out; it undoes the call where the amplitude is 1.
 * Errors: NULL_POINTER, BAD_BATCH, BAD_HEADS, BAD_SHAPE (the spec, the amplitude not finite),
 * MISALIGNED, CUDA. */
int exact_topk_rotary(const exact_topk_rotary_spec* spec, const exact_topk_batch* batch,
                      const int32_t* positions, int64_t num_tokens, int q_heads,
                      const exact_topk_rows* q, const exact_topk_rows* q_out, int k_heads,
                      const exact_topk_rows* k, const exact_topk_rows* k_out, int inverse,
                      struct CUstream_st* stream);

/* Sequences on the GPU: their page tables, lengths and row ranges (an exact_topk_batch is made
 * of them), and the pages that no sequence has.
 *   page_table  device int32 [num_seqs][table_pitch]; entries behind a sequence's pages are not looked at
 *   kv_len      device int32 [num_seqs]
 *   q_start     device int32 [num_seqs + 1], written
 *   applied     device int32 [num_seqs], written; may be NULL
 *   slots, positions  device int32 [max_tokens], written; may be NULL
 *   free_pages  device int32 [num_pages], a ring of page ids
 *   free_range  device int32 [2]: the first free page's place in the ring, and how many there are
 *   counters    device, 4 bytes or more, 4-byte aligned, all-zero on entry and on return
 * num_pages * page_size must be below 2^31. A page's id stands once: in the ring or in a table. */
typedef struct exact_topk_page_tables {
  int32_t* page_table;
  int32_t* kv_len;
  int32_t* q_start;
  int32_t* applied;
  int32_t* slots;
  int32_t* positions;
  int32_t* free_pages;
  int32_t* free_range;
  void* counters;
  size_t counter_bytes;
  int64_t table_pitch;
  int64_t max_tokens;
  int32_t num_seqs;
  int32_t table_width;
  int32_t num_pages;
  int32_t page_size;
} exact_topk_page_tables;

/* Sequence b grows by change[b] tokens (negative: loses its last -change[b], all it has where it
 * has fewer; with negate nonzero by -change[b]). Pages that are no longer reached go to the end of
 * the ring, in the sequences' order and each sequence's in ascending place; pages for new tokens
 * are taken from the front, in the same order, those given back in this call last. A sequence
 * gets all its tokens or none:
 * none where they do not fit its table, where it needs pages and they and those asked for
 * by the sequences before it are more than there are, or where its tokens and those asked for
 * before it are more than max_tokens. (What a refused sequence asked for counts for those
 * behind it; one that does not fit its table asks for nothing.)
 *   kv_len, free_pages, free_range, and the tables' new entries: as they are after the call
 *   q_start     ranges of the new tokens' rows, in the sequences' order
 *   applied     the change that was made, 0 for a refused sequence; may be `change` itself
 *   slots, positions  of each new row: page * page_size + offset, and its place in the
 *               sequence; rows behind the last are left as they were
 * change is device int32 [num_seqs]. Results do not depend on the order in which CTAs run. Calls on
 * the same tables or counters must not overlap on the GPU.
 * Errors: NULL_POINTER, BAD_CACHE (pages), BAD_BATCH, COUNTERS_TOO_SMALL, MISALIGNED, CUDA. */
int exact_topk_update_tables(const exact_topk_page_tables* tables, const int32_t* change,
                             int negate, struct CUstream_st* stream);

/* How many times the issuing threads of the prompts' kernels (page scores and attention) poll for
 * their operands before they give up, for the calls that this process makes from now on: at most
 * 2^20, which a negative number brings back. What a CTA has not computed then is computed again
 * without waits. With 0 they always give up, which is how that is tested.
 * Errors: BAD_SHAPE (more than 2^20). */
int exact_topk_set_wait_limit(int64_t polls);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_TOPK_CACHE_H_ */
