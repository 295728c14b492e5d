// Host side of the cache operators declared in include/exact_topk_cache.h:
// argument checks and the attention's launch plan.  Nothing here synchronizes,
// allocates or reads device memory.

#include <atomic>
#include <cmath>
#include <cstdint>

#include "cache_internal.h"

namespace etk {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

int check_cache(const exact_topk_cache* cache, CacheArgs* out) {
  if (cache == nullptr || cache->k == nullptr || cache->v == nullptr ||
      cache->k_scale == nullptr || cache->v_scale == nullptr)
    return EXACT_TOPK_ERR_NULL_POINTER;
  if (cache->num_pages < 1 || cache->kv_heads < 1 || cache->kv_heads > 1024 ||
      (int64_t)cache->num_pages * cache->kv_heads > 0x7FFFFFFF ||
      !page_size_ok(cache->page_size) || (cache->head_dim != 64 && cache->head_dim != 128) ||
      (cache->type != EXACT_TOPK_TYPE_BF16 && cache->type != EXACT_TOPK_TYPE_FP16))
    return EXACT_TOPK_ERR_BAD_CACHE;
  if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(cache->key_bounds, 16) ||
      !aligned(cache->k_scale, 4) || !aligned(cache->v_scale, 4))
    return EXACT_TOPK_ERR_MISALIGNED;
  out->k = static_cast<uint8_t*>(cache->k);
  out->v = static_cast<uint8_t*>(cache->v);
  out->k_scale = cache->k_scale;
  out->v_scale = cache->v_scale;
  out->bounds = cache->key_bounds;
  out->num_pages = cache->num_pages;
  out->heads = cache->kv_heads;
  out->page = cache->page_size;
  out->page_shift = 4;
  while ((1 << out->page_shift) < cache->page_size) ++out->page_shift;
  out->dim = cache->head_dim;
  out->fp16 = cache->type == EXACT_TOPK_TYPE_FP16;
  return EXACT_TOPK_OK;
}

int check_batch_shape(int64_t num_tokens, int num_seqs, int single_rows, int width, int page) {
  if (num_seqs < 1 || num_seqs > EXACT_TOPK_MAX_SEQS || num_tokens < 0 ||
      num_tokens > ((int64_t)1 << 24) || (single_rows && num_tokens != num_seqs) || width < 1 ||
      (int64_t)width * page > ((int64_t)1 << 30))
    return EXACT_TOPK_ERR_BAD_BATCH;
  return EXACT_TOPK_OK;
}

int check_batch(const exact_topk_batch* batch, int64_t num_tokens, int page, BatchArgs* out) {
  if (batch == nullptr || batch->page_table == nullptr || batch->kv_len == nullptr)
    return EXACT_TOPK_ERR_NULL_POINTER;
  const int rc = check_batch_shape(num_tokens, batch->num_seqs, batch->q_start == nullptr,
                                   batch->table_width, page);
  if (rc != EXACT_TOPK_OK) return rc;
  if (batch->table_pitch < batch->table_width) return EXACT_TOPK_ERR_BAD_BATCH;
  if (!aligned(batch->page_table, 4) || !aligned(batch->kv_len, 4) || !aligned(batch->q_start, 4))
    return EXACT_TOPK_ERR_MISALIGNED;
  out->table = batch->page_table;
  out->kv_len = batch->kv_len;
  out->q_start = batch->q_start;
  out->table_pitch = batch->table_pitch;
  out->num_tokens = num_tokens;
  out->num_seqs = batch->num_seqs;
  out->width = batch->table_width;
  return EXACT_TOPK_OK;
}

int check_rows(const exact_topk_rows* rows, int64_t num_tokens, RowArgs* out) {
  if (rows == nullptr || (rows->data == nullptr && num_tokens > 0))
    return EXACT_TOPK_ERR_NULL_POINTER;
  if (!aligned(rows->data, 16) || rows->token_stride % 8 != 0 || rows->head_stride % 8 != 0)
    return EXACT_TOPK_ERR_MISALIGNED;
  out->data = rows->data;
  out->token_stride = rows->token_stride;
  out->head_stride = rows->head_stride;
  return EXACT_TOPK_OK;
}

// CTAs of an attention launch: the join of a tile that all of them share holds a factor for each.
int most_workers(int columns, int dim) {
  return kMaxAttentionWorkers / 4 * attention_ctas_per_sm(columns, dim);
}

uint64_t partial_bytes(const exact_topk_attention_plan& p, int dim) {
  return (uint64_t)p.workers * 2 * partial_floats(p.columns, dim) * 4;
}

uint64_t again_bytes(const exact_topk_attention_plan& p, int group) {
  if (p.prompt_tokens == 0) return 0;
  return (uint64_t)p.num_tokens * p.kv_heads * ((group + p.prompt_heads - 1) / p.prompt_heads);
}

bool heads_ok(int q_heads, int kv_heads) {
  return q_heads >= 1 && q_heads <= 65536 && q_heads % kv_heads == 0;
}

// What the cache's writer and reader check alike.
int check_move(const exact_topk_cache* cache, const exact_topk_batch* batch, int64_t num_tokens,
               const exact_topk_rows* k, const exact_topk_rows* v, CacheArgs* c, BatchArgs* b,
               RowArgs* kr, RowArgs* vr) {
  int rc = check_cache(cache, c);
  if (rc == EXACT_TOPK_OK) rc = check_batch(batch, num_tokens, c->page, b);
  if (rc == EXACT_TOPK_OK) rc = check_rows(k, num_tokens, kr);
  if (rc == EXACT_TOPK_OK) rc = check_rows(v, num_tokens, vr);
  return rc;
}

std::atomic<uint32_t> g_wait_limit{kWaitLimit};

}  // namespace

uint32_t wait_limit() { return g_wait_limit.load(std::memory_order_relaxed); }

}  // namespace etk

using namespace etk;

extern "C" {

int exact_topk_cache_write(const exact_topk_cache* cache, const exact_topk_batch* batch,
                           int64_t num_tokens, const exact_topk_rows* k, const exact_topk_rows* v,
                           struct CUstream_st* stream) {
  CacheArgs c;
  BatchArgs b;
  RowArgs kr, vr;
  const int rc = check_move(cache, batch, num_tokens, k, v, &c, &b, &kr, &vr);
  if (rc != EXACT_TOPK_OK || num_tokens == 0) return rc;
  return launch_cache_write(c, b, kr, vr, reinterpret_cast<cudaStream_t>(stream));
}

int exact_topk_cache_read(const exact_topk_cache* cache, const exact_topk_batch* batch,
                          int64_t num_tokens, const exact_topk_rows* k, const exact_topk_rows* v,
                          struct CUstream_st* stream) {
  CacheArgs c;
  BatchArgs b;
  RowArgs kr, vr;
  const int rc = check_move(cache, batch, num_tokens, k, v, &c, &b, &kr, &vr);
  if (rc != EXACT_TOPK_OK || num_tokens == 0) return rc;
  return launch_cache_read(c, b, kr, vr, reinterpret_cast<cudaStream_t>(stream));
}

int exact_topk_block_scores(const exact_topk_cache* cache, const exact_topk_batch* batch,
                            int64_t num_tokens, int q_heads, const exact_topk_rows* q,
                            int keep_first, int keep_last, float* scores, int64_t row_pitch,
                            int32_t* ke, int32_t* num_valid_rows, struct CUstream_st* stream) {
  CacheArgs c;
  BatchArgs b;
  ScoreArgs a;
  int rc = check_cache(cache, &c);
  if (rc == EXACT_TOPK_OK) rc = check_batch(batch, num_tokens, c.page, &b);
  if (rc == EXACT_TOPK_OK) rc = check_rows(q, num_tokens, &a.q);
  if (rc != EXACT_TOPK_OK) return rc;
  if (c.bounds == nullptr || (num_tokens > 0 && (scores == nullptr || ke == nullptr)))
    return EXACT_TOPK_ERR_NULL_POINTER;
  if (!heads_ok(q_heads, c.heads)) return EXACT_TOPK_ERR_BAD_HEADS;
  if (row_pitch < b.width || keep_first < 0 || keep_last < 0 ||
      num_tokens * c.heads > 0x7FFFFFFF)
    return EXACT_TOPK_ERR_BAD_SHAPE;
  if (!aligned(scores, 4) || !aligned(ke, 4) || !aligned(num_valid_rows, 4))
    return EXACT_TOPK_ERR_MISALIGNED;
  a.scores = scores;
  a.ke = ke;
  a.num_valid_rows = num_valid_rows;
  a.row_pitch = row_pitch;
  a.group = q_heads / c.heads;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  if (num_tokens == 0) {  // no rows: only their count is asked for
    if (num_valid_rows != nullptr &&
        cudaMemsetAsync(num_valid_rows, 0, sizeof(int32_t),
                        reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return EXACT_TOPK_ERR_CUDA;
    return EXACT_TOPK_OK;
  }
  return launch_block_scores(c, b, a, reinterpret_cast<cudaStream_t>(stream));
}

int exact_topk_make_attention_plan(int64_t num_tokens, int num_seqs, int single_rows, int q_heads,
                                   int kv_heads, int head_dim, int page_size, int table_width,
                                   int num_blocks, int prompt,
                                   const exact_topk_device_info* info,
                                   exact_topk_attention_plan* plan) {
  if (info == nullptr || plan == nullptr) return EXACT_TOPK_ERR_NULL_POINTER;
  if (!page_size_ok(page_size) || (head_dim != 64 && head_dim != 128) || kv_heads < 1 ||
      kv_heads > 1024 || info->sm_count < 1)
    return EXACT_TOPK_ERR_BAD_CACHE;
  const int rc = check_batch_shape(num_tokens, num_seqs, single_rows, table_width, page_size);
  if (rc != EXACT_TOPK_OK) return rc;
  if (!heads_ok(q_heads, kv_heads) || num_tokens * q_heads > 0x7FFFFFFF)
    return EXACT_TOPK_ERR_BAD_HEADS;
  if (num_blocks < 0 || num_blocks > EXACT_TOPK_MAX_K) return EXACT_TOPK_ERR_BAD_K;
  if (num_blocks > 0 && table_width > EXACT_TOPK_MAX_LISTED_WIDTH) return EXACT_TOPK_ERR_BAD_BATCH;
  exact_topk_attention_plan p{};
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.head_dim = head_dim;
  p.page_size = page_size;
  p.table_width = table_width;
  p.num_blocks = num_blocks;
  // Columns of a tile: 8 as a rule, more only where a key head has more query heads. Wider
  // tiles share pages between tokens, but are fewer and their products and joins longer. Over
  // listed pages 8 columns were the fastest or within 4% of it from 1 to 256 tokens of a sequence
  // (8 tokens of 32 sequences x 16 heads over 32 pages: 50 us, 16 columns 58, 32 columns 56; 32
  // tokens of one: 17, 21 and 30; 256: 44, 53 and 49; 512: 84, 88 and 75). Over the whole cache
  // 16 columns win once passes of 8 would read 256 MB (65 MB: 20.5 us with 8, 23.3 with 16; 262 MB:
  // 43.7 and 44.4; 524 MB: 67.2 and 60.3; 2.1 GB: 230 and 161), and 32 lose to them (94 and 170).
  const int group = q_heads / kv_heads;
  const int64_t mean = single_rows ? 1 : (num_tokens + num_seqs - 1) / num_seqs;
  const int64_t passes = (mean * group + 7) / 8;
  const double read = (double)num_seqs * kv_heads * table_width * page_size * 2 * head_dim *
                      (double)passes;
  p.columns = group > 16 ? 32 : (group > 8 ? 16 : 8);
  if (group <= 8 && num_blocks == 0 && passes > 1 && read >= 256e6) p.columns = 16;
  p.tile_heads = group < p.columns ? group : p.columns;
  p.tile_tokens = p.columns / p.tile_heads < 8 ? p.columns / p.tile_heads : 8;
  if (single_rows) p.tile_tokens = 1;
  p.workers = info->sm_count * attention_ctas_per_sm(p.columns, head_dim);
  if (p.workers > most_workers(p.columns, head_dim)) p.workers = most_workers(p.columns, head_dim);
  // A CTA's four warps take 32 tokens each at a time; with 128 tokens a CTA its part of the join
  // outweighs its own work (four short sequences: 21.3 us, 17.0 with 256, 18.0 with 512).
  p.min_units = 256 / page_size;
  p.counter_bytes = ((uint64_t)p.workers * 4 + 15) / 16 * 16;
  // The prompt's kernel takes 128 rows (tokens x heads) at a time and does not split a tile: it
  // wants tiles that a sequence fills, and enough of them. Over the whole cache it wins from about
  // 5000 rows on (16 heads x 256 tokens over 8192: 132 us against 110, 512 tokens: 133 against
  // 203). Over listed pages it also depends on how many of them neighbours share: 16 heads x 512
  // tokens over 32 pages of 512 each take 54 us against 84 where most are shared, and 198 against
  // 84 where none are; 1024 tokens 55 against 138, 2048 tokens without any shared 248 against 288.
  const int prompt_heads = group < kPromptRows ? group : kPromptRows;
  const int prompt_tokens =
      kPromptRows / prompt_heads < kPromptTokens ? kPromptRows / prompt_heads : kPromptTokens;
  const int64_t prompt_rows = num_blocks > 0 ? 16384 : 5120;
  const bool prompt_fits = num_blocks == 0 || table_width <= kPromptListedWidth;
  if (prompt > 0 && !prompt_fits) return EXACT_TOPK_ERR_BAD_PLAN;
  if (prompt > 0 || (prompt < 0 && prompt_fits && !single_rows && mean >= prompt_tokens &&
                     num_tokens * q_heads >= prompt_rows)) {
    p.prompt_tokens = prompt_tokens;
    p.prompt_heads = prompt_heads;
  }
  p.workspace_bytes = partial_bytes(p, head_dim) + again_bytes(p, group);
  *plan = p;
  return EXACT_TOPK_OK;
}

int exact_topk_attention_run(const exact_topk_attention_plan* plan, const exact_topk_cache* cache,
                             const exact_topk_batch* batch, const exact_topk_rows* q,
                             const exact_topk_rows* out, const int32_t* blocks, float scale,
                             void* counters, size_t counter_bytes, void* workspace,
                             size_t workspace_bytes, struct CUstream_st* stream) {
  CacheArgs c;
  BatchArgs b;
  AttentionArgs a;
  if (plan == nullptr || counters == nullptr || workspace == nullptr)
    return EXACT_TOPK_ERR_NULL_POINTER;
  int rc = check_cache(cache, &c);
  if (rc == EXACT_TOPK_OK) rc = check_batch(batch, plan->num_tokens, c.page, &b);
  if (rc == EXACT_TOPK_OK) rc = check_rows(q, plan->num_tokens, &a.q);
  if (rc == EXACT_TOPK_OK) rc = check_rows(out, plan->num_tokens, &a.out);
  if (rc != EXACT_TOPK_OK) return rc;
  if (plan->num_blocks > 0 && blocks == nullptr) return EXACT_TOPK_ERR_NULL_POINTER;
  if (!heads_ok(plan->q_heads, c.heads) || plan->num_tokens * plan->q_heads > 0x7FFFFFFF)
    return EXACT_TOPK_ERR_BAD_HEADS;
  if (plan->num_blocks < 0 || plan->num_blocks > EXACT_TOPK_MAX_K) return EXACT_TOPK_ERR_BAD_K;
  const int group = plan->q_heads / c.heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  if (plan->kv_heads != c.heads || plan->head_dim != c.dim || plan->page_size != c.page ||
      plan->table_width != b.width || plan->num_seqs != b.num_seqs ||
      (plan->num_blocks == 0 && blocks != nullptr) ||
      (plan->num_blocks > 0 && b.width > EXACT_TOPK_MAX_LISTED_WIDTH) ||
      (plan->columns != 8 && plan->columns != 16 && plan->columns != 32) || plan->tile_heads < 1 ||
      plan->tile_heads > group || plan->tile_tokens < 1 || plan->tile_tokens > 8 ||
      plan->tile_tokens * plan->tile_heads > plan->columns || plan->workers < 1 ||
      plan->workers > most_workers(plan->columns, c.dim) || plan->min_units < 1 ||
      !std::isfinite(a.scale_log2) || plan->prompt_tokens < 0 ||
      plan->prompt_tokens > kPromptTokens)
    return EXACT_TOPK_ERR_BAD_PLAN;
  // A tile of the kernel that runs behind the prompt's lies within one of that one's.
  if (plan->prompt_tokens > 0 &&
      (plan->prompt_heads < 1 || plan->prompt_heads > group ||
       plan->prompt_tokens * plan->prompt_heads > kPromptRows ||
       (plan->prompt_heads != group && plan->prompt_heads % plan->tile_heads != 0) ||
       (plan->num_blocks > 0 && b.width > kPromptListedWidth)))
    return EXACT_TOPK_ERR_BAD_PLAN;
  if (counter_bytes < plan->counter_bytes || counter_bytes < (size_t)plan->workers * 4)
    return EXACT_TOPK_ERR_COUNTERS_TOO_SMALL;
  const uint64_t partial = partial_bytes(*plan, c.dim);
  if (workspace_bytes < plan->workspace_bytes ||
      workspace_bytes < partial + again_bytes(*plan, group))
    return EXACT_TOPK_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(counters, 16) || !aligned(workspace, 16) || !aligned(blocks, 4))
    return EXACT_TOPK_ERR_MISALIGNED;
  if (plan->num_tokens == 0) return EXACT_TOPK_OK;
  a.blocks = blocks;
  a.counters = static_cast<int32_t*>(counters);
  a.partial = static_cast<float*>(workspace);
  a.num_blocks = plan->num_blocks;
  a.group = group;
  a.columns = plan->columns;
  a.tile_tokens = plan->tile_tokens;
  a.tile_heads = plan->tile_heads;
  a.workers = plan->workers;
  a.min_units = plan->min_units;
  a.prompt_tokens = plan->prompt_tokens;
  a.prompt_heads = plan->prompt_heads;
  a.again = plan->prompt_tokens > 0 ? static_cast<uint8_t*>(workspace) + partial : nullptr;
  a.group_parts = (group + plan->tile_heads - 1) / plan->tile_heads;
  // a part of a listed tile: at least 128 tokens, 32 for each warp
  a.max_cut = plan->num_blocks * c.page / 128;
  if (a.max_cut < 1) a.max_cut = 1;
  return launch_attention(c, b, a, reinterpret_cast<cudaStream_t>(stream));
}

int exact_topk_set_wait_limit(int64_t polls) {
  if (polls > (int64_t)kWaitLimit) return EXACT_TOPK_ERR_BAD_SHAPE;
  g_wait_limit.store(polls < 0 ? kWaitLimit : (uint32_t)polls, std::memory_order_relaxed);
  return EXACT_TOPK_OK;
}

}  // extern "C"
