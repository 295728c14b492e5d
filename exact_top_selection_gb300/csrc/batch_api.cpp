// Host side of the operators on a batch declared in include/exact_topk_cache.h (rotary
// positions, page tables): argument checks.  Nothing here synchronizes, allocates or reads device
// memory.

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "batch_internal.h"

namespace etk {
namespace {

constexpr int64_t kMostTokens = (int64_t)1 << 24;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_rows(const exact_topk_rows* rows, int64_t num_tokens, RowArgs* out) {
  if (rows == nullptr || (rows->data == nullptr && num_tokens > 0))
    return EXACT_TOPK_ERR_NULL_POINTER;
  if (!aligned(rows->data, 16) || rows->token_stride % 8 != 0 || rows->head_stride % 8 != 0)
    return EXACT_TOPK_ERR_MISALIGNED;
  *out = RowArgs{rows->data, rows->token_stride, rows->head_stride};
  return EXACT_TOPK_OK;
}

bool same(const RowArgs& a, const RowArgs& b) {
  return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

}  // namespace
}  // namespace etk

using namespace etk;

extern "C" {

int exact_topk_rotary(const exact_topk_rotary_spec* spec, const exact_topk_batch* batch,
                      const int32_t* positions, int64_t num_tokens, int q_heads,
                      const exact_topk_rows* q, const exact_topk_rows* q_out, int k_heads,
                      const exact_topk_rows* k, const exact_topk_rows* k_out, int inverse,
                      struct CUstream_st* stream) {
  RotaryArgs a{};
  BatchArgs b{};
  if (spec == nullptr || spec->turns == nullptr) return EXACT_TOPK_ERR_NULL_POINTER;
  if (num_tokens < 0 || num_tokens > kMostTokens) return EXACT_TOPK_ERR_BAD_BATCH;
  if ((batch == nullptr) == (positions == nullptr) && num_tokens > 0)
    return EXACT_TOPK_ERR_NULL_POINTER;
  if (batch != nullptr) {
    if (batch->kv_len == nullptr) return EXACT_TOPK_ERR_NULL_POINTER;
    if (batch->num_seqs < 1 || batch->num_seqs > EXACT_TOPK_MAX_SEQS ||
        (batch->q_start == nullptr && num_tokens != batch->num_seqs))
      return EXACT_TOPK_ERR_BAD_BATCH;
    if (!aligned(batch->kv_len, 4) || !aligned(batch->q_start, 4))
      return EXACT_TOPK_ERR_MISALIGNED;
    b.kv_len = batch->kv_len;
    b.q_start = batch->q_start;
    b.num_tokens = num_tokens;
    b.num_seqs = batch->num_seqs;
    b.width = 1 << 30;  // lengths are clamped to this many tokens
    if (spec->page_size > 0) {
      const int64_t most = (int64_t)batch->table_width * spec->page_size;
      if (batch->table_width < 1 || most > b.width) return EXACT_TOPK_ERR_BAD_BATCH;
      b.width = (int)most;
    }
  }
  if (spec->head_dim < 8 || spec->head_dim > 1024 || spec->head_dim % 8 != 0 ||
      spec->rotary_dim < 2 || spec->rotary_dim % 2 != 0 || spec->rotary_dim > spec->head_dim ||
      spec->rotary_dim > EXACT_TOPK_MAX_ROTARY_DIM || !std::isfinite(spec->amplitude) ||
      !(spec->page_size == 0 || spec->page_size == 16 || spec->page_size == 32 ||
        spec->page_size == 64 || spec->page_size == 128) ||
      (spec->type != EXACT_TOPK_TYPE_BF16 && spec->type != EXACT_TOPK_TYPE_FP16))
    return EXACT_TOPK_ERR_BAD_SHAPE;
  if (q_heads < 1 || q_heads > 65536 || k_heads < 0 || k_heads > 65536)
    return EXACT_TOPK_ERR_BAD_HEADS;
  int rc = check_rows(q, num_tokens, &a.q);
  if (rc == EXACT_TOPK_OK) rc = check_rows(q_out, num_tokens, &a.q_out);
  if (rc == EXACT_TOPK_OK && k_heads > 0) rc = check_rows(k, num_tokens, &a.k);
  if (rc == EXACT_TOPK_OK && k_heads > 0) rc = check_rows(k_out, num_tokens, &a.k_out);
  if (rc != EXACT_TOPK_OK) return rc;
  if (!aligned(spec->turns, 8) || !aligned(positions, 4)) return EXACT_TOPK_ERR_MISALIGNED;
  if (num_tokens == 0) return EXACT_TOPK_OK;
  a.turns = spec->turns;
  a.positions = positions;
  a.num_tokens = num_tokens;
  a.amplitude = spec->amplitude;
  a.q_heads = q_heads;
  a.k_heads = k_heads;
  a.dim = spec->head_dim;
  a.pairs = spec->rotary_dim / 2;
  a.neighbours = spec->neighbours != 0;
  a.fp16 = spec->type == EXACT_TOPK_TYPE_FP16;
  a.inverse = inverse != 0;
  a.copy_q = !same(a.q, a.q_out);
  a.copy_k = k_heads > 0 && !same(a.k, a.k_out);
  return launch_rotary(a, b, reinterpret_cast<cudaStream_t>(stream));
}

int exact_topk_update_tables(const exact_topk_page_tables* t, const int32_t* change, int negate,
                             struct CUstream_st* stream) {
  if (t == nullptr || change == nullptr || t->page_table == nullptr || t->kv_len == nullptr ||
      t->q_start == nullptr || t->free_pages == nullptr || t->free_range == nullptr ||
      t->counters == nullptr)
    return EXACT_TOPK_ERR_NULL_POINTER;
  const int P = t->page_size;
  if ((P != 16 && P != 32 && P != 64 && P != 128) || t->num_pages < 1 ||
      (int64_t)t->num_pages * P > 0x7FFFFFFF)
    return EXACT_TOPK_ERR_BAD_CACHE;
  if (t->num_seqs < 1 || t->num_seqs > EXACT_TOPK_MAX_SEQS || t->table_width < 1 ||
      (int64_t)t->table_width * P > ((int64_t)1 << 30) || t->table_pitch < t->table_width ||
      t->max_tokens < 0 || t->max_tokens > kMostTokens)
    return EXACT_TOPK_ERR_BAD_BATCH;
  if (t->counter_bytes < 4) return EXACT_TOPK_ERR_COUNTERS_TOO_SMALL;
  for (const void* p : {(const void*)t->page_table, (const void*)t->kv_len,
                        (const void*)t->q_start, (const void*)t->applied, (const void*)t->slots,
                        (const void*)t->positions, (const void*)t->free_pages,
                        (const void*)t->free_range, (const void*)t->counters,
                        (const void*)change})
    if (!aligned(p, 4)) return EXACT_TOPK_ERR_MISALIGNED;
  TableArgs a{};
  a.table = t->page_table;
  a.kv_len = t->kv_len;
  a.q_start = t->q_start;
  a.applied = t->applied;
  a.slots = t->slots;
  a.positions = t->positions;
  a.free_pages = t->free_pages;
  a.free_range = t->free_range;
  a.arrived = static_cast<int32_t*>(t->counters);
  a.change = change;
  a.pitch = t->table_pitch;
  a.max_tokens = t->max_tokens;
  a.num_seqs = t->num_seqs;
  a.width = t->table_width;
  a.num_pages = t->num_pages;
  a.page_shift = P == 16 ? 4 : (P == 32 ? 5 : (P == 64 ? 6 : 7));
  a.negate = negate != 0;
  return launch_update_tables(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
