// Internal interface between the host checks of the operators on a batch (batch_api.cpp) and
// their kernels (rotary_kernels.cu, table_kernels.cu).  Not installed.
#pragma once

#include <cstdint>

#include "cache_internal.h"

namespace etk {

struct RotaryArgs {
  RowArgs q, k, q_out, k_out;
  const uint64_t* turns;     // of each pair in a position, as a fraction of 2^64
  const int32_t* positions;  // NULL: those of the batch
  int64_t num_tokens;
  float amplitude;
  int q_heads, k_heads, dim, pairs, neighbours, fp16, inverse;
  int copy_q, copy_k;  // the channels that do not turn have to be copied
};

struct TableArgs {
  int32_t* table;
  int32_t* kv_len;
  int32_t* q_start;
  int32_t* applied;
  int32_t* slots;
  int32_t* positions;
  int32_t* free_pages;
  int32_t* free_range;
  int32_t* arrived;  // CTAs of the call that have read its inputs
  const int32_t* change;
  int64_t pitch;
  int64_t max_tokens;
  int num_seqs, width, num_pages, page_shift, negate;
};

int launch_rotary(const RotaryArgs&, const BatchArgs&, cudaStream_t);
int launch_update_tables(const TableArgs&, cudaStream_t);

}  // namespace etk
