// Internal interface between the host checks of the cache operators
// (cache_api.cpp) and their kernels (cache_kernels.cu, score_kernels.cu,
// attention_kernels.cu).  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "exact_topk_cache.h"

namespace etk {

// The arguments of a checked call as the kernels take them.
struct CacheArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  void* bounds;
  int num_pages, heads, page, page_shift, dim, fp16;
};

struct BatchArgs {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* q_start;  // NULL: one row for each sequence
  int64_t table_pitch;
  int64_t num_tokens;
  int num_seqs, width;
};

struct RowArgs {
  void* data;
  int64_t token_stride, head_stride;
};

// Polls of a barrier after which a wait gives up, far beyond any real wait, and the limit that
// calls take now (exact_topk_set_wait_limit).
constexpr uint32_t kWaitLimit = 1u << 20;
uint32_t wait_limit();

struct ScoreArgs {
  RowArgs q;
  float* scores;
  int32_t* ke;
  int32_t* num_valid_rows;
  int64_t row_pitch;
  int group, keep_first, keep_last;
};

struct AttentionArgs {
  RowArgs q, out;
  const int32_t* blocks;  // NULL: the whole cache
  int32_t* counters;      // [workers] arrivals at the tile a worker starts and does not finish
  float* partial;         // [workers][2] partial tiles (partial_floats each)
  float scale_log2;       // softmax scale * log2(e)
  int num_blocks, group, group_parts, columns, tile_tokens, tile_heads, workers;
  // The prompt's kernel: tokens and heads of its tiles, 0 where it does not run; and which tokens
  // it leaves to the other one, [num_tokens][kv_heads][parts of a group] (NULL: all).
  int prompt_tokens, prompt_heads;
  uint8_t* again;
  int min_units, max_cut;  // least pages of a part of the whole cache; most parts of a listed tile
};

// Floats of one partial tile: running maxima and sums of the columns, and the outputs.
constexpr int64_t partial_floats(int columns, int dim) {
  return (int64_t)columns * 2 + (int64_t)columns * dim;
}

// Rows of a prompt's tile, its tokens at most (a bit of a word each), and the widest page table of
// a call with lists that it takes (a word for each page in shared memory).
constexpr int kPromptRows = 128;
constexpr int kPromptTokens = 32;
constexpr int kPromptListedWidth = 24576;

// Shared memory that a CTA may have.
constexpr size_t kMostShared = 227 * 1024;

// The most CTAs of an attention launch.
constexpr int kMaxAttentionWorkers = 608;

// Resident CTAs that the attention kernels are built for. They have to fit the SM's shared memory
// with 8 bytes for each sequence and, over lists, a byte for each page of the table: with 8
// columns of 128 channels one fewer fits from 384 sequences on, and over lists of 64 sequences
// from 2553 pages on. The prompt's kernel takes 4 bytes for each page over lists, and a second CTA
// fits up to about 2900. Beyond that all still runs, in more waves than the plan counts on.
constexpr int attention_ctas_per_sm(int columns, int dim) {
  return dim == 64 ? (columns == 32 ? 3 : 4) : (columns == 8 ? 4 : (columns == 16 ? 3 : 2));
}

int launch_cache_write(const CacheArgs&, const BatchArgs&, const RowArgs& k, const RowArgs& v,
                       cudaStream_t);
int launch_cache_read(const CacheArgs&, const BatchArgs&, const RowArgs& k, const RowArgs& v,
                      cudaStream_t);
int launch_block_scores(const CacheArgs&, const BatchArgs&, const ScoreArgs&, cudaStream_t);
int launch_prompt_attention(const CacheArgs&, const BatchArgs&, const AttentionArgs&,
                            cudaStream_t);
int launch_attention(const CacheArgs&, const BatchArgs&, const AttentionArgs&, cudaStream_t);

}  // namespace etk
