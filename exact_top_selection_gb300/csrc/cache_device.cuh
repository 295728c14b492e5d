// Device helpers shared by the cache operators' kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_internal.h"

namespace etk {

// Rows [begin, begin + count) of a sequence, its clamped length and the position of
// its first row (negative where it has more rows than tokens).
struct SeqRows {
  int64_t begin;
  int count, len, pos0;
};

__device__ __forceinline__ int64_t clamp_row(const BatchArgs& b, int i) {
  const int64_t r = b.q_start[i];
  return r < 0 ? 0 : (r > b.num_tokens ? b.num_tokens : r);
}

__device__ __forceinline__ SeqRows sequence_rows(const BatchArgs& b, int page_shift, int seq) {
  SeqRows s;
  if (b.q_start == nullptr) {
    s.begin = seq;
    s.count = 1;
  } else {
    s.begin = clamp_row(b, seq);
    const int64_t end = clamp_row(b, seq + 1);
    s.count = end > s.begin ? (int)(end - s.begin) : 0;
  }
  const int64_t most = (int64_t)b.width << page_shift;
  const int len = b.kv_len[seq];
  s.len = len < 0 ? 0 : (len > most ? (int)most : len);
  s.pos0 = s.len - s.count;
  return s;
}

// Work that comes in pieces of `piece` rows is laid over a grid that the host can
// size without the row ranges: sequence b's pieces start at slot
// floor(q_start[b] / piece) + extra * b.  A sequence of n rows that needs at most
// floor(n / piece) + extra pieces ends before the next one's first slot, since
// floor(x + n) >= floor(x) + floor(n).
__device__ __forceinline__ int64_t first_slot(const BatchArgs& b, int seq, int piece, int extra) {
  if (b.q_start == nullptr) return seq;
  return clamp_row(b, seq) / piece + (int64_t)extra * seq;
}

// The last sequence whose first slot is at or before `slot` (q_start ascends).
__device__ __forceinline__ int sequence_of_slot(const BatchArgs& b, int64_t slot, int piece,
                                                int extra) {
  if (b.q_start == nullptr) return (int)slot;
  int lo = 0, hi = b.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_slot(b, mid, piece, extra) <= slot)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

inline int64_t slot_count(const BatchArgs& b, int piece, int extra) {
  return b.q_start == nullptr ? b.num_seqs : b.num_tokens / piece + (int64_t)extra * b.num_seqs;
}

// Page id of table entry j, or -1 for an absent page.
__device__ __forceinline__ int page_of(const CacheArgs& c, const BatchArgs& b, int seq, int j) {
  const int p = b.table[(int64_t)seq * b.table_pitch + j];
  return (unsigned)p < (unsigned)c.num_pages ? p : -1;
}

template <bool kFp16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kFp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t w;
  if (kFp16) {
    const __half2 h = __floats2half2_rn(x, y);
    w = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w = *reinterpret_cast<const uint32_t*>(&h);
  }
  return w;
}

// Two e4m3 codes as a pair of halves: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t codes_to_half2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

__device__ __forceinline__ float2 codes_to_float2(uint16_t codes) {
  const uint32_t h = codes_to_half2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

inline int launch_status() {
  return cudaGetLastError() == cudaSuccess ? EXACT_TOPK_OK : EXACT_TOPK_ERR_CUDA;
}

}  // namespace etk
