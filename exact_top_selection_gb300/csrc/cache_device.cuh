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

// The part of a page that a slot's sequence reaches with its rows.
struct PagePart {
  SeqRows rows;
  int seq, block, first, end;  // offsets [first, end) of page `block` of the sequence
  int index;                   // 0: the sequence's first part
};

// False where the slot has no part (first == end may still hold for index 0).
__device__ __forceinline__ bool page_part(const BatchArgs& b, int page_shift, int64_t slot,
                                          PagePart* part) {
  const int P = 1 << page_shift;
  part->seq = sequence_of_slot(b, slot, P, 2);
  part->rows = sequence_rows(b, page_shift, part->seq);
  part->index = (int)(slot - first_slot(b, part->seq, P, 2));
  const int begin = part->rows.pos0 > 0 ? part->rows.pos0 : 0;
  part->block = (begin >> page_shift) + part->index;
  const int64_t base = (int64_t)part->block << page_shift;
  const int64_t left = (int64_t)part->rows.len - base;
  part->first = part->index == 0 ? begin & (P - 1) : 0;
  part->end = left < P ? (int)left : P;
  return part->index >= 0 && part->rows.count > 0 && part->end > part->first;
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

__device__ __forceinline__ float finite_magnitude(float x) {
  const float a = fabsf(x);
  return a < __uint_as_float(0x7F800000u) ? a : 0.f;
}

// Pairs of the rows' type.
template <bool kFp16>
__device__ __forceinline__ uint32_t larger2(uint32_t x, uint32_t y) {
  if (kFp16) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&x),
                                   *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool kFp16>
__device__ __forceinline__ uint32_t smaller2(uint32_t x, uint32_t y) {
  if (kFp16) {
    const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&x), *reinterpret_cast<__half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&x),
                                   *reinterpret_cast<__nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bit patterns: the type's infinity, in both halves.
template <bool kFp16>
constexpr uint32_t infinities() {
  return kFp16 ? 0x7C007C00u : 0x7F807F80u;
}

// NaN as 0 and infinities as the type's largest number, in both halves.
template <bool kFp16>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  uint32_t r = 0u;
#pragma unroll
  for (int s = 0; s < 32; s += 16) {
    uint32_t x = w >> s & 0xFFFFu;
    const uint32_t a = x & 0x7FFFu, inf = infinities<kFp16>() & 0xFFFFu;
    if (a == inf) x -= 1u;  // the pattern before infinity
    if (a > inf) x = 0u;
    r |= x << s;
  }
  return r;
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

// Eight e2m1 codes as four pairs of halves, the lower four bits of a byte in a pair's lower half.
__device__ __forceinline__ void codes4_to_half2(uint32_t codes, uint32_t (&y)[4]) {
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
      : "r"(codes));
}

__device__ __forceinline__ uint32_t times2(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x),
                            *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// An e4m3 scale in both halves of a pair.
__device__ __forceinline__ uint32_t scale_to_half2(uint32_t code) {
  return __byte_perm(codes_to_half2((uint16_t)code), 0u, 0x1010);
}

inline int launch_status() {
  return cudaGetLastError() == cudaSuccess ? EXACT_TOPK_OK : EXACT_TOPK_ERR_CUDA;
}

}  // namespace etk
