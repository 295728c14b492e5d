// Page scores (exact_topk_block_scores): S[t][h][j] = max over the key head's
// query heads g of relu(q_g) . hi_j + min(q_g, 0) . lo_j, since for each channel
// max(q * hi, q * lo) is q * hi where q >= 0 and q * lo where q < 0 (hi >= lo).
// That is one product over 2 D channels of [relu(q) | min(q, 0)] with [hi | lo], both
// exact in the input type, so the tensor cores' FP32 sums of exact products are
// as good as an FP32 evaluation.

#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPages = 16;  // pages of a warp's step: the rows of one matrix instruction

template <bool kFp16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if (kFp16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Both halves' positive or negative part; NaN stays NaN.
template <bool kFp16>
__device__ __forceinline__ uint32_t clamp_sign(uint32_t w, bool positive) {
  if (kFp16) {
    const __half2 x = *reinterpret_cast<const __half2*>(&w), zero = __floats2half2_rn(0.f, 0.f);
    const __half2 r = positive ? __hmax2_nan(x, zero) : __hmin2_nan(x, zero);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w);
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 r = positive ? __hmax2_nan(x, zero) : __hmin2_nan(x, zero);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A tile: up to 8 query columns (tile_tokens tokens x tile_heads heads of one key head)
// against a range of pages, 16 pages a warp at a time. Pages are the rows of the
// matrix instruction, so that the few columns of a decoding step fill its 8.
// Both operands come from global memory straight into fragments: the order of the
// contraction is free, so each lane takes 16 contiguous bytes of a page's row and of a
// column (lane % 4 chunks of 8 channels), which makes 64-byte segments of every load.
// A group of more than 8 heads takes several passes; the maxima are kept between them.
template <bool kFp16, int D>
__global__ void __launch_bounds__(kThreads) score_step_kernel(CacheArgs c, BatchArgs b,
                                                              ScoreArgs a, int tile_tokens) {
  constexpr int kChunks = D / 16;  // 16-byte chunks of [hi | lo] for each of 4 lanes
  __shared__ float s_out[kWarps][kPages][9];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const int h = blockIdx.z;
  const int64_t slot = blockIdx.x;
  if (a.num_valid_rows != nullptr && slot == 0 && blockIdx.y == 0 && h == 0 && threadIdx.x == 0)
    *a.num_valid_rows =
        (int32_t)((b.q_start == nullptr ? b.num_seqs : clamp_row(b, b.num_seqs)) * c.heads);
  const int seq = sequence_of_slot(b, slot, tile_tokens, 1);
  const SeqRows rows = sequence_rows(b, c.page_shift, seq);
  const int64_t index = slot - first_slot(b, seq, tile_tokens, 1);
  const int64_t token0 = index * tile_tokens;  // within the sequence
  if (index < 0 || token0 >= rows.count) return;
  const int tokens = rows.count - token0 < tile_tokens ? (int)(rows.count - token0) : tile_tokens;
  const int last = rows.pos0 + (int)token0 + tokens - 1;  // the tile's last position
  const int seen = last < 0 ? 0 : (last >> c.page_shift) + 1;

  if (blockIdx.y == 0 && threadIdx.x < tokens) {
    const int pos = rows.pos0 + (int)token0 + (int)threadIdx.x;
    a.ke[(rows.begin + token0 + threadIdx.x) * c.heads + h] =
        pos < 0 ? 0 : (pos >> c.page_shift) + 1;
  }
  const uint16_t* const bounds = static_cast<const uint16_t*>(c.bounds);
  const uint16_t* const queries = static_cast<const uint16_t*>(a.q.data);
  const int group = a.group;

  for (int page0 = ((int)blockIdx.y * kWarps + warp) * kPages; page0 < seen;
       page0 += (int)gridDim.y * kWarps * kPages) {
    int id[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = page0 + g + 8 * r;
      id[r] = j < seen ? page_of(c, b, seq, j) : -1;
    }
    uint4 x[2][kChunks];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint16_t* const at = bounds + ((int64_t)id[r] * c.heads + h) * (2 * D) + q4 * 8;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        x[r][j] = id[r] >= 0 ? __ldg(reinterpret_cast<const uint4*>(at + j * 32))
                             : make_uint4(0u, 0u, 0u, 0u);
    }
    // columns of a pass: tokens x the group's heads when they fit, else 8 heads of one token
    const int heads = group < 8 ? group : 8;
    const int columns = tokens * heads;
    float best = -__uint_as_float(0x7F800000u);
    for (int head0 = 0; head0 < group; head0 += heads) {
      const bool live = g < columns && head0 + g % heads < group;
      const uint16_t* const q =
          queries + (rows.begin + token0 + g / heads) * a.q.token_stride +
          ((int64_t)h * group + head0 + g % heads) * a.q.head_stride + q4 * 8;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const bool positive = j < kChunks / 2;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (live) w = __ldg(reinterpret_cast<const uint4*>(q + (j % (kChunks / 2)) * 32));
        const uint32_t a0[4] = {x[0][j].x, x[1][j].x, x[0][j].y, x[1][j].y};
        const uint32_t a1[4] = {x[0][j].z, x[1][j].z, x[0][j].w, x[1][j].w};
        mma<kFp16>(s, a0, clamp_sign<kFp16>(w.x, positive), clamp_sign<kFp16>(w.y, positive));
        mma<kFp16>(s, a1, clamp_sign<kFp16>(w.z, positive), clamp_sign<kFp16>(w.w, positive));
      }
      __syncwarp();
      s_out[warp][g][2 * q4] = s[0];
      s_out[warp][g][2 * q4 + 1] = s[1];
      s_out[warp][g + 8][2 * q4] = s[2];
      s_out[warp][g + 8][2 * q4 + 1] = s[3];
      __syncwarp();
      const int here = group - head0 < heads ? group - head0 : heads;
      if (group > 8) {  // one token a tile: its maximum goes from pass to pass
        if (lane < kPages)
          for (int i = 0; i < here; ++i) {
            const float v = s_out[warp][lane][i];
            best = best != best || v <= best ? best : v;
          }
        if (head0 + heads < group) continue;
      }
      for (int i = lane; i < tokens * kPages; i += 32) {
        const int t = i / kPages, j = page0 + i % kPages;
        const int pos = rows.pos0 + (int)token0 + t;
        const int newest = pos >> c.page_shift;
        if (pos < 0 || j > newest) continue;
        float v = best;
        if (group <= 8) {
          v = s_out[warp][i % kPages][t * heads];
          for (int k = 1; k < heads; ++k) {
            const float u = s_out[warp][i % kPages][t * heads + k];
            v = v != v || u <= v ? v : u;
          }
        }
        if (j < a.keep_first || j > newest - a.keep_last) v = __uint_as_float(0x7F800000u);
        if (page_of(c, b, seq, j) < 0) v = -__uint_as_float(0x7F800000u);
        a.scores[((rows.begin + token0 + t) * c.heads + h) * a.row_pitch + j] = v;
      }
    }
  }
}

}  // namespace

int launch_block_scores(const CacheArgs& c, const BatchArgs& b, const ScoreArgs& a,
                        cudaStream_t stream) {
  const int tile_tokens = a.group >= 8 ? 1 : 8 / a.group;
  const int64_t slots = slot_count(b, tile_tokens, 1);
  const int steps = (b.width + kWarps * kPages - 1) / (kWarps * kPages);
  const dim3 grid((unsigned)slots, (unsigned)(steps < 65535 ? steps : 65535), (unsigned)c.heads);
  if (c.dim == 128) {
    if (c.fp16)
      score_step_kernel<true, 128><<<grid, kThreads, 0, stream>>>(c, b, a, tile_tokens);
    else
      score_step_kernel<false, 128><<<grid, kThreads, 0, stream>>>(c, b, a, tile_tokens);
  } else {
    if (c.fp16)
      score_step_kernel<true, 64><<<grid, kThreads, 0, stream>>>(c, b, a, tile_tokens);
    else
      score_step_kernel<false, 64><<<grid, kThreads, 0, stream>>>(c, b, a, tile_tokens);
  }
  return launch_status();
}

}  // namespace etk
