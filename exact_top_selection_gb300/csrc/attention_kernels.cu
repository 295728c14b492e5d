// Attention over the paged 8-bit cache (exact_topk_attention_run): a row's
// running maximum m (up to an offset), sum l and output O, in FP32, over its pages in one pass,
//
//   x_p = scale * (q . k_p) * k_scale,  m' = max(m, x_p),
//   l' = l e^(m - m') + e^(x_p - m'),   O' = O e^(m - m') + e^(x_p - m') v_p.
//
// What bounds it: the cached bytes where a page serves the few columns of a decoding
// step; the conversion of codes and the matrix instructions where neighbouring tokens
// of a prompt read the same pages.
//
// Layout. A tile is up to 8, 16 or 32 columns: tokens x heads of one key head. Cached
// tokens are the ROWS of both products, S^T = K Q^T (16 tokens x 8 columns) and O^T =
// V^T P^T (16 channels x 8 columns), so that the few query columns of a key head fill
// the 8 columns of m16n8k16. The order of a contraction is free, so fragments are read in
// 16-byte pieces: for the first product each lane holds 32 (16) channels of two tokens, for
// the second 16 (8) channels of four tokens, whose codes are paired by byte permutes before
// they are converted. S^T's accumulators, packed to halves and transposed in registers, are
// P^T's fragments. Codes come through a ring in shared memory of each warp's own
// (cp.async), which keeps 32 KB of 48 on their way in each of an SM's four CTAs: loads into
// registers instead kept 48 KB an SM and reached 5.0 TB/s.
//
// Types. Codes are exact in FP16, so both products run in FP16 with FP32 sums. A
// query row is brought to [2^8, 2^9) by a power of two: what is then below FP16's
// normal range is off by 2^-25, against 2^8, less than FP32's own rounding of
// the sum. Probabilities are held in FP16 with the largest between 2^6 and 2^14: 11 bits
// (against the 8 or 11 of the output) down to 2^-20 of it, below that off by at most 2^-31 of it.
// The factor cancels in the quotient. With the largest between 1 and 2^8 instead, a flat tail
// of 2^-26 each was lost from the outputs, but not from the sum that divides them.
//
// Work. Over the whole cache, all pages of all tiles form one line that the CTAs cut into
// equal parts, whatever the lengths; a CTA's part may cover several tiles. Listed pages
// are as many for each tile: a tile is cut into as many equal parts as there are
// CTAs for it, one where there are more tiles than CTAs. Inside a CTA each warp takes
// 32 tokens of a page, and its four warps' results are joined through shared memory. A
// tile that several CTAs share is joined from their partial results by the last of
// them to arrive, in the order of their parts, so that results do not depend on timing.
//
// Measured: 64 sequences of 2048 to 65536 tokens, 4 key heads x 8 query heads of 128 channels
// (2.4 GB): 360 to 370 us from GPU to GPU, 95 to 98% of the rate of a copy. 8 sequences of 512 K
// tokens, 3 new ones, 2 x 4 heads of 64 channels (1.06 GB): 209 us. 32 listed pages of 64
// sequences (134 MB): 34 us.

#include <climits>

#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 128;   // pages whose ids are held in shared memory at a time
// m, the exponent that a row's probabilities are relative to, is put kRoom powers of two below the
// largest score so far, and moved again only when a score is more than kMost above it:
// probabilities reach 2^14 at most, and the sums are rescaled a few times in a row's life
// instead of at each step.
constexpr float kRoom = 6.f;
constexpr float kMost = 14.f;

__device__ __forceinline__ float infinity() { return __uint_as_float(0x7F800000u); }

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 16 bytes to shared memory, asynchronously; zeros where !there.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(there ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Any of four codes NaN (0x7F or 0xFF)?
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Which sequence, tokens and heads a tile has.
struct Tile {
  int64_t row0;    // first token's row
  int seq, head, head0, heads;  // key head; its query heads [head0, head0 + heads)
  int tokens, pos0;             // tokens and the first one's position
  int64_t start;   // its place on the line of units
  int units;
};

// A sequence's tiles: groups of tokens x key heads x parts of a key head's group.
__device__ __forceinline__ int64_t tile_count(const AttentionArgs& a, const CacheArgs& c,
                                              int rows) {
  return (int64_t)((rows + a.tile_tokens - 1) / a.tile_tokens) * c.heads * a.group_parts;
}

// Units of each of a sequence's tiles over the whole cache: pages, at least one.
__device__ __forceinline__ int page_units(const CacheArgs& c, const SeqRows& s) {
  const int pages = (s.len + c.page - 1) >> c.page_shift;
  return pages > 0 ? pages : 1;
}

// Steps that a warp holds in shared memory, all but one of them on their way: 48 KB of a
// CTA where four share an SM, more where fewer do.
constexpr int ring_steps(int dim, int tiles, int blocks) {
  const int ctas = attention_ctas_per_sm(tiles * 8, dim);
  const int tokens = ctas == 4 ? 48 : (ctas == 3 ? 64 : 80);  // of 128 channels
  const int steps = tokens * 128 / dim / (16 * blocks);
  return steps;
}

// ST: blocks of 16 tokens in a step.
template <int D, int NT, int ST>
struct alignas(128) Shared {
  static constexpr int kRegs = D / 16 * NT * 4;  // output registers of a lane
  static constexpr int kRow = D + 8;             // halves of a query row, padded by 16 bytes
  static constexpr int kRing = ring_steps(D, NT, ST);
  static constexpr int kRingBytes = kWarps * kRing * 2 * 16 * ST * D;
  static constexpr int kOutBytes = kWarps * kRegs * 32 * 4;
  union {
    uint8_t ring[kWarps][kRing][2][16 * ST * D];  // codes of keys and values
    float out[kWarps][kRegs][32];                 // after the last step
    // after the outputs: each partial result's factor for each column
    float weight[(kRingBytes > kOutBytes ? kRingBytes : kOutBytes) / 4];
  };
  float stat[kWarps][2][NT * 8];   // m and l of the columns
  __half q[NT * 8][kRow];
  float factor[NT * 8];
  float sum[NT * 8];               // of a tile that several CTAs share
  int64_t offset[kChunk];          // of a page's codes; -1 for an absent page
  uint32_t entry[kChunk];          // place in the sequence | members << 24
  float2 scale[kChunk];            // of keys and values
  int scan[kWarps];
  int last;
  static_assert(sizeof(weight) >= kMaxAttentionWorkers * NT * 8 * 4 ||
                    attention_ctas_per_sm(NT * 8, D) < 4,
                "a factor for each CTA and column");
  static_assert(sizeof(weight) >= kMaxAttentionWorkers * 3 / 4 * NT * 8 * 4 ||
                    attention_ctas_per_sm(NT * 8, D) != 3,
                "a factor for each CTA and column");
  static_assert(sizeof(weight) >= kMaxAttentionWorkers / 2 * NT * 8 * 4 ||
                    attention_ctas_per_sm(NT * 8, D) != 2,
                "a factor for each CTA and column");
};

// Where a tile's outputs go.
struct OutPlace {
  uint16_t* data;  // the tile's first token and head
  int64_t token_stride, head_stride;
  int heads, columns, fp16;
};

// A lane's outputs of column n * 8 + 2 c + j: 2 * kOwn neighbouring channels for each warp.
template <int D, int NT>
__device__ __forceinline__ void write_outputs(const OutPlace& out, int col, int token, float l,
                                              const float (&y)[D / 16 / kWarps][2]) {
  constexpr int kOwn = D / 16 / kWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint16_t* const at = out.data + token * out.token_stride +
                       (col - token * out.heads) * out.head_stride + (lane >> 2) * (D / 8) +
                       warp * kOwn * 2;
  const float by = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const float y0 = l == 0.f ? 0.f : y[i][0] * by, y1 = l == 0.f ? 0.f : y[i][1] * by;
    *reinterpret_cast<uint32_t*>(at + i * 2) =
        out.fp16 ? pack2<true>(y0, y1) : pack2<false>(y0, y1);
  }
}

// Joins the partial results of a tile, in the order of its parts, and writes its outputs. Part 0
// is at `first`, part 1 `second` floats behind it, and each further one `step` behind the one
// before. `weight` is shared memory for a factor of each part and column, `sums` for a sum of
// each column. Apart from the kernel's body, whose registers its own would crowd.
template <int D, int NT>
__device__ __noinline__ void join_parts(const float* first, int parts, int64_t second,
                                        int64_t step, float* weight, float* sums, OutPlace out) {
  constexpr int kColumns = NT * 8, kOwn = D / 16 / kWarps, kOwnRegs = kOwn * NT * 4;
  constexpr int kCols = kColumns / kWarps;
  constexpr int kBatch = kOwnRegs < 64 ? 64 / kOwnRegs : 1;  // parts on their way
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q4 = lane & 3;
  const auto slot = [&](int i) { return first + (i == 0 ? 0 : second + (i - 1) * step); };
  const int own = 2 * kColumns + warp * kOwnRegs * 32 + lane;
  float v[kBatch][kOwnRegs];
  const auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* const p = slot(i0 + k) + own;
#pragma unroll
      for (int i = 0; i < kOwnRegs; ++i) v[k][i] = i0 + k < parts ? __ldcg(p + i * 32) : 0.f;
    }
  };
  load(0);
  // Every warp takes a quarter of the columns, a part a lane: maxima, then factors and sums.
  float top[kCols], sum[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    top[k] = -infinity();
    sum[k] = 0.f;
  }
  for (int i = lane; i < parts; i += 32) {
    const float* const p = slot(i) + warp * kCols;
    float pm[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k) pm[k] = __ldcg(p + k);
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      top[k] = fmaxf(top[k], pm[k]);
      weight[i * kColumns + warp * kCols + k] = pm[k];
    }
  }
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], d));
    if (top[k] == -infinity()) top[k] = 0.f;
  }
  for (int i = lane; i < parts; i += 32) {
    const float* const p = slot(i) + kColumns + warp * kCols;
    float pl[kCols];
#pragma unroll
    for (int k = 0; k < kCols; ++k) pl[k] = __ldcg(p + k);
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
      float* const w = weight + i * kColumns + warp * kCols + k;
      const float by = exp2_fast(*w - top[k]);
      *w = by;
      sum[k] += by * pl[k];
    }
  }
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum[k] += __shfl_xor_sync(~0u, sum[k], d);
    if (lane == 0) sums[warp * kCols + k] = sum[k];
  }
  __syncthreads();
  float r[kOwnRegs];
#pragma unroll
  for (int i = 0; i < kOwnRegs; ++i) r[i] = 0.f;
  for (int i0 = 0; i0 < parts; i0 += kBatch) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* const by = weight + (i0 + k < parts ? i0 + k : 0) * kColumns + q4 * 2;
#pragma unroll
      for (int i = 0; i < kOwnRegs; ++i) r[i] += v[k][i] * by[i / 4 % NT * 8 + (i & 1)];
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = n * 8 + q4 * 2 + j;
      if (col >= out.columns) continue;
      float y[kOwn][2];
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        y[i][0] = r[(i * NT + n) * 4 + j];
        y[i][1] = r[(i * NT + n) * 4 + 2 + j];
      }
      write_outputs<D, NT>(out, col, col / out.heads, sums[col], y);
    }
}

template <int D, int NT, int ST>
__global__ void __launch_bounds__(kThreads, attention_ctas_per_sm(NT * 8, D))
    attention_kernel(CacheArgs c, BatchArgs b, AttentionArgs a) {
  constexpr int kTiles = D / 16;    // channel tiles of the output
  constexpr int kHalf = D / 64;     // 64-byte parts of a token's codes
  constexpr int kTokens = 16 * ST;  // of a step
  constexpr int kColumns = NT * 8;
  // query fragments in registers where there is room; else read at each step
  constexpr bool kHoldQ = D * NT <= 128;
  using Smem = Shared<D, NT, ST>;
  extern __shared__ __align__(128) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  // behind it: prefix sums of the sequences' units, then the members of each page (listed pages)
  int64_t* const prefix = reinterpret_cast<int64_t*>(raw + sizeof(Smem));
  uint32_t* const marks = reinterpret_cast<uint32_t*>(prefix + b.num_seqs + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const bool listed = a.blocks != nullptr;

  // Behind the prompt's kernel: nothing to do, most of the time. Marks of up to 64 KB are looked
  // over at once (3.5 us where none is set, 5 at 64 KB), and each tile's again below, all that
  // there are where there are more marks: 229 us for 16384 tokens x 8 key heads, 453 for 32768.
  if (a.again != nullptr) {
    const int64_t marks_count = (b.q_start == nullptr ? b.num_seqs : clamp_row(b, b.num_seqs)) *
                                c.heads * ((a.group + a.prompt_heads - 1) / a.prompt_heads);
    if (marks_count <= 65536) {
      uint32_t any = 0u;
      int i = tid * 16;
      for (; i + 16 <= marks_count; i += kThreads * 16) {
        const uint4 w = *reinterpret_cast<const uint4*>(a.again + i);
        any |= w.x | w.y | w.z | w.w;
      }
      for (; i < marks_count; ++i) any |= a.again[i];
      if (!__syncthreads_or(any != 0u)) return;
    }
  }

  // ---- the line of units: pages over the whole cache, tiles for listed pages ----
  const bool even = listed && b.q_start == nullptr;  // every sequence has one row
  int64_t total = (int64_t)b.num_seqs * c.heads * a.group_parts;
  if (!even) {
    int64_t carry = 0;
    for (int base = 0; base < b.num_seqs; base += kThreads) {
      int64_t mine = 0;
      if (base + tid < b.num_seqs) {
        const SeqRows s = sequence_rows(b, c.page_shift, base + tid);
        mine = tile_count(a, c, s.count) * (listed ? 1 : page_units(c, s));
      }
      int64_t sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += up;
      }
      int64_t* const totals = reinterpret_cast<int64_t*>(sm.stat);
      if (lane == 31) totals[warp] = sum;
      __syncthreads();
      int64_t before = carry;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += totals[w];
        carry += totals[w];
      }
      if (base + tid < b.num_seqs) prefix[base + tid + 1] = before + sum;
      if (base + tid == 0) prefix[0] = 0;
      __syncthreads();
    }
    total = carry;
  }
  // Listed pages: `cut` parts of each tile, one unit each. Whole cache: parts of `part` units.
  int64_t part = 1;
  int cut = 1;
  if (listed) {
    const int64_t fit = total > 0 ? a.workers / total : 1;
    cut = fit < 1 ? 1 : (fit < a.max_cut ? (int)fit : a.max_cut);
    total *= cut;
  } else {
    part = (total + a.workers - 1) / a.workers;
    if (part < a.min_units) part = a.min_units;
  }
  const int64_t line_end =
      listed ? total : ((blockIdx.x + 1) * part < total ? (blockIdx.x + 1) * part : total);

  for (int64_t u = blockIdx.x * part; u < line_end;) {
    // ---- the tile that unit u belongs to ----
    Tile t;
    {
      const int64_t at = listed ? u / cut : u;
      int64_t index;
      if (even) {
        const int each = c.heads * a.group_parts;
        t.seq = (int)(at / each);
        index = at - (int64_t)t.seq * each;
      } else {
        int lo = 0, hi = b.num_seqs - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (prefix[mid + 1] > at)
            hi = mid;
          else
            lo = mid + 1;
        }
        t.seq = lo;
        index = at - prefix[lo];
      }
      const SeqRows s = sequence_rows(b, c.page_shift, t.seq);
      if (listed) {
        t.units = cut;
        t.start = at * cut;
      } else {
        t.units = page_units(c, s);
        const int64_t start = index / t.units;
        t.start = prefix[t.seq] + start * t.units;
        index = start;
      }
      int rest = (int)index;  // rows x query heads are below 2^31
      const int group_part = a.group_parts > 1 ? rest % a.group_parts : 0;
      rest /= a.group_parts;
      t.head = rest % c.heads;
      const int token0 = rest / c.heads * a.tile_tokens;
      t.tokens = s.count - token0 < a.tile_tokens ? s.count - token0 : a.tile_tokens;
      t.row0 = s.begin + token0;
      t.pos0 = s.pos0 + token0;
      t.head0 = group_part * a.tile_heads;
      t.heads = a.group - t.head0 < a.tile_heads ? a.group - t.head0 : a.tile_heads;
    }
    if (a.again != nullptr) {  // behind the prompt's kernel: only what it has left
      const int parts = (a.group + a.prompt_heads - 1) / a.prompt_heads;
      bool left = false;
      for (int i = 0; i < t.tokens; ++i)
        left |= a.again[((t.row0 + i) * c.heads + t.head) * parts + t.head0 / a.prompt_heads] != 0;
      if (!left) {
        u = listed ? u + gridDim.x
                   : (line_end < t.start + t.units ? line_end : t.start + t.units);
        continue;
      }
    }
    const int64_t u_end =
        listed ? u + 1 : (line_end < t.start + t.units ? line_end : t.start + t.units);
    const int columns = t.tokens * t.heads;
    // tokens of the cache that the tile's last and first token see
    const int most = t.pos0 + t.tokens > 0 ? t.pos0 + t.tokens : 0;
    const int least = t.pos0 + 1 > 0 ? t.pos0 + 1 : 0;
    const int pages = (most + c.page - 1) >> c.page_shift;

    // ---- pages of a list: which tokens of the tile take each ----
    const int words = (pages + 3) >> 2;
    const int per_thread = (words + kThreads - 1) / kThreads;
    if (listed) {
      for (int i = tid; i < words; i += kThreads) marks[i] = 0u;
      __syncthreads();
      for (int token = warp; token < t.tokens; token += kWarps) {
        const int newest = t.pos0 + token >= 0 ? (t.pos0 + token) >> c.page_shift : -1;
        const int32_t* const list =
            a.blocks + ((t.row0 + token) * c.heads + t.head) * a.num_blocks;
        for (int i = lane; i < a.num_blocks; i += 32) {
          const int j = __ldg(list + i);
          if (j >= 0 && j <= newest) atomicOr(&marks[j >> 2], 1u << ((j & 3) * 8 + token));
        }
      }
    }

    // ---- queries: one column a warp at a time ----
    const int lane_token = lane / t.heads;  // of column `lane`
#pragma unroll
    for (int k = 0; k < kColumns / kWarps; ++k) {
      const int col = warp + k * kWarps;
      const int token = __shfl_sync(~0u, lane_token, col);
      float2 x[D / 64];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) x[i] = make_float2(0.f, 0.f);
      if (col < columns) {
        const uint16_t* const at =
            static_cast<const uint16_t*>(a.q.data) + (t.row0 + token) * a.q.token_stride +
            ((int64_t)t.head * a.group + t.head0 + col - token * t.heads) * a.q.head_stride;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(at + i * 64 + lane * 2));
          x[i] = c.fp16 ? unpack2<true>(w) : unpack2<false>(w);
          top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      // 2^(8 - exponent of the largest); 1 for rows of zeros and infinities
      int e = (int)(__float_as_uint(top) >> 23) - 127;
      if (e == 128 || top == 0.f) e = 8;
      int up = 8 - e;
      up = up < -120 ? -120 : (up > 120 ? 120 : up);
      const float by = __uint_as_float((uint32_t)(up + 127) << 23);
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        *reinterpret_cast<__half2*>(&sm.q[col][i * 64 + lane * 2]) =
            __floats2half2_rn(x[i].x * by, x[i].y * by);
      if (lane == 0)
        sm.factor[col] =
            col < columns ? __uint_as_float((uint32_t)(127 - up) << 23) * a.scale_log2 : 0.f;
    }
    __syncthreads();  // queries and marks are in place

    // this CTA's entries of the tile
    int from, to;
    int mine = 0;  // entries before this thread's words
    if (listed) {
      int have = 0;
      for (int i = tid * per_thread; i < (tid + 1) * per_thread && i < words; ++i) {
        const uint32_t w = marks[i];
#pragma unroll
        for (int k = 0; k < 4; ++k) have += (w >> (8 * k) & 255u) != 0u;
      }
      int sum = have;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += up;
      }
      if (lane == 31) sm.scan[warp] = sum;
      __syncthreads();
      mine = sum - have;
      int count = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) mine += sm.scan[w];
        count += sm.scan[w];
      }
      const int which = (int)(u - t.start);
      from = (int)((int64_t)count * which / cut);
      to = (int)((int64_t)count * (which + 1) / cut);
    } else {
      from = (int)(u - t.start);
      to = (int)(u_end - t.start);
      from = from < pages ? from : pages;
      to = to < pages ? to : pages;
    }

    // ---- a lane's columns ----
    float m[NT][2], l[NT][2], o[kTiles][NT][4];
    uint32_t shift[NT][2], have[NT];  // token of a column; tokens of each 8 columns
    uint4 held[kHoldQ ? NT : 1][kHalf][2];  // query fragments
    {
      uint32_t bits = lane < columns ? 1u << lane_token : 0u;
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) bits |= __shfl_xor_sync(~0u, bits, d);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        have[n] = __shfl_sync(~0u, bits, n * 8);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = n * 8 + q4 * 2 + j;
          const int token = __shfl_sync(~0u, lane_token, col);
          m[n][j] = -infinity();
          l[n][j] = 0.f;
          shift[n][j] = col < columns ? (uint32_t)token : 31u;  // no token: never a member
        }
        if (kHoldQ)
#pragma unroll
          for (int p = 0; p < kHalf; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              held[n][p][i] = *reinterpret_cast<const uint4*>(
                  &sm.q[n * 8 + g][p * 64 + q4 * 16 + i * 8]);
#pragma unroll
        for (int k = 0; k < kTiles; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[k][n][r] = 0.f;
      }
    }
    const uint32_t everyone = (1u << t.tokens) - 1u;
    float unit = 1.f;  // the values' scale that o is held in

    // A warp keeps to 32 tokens of a page (a page of 16: all of it), in `per_page` steps:
    // those from `row0` on, of entries first_entry, first_entry + entry_step, ...
    const int sub_shift = c.page_shift > 5 ? c.page_shift - 5 : 0;
    const int row0 = (warp & ((1 << sub_shift) - 1)) * 32;
    const int first_entry = warp >> sub_shift, entry_step = kWarps >> sub_shift;
    const int per_page = (c.page < 32 ? c.page : 32) / kTokens;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sm.ring[warp][0][0][0]);

    for (int chunk0 = from; chunk0 < to; chunk0 += kChunk) {
      const int entries = to - chunk0 < kChunk ? to - chunk0 : kChunk;
      // ---- the chunk's pages ----
      if (chunk0 > from) __syncthreads();
      if (listed) {
        int at = mine;
        for (int i = tid * per_thread; i < (tid + 1) * per_thread && i < words; ++i) {
          const uint32_t w = marks[i];
          if (w == 0u) continue;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t who = w >> (8 * k) & 255u;
            if (who == 0u) continue;
            if (at >= chunk0 && at < chunk0 + entries)
              sm.entry[at - chunk0] = (uint32_t)(i * 4 + k) | who << 24;
            ++at;
          }
        }
        __syncthreads();
      }
      for (int i = tid; i < entries; i += kThreads) {
        const int place = listed ? (int)(sm.entry[i] & 0xFFFFFFu) : chunk0 + i;
        const int page = page_of(c, b, t.seq, place);
        if (!listed) sm.entry[i] = (uint32_t)place;
        const int64_t tile = (int64_t)page * c.heads + t.head;
        sm.offset[i] = page >= 0 ? tile * c.page * D : -1;
        if (page >= 0)
          sm.scale[i] = make_float2(__ldg(c.k_scale + tile), __ldg(c.v_scale + tile));
      }
      __syncthreads();

      // Codes of a step into a place of the ring. A step is contiguous in memory. In
      // shared memory its 16-byte pieces are exchanged within lines of 128 bytes so
      // that the reads below touch every bank once.
      int fetch_entry = first_entry, fetch_step = 0;
      const auto fetch = [&](int place_in_ring) {
        if (fetch_entry < entries) {
          const int64_t offset = sm.offset[fetch_entry];
          const uint32_t entry = sm.entry[fetch_entry];
          const int place = listed ? (int)(entry & 0xFFFFFFu) : (int)entry;
          const int row = row0 + fetch_step * kTokens;
          const int rows = most - (place << c.page_shift) - row;  // tokens that anyone sees
          if (offset >= 0 && rows > 0) {
            const int64_t at = offset + row * D + lane * 16;
            const uint32_t to = ring + place_in_ring * (2 * kTokens * D);
#pragma unroll
            for (int j = 0; j < kTokens * D / 512; ++j) {
              const int piece = lane + 32 * j, line = piece >> 3, p = piece & 7;
              const bool there = (D == 128 ? line : piece >> 2) < rows;
              const int pk = D == 128 ? p ^ ((line & 1) << 2) : p;
              const int pv = D == 128 ? p ^ ((line >> 1 & 3) << 1) : p ^ ((line & 3) << 1);
              copy16(to + line * 128 + pk * 16, c.k + at + j * 512, there);
              copy16(to + kTokens * D + line * 128 + pv * 16, c.v + at + j * 512, there);
            }
          }
          if (++fetch_step == per_page) {
            fetch_step = 0;
            fetch_entry += entry_step;
          }
        }
        copy_commit();
      };

      const auto compute = [&](int e, int step, int place_in_ring) {
        const uint32_t entry = sm.entry[e];
        const int place = listed ? (int)(entry & 0xFFFFFFu) : (int)entry;
        const int pos = (place << c.page_shift) + row0 + step * kTokens;
        if (sm.offset[e] < 0 || pos >= most) return;
        const uint32_t members = listed ? entry >> 24 : everyone;
        const float2 scale = sm.scale[e];
        const uint8_t* const codes = &sm.ring[warp][place_in_ring][0][0];
        // Eight columns of which no token takes the page are left out. Where some do and
        // some do not, or the step ends beyond a token, scores are masked.
        bool takes[NT];
        bool masked = pos + kTokens > least;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          takes[n] = NT == 1 || (members & have[n]) != 0u;
          masked |= takes[n] && (members & have[n]) != have[n];
        }

        // ---- S^T ----
        float x[NT][4 * ST];
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          uint32_t f[D / 16][4];
#pragma unroll
          for (int p = 0; p < kHalf; ++p) {
            uint4 w[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int row = st * 16 + g + 8 * r;
              w[r] = *reinterpret_cast<const uint4*>(
                  codes + row * D + (D == 128 ? (p * 4 + q4) ^ ((row & 1) << 2) : q4) * 16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w0 = word(w[0], k), w1 = word(w[1], k);
              f[p * 4 + k][0] = codes_to_half2((uint16_t)w0);
              f[p * 4 + k][2] = codes_to_half2((uint16_t)(w0 >> 16));
              f[p * 4 + k][1] = codes_to_half2((uint16_t)w1);
              f[p * 4 + k][3] = codes_to_half2((uint16_t)(w1 >> 16));
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (!takes[n]) continue;
            // two sums, for shorter chains
            float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < kHalf; ++p)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint4 q;
                if (kHoldQ)
                  q = held[n][p][k];
                else
                  q = *reinterpret_cast<const uint4*>(
                      &sm.q[n * 8 + g][p * 64 + q4 * 16 + k * 8]);
                const uint32_t(&f0)[4] = f[p * 4 + k * 2];
                const uint32_t(&f1)[4] = f[p * 4 + k * 2 + 1];
                mma(s0, f0[0], f0[1], f0[2], f0[3], q.x, q.y);
                mma(s1, f1[0], f1[1], f1[2], f1[3], q.z, q.w);
              }
#pragma unroll
            for (int r = 0; r < 4; ++r) x[n][st * 4 + r] = s0[r] + s1[r];
          }
        }

        // ---- probabilities ----
        if (scale.y != unit) {
          const float by = unit / scale.y;
          unit = scale.y;
#pragma unroll
          for (int k = 0; k < kTiles; ++k)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r) o[k][n][r] *= by;
        }
        uint32_t pt[NT][2 * ST];
        uint32_t seen[ST];  // 4 bits for each 8 columns: this lane's scores that count
#pragma unroll
        for (int st = 0; st < ST; ++st) seen[st] = 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (!takes[n]) continue;
          const float2 factor = *reinterpret_cast<const float2*>(&sm.factor[n * 8 + q4 * 2]);
          const float fx = factor.x * scale.x, fy = factor.y * scale.x;
          float y[4 * ST];
          float high = -infinity();
#pragma unroll
          for (int r = 0; r < 4 * ST; ++r) {
            x[n][r] *= r & 1 ? fy : fx;
            y[r] = x[n][r] - m[n][r & 1];
          }
          if (masked) {
#pragma unroll
            for (int r = 0; r < 4 * ST; ++r) {
              const uint32_t token = shift[n][r & 1];
              if (pos + (r >> 2) * 16 + g + (r >> 1 & 1) * 8 > t.pos0 + (int)token ||
                  (members >> token & 1u) == 0u)
                x[n][r] = y[r] = -infinity();
              else
                seen[r >> 2] |= 1u << (n * 4 + (r & 3));
            }
          }
#pragma unroll
          for (int r = 0; r < 4 * ST; ++r) high = fmaxf(high, y[r]);
          if (__any_sync(~0u, high > kMost)) {
            float by[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float best = -infinity();
#pragma unroll
              for (int r = j; r < 4 * ST; r += 2) best = fmaxf(best, x[n][r]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1)
                best = fmaxf(best, __shfl_xor_sync(~0u, best, d));
              best = fmaxf(m[n][j], best - kRoom);
              by[j] = m[n][j] == -infinity() ? 0.f : exp2_fast(m[n][j] - best);
              m[n][j] = best;
              l[n][j] *= by[j];
            }
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
#pragma unroll
              for (int r = 0; r < 4; ++r) o[k][n][r] *= by[r & 1];
            // a masked score stays -inf, also where its column has seen nothing yet
#pragma unroll
            for (int r = 0; r < 4 * ST; ++r)
              y[r] = x[n][r] == -infinity() ? x[n][r] : x[n][r] - m[n][r & 1];
          }
#pragma unroll
          for (int r = 0; r < 4 * ST; ++r) {
            y[r] = exp2_fast(y[r]);
            l[n][r & 1] += y[r];
          }
#pragma unroll
          for (int r = 0; r < 2 * ST; ++r)
            pt[n][r] = transpose8(pack2<true>(y[2 * r], y[2 * r + 1]));
        }

#pragma unroll
        for (int st = 0; st < ST; ++st) {
          // ---- values: tokens 2c, 2c+1, 2c+8, 2c+9 of 16 (8) channels ----
          uint4 v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = st * 16 + q4 * 2 + (r & 1) + (r >> 1) * 8;
            const uint8_t* const at = codes + kTokens * D;
            if (D == 128) {
              v[r] = *reinterpret_cast<const uint4*>(at + row * 128 +
                                                     (g ^ ((row >> 1 & 3) << 1)) * 16);
            } else {
              const int line = row >> 1, p = (row & 1) * 4 + (g >> 1);
              const uint2 half = *reinterpret_cast<const uint2*>(
                  at + line * 128 + (p ^ ((line & 3) << 1)) * 16 + (g & 1) * 8);
              v[r] = make_uint4(half.x, half.y, 0u, 0u);
            }
          }
          // A value that is NaN makes NaN of the columns that see its token, and of no
          // other: where not every column sees every token, such values are taken out
          // of the product, and a product of ones marks the outputs that they reach.
          if (masked) {
            uint32_t bad = 0u;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int k = 0; k < D / 32; ++k) bad |= nan_codes(word(v[r], k));
            if (__any_sync(~0u, bad != 0u)) {
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (!takes[n]) continue;
                const uint32_t bits = seen[st] >> (n * 4);
                const uint32_t s0 = transpose8((bits & 1u ? 0x3C00u : 0u) |
                                               (bits & 2u ? 0x3C000000u : 0u));
                const uint32_t s1 = transpose8((bits & 4u ? 0x3C00u : 0u) |
                                               (bits & 8u ? 0x3C000000u : 0u));
#pragma unroll
                for (int k = 0; k < kTiles; ++k) {
                  uint32_t one[4];
#pragma unroll
                  for (int r = 0; r < 4; ++r) {  // channel 2k + (r & 1), token pair r >> 1
                    const int byte = (k & 1) * 2 + (r & 1);
                    const uint32_t w0 = word(v[(r >> 1) * 2], k >> 1) >> (8 * byte);
                    const uint32_t w1 = word(v[(r >> 1) * 2 + 1], k >> 1) >> (8 * byte);
                    one[r] = ((w0 & 0x7Fu) == 0x7Fu ? 0x3C00u : 0u) |
                             ((w1 & 0x7Fu) == 0x7Fu ? 0x3C000000u : 0u);
                  }
                  float hit[4] = {0.f, 0.f, 0.f, 0.f};
                  mma(hit, one[0], one[1], one[2], one[3], s0, s1);
#pragma unroll
                  for (int r = 0; r < 4; ++r)
                    if (hit[r] > 0.f) o[k][n][r] = __uint_as_float(0x7FFFFFFFu);
                }
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                  const uint32_t nan = nan_codes(w[k]) >> 7;  // 1 in each byte that is NaN
                  w[k] &= ~(nan * 255u);
                }
                v[r] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }

          // ---- O^T, half of the channels at a time ----
          constexpr int kPart = kTiles / 2;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t f[kPart][4];
#pragma unroll
            for (int k = 0; k < kPart; ++k) {
              const int tile = half * kPart + k;
              const uint32_t w0 = __byte_perm(word(v[0], tile >> 1), word(v[1], tile >> 1),
                                              tile & 1 ? 0x7362 : 0x5140);
              const uint32_t w1 = __byte_perm(word(v[2], tile >> 1), word(v[3], tile >> 1),
                                              tile & 1 ? 0x7362 : 0x5140);
              f[k][0] = codes_to_half2((uint16_t)w0);
              f[k][1] = codes_to_half2((uint16_t)(w0 >> 16));
              f[k][2] = codes_to_half2((uint16_t)w1);
              f[k][3] = codes_to_half2((uint16_t)(w1 >> 16));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (!takes[n]) continue;
#pragma unroll
              for (int k = 0; k < kPart; ++k)
                mma(o[half * kPart + k][n], f[k][0], f[k][1], f[k][2], f[k][3],
                    pt[n][st * 2], pt[n][st * 2 + 1]);
            }
          }
        }
      };

#pragma unroll
      for (int i = 0; i < Smem::kRing - 1; ++i) fetch(i);
      int now = 0, behind = Smem::kRing - 1;
      for (int e = first_entry; e < entries; e += entry_step) {
        for (int step = 0; step < per_page; ++step) {
          copy_wait<Smem::kRing - 2>();
          __syncwarp();
          compute(e, step, now);
          __syncwarp();
          fetch(behind);
          behind = now;
          now = now + 1 == Smem::kRing ? 0 : now + 1;
        }
      }
      copy_wait<0>();
    }
    __syncthreads();  // the ring's memory is used for the outputs now

    // ---- join the warps ----
    // Each lane's sums cover its own tokens: add over the lanes of a column. Then
    // bring every warp to the columns' common maximum and to a scale of 1.
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][j] += __shfl_xor_sync(~0u, l[n][j], d);
        if (g == 0) {
          sm.stat[warp][0][n * 8 + q4 * 2 + j] = m[n][j];
          sm.stat[warp][1][n * 8 + q4 * 2 + j] = l[n][j];
        }
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = n * 8 + q4 * 2 + j;
        float top = -infinity();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.stat[w][0][col]);
        const float base = top == -infinity() ? 0.f : top;
        const float by = exp2_fast(m[n][j] - base) * unit;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          sm.out[warp][(i * NT + n) * 4 + j][lane] = o[i][n][j] * by;
          sm.out[warp][(i * NT + n) * 4 + 2 + j][lane] = o[i][n][2 + j] * by;
        }
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          sum += sm.stat[w][1][col] * exp2_fast(sm.stat[w][0][col] - base);
        m[n][j] = top;
        l[n][j] = sum;
      }
    __syncthreads();
    // each warp keeps a quarter of the channel tiles
    constexpr int kOwn = kTiles / kWarps;
    float r[kOwn][NT][4];
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w)
            sum += sm.out[w][((warp * kOwn + i) * NT + n) * 4 + k][lane];
          r[i][n][k] = sum;
        }

    // ---- join the CTAs ----
    OutPlace out;
    out.data = static_cast<uint16_t*>(a.out.data) + t.row0 * a.out.token_stride +
               ((int64_t)t.head * a.group + t.head0) * a.out.head_stride;
    out.token_stride = a.out.token_stride;
    out.head_stride = a.out.head_stride;
    out.heads = t.heads;
    out.columns = columns;
    out.fp16 = c.fp16;
    const int first_cta = (int)(t.start / part);
    const int last_cta = (int)((t.start + t.units - 1) / part);
    if (first_cta != last_cta) {
      constexpr int64_t kFloats = partial_floats(kColumns, D);
      // a CTA's first slot holds the tile it continues, its second the tile it starts
      float* const at = a.partial +
                        ((int64_t)blockIdx.x * 2 + (first_cta == (int)blockIdx.x)) * kFloats;
      if (warp == 0 && g == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            at[n * 8 + q4 * 2 + j] = m[n][j];
            at[kColumns + n * 8 + q4 * 2 + j] = l[n][j];
          }
      }
      float* const mine_at = at + 2 * kColumns + (warp * kOwn * NT * 4) * 32 + lane;
#pragma unroll
      for (int i = 0; i < kOwn * NT * 4; ++i)
        mine_at[i * 32] = r[i / (NT * 4)][i / 4 % NT][i % 4];
      __syncthreads();
      if (tid == 0) {
        __threadfence();  // the CTA's partial result before its arrival
        const int arrived = atomicAdd(a.counters + first_cta, 1);
        sm.last = arrived == last_cta - first_cta;
        if (sm.last) a.counters[first_cta] = 0;
        __threadfence();  // the others' arrivals before their partial results
      }
      __syncthreads();
      if (sm.last)
        join_parts<D, NT>(a.partial + ((int64_t)first_cta * 2 + 1) * kFloats,
                          last_cta - first_cta + 1, kFloats, 2 * kFloats, sm.weight, sm.sum, out);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = n * 8 + q4 * 2 + j;
          if (col >= columns) continue;
          float y[kOwn][2];
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            y[i][0] = r[i][n][j];
            y[i][1] = r[i][n][2 + j];
          }
          write_outputs<D, NT>(out, col, (int)(shift[n][j] & 7u), l[n][j], y);
        }
    }
    u = listed ? u + gridDim.x : u_end;
    __syncthreads();  // shared memory is free for the next tile
  }
}

template <int D, int NT, int ST>
int launch_tile(const CacheArgs& c, const BatchArgs& b, const AttentionArgs& a,
                cudaStream_t stream) {
  constexpr size_t most = sizeof(Shared<D, NT, ST>) + sizeof(int64_t) * (EXACT_TOPK_MAX_SEQS + 1) +
                          EXACT_TOPK_MAX_LISTED_WIDTH;
  static_assert(most <= kMostShared, "every call that the checks let through");
  const size_t smem = sizeof(Shared<D, NT, ST>) + sizeof(int64_t) * ((size_t)b.num_seqs + 1) +
                      (a.blocks != nullptr ? ((size_t)b.width + 3) / 4 * 4 : 0);
  // Set on every call: a host-side table entry, cheaper than remembering it per device. The limit
  // belongs to the kernel and not to the call, so it is the largest call's: another thread's
  // launch may come between this thread's setting and its own launch.
  if (smem > 48 * 1024 && cudaFuncSetAttribute(attention_kernel<D, NT, ST>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)most) != cudaSuccess) {
    cudaGetLastError();
    return EXACT_TOPK_ERR_CUDA;
  }
  attention_kernel<D, NT, ST><<<a.workers, kThreads, smem, stream>>>(c, b, a);
  return launch_status();
}

}  // namespace

int launch_attention(const CacheArgs& c, const BatchArgs& b, const AttentionArgs& a,
                     cudaStream_t stream) {
  if (a.prompt_tokens > 0) {
    const int rc = launch_prompt_attention(c, b, a, stream);
    if (rc != EXACT_TOPK_OK) return rc;
  }
  if (c.dim == 128) {
    if (a.columns == 8) return launch_tile<128, 1, 1>(c, b, a, stream);
    if (a.columns == 16) return launch_tile<128, 2, 1>(c, b, a, stream);
    return launch_tile<128, 4, 1>(c, b, a, stream);
  }
  // Steps of 2 KB of keys and of values. Pages of 16 tokens have half of that.
  if (c.page == 16) {
    if (a.columns == 8) return launch_tile<64, 1, 1>(c, b, a, stream);
    if (a.columns == 16) return launch_tile<64, 2, 1>(c, b, a, stream);
    return launch_tile<64, 4, 1>(c, b, a, stream);
  }
  if (a.columns == 8) return launch_tile<64, 1, 2>(c, b, a, stream);
  if (a.columns == 16) return launch_tile<64, 2, 2>(c, b, a, stream);
  return launch_tile<64, 4, 2>(c, b, a, stream);
}

}  // namespace etk
