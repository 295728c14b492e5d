// Page scores (exact_topk_block_scores): S[t][h][j] = max over the key head's
// query heads g of relu(q_g) . hi_j + min(q_g, 0) . lo_j, since for each channel
// max(q * hi, q * lo) is q * hi where q >= 0 and q * lo where q < 0 (hi >= lo).
// That is one product over 2 D channels of [relu(q) | min(q, 0)] with [hi | lo], both
// exact in the input type, so the tensor cores' FP32 sums of exact products are
// as good as an FP32 evaluation.

#include "cache_device.cuh"
#include "tensor_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kPromptColumns = 64;
constexpr int kSms = 152;  // of a GB300; with fewer or more the items are shared out all the same
constexpr int kStepCtas = 4;  // resident on an SM
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

// The larger one; NaN where either is.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

__device__ __forceinline__ float max_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "l"(p));
  return r;
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
// 64 sequences of up to 1024 pages, 4 x 8 heads of 128 channels (75 MB): 15.5 us; with a CTA for
// every 64 pages, and their ids not asked for ahead, 19.9.
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
  // columns of a pass: tokens x the group's heads when they fit, else 8 heads of one token
  const int heads = group < 8 ? group : 8;
  const int columns = tokens * heads;
  const int own_token = g / heads, own_head = g - own_token * heads;
  const uint16_t* const own = queries + (rows.begin + token0 + own_token) * a.q.token_stride +
                              ((int64_t)h * group + own_head) * a.q.head_stride + q4 * 8;
  uint4 w[kChunks / 2];
  const auto load_queries = [&](int head0) {
    const bool live = g < columns && head0 + own_head < group;
#pragma unroll
    for (int j = 0; j < kChunks / 2; ++j)
      w[j] = live ? __ldg(reinterpret_cast<const uint4*>(own + head0 * a.q.head_stride + j * 32))
                  : make_uint4(0u, 0u, 0u, 0u);
  };
  load_queries(0);

  const int step = (int)gridDim.y * kWarps * kPages;
  int page0 = ((int)blockIdx.y * kWarps + warp) * kPages;
  int next[2];  // ids of the pages after these
  const auto find = [&](int p) {
#pragma unroll
    for (int r = 0; r < 2; ++r)
      next[r] = p + g + 8 * r < seen ? page_of(c, b, seq, p + g + 8 * r) : -1;
  };
  find(page0);
  for (; page0 < seen; page0 += step) {
    uint4 x[2][kChunks];
    uint32_t absent = 0u;  // of the warp's 16 pages
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int id = next[r];
      const uint16_t* const at = bounds + ((int64_t)id * c.heads + h) * (2 * D) + q4 * 8;
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
        x[r][j] = id >= 0 ? load_once(at + j * 32) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t lanes = __ballot_sync(~0u, id < 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) absent |= (lanes >> (4 * k) & 1u) << (8 * r + k);
    }
    find(page0 + step);
    float best = -__uint_as_float(0x7F800000u);
    for (int head0 = 0; head0 < group; head0 += heads) {
      if (group > 8) load_queries(head0);
      float s[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const bool positive = j < kChunks / 2;
        const uint4& u = w[j % (kChunks / 2)];
        const uint32_t a0[4] = {x[0][j].x, x[1][j].x, x[0][j].y, x[1][j].y};
        const uint32_t a1[4] = {x[0][j].z, x[1][j].z, x[0][j].w, x[1][j].w};
        mma<kFp16>(s, a0, clamp_sign<kFp16>(u.x, positive), clamp_sign<kFp16>(u.y, positive));
        mma<kFp16>(s1, a1, clamp_sign<kFp16>(u.z, positive), clamp_sign<kFp16>(u.w, positive));
      }
      __syncwarp();
      s_out[warp][g][2 * q4] = s[0] + s1[0];
      s_out[warp][g][2 * q4 + 1] = s[1] + s1[1];
      s_out[warp][g + 8][2 * q4] = s[2] + s1[2];
      s_out[warp][g + 8][2 * q4 + 1] = s[3] + s1[3];
      __syncwarp();
      const int here = group - head0 < heads ? group - head0 : heads;
      if (group > 8) {  // one token a tile: its maximum goes from pass to pass
        if (lane < kPages)
          for (int i = 0; i < here; ++i) best = max_nan(best, s_out[warp][lane][i]);
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
          for (int k = 1; k < heads; ++k)
            v = max_nan(v, s_out[warp][i % kPages][t * heads + k]);
        }
        if (j < a.keep_first || j > newest - a.keep_last) v = __uint_as_float(0x7F800000u);
        if (absent >> (i % kPages) & 1u) v = -__uint_as_float(0x7F800000u);
        a.scores[((rows.begin + token0 + t) * c.heads + h) * a.row_pitch + j] = v;
      }
    }
  }
}

// ---- prompts ----
//
// Many columns against many pages: bound by the matrix products, so they run on the
// fifth-generation tensor cores. A CTA keeps 256 columns (tokens x heads of one key
// head, [relu(q) | min(q, 0)]) in shared memory and streams pages past them, 128 at a
// time: D[128 pages][256 columns] in tensor memory, two of them, so that one is
// read out while the next is computed. Pages are the accumulator's lanes: the largest over a
// token's heads is a maximum over neighbouring columns of one lane, and a warp's 32 lanes
// write 32 neighbouring scores.
//
// One CTA an SM takes items (256 columns x a run of pages) in turn; where they lie is worked
// out for up to 16 of them at once. Its warps keep to one role each: four gather page rows,
// which lie anywhere in memory, in lines of 64 channels through a ring; eight bring the next
// item's columns, line by line as the products let go of the old ones; one thread issues
// the products; four warps read the results out. Every wait is bounded; a CTA whose wait
// ran out computes its items again, one score a thread (score_again).
//
// The products alone, with nothing to wait for, take 87 us of a chunk of 4096 tokens x 32 heads
// over 2048 pages (an SM's shared memory feeds both operands: 96 of its 128 bytes a clock). A
// TMA gather of four rows at a time brought lines at a fifth of that rate.
constexpr int kReadOut = 128;            // threads of each role
constexpr int kGather = 128;
constexpr int kFill = 256;
constexpr int kItems = 16;               // items whose places are held
constexpr int kPromptThreads = kReadOut + kGather + kFill + 32;
constexpr int kIssueWarp = (kPromptThreads - 32) / 32;
constexpr int kColumns = 256;
constexpr int kLanes = 128;              // pages of a tile
constexpr int kLine = 64;                // channels of a line
constexpr int kLineBytes = kLanes * kLine * 2;

// An item: a column tile of a sequence and key head, and a run of page tiles (none where there
// are no rows, or no pages left for the run).
struct PromptItem {
  int64_t row0;
  int seq, head, pos0, tokens, seen, first_page, tiles, first_run;
};

// Lines are in the order hi, lo of channels 0-63, then hi, lo of channels 64-127.
template <int D>
struct PromptShared {
  static constexpr int kChunks = 2 * D / kLine;
  static constexpr int kStages = 6;
  uint8_t columns[kChunks][kColumns * kLine * 2];
  uint8_t pages[kStages][kLineBytes];
  uint64_t full[kStages], empty[kStages];       // page lines
  uint64_t filled[kChunks], released[kChunks];  // column lines
  uint64_t done[2], free[2];                    // accumulators
  uint64_t drained;
  PromptItem item[kItems];
  uint32_t tensor;
  int failed;
};

struct PromptWork {
  int64_t slots, items;
  int groups, each;  // runs of page tiles, and the tiles of one
};

__device__ __forceinline__ PromptItem prompt_item(const CacheArgs& c, const BatchArgs& b,
                                                  const PromptWork& w, int tile_tokens,
                                                  int64_t i) {
  PromptItem item = {};
  const int group = (int)(i % w.groups);
  const int64_t rest = i / w.groups;
  item.head = (int)(rest % c.heads);
  item.first_run = group == 0;
  const int64_t slot = rest / c.heads;
  item.seq = sequence_of_slot(b, slot, tile_tokens, 1);
  const SeqRows rows = sequence_rows(b, c.page_shift, item.seq);
  const int64_t token0 = (slot - first_slot(b, item.seq, tile_tokens, 1)) * tile_tokens;
  if (token0 < 0 || token0 >= rows.count) return item;
  item.tokens = rows.count - token0 < tile_tokens ? (int)(rows.count - token0) : tile_tokens;
  item.row0 = rows.begin + token0;
  item.pos0 = rows.pos0 + (int)token0;
  const int last = item.pos0 + item.tokens - 1;
  item.seen = last < 0 ? 0 : (last >> c.page_shift) + 1;
  item.first_page = group * w.each * kLanes;
  if (item.first_page >= item.seen) return item;
  const int all = (item.seen - item.first_page + kLanes - 1) / kLanes;
  item.tiles = all < w.each ? all : w.each;
  return item;
}

// All scores of a CTA's items from their definition, without waits. Apart from the kernel's body,
// whose registers its own would crowd.
template <bool kFp16, int D>
__device__ __noinline__ void score_again(const CacheArgs& c, const BatchArgs& b,
                                         const ScoreArgs& a, const PromptWork& work,
                                         int tile_tokens) {
  const uint16_t* const bounds = static_cast<const uint16_t*>(c.bounds);
  const uint16_t* const queries = static_cast<const uint16_t*>(a.q.data);
  for (int64_t i = blockIdx.x; i < work.items; i += gridDim.x) {
    const PromptItem item = prompt_item(c, b, work, tile_tokens, i);
    if (item.tiles == 0) continue;
    const int left = item.seen - item.first_page;
    const int pages = left < item.tiles * kLanes ? left : item.tiles * kLanes;
    for (int n = threadIdx.x; n < item.tokens * pages; n += kPromptThreads) {
      const int token = n / pages, j = item.first_page + n % pages;
      const int pos = item.pos0 + token, newest = pos >> c.page_shift;
      if (pos < 0 || j > newest) continue;
      const int page = page_of(c, b, item.seq, j);
      float best = -__uint_as_float(0x7F800000u);
      if (page >= 0 && (j < a.keep_first || j > newest - a.keep_last)) {
        best = __uint_as_float(0x7F800000u);
      } else if (page >= 0) {
        const uint4* const at = reinterpret_cast<const uint4*>(
            bounds + ((int64_t)page * c.heads + item.head) * (2 * D));
        for (int g = 0; g < a.group; ++g) {
          const uint4* const q = reinterpret_cast<const uint4*>(
              queries + (item.row0 + token) * a.q.token_stride +
              ((int64_t)item.head * a.group + g) * a.q.head_stride);
          float sum = 0.f;
#pragma unroll 1
          for (int k = 0; k < D / 8; ++k) {
            const uint4 x = __ldg(q + k), y = __ldg(at + k), z = __ldg(at + D / 8 + k);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w}, hi[4] = {y.x, y.y, y.z, y.w},
                           lo[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const float2 up = unpack2<kFp16>(clamp_sign<kFp16>(u[m], true));
              const float2 down = unpack2<kFp16>(clamp_sign<kFp16>(u[m], false));
              const float2 most = unpack2<kFp16>(hi[m]), least = unpack2<kFp16>(lo[m]);
              sum = fmaf(up.x, most.x, fmaf(down.x, least.x, sum));
              sum = fmaf(up.y, most.y, fmaf(down.y, least.y, sum));
            }
          }
          best = g == 0 ? sum : max_nan(best, sum);
        }
      }
      a.scores[((item.row0 + token) * c.heads + item.head) * a.row_pitch + j] = best;
    }
  }
}

// kPadded: the group's heads rounded up to a power of two, at most 32; a column beyond
// the group repeats its last head, which leaves the maximum as it is.
template <bool kFp16, int D, int kPadded>
__global__ void __launch_bounds__(kPromptThreads, 1)
    score_prompt_kernel(const __grid_constant__ CacheArgs c, const __grid_constant__ BatchArgs b,
                        const __grid_constant__ ScoreArgs a,
                        const __grid_constant__ PromptWork work, uint32_t wait_limit) {
  using Smem = PromptShared<D>;
  constexpr int kChunks = Smem::kChunks, kStages = Smem::kStages;
  constexpr int kTileTokens = kColumns / kPadded;
  extern __shared__ unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      raw + ((1024u - (shared_address(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.num_valid_rows != nullptr && blockIdx.x == 0 && tid == 0)
    *a.num_valid_rows =
        (int32_t)((b.q_start == nullptr ? b.num_seqs : clamp_row(b, b.num_seqs)) * c.heads);
  if (tid == 0) {
    sm.failed = 0;
    for (int i = 0; i < kStages; ++i) {
      barrier_init(&sm.full[i], kGather);
      barrier_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kChunks; ++i) {
      barrier_init(&sm.filled[i], kFill);
      barrier_init(&sm.released[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      barrier_init(&sm.done[i], 1);
      barrier_init(&sm.free[i], kReadOut);
    }
    barrier_init(&sm.drained, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     shared_address(&sm.tensor))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tensor = sm.tensor;
  volatile int* const failed = &sm.failed;

  // Each role's own counts go on from batch to batch of items, as the barriers' phases do.
  bool ok = true;
  int steps = 0, tiles = 0, columns_filled = 0;
  for (int64_t item0 = blockIdx.x; item0 < work.items; item0 += (int64_t)kItems * gridDim.x) {
    const int items = (int)((work.items - item0 + gridDim.x - 1) / gridDim.x < kItems
                                ? (work.items - item0 + gridDim.x - 1) / gridDim.x
                                : kItems);
    __syncthreads();
    if (tid < items)
      sm.item[tid] = prompt_item(c, b, work, kTileTokens, item0 + (int64_t)tid * gridDim.x);
    __syncthreads();
    if (tid < kReadOut) {
      // ---- read out ----
      constexpr int kEach = 32 / kPadded;  // tokens of 32 columns
      const int64_t row_step = (int64_t)c.heads * a.row_pitch;
      for (int i = 0; i < items && ok; ++i) {
        const PromptItem& item = sm.item[i];
        if (item.tiles == 0) continue;
        const int first_newest = item.pos0 >> c.page_shift;  // the first token's newest page
        const int parts = (item.tokens + kEach - 1) / kEach;
        int j0 = item.first_page + warp * 32;
        bool there = j0 + lane < item.seen && page_of(c, b, item.seq, j0 + lane) >= 0;
        for (int tile = 0; tile < item.tiles; ++tile, ++tiles, j0 += kLanes) {
          const int buffer = tiles & 1, j = j0 + lane;
          // all of the warp's pages are seen by every token, and scored
          const bool plain = item.pos0 >= 0 && j0 >= a.keep_first &&
                             j0 + 31 <= first_newest - a.keep_last && __all_sync(~0u, there);
          float* at = a.scores + (item.row0 * c.heads + item.head) * a.row_pitch + j;
          ok = barrier_wait(&sm.done[buffer], (tiles >> 1) & 1, failed);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t from = tensor + ((uint32_t)(warp * 32) << 16) + buffer * kColumns;
          const auto largest = [&](const float (&v)[32], int t) {
            float best = v[t * kPadded];
            if (kPadded == 2) best = max_nan(best, v[t * kPadded + 1]);
#pragma unroll
            for (int k = 1; k + 1 < kPadded; k += 2)
              best = max_nan(best, v[t * kPadded + k], v[t * kPadded + k + 1]);
            if (kPadded > 2) best = max_nan(best, v[t * kPadded + kPadded - 1]);
            return best;
          };
          const auto write = [&](int part, const float (&v)[32]) {
            const int left = item.tokens - part * kEach;
            if (plain && left >= kEach) {
#pragma unroll
              for (int t = 0; t < kEach; ++t, at += row_step) *at = largest(v, t);
              return;
            }
#pragma unroll
            for (int t = 0; t < kEach; ++t, at += row_step) {
              float best = largest(v, t);
              const int pos = item.pos0 + part * kEach + t;
              const int newest = pos >> c.page_shift;
              if (j < a.keep_first || j > newest - a.keep_last)
                best = __uint_as_float(0x7F800000u);
              if (!there) best = -__uint_as_float(0x7F800000u);
              if (t < left && pos >= 0 && j <= newest) *at = best;
            }
          };
          bool next = false;  // the next tile's page, asked for before it is needed
          if (tile + 1 < item.tiles && j + kLanes < item.seen)
            next = page_of(c, b, item.seq, j + kLanes) >= 0;
          for (int part = 0; part < parts; ++part) {
            float v[32];
            tensor_load32(from + part * 32, v);
            tensor_wait(v);
            write(part, v);
          }
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          barrier_arrive(&sm.free[buffer]);
          there = next;
        }
      }
    } else if (tid < kReadOut + kGather) {
      // ---- gather: thread i takes piece i % 8 of the lines of pages i / 8 + 16 k ----
      constexpr int kRows = kLanes / (kGather / 8);
      const int piece = tid & 7, line0 = (tid - kReadOut) >> 3;
      const uint16_t* const bounds = static_cast<const uint16_t*>(c.bounds);
      for (int i = 0; i < items && ok; ++i) {
        const PromptItem& item = sm.item[i];
        // where the lines of the tile after this one are; those of absent pages and ones that
        // nobody sees are the first page's, whose results are not written
        const uint16_t* next[kRows];
        const auto find = [&](int tile) {
#pragma unroll
          for (int k = 0; k < kRows; ++k) {
            const int j = item.first_page + tile * kLanes + line0 + k * (kGather / 8);
            const int page = tile < item.tiles && j < item.seen ? page_of(c, b, item.seq, j) : 0;
            next[k] = bounds + ((int64_t)(page < 0 ? 0 : page) * c.heads + item.head) * (2 * D) +
                      piece * 8;
          }
        };
        find(0);
        for (int tile = 0; tile < item.tiles && ok; ++tile) {
          const uint16_t* from[kRows];
#pragma unroll
          for (int k = 0; k < kRows; ++k) from[k] = next[k];
          find(tile + 1);
          for (int chunk = 0; chunk < kChunks; ++chunk, ++steps) {
            const int s = steps % kStages;
            if (steps >= kStages &&
                !barrier_wait(&sm.empty[s], (steps / kStages - 1) & 1, failed)) {
              ok = false;
              break;
            }
            const uint32_t to =
                shared_address(sm.pages[s]) + line0 * (kLine * 2) + ((piece ^ (line0 & 7)) << 4);
            const int channel = (chunk & 1) * D + (chunk >> 1) * kLine;
#pragma unroll
            for (int k = 0; k < kRows; ++k)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                               to + k * (kGather / 8) * (kLine * 2)),
                           "l"(from[k] + channel)
                           : "memory");
            // arrives when this thread's copies have; the issuing thread orders them before its
            // reads
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                             shared_address(&sm.full[s]))
                         : "memory");
          }
        }
      }
    } else if (warp < kIssueWarp) {
      // ---- columns: 8 channels at a time, the positive and the negative part to their lines ----
      constexpr int kLines = D / kLine;                    // of a column of q
      constexpr int kPieces = kColumns * kLine / 8 / kFill;  // a thread's pieces of a line
      const int thread = tid - kReadOut - kGather;
      const int piece = thread & 7;
      for (int i = 0; i < items; ++i) {
        const PromptItem& item = sm.item[i];
        // lengths, by the threads of each column tile's first run, whether or not a wait ran out
        if (item.first_run && thread < item.tokens) {
          const int pos = item.pos0 + thread;
          a.ke[(item.row0 + thread) * c.heads + item.head] =
              pos < 0 ? 0 : (pos >> c.page_shift) + 1;
        }
        if (item.tiles == 0 || !ok) continue;
        uint4 w[kLines][kPieces];
#pragma unroll
        for (int line = 0; line < kLines; ++line)
#pragma unroll
          for (int n = 0; n < kPieces; ++n) {
            const int col = (thread >> 3) + n * (kFill / 8);
            const int token = col / kPadded;
            const int head = col % kPadded < a.group ? col % kPadded : a.group - 1;
            w[line][n] = make_uint4(0u, 0u, 0u, 0u);
            if (token < item.tokens)
              w[line][n] = __ldg(reinterpret_cast<const uint4*>(
                  static_cast<const uint16_t*>(a.q.data) + (item.row0 + token) * a.q.token_stride +
                  ((int64_t)item.head * a.group + head) * a.q.head_stride + line * kLine +
                  piece * 8));
          }
#pragma unroll
        for (int chunk = 0; chunk < kChunks; ++chunk) {
          if (columns_filled > 0)
            ok = barrier_wait(&sm.released[chunk], (columns_filled - 1) & 1, failed);
          if (!ok) break;
          const bool positive = (chunk & 1) == 0;
#pragma unroll
          for (int n = 0; n < kPieces; ++n) {
            const int col = (thread >> 3) + n * (kFill / 8);
            const uint4 u = w[chunk >> 1][n];
            *reinterpret_cast<uint4*>(
                &sm.columns[chunk][col * (kLine * 2) + ((piece ^ (col & 7)) << 4)]) =
                make_uint4(clamp_sign<kFp16>(u.x, positive), clamp_sign<kFp16>(u.y, positive),
                           clamp_sign<kFp16>(u.z, positive), clamp_sign<kFp16>(u.w, positive));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          barrier_arrive(&sm.filled[chunk]);
        }
        ++columns_filled;
      }
    } else {
      // ---- products, by one thread ----
      // The waits for operands are the ones whose limit the host sets: once one has run out, the
      // others give up as well.
      constexpr uint32_t kType = kFp16 ? 0u : 1u;
      constexpr uint32_t kind = 1u << 4 | kType << 7 | kType << 10 | (kColumns / 8) << 17 |
                                (kLanes / 16) << 24;
      const bool leader = elected();
      for (int i = 0; i < items && ok; ++i) {
        const int item_tiles = sm.item[i].tiles;
        if (item_tiles == 0) continue;
        for (int tile = 0; tile < item_tiles && ok; ++tile, ++tiles) {
          const int buffer = tiles & 1;
          if (tiles >= 2) ok = barrier_wait(&sm.free[buffer], ((tiles >> 1) - 1) & 1, failed);
          for (int chunk = 0; chunk < kChunks; ++chunk, ++steps) {
            const int s = steps % kStages;
            if (tile == 0)
              ok = ok && barrier_wait(&sm.filled[chunk], columns_filled & 1, failed, wait_limit);
            ok = ok && barrier_wait(&sm.full[s], (steps / kStages) & 1, failed, wait_limit);
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            if (leader) {
              const uint64_t pages = operand(shared_address(sm.pages[s]));
              const uint64_t columns = operand(shared_address(sm.columns[chunk]));
#pragma unroll
              for (int k = 0; k < kLine / 16; ++k)  // 32 bytes of a line each
                tensor_mma(tensor + buffer * kColumns, pages + 2 * k, columns + 2 * k, kind,
                           chunk > 0 || k > 0);
              tensor_commit(&sm.empty[s]);
              if (tile == item_tiles - 1) tensor_commit(&sm.released[chunk]);
              if (chunk == kChunks - 1) tensor_commit(&sm.done[buffer]);
            }
            __syncwarp();
          }
        }
        ++columns_filled;
      }
    }
  }
  if (warp == kIssueWarp) {
    // what was issued ends before the shared memory and the tensor memory go
    int none = 0;
    if (elected()) tensor_commit(&sm.drained);
    __syncwarp();
    barrier_wait(&sm.drained, 0, &none);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tensor)
                 : "memory");
  if (*failed) score_again<kFp16, D>(c, b, a, work, kTileTokens);
}

template <bool kFp16, int D, int kPadded>
int launch_prompt(const CacheArgs& c, const BatchArgs& b, const ScoreArgs& a,
                  cudaStream_t stream) {
  constexpr size_t smem = sizeof(PromptShared<D>) + 1024;
  const auto kernel = score_prompt_kernel<kFp16, D, kPadded>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess) {
    cudaGetLastError();
    return EXACT_TOPK_ERR_CUDA;
  }
  PromptWork work;
  work.slots = slot_count(b, kColumns / kPadded, 1);
  const int tiles = (b.width + kLanes - 1) / kLanes;
  // Runs of page tiles of equal length, as few of them as make six items for each CTA, so that the
  // last ones end together; of at least 2 tiles, behind which an item's columns come in, and of at
  // most 16.
  const int64_t column_tiles = work.slots * c.heads;
  int64_t groups = (kSms * 6 + column_tiles - 1) / column_tiles;
  groups = groups < (tiles + 15) / 16 ? (tiles + 15) / 16 : groups;
  groups = groups > (tiles + 1) / 2 ? (tiles + 1) / 2 : groups;
  work.each = (int)((tiles + groups - 1) / groups);
  work.groups = (tiles + work.each - 1) / work.each;
  work.items = work.slots * c.heads * work.groups;
  const unsigned grid = (unsigned)(work.items < kSms ? work.items : kSms);
  kernel<<<grid, kPromptThreads, smem, stream>>>(c, b, a, work, wait_limit());
  return launch_status();
}

template <bool kFp16, int D>
int launch_prompt_group(const CacheArgs& c, const BatchArgs& b, const ScoreArgs& a,
                        cudaStream_t stream) {
  if (a.group == 1) return launch_prompt<kFp16, D, 1>(c, b, a, stream);
  if (a.group == 2) return launch_prompt<kFp16, D, 2>(c, b, a, stream);
  if (a.group <= 4) return launch_prompt<kFp16, D, 4>(c, b, a, stream);
  if (a.group <= 8) return launch_prompt<kFp16, D, 8>(c, b, a, stream);
  if (a.group <= 16) return launch_prompt<kFp16, D, 16>(c, b, a, stream);
  return launch_prompt<kFp16, D, 32>(c, b, a, stream);
}

}  // namespace

int launch_block_scores(const CacheArgs& c, const BatchArgs& b, const ScoreArgs& a,
                        cudaStream_t stream) {
  // Rows of a sequence (their mean number) times its group's heads: from 64 columns on the
  // tensor cores' tiles are filled well enough.
  const int64_t mean = (b.num_tokens + b.num_seqs - 1) / b.num_seqs;
  if (a.group <= 32 && mean * a.group >= kPromptColumns) {
    if (c.dim == 128)
      return c.fp16 ? launch_prompt_group<true, 128>(c, b, a, stream)
                    : launch_prompt_group<false, 128>(c, b, a, stream);
    return c.fp16 ? launch_prompt_group<true, 64>(c, b, a, stream)
                  : launch_prompt_group<false, 64>(c, b, a, stream);
  }
  const int tile_tokens = a.group >= 8 ? 1 : 8 / a.group;
  const int64_t slots = slot_count(b, tile_tokens, 1);
  // CTAs of a tile: two waves of them over all tiles, each with a few steps of 64 pages whose
  // next page ids come while the last ones' bounds are used.
  int64_t steps = ((int64_t)b.width + kWarps * kPages - 1) / (kWarps * kPages);
  const int64_t wanted = (2 * kSms * kStepCtas + slots * c.heads - 1) / (slots * c.heads);
  steps = steps < wanted ? steps : wanted;
  const dim3 grid((unsigned)slots, (unsigned)steps, (unsigned)c.heads);
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
