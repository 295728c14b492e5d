// Attention of many neighbouring tokens over the paged 4-bit cache: two tiles of 128 rows on one
// conversion of its keys and values (a form of exact_topk_cache4_attention_run).
//
// As prompt_attention_kernels.cu, whose description holds: S = Q K^T, P = e^(S - m), O += P V in
// blocks of 64 cached tokens on the fifth-generation tensor cores, a row a thread. There a
// CTA has one tile, and two CTAs an SM each convert the same codes; with a product by a scale
// for each pair of codes that conversion is as long as the softmax. Here a CTA has an SM to itself
// and two tiles, of neighbouring tokens, with two warps each to issue their products, and eight
// warps convert each block once for both.
//
// Scales are part of the FP16 operands (a code times its scale is exact in FP16), units part of the
// scores' factor and of the outputs. A NaN scale shows as a NaN among a row's sums or outputs; its
// tile is left to the kernel that runs behind, as is one whose wait ran out.
//
// What bounds it: 664 clocks of products for a block and tile (8 of 50, limited by shared memory's
// reads of both operands, and 4 of 66), so 1328 of the 1980 that a block of both takes, and the
// chain of a tile's probabilities, outputs and scores of the block after the next, which take the
// probabilities' place: tensor memory has no room for scores that would not wait. 2048 tokens x 16
// query heads (2 key heads of 128 channels) over 16384: 267 us (965 TFLOP/s); 4096 over 32 pages of
// 64 tokens each: 122 us. With a warp a tile for both kinds of products it took 274 us, and with 32
// scores loaded at a time, none of them while others are weighed, 280.
//
// Measured and not kept: two threads a row (twice the votes and barriers); two groups of softmax
// warps for a tile, a block each in turn; the next block's scores waited for while this one's are
// weighed (+40: they are late as a rule); the maximum looked for only where a block's sum is too
// large (+20); an arrival for each warp instead of each thread (+6); waits that poll without a pause
// (+4); probabilities stored 64 tokens at a time (+7); converted pieces exchanged between lanes
// against bank conflicts, where lanes by token have none (+22); the line of all tiles' blocks cut
// evenly over the SMs, of which 128 CTAs leave 24 idle: to begin and to join parts of tiles, and
// the registers for it, cost more than the 16% (290, over lists 168).

#include "cache_device.cuh"
#include "prompt_device.cuh"

namespace etk {
namespace {

constexpr int kTiles = 2;
constexpr int kRows = 128;                       // of a tile
constexpr int kConvert = 128;                    // threads for keys, and as many for values
constexpr int kSoftmaxWarps = kTiles * kRows / 32;
constexpr int kConvertWarps = 2 * kConvert / 32;
constexpr int kWarps = kSoftmaxWarps + kConvertWarps + 2 * kTiles;
constexpr int kThreads = kWarps * 32;
constexpr int kBlock = 64;                       // cached tokens of a block
constexpr int kEntries = 128;                    // parts of pages held at a time
constexpr float kRoom = 6.f, kMost = 14.f;       // see attention_kernels.cu

__device__ __forceinline__ void tensor_store16(uint32_t address, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(address)
      : "memory");
}

// Stores issued so far are complete.
__device__ __forceinline__ void tensor_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// A part of a page: at most 64 tokens.
struct alignas(16) Entry {
  int pos;           // position of its first token
  uint32_t members;  // tokens of the tiles that take it; 0 for an absent page
  int64_t first;     // its first number's place in the cache; -1 for an absent page
};

template <int D>
struct Shared {
  uint8_t q[kTiles][D / 64][kRows * 128];  // lines of 64 channels, in swizzled blocks of 8
  uint8_t k[2][D / 64][kBlock * 128];
  uint8_t v[2][D / 64][kBlock * 128];
  Entry entry[kEntries];
  float factor[kTiles * kRows];
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t scored[kTiles][2], weighed[kTiles][2], added[kTiles][2], drained[2 * kTiles];
  uint32_t tensor;
  int scan[kWarps];
  int failed, again;
};

// kPartShift: log2 of the parts of a block (1 of pages of 64 and 128 tokens, 2 of 32, 4 of 16).
template <int D, int kPartShift>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_pair_kernel(Cache4Args c, BatchArgs b, AttentionArgs a, uint32_t wait_limit) {
  using Smem = Shared<D>;
  constexpr int kLines = D / 64;
  // tensor memory: O of both tiles, then two blocks' S of each, which its P replaces
  constexpr uint32_t kS = kTiles * 128, kTensorColumns = 512;
  extern __shared__ unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      raw + ((1024u - (shared_address(raw) & 1023u)) & 1023u));
  uint32_t* const marks = reinterpret_cast<uint32_t*>(&sm + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool listed = a.blocks != nullptr;
  const int head = blockIdx.y, head0 = (int)blockIdx.z * a.prompt_heads;
  const int heads = a.group - head0 < a.prompt_heads ? a.group - head0 : a.prompt_heads;
  const int piece = kTiles * a.prompt_tokens;  // tokens of a CTA
  const int64_t slot = blockIdx.x;
  const int seq = sequence_of_slot(b, slot, piece, 1);
  const SeqRows rows = sequence_rows(b, c.page_shift, seq);
  const int64_t index = slot - first_slot(b, seq, piece, 1);
  const int64_t token0 = index * piece;
  if (index < 0 || token0 >= rows.count) return;
  const int tokens = rows.count - token0 < piece ? (int)(rows.count - token0) : piece;
  const int64_t row0 = rows.begin + token0;
  const int pos0 = rows.pos0 + (int)token0;
  const int most = pos0 + tokens > 0 ? pos0 + tokens : 0;
  const int pages = (most + c.page - 1) >> c.page_shift;
  const int tiles = tokens > a.prompt_tokens ? 2 : 1;  // that have rows

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      barrier_init(&sm.k_full[i], kConvert);
      barrier_init(&sm.v_full[i], kConvert);
      barrier_init(&sm.k_free[i], tiles);
      barrier_init(&sm.v_free[i], tiles);
      for (int t = 0; t < kTiles; ++t) {
        barrier_init(&sm.scored[t][i], 1);
        barrier_init(&sm.weighed[t][i], kRows);
        barrier_init(&sm.added[t][i], 1);
      }
    }
    for (int t = 0; t < 2 * kTiles; ++t) barrier_init(&sm.drained[t], 1);
    sm.failed = 0;
    sm.again = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps - 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     shared_address(&sm.tensor)),
                 "r"(kTensorColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- queries: 8 channels a lane, all of a warp's 16 rows on their way ----
  constexpr int kLanes = D / 8, kStepRows = 32 / kLanes;  // lanes of a row, rows of a step
  constexpr int kSteps = 16 / kStepRows;
  const bool loads = warp < kTiles * kRows / 16;
  const int chunk = lane % kLanes, loads_tile = warp / (kRows / 16);
  const int first_row = warp * 16 % kRows + lane / kLanes;  // in its tile
  uint32_t there = 0u;  // steps whose row has a token
  uint4 w[kSteps];
  if (loads) {
    int token = first_row / heads, in_token = first_row - token * heads;
    const uint16_t* const from =
        static_cast<const uint16_t*>(a.q.data) +
        (row0 + loads_tile * a.prompt_tokens) * a.q.token_stride +
        ((int64_t)head * a.group + head0) * a.q.head_stride + chunk * 8;
    const int have = tokens - loads_tile * a.prompt_tokens;
    const int some = have < a.prompt_tokens ? have : a.prompt_tokens;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (token < some) {
        there |= 1u << k;
        w[k] = __ldg(reinterpret_cast<const uint4*>(from + token * a.q.token_stride +
                                                    in_token * a.q.head_stride));
      }
      in_token += kStepRows;
      while (in_token >= heads) {
        in_token -= heads;
        ++token;
      }
    }
  }

  // ---- pages of a list: which tokens of the tiles take each ----
  if (listed)
    for (int i = tid; i < pages; i += kThreads) marks[i] = 0u;
  __syncthreads();
  if (listed)
    for (int token = warp; token < tokens; token += kWarps) {
      const int newest = pos0 + token >= 0 ? (pos0 + token) >> c.page_shift : -1;
      const int32_t* const list = a.blocks + ((row0 + token) * c.heads + head) * a.num_blocks;
      for (int i = lane; i < a.num_blocks; i += 32) {
        const int j = __ldg(list + i);
        if (j >= 0 && j <= newest) atomicOr(&marks[j], 1u << token);
      }
    }

  if (loads) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      float2 x[4];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = c.fp16 ? unpack2<true>(u[i]) : unpack2<false>(u[i]);
        top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
      int e = (int)(__float_as_uint(top) >> 23) - 127;
      if (e == 128 || top == 0.f) e = 8;
      int up = 8 - e;
      up = up < -120 ? -120 : (up > 120 ? 120 : up);
      // the scale's sign goes into the queries, so that a row's largest score is its largest
      // product
      const float by = copysignf(__uint_as_float((uint32_t)(up + 127) << 23), a.scale_log2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i].x *= by;
        x[i].y *= by;
      }
      const int in_tile = first_row + k * kStepRows;
      *reinterpret_cast<uint4*>(&sm.q[loads_tile][chunk / 8]
                                     [in_tile * 128 + (((chunk & 7) ^ (in_tile & 7)) << 4)]) =
          make_uint4(pack2<true>(x[0].x, x[0].y), pack2<true>(x[1].x, x[1].y),
                     pack2<true>(x[2].x, x[2].y), pack2<true>(x[3].x, x[3].y));
      // NaN where the row has an infinity (see attention_kernels.cu)
      if (chunk == 0)
        sm.factor[loads_tile * kRows + in_tile] =
            (there >> k & 1u) != 0u
                ? __uint_as_float(top == infinity() ? 0x7FFFFFFFu : (uint32_t)(127 - up) << 23) *
                      fabsf(a.scale_log2)
                : 0.f;
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tensor = sm.tensor;
  volatile int* const failed = &sm.failed;

  // ---- how many parts of pages there are, and how many before this thread's ----
  const int part_shift = c.page_shift > 6 ? c.page_shift - 6 : 0;  // parts of a page
  constexpr int part_tokens_shift = 6 - kPartShift, per_block_shift = kPartShift;
  const int per_thread = (pages + kThreads - 1) / kThreads;
  int mine = 0, count = pages;
  if (listed) {
    int have = 0;
    for (int i = tid * per_thread; i < (tid + 1) * per_thread && i < pages; ++i)
      have += marks[i] != 0u;
    int sum = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) sm.scan[warp] = sum;
    __syncthreads();
    mine = sum - have;
    count = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) mine += sm.scan[w];
      count += sm.scan[w];
    }
  }

  // a row's state, kept by its thread
  const int tile = warp < kSoftmaxWarps ? warp / (kRows / 32) : warp & 1;  // of this warp
  const int row = tid & (kRows - 1);
  const int row_token = tile * a.prompt_tokens + row / heads;
  const bool live = warp < kSoftmaxWarps && row / heads < a.prompt_tokens && row_token < tokens;
  const int row_pos = live ? pos0 + row_token : -1;
  const uint32_t row_bit = live ? 1u << (row_token & 31) : 0u;  // without lists any bit does
  const float row_factor = warp < kSoftmaxWarps ? sm.factor[tid] : 0.f;
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  const uint32_t outputs = tensor + tile * 128, scores_at = tensor + kS + tile * 2 * kBlock;
  float m = -infinity(), l = 0.f;
  int done = 0;  // blocks so far, the same for every role
  bool ok = true;

  // Block n's barriers are those of its parity, so that who waits for one may be a block behind:
  // all that is known of the others then is that block n - 2 is done.
  const auto was_added = [&](int n) {
    return barrier_wait(&sm.added[tile][n & 1], (n >> 1) & 1, failed);
  };

  // O times a factor for each row
  const auto scale_outputs = [&](float by) {
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      float v[32];
      uint32_t w[32];
      tensor_load32(outputs + lane_base + i, v);
      tensor_wait(v);
#pragma unroll
      for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(v[k] * by);
      tensor_store32(outputs + lane_base + i, w);
    }
  };

  // 32 tokens' probabilities times a power of two: what falls below FP16's normal numbers is off by
  // 2^-25, against a largest one of 2^kRoom
  const auto scale_probabilities = [&](uint32_t at, float by) {
    float v[16];
    uint32_t w[16];
    tensor_stored();
    tensor_load16(at, v);
    tensor_wait(v);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 x = unpack2<true>(__float_as_uint(v[k]));
      w[k] = pack2<true>(x.x * by, x.y * by);
    }
    tensor_store16(at, w);
  };

  for (int chunk0 = 0; chunk0 < (count << part_shift); chunk0 += kEntries) {
    const int left = (count << part_shift) - chunk0;
    const int entries = left < kEntries ? left : kEntries;
    const int blocks = (entries + (1 << per_block_shift) - 1) >> per_block_shift;
    // ---- the chunk's parts of pages ----
    __syncthreads();
    if (listed) {
      int at = mine << part_shift;
      for (int i = tid * per_thread; i < (tid + 1) * per_thread && i < pages; ++i) {
        const uint32_t who = marks[i];
        if (who == 0u) continue;
        for (int k = 0; k < 1 << part_shift; ++k, ++at)
          if (at >= chunk0 && at < chunk0 + entries) {
            sm.entry[at - chunk0].pos = (i << c.page_shift) + (k << 6);
            sm.entry[at - chunk0].members = who;
          }
      }
      __syncthreads();
    }
    for (int i = tid; i < kEntries; i += kThreads) {
      Entry& e = sm.entry[i];
      e.first = -1;
      if (i >= entries) {
        e.members = 0u;
        e.pos = most;
        continue;
      }
      if (!listed) {
        e.pos = (chunk0 + i) << part_tokens_shift;
        e.members = ~0u;
      }
      const int page = page_of(c, b, seq, e.pos >> c.page_shift);
      if (page < 0) {
        e.members = 0u;
        continue;
      }
      const int64_t place = (int64_t)page * c.heads + head;
      e.first = ((place << c.page_shift) + (e.pos & (c.page - 1))) * D;
    }
    __syncthreads();

    if (warp < kSoftmaxWarps) {
      // ---- softmax: a row a thread ----
      for (int block = 0; block < blocks && tile < tiles; ++block) {
        const int n = done + block;
        // A part that this row does not take, and tokens behind its own, have probability 0: an
        // offset of -inf does it for whole parts.
        constexpr int kParts = 1 << kPartShift;
        int seen[kParts];
        bool cuts = false;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const Entry& e = sm.entry[(block << per_block_shift) + k];
          const bool takes = row_pos >= e.pos && (e.members & row_bit) != 0u;
          seen[k] = takes ? row_pos + 1 - e.pos : 0;
          cuts |= takes && seen[k] < 1 << part_tokens_shift;
        }
        cuts = __any_sync(~0u, cuts);
        ok = ok && barrier_wait(&sm.scored[tile][n & 1], (n >> 1) & 1, failed);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t from = scores_at + lane_base + (n & 1) * kBlock;
        // Probabilities under the running maximum, 32 tokens at a time. They take the place of
        // scores that have been read. Where a score turns out too far above the maximum, that is
        // raised by a whole number and the 32 are done again: it is seldom.
        float by = 1.f;
        bool some = false;
        float s[2][16];
        uint32_t p[16];
        float high = 0.f, base = 0.f;
        float2 sum = make_float2(0.f, 0.f);
        // 16 tokens: the first or second half of p
        const auto weigh = [&](const float (&x)[16], int group) {
          constexpr int kPartGroups = 4 >> kPartShift;  // 16 tokens of a part
          const int part = group / kPartGroups;
          const float offset = seen[part] > 0 ? -base : -infinity();
          float2 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            y[i] = fma2(make_float2(x[2 * i], x[2 * i + 1]), row_factor, offset);
          if (cuts) {
            const int left = seen[part] - group % kPartGroups * 16;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              y[i].x = 2 * i < left ? y[i].x : -infinity();
              y[i].y = 2 * i + 1 < left ? y[i].y : -infinity();
            }
          }
          const float high0 =
              max3(max3(y[0].x, y[0].y, y[1].x), y[1].y, max3(y[2].x, y[2].y, y[3].x));
          const float high1 =
              max3(max3(y[3].y, y[4].x, y[4].y), y[5].x, max3(y[5].y, y[6].x, y[6].y));
          high = max3(high, max3(high0, y[7].x, y[7].y), high1);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y[i].x = exp2_fast(y[i].x);
            y[i].y = exp2_fast(y[i].y);
          }
          const float2 sum0 = add2(add2(y[0], y[1]), add2(y[2], y[3]));
          const float2 sum1 = add2(add2(y[4], y[5]), add2(y[6], y[7]));
          sum = add2(sum, add2(sum0, sum1));
#pragma unroll
          for (int i = 0; i < 8; ++i) p[group % 2 * 8 + i] = pack2<true>(y[i].x, y[i].y);
        };
        const auto begin = [&] {
          base = m == -infinity() ? 0.f : m;
          high = -infinity();
          sum = make_float2(0.f, 0.f);
        };
        tensor_load16(from, s[0]);
        tensor_wait(s[0]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // each 16 are on their way while those before them are weighed
          begin();
          tensor_load16(from + half * 32 + 16, s[1]);
          weigh(s[0], half * 2);
          tensor_wait(s[1]);
          if (half == 0) tensor_load16(from + 32, s[0]);
          weigh(s[1], half * 2 + 1);
          const bool raise = high > (m == -infinity() ? m : kMost);
          if (__any_sync(~0u, raise)) {
            some = true;
            float less = 1.f;
            if (raise) {
              if (m == -infinity()) {
                m = high - kRoom;
                less = 0.f;
              } else {
                const float up = floorf(high - kRoom);
                m += up;
                less = exp2_fast(-up);  // a power of two
              }
              l *= less;
              by *= less;
            }
            if (half > 0) scale_probabilities(from, less);
            begin();
            float again[16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              tensor_load16(from + half * 32 + k * 16, again);
              tensor_wait(again);
              weigh(again, half * 2 + k);
            }
          }
          l += sum.x + sum.y;
          if (half == 0) tensor_wait(s[0]);
          tensor_store16(from + half * 16, p);
        }
        tensor_stored();
        if (some && n > 0) {  // O is in place up to the block before
          ok = was_added(n - 1);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          scale_outputs(by);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        barrier_arrive(&sm.weighed[tile][n & 1]);  // a warp may be a block ahead of another
      }
    } else if (warp < kSoftmaxWarps + kConvertWarps) {
      // ---- codes to operands: four warps for keys, four for values ----
      // A warp has 16 tokens of the block, 8 at a time: 4 lanes for a token, a lane with D / 4
      // neighbouring channels. A quarter of the warp has the same channels of 8 tokens, whose
      // swizzled pieces of 16 bytes touch every bank once.
      const bool keys = warp < kSoftmaxWarps + kConvertWarps / 2;
      const uint8_t* const codes = keys ? c.k : c.v;
      const uint8_t* const scales =
          reinterpret_cast<const uint8_t*>(keys ? c.k_scale : c.v_scale);
      uint64_t* const full = keys ? sm.k_full : sm.v_full;
      uint64_t* const free_again = keys ? sm.k_free : sm.v_free;
      const int first = (warp & 3) * 16 + (lane & 7), quarter = lane >> 3;
      uint4 x[2];         // 32 (16) codes of tokens first, first + 8
      uint32_t scale[2];  // and their two scales (one)
      const auto entry_of = [&](int block, int i) -> const Entry& {
        return sm.entry[(block << per_block_shift) + ((first + i * 8) >> part_tokens_shift)];
      };
      // Loads without branches, so that nothing waits for them: of an absent part they take the
      // cache's first page, behind the last block its last one, behind the sequence's end what
      // the page holds; zeros are put for the first and the last.
      const auto load = [&](int block) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Entry& e = entry_of(block < blocks ? block : blocks - 1, i);
          const int in_part = (first + i * 8) & ((1 << part_tokens_shift) - 1);
          const int64_t at = (e.first < 0 ? 0 : e.first) + in_part * D + quarter * (D / 4);
          if constexpr (D == 128) {
            x[i] = __ldg(reinterpret_cast<const uint4*>(codes + at / 2));
            scale[i] = __ldg(reinterpret_cast<const uint16_t*>(scales + at / 16));
          } else {
            const uint2 both = __ldg(reinterpret_cast<const uint2*>(codes + at / 2));
            x[i] = make_uint4(both.x, both.y, 0u, 0u);
            scale[i] = __ldg(scales + at / 16);
          }
        }
      };
      // the line of a lane's channels (of 128: the first or second 64), its first piece there
      const int line = D == 128 ? quarter >> 1 : 0;
      const int piece0 = D == 128 ? (quarter & 1) * 4 : quarter * 2;
      const auto place = [&](uint8_t (&lines)[kLines][kBlock * 128], int i) {
        const uint32_t both = codes_to_half2((uint16_t)scale[i]);
        const uint32_t by[2] = {__byte_perm(both, 0u, 0x1010), __byte_perm(both, 0u, 0x3232)};
        const int token = first + i * 8;
        uint8_t* const to = &lines[line][token * 128];
        constexpr int kPieces = D / 32;
        uint32_t y[kPieces][4];
        codes4_to_half2(x[i].x, y[0]);
        codes4_to_half2(x[i].y, y[1]);
        if constexpr (D == 128) {
          codes4_to_half2(x[i].z, y[2]);
          codes4_to_half2(x[i].w, y[3]);
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
#pragma unroll
          for (int n = 0; n < 4; ++n) y[j][n] = times2(y[j][n], by[j >> 1]);
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
          *reinterpret_cast<uint4*>(to + (((piece0 + j) ^ (token & 7)) << 4)) =
              make_uint4(y[j][0], y[j][1], y[j][2], y[j][3]);
      };
      load(0);
      for (int block = 0; block < blocks; ++block) {
        const int n = done + block, buffer = n & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Entry& e = entry_of(block, i);
          const bool there =
              e.first >= 0 && e.pos + ((first + i * 8) & ((1 << part_tokens_shift) - 1)) < most;
          if (!there) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            scale[i] = 0u;
          }
        }
        if (n >= 2) ok = ok && barrier_wait(&free_again[buffer], ((n >> 1) - 1) & 1, failed);
        if (!ok) break;
        if (keys) {
          place(sm.k[buffer], 0);
          place(sm.k[buffer], 1);
        } else {
          place(sm.v[buffer], 0);
          place(sm.v[buffer], 1);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        barrier_arrive(&full[buffer]);
        load(block + 1);
      }
    } else if (tile < tiles) {
      // ---- products, of scores and of outputs: a warp for each tile ----
      // The waits for operands are the ones whose limit the host sets: once one has run out, the
      // others give up as well.
      const bool leader = elected();
      if (warp < kWarps - kTiles) {
        constexpr uint32_t kScores = 1u << 4 | (kBlock / 8) << 17 | (kRows / 16) << 24;
        constexpr int kLine = kBlock * 128 / 16;  // a line's place in an operand's
        const uint64_t q = operand(shared_address(sm.q[tile][0]));
        const uint64_t k0 = operand(shared_address(sm.k[0][0]));
        for (int block = 0; block < blocks; ++block) {
          const int n = done + block, buffer = n & 1;
          ok = ok && barrier_wait(&sm.k_full[buffer], (n >> 1) & 1, failed, wait_limit);
          if (n >= 2) ok = ok && was_added(n - 2);  // the P that these scores replace has been used
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint64_t k = k0 + buffer * (kLines * kLine);
#pragma unroll
            for (int line = 0; line < kLines; ++line)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                tensor_mma(scores_at + buffer * kBlock, q + line * (kRows * 128 / 16) + 2 * i,
                           k + line * kLine + 2 * i, kScores, line > 0 || i > 0);
            tensor_commit(&sm.scored[tile][buffer]);
            tensor_commit(&sm.k_free[buffer]);
          }
          __syncwarp();
        }
      } else {
        constexpr uint32_t kOutputs = 1u << 4 | 1u << 16 | (D / 8) << 17 | (kRows / 16) << 24;
        const uint64_t v0 = operand_across(shared_address(sm.v[0][0]), kBlock * 128);
        for (int block = 0; block < blocks; ++block) {
          const int n = done + block, buffer = n & 1;
          ok = ok && barrier_wait(&sm.v_full[buffer], (n >> 1) & 1, failed, wait_limit);
          ok = ok && barrier_wait(&sm.weighed[tile][buffer], (n >> 1) & 1, failed);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (leader) {
            const uint64_t v = v0 + buffer * (kLines * kBlock * 128 / 16);
#pragma unroll
            for (int k = 0; k < kBlock / 16; ++k)  // 16 tokens: 8 columns of P, 2 KB of V
              tensor_mma_from(outputs, scores_at + buffer * kBlock + 8 * k, v + 128 * k, kOutputs,
                              n > 0 || k > 0);
            tensor_commit(&sm.added[tile][buffer]);
            tensor_commit(&sm.v_free[buffer]);
          }
          __syncwarp();
        }
      }
    }
    __syncwarp();
    done += blocks;
  }

  // ---- outputs ----
  if (warp < kSoftmaxWarps && tile < tiles) {
    float nan = l;  // NaN among scores, of this row's own or of a part that it does not take
    if (done > 0) {
      ok = ok && was_added(done - 1);
      ok = __all_sync(~0u, ok);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    const float by = l == 0.f ? 0.f : c.v_unit / l;
    uint16_t* const at =
        static_cast<uint16_t*>(a.out.data) + (row0 + row_token) * a.out.token_stride +
        ((int64_t)head * a.group + head0 + row % heads) * a.out.head_stride;
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      float v[32];
      if (done > 0) {
        tensor_load32(outputs + lane_base + i, v);
        tensor_wait(v);
        // a NaN among the values has reached every row by now
#pragma unroll
        for (int k = 0; k < 32; ++k) nan = fmaf(v[k], 0.f, nan);
      }
      if (live && ok) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x = l == 0.f ? 0.f : v[j * 8 + k * 2] * by;
            const float y = l == 0.f ? 0.f : v[j * 8 + k * 2 + 1] * by;
            w[k] = c.fp16 ? pack2<true>(x, y) : pack2<false>(x, y);
          }
          *reinterpret_cast<uint4*>(at + i + j * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (nan != nan) sm.again = 1;
  }
  if (warp >= kSoftmaxWarps + kConvertWarps) {
    // what was issued ends before the shared memory and the tensor memory go
    int none = 0;
    uint64_t* const drained = &sm.drained[warp - (kSoftmaxWarps + kConvertWarps)];
    if (elected()) tensor_commit(drained);
    __syncwarp();
    barrier_wait(drained, 0, &none);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  // tiles that the kernel behind this one has to do
  if (tid < tokens)
    a.again[((row0 + tid) * c.heads + head) * gridDim.z + blockIdx.z] =
        sm.again != 0 || sm.failed != 0;
  if (warp == kWarps - 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor),
                 "r"(kTensorColumns)
                 : "memory");
}

template <int D, int kPartShift>
int launch(const Cache4Args& c, const BatchArgs& b, const AttentionArgs& a, cudaStream_t stream) {
  constexpr size_t most = sizeof(Shared<D>) + 1024 + (size_t)kPairListedWidth * 4;
  static_assert(most <= kMostShared, "every call that is sent here");
  const size_t smem =
      sizeof(Shared<D>) + 1024 + (a.blocks != nullptr ? (size_t)b.width * 4 : 0);
  const auto kernel = prompt_pair_kernel<D, kPartShift>;
  // the largest call's size: the limit is the kernel's, whichever thread launches it
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) !=
      cudaSuccess) {
    cudaGetLastError();
    return EXACT_TOPK_ERR_CUDA;
  }
  const dim3 grid((unsigned)slot_count(b, kTiles * a.prompt_tokens, 1), (unsigned)c.heads,
                  (unsigned)((a.group + a.prompt_heads - 1) / a.prompt_heads));
  kernel<<<grid, kThreads, smem, stream>>>(c, b, a, wait_limit());
  return launch_status();
}

template <int D>
int launch_parts(const Cache4Args& c, const BatchArgs& b, const AttentionArgs& a,
                 cudaStream_t stream) {
  if (c.page == 16) return launch<D, 2>(c, b, a, stream);
  if (c.page == 32) return launch<D, 1>(c, b, a, stream);
  return launch<D, 0>(c, b, a, stream);
}

}  // namespace

int launch_prompt_pair(const Cache4Args& c, const BatchArgs& b, const AttentionArgs& a,
                       cudaStream_t stream) {
  return c.dim == 128 ? launch_parts<128>(c, b, a, stream) : launch_parts<64>(c, b, a, stream);
}

}  // namespace etk
