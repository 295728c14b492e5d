// Attention of many neighbouring tokens over the paged 8-bit cache, on the fifth-generation
// tensor cores (the prompt's form of exact_topk_attention_run).
//
// A CTA's tile is up to 128 rows: tokens x heads of one key head. It goes over the pages that
// any of its tokens takes (all of them, or the union of the tokens' lists) in blocks of 64
// cached tokens, with each row's running maximum m, sum l and output O:
//
//   S = Q K^T          [128 rows][64 tokens], FP32, in tensor memory
//   P = e^(S - m)      in FP16, in tensor memory
//   O += P V           [128 rows][D channels], FP32, in tensor memory
//
// A lane of tensor memory is a row, so a thread has a whole row of S to itself: its
// maximum and sum need no exchange, and a token that does not take a page is a row whose
// probabilities there are zero. Neighbouring tokens of a prompt share most of their
// pages; where they share none, a block costs as much as if they did, which the tensor cores
// still do faster than a kernel that leaves the others out.
//
// Codes are exact in FP16, so four warps turn them into FP16 operands on their way to
// shared memory, while four warps do the softmax of the block before and one thread issues the
// products: two CTAs share an SM, so that one's exponentials fill the other's waits. Values
// are brought to the tile's largest scale by the power of two between (an exact product), so
// O stays in one unit.
//
// Queries, probabilities and the running maximum are as in attention_kernels.cu. Three
// things are left to that kernel, which runs behind this one on the tiles that are marked: a
// NaN among scores or values (which would reach rows that do not see it), scales of values
// more than 2^12 apart, and a wait that ran out.
//
// A block's exponentials are 512 clocks of an SM and its products about as many; what bounds
// it is the latency from scores over softmax to outputs, with two CTAs to fill it. 4096
// tokens x 16 query heads (2 key heads of 128 channels), 32 pages of 64 tokens each, 40 in a
// tile's union: 133 us in a graph (520 TFLOP/s of the products that count), 137 by calls.

#include "cache_device.cuh"
#include "prompt_device.cuh"

namespace etk {
namespace {

constexpr int kRows = 128;           // threads of each role
constexpr int kConvert = 128;
constexpr int kThreads = kRows + kConvert + 32;
constexpr int kIssueWarp = (kRows + kConvert) / 32;
constexpr int kBlock = 64;           // cached tokens of a block
constexpr int kEntries = 128;        // parts of pages held at a time
constexpr float kRoom = 6.f;         // see attention_kernels.cu; with the part of a value's scale
constexpr float kMost = 14.f;        // that is no power of two, below 2, all stays under 2^15
constexpr int kFarthest = 12;        // powers of two between scales of values

// A part of a page: at most 64 tokens.
struct alignas(16) Entry {
  int pos;           // position of its first token
  uint32_t members;  // tokens of the tile that take it; 0 for an absent page
  float k_scale;
  float v_part;      // the values' scale without its power of two
  int64_t offset;    // of its codes; -1 for an absent page
  uint32_t v_power;  // that power of two over the tile's unit, twice in FP16
};

template <int D>
struct Shared {
  uint8_t q[D / 64][kRows * 128];       // lines of 64 channels, in swizzled blocks of 8
  uint8_t k[2][D / 64][kBlock * 128];
  uint8_t v[2][D / 64][kBlock * 128];
  Entry entry[kEntries];
  float factor[kRows];
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t scored[2], weighed[2], added[2], drained;
  uint32_t tensor;
  int scan[kIssueWarp];
  int failed, again, unit, odd;
};

// kPartShift: log2 of the parts of a block (1 of pages of 64 and 128 tokens, 2 of 32, 4 of 16).
// wait_limit stands apart from the other arguments: one field more among them cost 4% of the sparse
// chunk's time by the order that instructions then came in.
// kBits: of a code.
template <int D, int kPartShift, int kBits>
__global__ void __launch_bounds__(kThreads, 2)
    prompt_attention_kernel(typename CacheOf<kBits>::Args c, BatchArgs b, AttentionArgs a,
                            uint32_t wait_limit) {
  using Smem = Shared<D>;
  constexpr int kLines = D / 64;
  // tensor memory: O, then two blocks' S, each of which its P replaces
  constexpr uint32_t kS = 128, kTensorColumns = 256;
  extern __shared__ unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      raw + ((1024u - (shared_address(raw) & 1023u)) & 1023u));
  uint32_t* const marks = reinterpret_cast<uint32_t*>(&sm + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool listed = a.blocks != nullptr;
  const int head = blockIdx.y, head0 = (int)blockIdx.z * a.prompt_heads;
  const int heads = a.group - head0 < a.prompt_heads ? a.group - head0 : a.prompt_heads;
  const int64_t slot = blockIdx.x;
  const int seq = sequence_of_slot(b, slot, a.prompt_tokens, 1);
  const SeqRows rows = sequence_rows(b, c.page_shift, seq);
  const int64_t index = slot - first_slot(b, seq, a.prompt_tokens, 1);
  const int64_t token0 = index * a.prompt_tokens;
  if (index < 0 || token0 >= rows.count) return;
  const int tokens =
      rows.count - token0 < a.prompt_tokens ? (int)(rows.count - token0) : a.prompt_tokens;
  const int64_t row0 = rows.begin + token0;
  const int pos0 = rows.pos0 + (int)token0;
  const int live = tokens * heads;  // rows of the tile
  const int most = pos0 + tokens > 0 ? pos0 + tokens : 0;
  const int pages = (most + c.page - 1) >> c.page_shift;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      barrier_init(&sm.k_full[i], kConvert);
      barrier_init(&sm.v_full[i], kConvert);
      barrier_init(&sm.k_free[i], 1);
      barrier_init(&sm.v_free[i], 1);
      barrier_init(&sm.scored[i], 1);
      barrier_init(&sm.weighed[i], kRows);
      barrier_init(&sm.added[i], 1);
    }
    barrier_init(&sm.drained, 1);
    sm.failed = 0;
    sm.again = 0;
    sm.unit = -1000;
    sm.odd = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     shared_address(&sm.tensor)),
                 "r"(kTensorColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- pages of a list: which tokens of the tile take each ----
  if (listed)
    for (int i = tid; i < pages; i += kThreads) marks[i] = 0u;
  __syncthreads();
  if (listed)
    for (int token = warp; token < tokens; token += kThreads / 32) {
      const int newest = pos0 + token >= 0 ? (pos0 + token) >> c.page_shift : -1;
      const int32_t* const list = a.blocks + ((row0 + token) * c.heads + head) * a.num_blocks;
      for (int i = lane; i < a.num_blocks; i += 32) {
        const int j = __ldg(list + i);
        if (j >= 0 && j <= newest) atomicOr(&marks[j], 1u << token);
      }
    }

  // ---- queries: 8 channels a lane, all of a warp's 16 rows on their way ----
  if (warp < kIssueWarp) {
    constexpr int kLanes = D / 8, kStepRows = 32 / kLanes;  // lanes of a row, rows of a step
    constexpr int kSteps = kRows / kIssueWarp / kStepRows;
    const int piece = lane % kLanes;
    uint4 w[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int row = (warp * kSteps + k) * kStepRows + lane / kLanes;
      const int token = row / heads;
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (row < live)
        w[k] = __ldg(reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q.data) + (row0 + token) * a.q.token_stride +
            ((int64_t)head * a.group + head0 + row - token * heads) * a.q.head_stride +
            piece * 8));
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int row = (warp * kSteps + k) * kStepRows + lane / kLanes;
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
      *reinterpret_cast<uint4*>(
          &sm.q[piece / 8][row * 128 + (((piece & 7) ^ (row & 7)) << 4)]) =
          make_uint4(pack2<true>(x[0].x, x[0].y), pack2<true>(x[1].x, x[1].y),
                     pack2<true>(x[2].x, x[2].y), pack2<true>(x[3].x, x[3].y));
      // NaN where the row has an infinity (see attention_kernels.cu)
      if (piece == 0)
        sm.factor[row] =
            row < live ? __uint_as_float(top == infinity() ? 0x7FFFFFFFu
                                                           : (uint32_t)(127 - up) << 23) *
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
  const int per_thread = (pages + kIssueWarp * 32 - 1) / (kIssueWarp * 32);
  int mine = 0, count = pages;
  if (listed) {
    int have = 0;
    if (warp < kIssueWarp)
      for (int i = tid * per_thread; i < (tid + 1) * per_thread && i < pages; ++i)
        have += marks[i] != 0u;
    int sum = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31 && warp < kIssueWarp) sm.scan[warp] = sum;
    __syncthreads();
    mine = sum - have;
    count = 0;
    for (int w = 0; w < kIssueWarp; ++w) {
      if (w < warp) mine += sm.scan[w];
      count += sm.scan[w];
    }
  }

  // a row's state, kept by its thread
  const int row = tid;
  const int row_token = row < live ? row / heads : 0;
  const int row_pos = row < live ? pos0 + row_token : -1;
  const float row_factor = tid < kRows ? sm.factor[row] : 0.f;
  const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
  float m = -infinity(), l = 0.f;
  int done = 0;  // blocks so far, the same for every role
  bool ok = true;

  // Block n's barriers are those of its parity, so that who waits for one may be a block behind:
  // all that is known of the others then is that block n - 2 is done.
  const auto was_added = [&](int n) {
    return barrier_wait(&sm.added[n & 1], (n >> 1) & 1, failed);
  };

  // O times a factor for each row
  const auto scale_outputs = [&](float by) {
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      float v[32];
      uint32_t w[32];
      tensor_load32(tensor + lane_base + i, v);
      tensor_wait(v);
#pragma unroll
      for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(v[k] * by);
      tensor_store32(tensor + lane_base + i, w);
    }
  };

  for (int chunk0 = 0; chunk0 < (count << part_shift); chunk0 += kEntries) {
    const int left = (count << part_shift) - chunk0;
    const int entries = left < kEntries ? left : kEntries;
    const int blocks = (entries + (1 << per_block_shift) - 1) >> per_block_shift;
    // ---- the chunk's parts of pages ----
    __syncthreads();
    if (listed) {
      if (warp < kIssueWarp) {
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
      }
      __syncthreads();
    }
    int high = -1000;  // the largest power of two among the chunk's scales of values
    for (int i = tid; i < kEntries; i += kThreads) {
      Entry& e = sm.entry[i];
      if (i >= entries) {
        e.offset = -1;
        e.members = 0u;
        e.pos = most;
        e.k_scale = 0.f;
        e.v_part = 1.f;
        e.v_power = 0x3C003C00u;
        continue;
      }
      if (!listed) {
        e.pos = (chunk0 + i) << part_tokens_shift;
        e.members = ~0u;
      }
      const int page = page_of(c, b, seq, e.pos >> c.page_shift);
      e.offset = -1;
      if (page < 0) {
        e.members = 0u;
        e.k_scale = 0.f;
        e.v_part = 1.f;
        e.v_power = 0x3C003C00u;
        continue;
      }
      const int64_t tile = (int64_t)page * c.heads + head;
      e.offset = ((tile << c.page_shift) + (e.pos & (c.page - 1))) * D;
      if constexpr (kBits == 4) {  // scales are part of the operands, and the unit of the outputs
        e.k_scale = e.v_part = 1.f;
        continue;
      }
      e.k_scale = __ldg(c.k_scale + tile);
      const uint32_t v = __float_as_uint(__ldg(c.v_scale + tile));
      e.v_part = __uint_as_float((v & 0x7FFFFFu) | 127u << 23);
      if (e.v_part != 1.f) sm.odd = 1;
      const int power = (int)(v >> 23 & 255u) - 127;
      e.v_power = (uint32_t)power;  // for now
      high = high > power ? high : power;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const int other = __shfl_xor_sync(~0u, high, o);
      high = high > other ? high : other;
    }
    const int unit_before = sm.unit;
    __syncthreads();
    if (lane == 0 && high > unit_before) atomicMax(&sm.unit, high);
    __syncthreads();
    const int unit = sm.unit;
    for (int i = tid; kBits == 8 && i < entries; i += kThreads) {
      Entry& e = sm.entry[i];
      if (e.offset < 0) continue;
      const int below = unit - (int)e.v_power;
      if (below > kFarthest) sm.again = 1;
      const uint32_t half = (uint32_t)(15 - (below > kFarthest ? kFarthest : below)) << 10;
      e.v_power = half | half << 16;
    }
    // O so far is in the unit before
    if (tid < kRows && done > 0 && unit > unit_before) {
      ok = ok && was_added(done - 1);
      ok = __all_sync(~0u, ok);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      scale_outputs(exp2f((float)(unit_before - unit)));
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    __syncthreads();

    const bool odd = sm.odd != 0;
    if (tid < kRows) {
      // ---- softmax: a row a thread ----
      for (int block = 0; block < blocks; ++block) {
        const int n = done + block;
        ok = ok && barrier_wait(&sm.scored[n & 1], (n >> 1) & 1, failed);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t from = tensor + lane_base + kS + (n & 1) * kBlock;
        // A part that this row does not take, and tokens behind its own, have probability 0: an
        // offset of -inf does it for whole parts.
        constexpr int kParts = 1 << kPartShift;
        float scale[kParts], v_part[kParts];
        int seen[kParts];
        bool cuts = false;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          const Entry& e = sm.entry[(block << per_block_shift) + k];
          const bool takes = row_pos >= e.pos && (e.members >> row_token & 1u) != 0u;
          seen[k] = takes ? row_pos + 1 - e.pos : 0;
          scale[k] = row_factor * e.k_scale;
          v_part[k] = e.v_part;
          cuts |= takes && seen[k] < 1 << part_tokens_shift;
        }
        cuts = __any_sync(~0u, cuts);
        // Probabilities under the running maximum, 16 tokens at a time, the next ones' scores on
        // their way. Where a score turns out too far above the maximum, that is raised and
        // the block done again: it is seldom.
        uint32_t p[32];
        float2 sum;
        float by = 1.f;
        bool some = false;
        for (int attempt = 0; attempt < 2; ++attempt) {
          const float base = m == -infinity() ? 0.f : m;
          float high = -infinity();
          sum = make_float2(0.f, 0.f);
          float s[2][16];
          tensor_load16(from, s[0]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            constexpr int kPartGroups = 4 >> kPartShift;  // 16 tokens of a part
            const int part = k / kPartGroups;
            const float(&x)[16] = s[k & 1];
            tensor_wait(s[k & 1]);
            if (k < 3) tensor_load16(from + (k + 1) * 16, s[(k + 1) & 1]);
            const float offset = seen[part] > 0 ? -base : -infinity();
            float2 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y[i] = fma2(make_float2(x[2 * i], x[2 * i + 1]), scale[part], offset);
            if (cuts) {
              const int left = seen[part] - k % kPartGroups * 16;
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
            if (odd) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                y[i].x *= v_part[part];
                y[i].y *= v_part[part];
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) p[k * 8 + i] = pack2<true>(y[i].x, y[i].y);
          }
          const bool raise = high > (m == -infinity() ? m : kMost);
          if (!__any_sync(~0u, raise)) break;
          some = true;
          if (raise) {
            const float best = base + high - kRoom;
            by = m == -infinity() ? 0.f : exp2_fast(m - best);
            m = best;
            l *= by;
          }
        }
        l += sum.x + sum.y;
        if (some && n > 0) {  // O is in place up to the block before
          ok = was_added(n - 1);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          scale_outputs(by);
        }
        tensor_store32(from, p);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        barrier_arrive(&sm.weighed[n & 1]);  // a warp may be a block ahead of another
      }
    } else if (tid < kRows + kConvert) {
      // ---- codes to operands ----
      // A warp has 16 tokens of the block, 8 at a time: 4 lanes with 16 codes each for a line of 64
      // channels. Of a token's line they write every other piece of 16 bytes, of an odd token's
      // the other ones, so that a quarter of a warp touches every bank once.
      const int first = (warp - kRows / 32) * 16 + (lane >> 2), chunk = lane & 3;
      // tokens first, first + 8; 4-bit codes with their scale in the third word
      uint4 k[2][kLines], v[2][kLines];
      const auto entry_of = [&](int block, int i) -> const Entry& {
        return sm.entry[(block << per_block_shift) + ((first + i * 8) >> part_tokens_shift)];
      };
      // Loads without branches, so that nothing waits for them: of an absent part they take the
      // cache's first page, behind the last block its last one, behind the sequence's end what
      // the page holds. `clear` puts zeros for the first and the last.
      const auto load = [&](int block, const uint8_t* codes, const float* scales,
                            uint4 (&x)[2][kLines]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Entry& e = entry_of(block < blocks ? block : blocks - 1, i);
          const int in_part = (first + i * 8) & ((1 << part_tokens_shift) - 1);
          const int64_t at = (e.offset < 0 ? 0 : e.offset) + in_part * D + chunk * 16;
#pragma unroll
          for (int line = 0; line < kLines; ++line) {
            if constexpr (kBits == 8) {
              x[i][line] = __ldg(reinterpret_cast<const uint4*>(codes + at + line * 64));
            } else {
              const int64_t group = at / 16 + line * 4;
              const uint2 both = __ldg(reinterpret_cast<const uint2*>(codes + group * 8));
              x[i][line] = make_uint4(
                  both.x, both.y, __ldg(reinterpret_cast<const uint8_t*>(scales) + group), 0u);
            }
          }
        }
      };
      const auto there = [&](int block, int i) {
        const Entry& e = entry_of(block, i);
        return e.offset >= 0 && e.pos + ((first + i * 8) & ((1 << part_tokens_shift) - 1)) < most;
      };
      // Zeros for what is not there; most blocks have everything. Lanes part ways here without a
      // vote: where a wait runs out, it may do so for some of a warp's lanes alone.
      const auto clear = [&](int block, uint4 (&x)[2][kLines]) {
        const bool in_place[2] = {there(block, 0), there(block, 1)};
        if (in_place[0] && in_place[1]) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (!in_place[i])
#pragma unroll
            for (int line = 0; line < kLines; ++line) x[i][line] = make_uint4(0u, 0u, 0u, 0u);
      };
      const int place0 = first * 128 + (((chunk * 2) ^ (first & 7)) << 4);  // + 8 tokens: 1024
      const auto place = [&](uint8_t (&lines)[kLines][kBlock * 128], int i,
                             const uint4 (&x)[kLines], uint32_t power) {
#pragma unroll
        for (int line = 0; line < kLines; ++line) {
          uint32_t y[8];
          if constexpr (kBits == 4) {
            uint32_t z[2][4];
            codes4_to_half2(x[line].x, z[0]);
            codes4_to_half2(x[line].y, z[1]);
            const uint32_t by = scale_to_half2(x[line].z);
#pragma unroll
            for (int n = 0; n < 8; ++n) y[n] = times2(z[n >> 2][n & 3], by);
          } else {
            const uint32_t w[4] = {x[line].x, x[line].y, x[line].z, x[line].w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              y[2 * n] = codes_to_half2((uint16_t)w[n]);
              y[2 * n + 1] = codes_to_half2((uint16_t)(w[n] >> 16));
            }
          }
          if (kBits == 8 && power != 0x3C003C00u) {
            const __half2 by = *reinterpret_cast<const __half2*>(&power);
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&y[n]), by);
              y[n] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          uint8_t* const to = &lines[line][0];
          *reinterpret_cast<uint4*>(to + place0 + i * 1024) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(to + (place0 ^ 16) + i * 1024) =
              make_uint4(y[4], y[5], y[6], y[7]);
        }
      };
      const auto keys = [&](int block) {
        const int n = done + block, buffer = n & 1;
        if (n >= 2) ok = ok && barrier_wait(&sm.k_free[buffer], ((n >> 1) - 1) & 1, failed);
        if (!ok) return;
        clear(block, k);
#pragma unroll
        for (int i = 0; i < 2; ++i) place(sm.k[buffer], i, k[i], 0x3C003C00u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        barrier_arrive(&sm.k_full[buffer]);
        load(block + 1, c.k, c.k_scale, k);
      };
      load(0, c.k, c.k_scale, k);
      load(0, c.v, c.v_scale, v);
      keys(0);
      for (int block = 0; block < blocks; ++block) {
        // keys are a block ahead: their place is free as soon as the scores are there, the
        // values' not before the probabilities have been used
        if (block + 1 < blocks) keys(block + 1);
        const int n = done + block, buffer = n & 1;
        if (n >= 2) ok = ok && barrier_wait(&sm.v_free[buffer], ((n >> 1) - 1) & 1, failed);
        if (!ok) break;
        clear(block, v);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          place(sm.v[buffer], i, v[i], kBits == 8 ? entry_of(block, i).v_power : 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        barrier_arrive(&sm.v_full[buffer]);
        load(block + 1, c.v, c.v_scale, v);
      }
    } else {
      // ---- products ----
      // The waits for operands are the ones whose limit the host sets: once one has run out, the
      // others give up as well.
      const bool leader = elected();
      constexpr uint32_t kScores = 1u << 4 | (kBlock / 8) << 17 | (kRows / 16) << 24;
      constexpr uint32_t kOutputs = 1u << 4 | 1u << 16 | (D / 8) << 17 | (kRows / 16) << 24;
      const auto scores = [&](int block) {
        const int n = done + block, buffer = n & 1;
        ok = ok && barrier_wait(&sm.k_full[buffer], (n >> 1) & 1, failed, wait_limit);
        // the P that these scores replace has been used; a chunk's first block waits for all
        const int used = block == 0 ? n - 1 : n - 2;
        if (used >= 0) ok = ok && was_added(used);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (leader) {
#pragma unroll
          for (int line = 0; line < kLines; ++line) {
            const uint64_t q = operand(shared_address(sm.q[line]));
            const uint64_t k = operand(shared_address(sm.k[buffer][line]));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tensor_mma(tensor + kS + buffer * kBlock, q + 2 * i, k + 2 * i, kScores,
                         line > 0 || i > 0);
          }
          tensor_commit(&sm.k_free[buffer]);
          tensor_commit(&sm.scored[buffer]);
        }
        __syncwarp();
      };
      scores(0);
      if (blocks > 1) scores(1);
      for (int block = 0; block < blocks && ok; ++block) {
        const int n = done + block, buffer = n & 1;
        ok = barrier_wait(&sm.v_full[buffer], (n >> 1) & 1, failed, wait_limit);
        ok = ok && barrier_wait(&sm.weighed[buffer], (n >> 1) & 1, failed);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (leader) {
          const uint64_t v = operand_across(shared_address(sm.v[buffer][0]), kBlock * 128);
#pragma unroll
          for (int k = 0; k < kBlock / 16; ++k)  // 16 tokens: 8 columns of P, 2 KB of V
            tensor_mma_from(tensor, tensor + kS + buffer * kBlock + 8 * k, v + 128 * k, kOutputs,
                            n > 0 || k > 0);
          tensor_commit(&sm.v_free[buffer]);
          tensor_commit(&sm.added[buffer]);
        }
        __syncwarp();
        if (block + 2 < blocks) scores(block + 2);
      }
    }
    __syncwarp();
    done += blocks;
  }

  // ---- outputs ----
  if (tid < kRows) {
    float nan = l;  // NaN among scores, of this row's own or of a part that it does not take
    if (done > 0) {
      ok = ok && was_added(done - 1);
      ok = __all_sync(~0u, ok);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    float by = l == 0.f ? 0.f : 1.f / l;
    if constexpr (kBits == 4)
      by *= c.v_unit;
    else
      by = l == 0.f ? 0.f : exp2f((float)(done > 0 ? sm.unit : 0)) / l;
    uint16_t* const at =
        static_cast<uint16_t*>(a.out.data) + (row0 + row_token) * a.out.token_stride +
        ((int64_t)head * a.group + head0 + row - row_token * heads) * a.out.head_stride;
#pragma unroll 1
    for (int i = 0; i < D; i += 32) {
      float v[32];
      if (done > 0) {
        tensor_load32(tensor + lane_base + i, v);
        tensor_wait(v);
        // a NaN among the values has reached every row by now
#pragma unroll
        for (int k = 0; k < 32; ++k) nan = fmaf(v[k], 0.f, nan);
      }
      if (row < live && ok) {
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
  if (warp == kIssueWarp) {
    // what was issued ends before the shared memory and the tensor memory go
    int none = 0;
    if (elected()) tensor_commit(&sm.drained);
    __syncwarp();
    barrier_wait(&sm.drained, 0, &none);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  // tiles that the kernel behind this one has to do
  if (tid < tokens)
    a.again[((row0 + tid) * c.heads + head) * gridDim.z + blockIdx.z] =
        sm.again != 0 || sm.failed != 0;
  if (warp == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tensor),
                 "r"(kTensorColumns)
                 : "memory");
}

template <int D, int kPartShift, int kBits>
int launch(const typename CacheOf<kBits>::Args& c, const BatchArgs& b, const AttentionArgs& a,
           cudaStream_t stream) {
  constexpr size_t most = sizeof(Shared<D>) + 1024 + (size_t)kPromptListedWidth * 4;
  static_assert(most <= kMostShared, "every call that the checks let through");
  const size_t smem =
      sizeof(Shared<D>) + 1024 + (a.blocks != nullptr ? (size_t)b.width * 4 : 0);
  const auto kernel = prompt_attention_kernel<D, kPartShift, kBits>;
  // the largest call's size: the limit is the kernel's, whichever thread launches it
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) !=
      cudaSuccess) {
    cudaGetLastError();
    return EXACT_TOPK_ERR_CUDA;
  }
  const dim3 grid((unsigned)slot_count(b, a.prompt_tokens, 1), (unsigned)c.heads,
                  (unsigned)((a.group + a.prompt_heads - 1) / a.prompt_heads));
  kernel<<<grid, kThreads, smem, stream>>>(c, b, a, wait_limit());
  return launch_status();
}

template <int D, int kBits>
int launch_parts(const typename CacheOf<kBits>::Args& c, const BatchArgs& b,
                 const AttentionArgs& a, cudaStream_t stream) {
  if (c.page == 16) return launch<D, 2, kBits>(c, b, a, stream);
  if (c.page == 32) return launch<D, 1, kBits>(c, b, a, stream);
  return launch<D, 0, kBits>(c, b, a, stream);
}

}  // namespace

int launch_prompt_attention(const CacheArgs& c, const BatchArgs& b, const AttentionArgs& a,
                            cudaStream_t stream) {
  return c.dim == 128 ? launch_parts<128, 8>(c, b, a, stream)
                      : launch_parts<64, 8>(c, b, a, stream);
}

int launch_prompt_attention4(const Cache4Args& c, const BatchArgs& b, const AttentionArgs& a,
                             cudaStream_t stream) {
  return c.dim == 128 ? launch_parts<128, 4>(c, b, a, stream)
                      : launch_parts<64, 4>(c, b, a, stream);
}

}  // namespace etk
