// Attention over the paged 8-bit cache (exact_topk_attention_run): a row's
// running maximum m, sum l and output O, in FP32, over its pages in one pass,
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
// the 8 columns of m16n8k16. The order of a contraction is free, so fragments
// come from global memory in 16-byte pieces with no shared memory between: for
// the first product each lane holds 32 (16) channels of two tokens, for the second 16 (8)
// channels of four tokens, whose codes are paired by byte permutes before they are
// converted. S^T's accumulators, packed to halves and transposed in registers, are
// P^T's fragments.
//
// Types. Codes are exact in FP16, so both products run in FP16 with FP32 sums. A
// query row is brought to [2^8, 2^9) by a power of two: what is then below FP16's
// normal range is off by 2^-25, against 2^8, less than FP32's own rounding of
// the sum. Probabilities are at most 2^8 in FP16 (11 bits, against the 8 or 11 of
// the output).
//
// Work. All pages of all tiles form one line that the CTAs cut into equal parts,
// whatever the lengths; a CTA's part may cover several tiles. Inside a CTA
// each warp takes 32 tokens at a time, and its four warps' results are joined through
// shared memory. A tile that several CTAs share is joined from their partial results
// by the last of them to arrive, in the order of their parts, so that results do not
// depend on timing.

#include <climits>

#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 128;   // pages whose ids are held in shared memory at a time
constexpr int kStep = 16;     // tokens of a matrix instruction
// The running maximum is raised only when a score is more than this above it (in
// powers of two): probabilities then reach 2^8, and the sums are rescaled a few
// times in a row's life instead of at each step.
constexpr float kSlack = 8.f;

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

// Sequence b's tiles and the units (pages) of each.
__device__ __forceinline__ void tile_shape(const AttentionArgs& a, const CacheArgs& c,
                                           const SeqRows& s, int64_t* tiles, int* units) {
  const int splits = (a.group + a.tile_heads - 1) / a.tile_heads;
  *tiles = (int64_t)((s.count + a.tile_tokens - 1) / a.tile_tokens) * c.heads * splits;
  const int pages = (s.len + c.page - 1) >> c.page_shift;
  const int n = a.blocks != nullptr ? a.num_blocks : pages;
  *units = n > 0 ? n : 1;
}

// Steps of 16 tokens that a warp holds in shared memory, all but one of them on their
// way: 40 to 48 KB of a CTA where four share an SM, more where fewer do.
constexpr int ring_steps(int dim, int tiles) {
  const int ctas = attention_ctas_per_sm(tiles * 8, dim);
  return dim == 128 ? (ctas == 4 ? 3 : (ctas == 3 ? 4 : 5)) : (ctas == 4 ? 5 : 8);
}

template <int D, int NT>
struct alignas(128) Shared {
  static constexpr int kRegs = D / 16 * NT * 4;  // output registers of a lane
  static constexpr int kRow = D + 8;             // halves of a query row, padded by 16 bytes
  static constexpr int kRing = ring_steps(D, NT);
  union {
    uint8_t ring[kWarps][kRing][2][kStep * D];  // codes of keys and values
    float out[kWarps][kRegs][32];               // after the last step
  };
  float stat[kWarps][NT * 4][32];  // m and l of a lane's two columns of every 8
  __half q[NT * 8][kRow];
  float factor[NT * 8];
  int page[kChunk];
  uint32_t entry[kChunk];          // place in the sequence | members << 24
  float2 scale[kChunk];            // of keys and values
  int scan[kWarps];
  int last;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, attention_ctas_per_sm(NT * 8, D))
    attention_kernel(CacheArgs c, BatchArgs b, AttentionArgs a) {
  constexpr int kTiles = D / 16;    // channel tiles of the output
  constexpr int kHalf = D / 64;     // 64-byte parts of a token's codes
  // query fragments in registers where there is room; else read at each step
  constexpr bool kHoldQ = D * NT <= 128;
  using Smem = Shared<D, NT>;
  extern __shared__ __align__(16) unsigned char raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  // behind it: prefix sums of the sequences' units, then the members of each page (listed pages)
  int64_t* const prefix = reinterpret_cast<int64_t*>(raw + sizeof(Smem));
  uint32_t* const marks = reinterpret_cast<uint32_t*>(prefix + b.num_seqs + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q4 = lane & 3;
  const bool listed = a.blocks != nullptr;

  // ---- the line of units ----
  {
    int64_t carry = 0;
    for (int base = 0; base < b.num_seqs; base += kThreads) {
      int64_t mine = 0;
      if (base + tid < b.num_seqs) {
        int64_t tiles;
        int units;
        tile_shape(a, c, sequence_rows(b, c.page_shift, base + tid), &tiles, &units);
        mine = tiles * units;
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
      for (int w = 0; w < warp; ++w) before += totals[w];
      if (base + tid < b.num_seqs) prefix[base + tid + 1] = before + sum;
      for (int w = 0; w < kWarps; ++w) carry += totals[w];
      __syncthreads();
    }
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
  }
  const int64_t total = prefix[b.num_seqs];
  int64_t part = (total + a.workers - 1) / a.workers;
  if (part < a.min_units) part = a.min_units;
  const int64_t line_end = (blockIdx.x + 1) * part < total ? (blockIdx.x + 1) * part : total;

  for (int64_t u = blockIdx.x * part; u < line_end;) {
    // ---- the tile that unit u belongs to ----
    Tile t;
    {
      int lo = 0, hi = b.num_seqs - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid + 1] > u)
          hi = mid;
        else
          lo = mid + 1;
      }
      const SeqRows s = sequence_rows(b, c.page_shift, lo);
      int64_t tiles;
      tile_shape(a, c, s, &tiles, &t.units);
      const int64_t index = (u - prefix[lo]) / t.units;
      t.start = prefix[lo] + index * t.units;
      const int splits = (a.group + a.tile_heads - 1) / a.tile_heads;
      const int split = (int)(index % splits);
      const int64_t rest = index / splits;
      t.seq = lo;
      t.head = (int)(rest % c.heads);
      const int64_t token0 = rest / c.heads * a.tile_tokens;
      t.tokens = s.count - token0 < a.tile_tokens ? (int)(s.count - token0) : a.tile_tokens;
      t.row0 = s.begin + token0;
      t.pos0 = s.pos0 + (int)token0;
      t.head0 = split * a.tile_heads;
      t.heads = a.group - t.head0 < a.tile_heads ? a.group - t.head0 : a.tile_heads;
    }
    const int64_t u_end = line_end < t.start + t.units ? line_end : t.start + t.units;
    const int columns = t.tokens * t.heads;
    // tokens of the cache that the tile's last and first token see
    const int most = t.pos0 + t.tokens > 0 ? t.pos0 + t.tokens : 0;
    const int least = t.pos0 + 1 > 0 ? t.pos0 + 1 : 0;
    const int pages = (most + c.page - 1) >> c.page_shift;

    // ---- queries: one column a warp at a time ----
    for (int col = warp; col < NT * 8; col += kWarps) {
      float2 x[D / 64];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) x[i] = make_float2(0.f, 0.f);
      if (col < columns) {
        const uint16_t* const at =
            static_cast<const uint16_t*>(a.q.data) +
            (t.row0 + col / t.heads) * a.q.token_stride +
            ((int64_t)t.head * a.group + t.head0 + col % t.heads) * a.q.head_stride;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(at + i * 64 + lane * 2);
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

    // ---- pages of a list: which tokens of the tile take each ----
    int count = 0;       // entries of the tile
    int mine = 0;        // entries before this thread's words
    const int words = (pages + 3) >> 2;
    const int per_thread = (words + kThreads - 1) / kThreads;
    if (listed) {
      for (int i = tid; i < words; i += kThreads) marks[i] = 0u;
      __syncthreads();
      for (int i = tid; i < t.tokens * a.num_blocks; i += kThreads) {
        const int token = i / a.num_blocks;
        const int pos = t.pos0 + token;
        const int j = a.blocks[((t.row0 + token) * c.heads + t.head) * a.num_blocks +
                               i % a.num_blocks];
        if (pos >= 0 && j >= 0 && j <= pos >> c.page_shift)
          atomicOr(&marks[j >> 2], 1u << ((j & 3) * 8 + token));
      }
      __syncthreads();
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
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) mine += sm.scan[w];
        count += sm.scan[w];
      }
    }
    // this CTA's entries of the tile
    int from, to;
    if (listed) {
      from = (int)((int64_t)count * (u - t.start) / t.units);
      to = (int)((int64_t)count * (u_end - t.start) / t.units);
    } else {
      from = (int)(u - t.start);
      to = (int)(u_end - t.start);
      from = from < pages ? from : pages;
      to = to < pages ? to : pages;
    }
    __syncthreads();  // queries are in place

    // ---- a lane's columns ----
    float m[NT][2], l[NT][2], o[kTiles][NT][4];
    uint32_t shift[NT][2], have[NT];  // token of a column; tokens of each 8 columns
    uint4 held[kHoldQ ? NT : 1][kHalf][2];  // query fragments
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      have[n] = 0u;
      for (int i = 0; i < 8; ++i)
        if (n * 8 + i < columns) have[n] |= 1u << ((n * 8 + i) / t.heads);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = n * 8 + q4 * 2 + j;
        const int token = col / t.heads;
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
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[i][n][r] = 0.f;
    }
    const uint32_t everyone = (1u << t.tokens) - 1u;
    float unit = 1.f;  // the values' scale that o is held in

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sm.ring[warp][0][0][0]);
    // steps of 16 tokens: a warp takes two in a row (a page of 16 has one)
    const int pair_shift = c.page >= 32 ? 1 : 0;
    const int sub_shift = c.page_shift - 4 - pair_shift;  // log2 of (pairs of) steps a page

    for (int chunk0 = from; chunk0 < to; chunk0 += kChunk) {
      const int entries = to - chunk0 < kChunk ? to - chunk0 : kChunk;
      // ---- ids of the chunk's pages ----
      if (chunk0 > from) __syncthreads();
      if (listed) {
        int at = mine;
        for (int i = tid * per_thread; i < (tid + 1) * per_thread && i < words; ++i) {
          const uint32_t w = marks[i];
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
        sm.page[i] = page;
        if (!listed) sm.entry[i] = (uint32_t)place;
        if (page >= 0) {
          const int64_t tile = (int64_t)page * c.heads + t.head;
          sm.scale[i] = make_float2(__ldg(c.k_scale + tile), __ldg(c.v_scale + tile));
        }
      }
      __syncthreads();

      const int subs = entries << sub_shift;
      const int steps = warp < subs ? ((subs - warp + kWarps - 1) / kWarps) << pair_shift : 0;

      // Step i of this warp: its entry, and its first row in the page.
      const auto find = [&](int i, int* e, int* row0) {
        const int sub = warp + (i >> pair_shift) * kWarps;
        *e = sub >> sub_shift;
        *row0 = ((sub & ((1 << sub_shift) - 1)) << (4 + pair_shift)) +
                ((i & ((1 << pair_shift) - 1)) << 4);
      };
      const auto position = [&](int e, int row0) {
        const int place = listed ? (int)(sm.entry[e] & 0xFFFFFFu) : (int)sm.entry[e];
        return (place << c.page_shift) + row0;
      };

      // Codes of step i into its place of the ring. A step is contiguous in memory. In
      // shared memory its 16-byte pieces are exchanged within lines of 128 bytes so
      // that the reads below touch every bank once.
      const auto fetch = [&](int i, int place_in_ring) {
        if (i < steps) {
          int e, row0;
          find(i, &e, &row0);
          const int page = sm.page[e];
          const int rows = most - position(e, row0);  // tokens that anyone sees
          if (page >= 0 && rows > 0) {
            const int64_t at =
                (((int64_t)page * c.heads + t.head) * c.page + row0) * D + lane * 16;
            const uint32_t to = ring + place_in_ring * (2 * kStep * D);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              const int piece = lane + 32 * j, line = piece >> 3, p = piece & 7;
              const bool there = (D == 128 ? line : piece >> 2) < rows;
              const int pk = D == 128 ? p ^ ((line & 1) << 2) : p;
              const int pv = D == 128 ? p ^ ((line >> 1 & 3) << 1) : p ^ ((line & 3) << 1);
              copy16(to + line * 128 + pk * 16, c.k + at + j * 512, there);
              copy16(to + kStep * D + line * 128 + pv * 16, c.v + at + j * 512, there);
            }
          }
        }
        copy_commit();
      };

      const auto compute = [&](int i, int place_in_ring) {
        int e, row0;
        find(i, &e, &row0);
        const int pos = position(e, row0);
        if (sm.page[e] < 0 || pos >= most) return;
        const uint32_t members = listed ? sm.entry[e] >> 24 : everyone;
        const float2 scale = sm.scale[e];
        const uint8_t* const codes = &sm.ring[warp][place_in_ring][0][0];
        // Eight columns of which no token takes the page are left out. Where some do and
        // some do not, or the step ends beyond a token, scores are masked.
        bool takes[NT];
        bool masked = pos + kStep > least;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          takes[n] = NT == 1 || (members & have[n]) != 0u;
          masked |= takes[n] && (members & have[n]) != have[n];
        }

        // ---- S^T ----
        float x[NT][4];
        {
          uint32_t a[D / 16][4];
#pragma unroll
          for (int p = 0; p < kHalf; ++p) {
            uint4 w[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int row = g + 8 * r;
              w[r] = *reinterpret_cast<const uint4*>(
                  codes + row * D + (D == 128 ? (p * 4 + q4) ^ ((row & 1) << 2) : q4) * 16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w0 = word(w[0], k), w1 = word(w[1], k);
              a[p * 4 + k][0] = codes_to_half2((uint16_t)w0);
              a[p * 4 + k][2] = codes_to_half2((uint16_t)(w0 >> 16));
              a[p * 4 + k][1] = codes_to_half2((uint16_t)w1);
              a[p * 4 + k][3] = codes_to_half2((uint16_t)(w1 >> 16));
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (!takes[n]) continue;
            float other[4] = {0.f, 0.f, 0.f, 0.f};  // two sums, for shorter chains
#pragma unroll
            for (int r = 0; r < 4; ++r) x[n][r] = 0.f;
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
                const uint32_t(&a0)[4] = a[p * 4 + k * 2];
                const uint32_t(&a1)[4] = a[p * 4 + k * 2 + 1];
                mma(x[n], a0[0], a0[1], a0[2], a0[3], q.x, q.y);
                mma(other, a1[0], a1[1], a1[2], a1[3], q.z, q.w);
              }
#pragma unroll
            for (int r = 0; r < 4; ++r) x[n][r] += other[r];
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
        uint32_t pt[NT][2];
        uint32_t seen = 0u;  // 4 bits for each 8 columns: this lane's scores that count
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (!takes[n]) continue;
          const float2 factor = *reinterpret_cast<const float2*>(&sm.factor[n * 8 + q4 * 2]);
          float y[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[n][r] *= (r & 1 ? factor.y : factor.x) * scale.x;
            y[r] = x[n][r] - m[n][r & 1];
          }
          if (masked) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t token = shift[n][r & 1];
              if (pos + g + (r >> 1) * 8 > t.pos0 + (int)token || (members >> token & 1u) == 0u)
                x[n][r] = y[r] = -infinity();
              else
                seen |= 1u << (n * 4 + r);
            }
          }
          const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
          if (__any_sync(~0u, top > kSlack)) {
            float by[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float high = fmaxf(fmaxf(x[n][j], x[n][j + 2]), m[n][j]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1)
                high = fmaxf(high, __shfl_xor_sync(~0u, high, d));
              by[j] = m[n][j] == -infinity() ? 0.f : exp2_fast(m[n][j] - high);
              m[n][j] = high;
              l[n][j] *= by[j];
            }
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
#pragma unroll
              for (int r = 0; r < 4; ++r) o[k][n][r] *= by[r & 1];
            // a masked score stays -inf, also where its column has seen nothing yet
#pragma unroll
            for (int r = 0; r < 4; ++r)
              y[r] = x[n][r] == -infinity() ? x[n][r] : x[n][r] - m[n][r & 1];
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            y[r] = exp2_fast(y[r]);
            l[n][r & 1] += y[r];
          }
          pt[n][0] = transpose8(pack2<true>(y[0], y[1]));
          pt[n][1] = transpose8(pack2<true>(y[2], y[3]));
        }

        // ---- values: tokens 2c, 2c+1, 2c+8, 2c+9 of 16 (8) channels ----
        uint4 v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = q4 * 2 + (r & 1) + (r >> 1) * 8;
          const uint8_t* const at = codes + kStep * D;
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
              const uint32_t bits = seen >> (n * 4);
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
          uint32_t a[kPart][4];
#pragma unroll
          for (int k = 0; k < kPart; ++k) {
            const int tile = half * kPart + k;
            const uint32_t w0 = __byte_perm(word(v[0], tile >> 1), word(v[1], tile >> 1),
                                            tile & 1 ? 0x7362 : 0x5140);
            const uint32_t w1 = __byte_perm(word(v[2], tile >> 1), word(v[3], tile >> 1),
                                            tile & 1 ? 0x7362 : 0x5140);
            a[k][0] = codes_to_half2((uint16_t)w0);
            a[k][1] = codes_to_half2((uint16_t)(w0 >> 16));
            a[k][2] = codes_to_half2((uint16_t)w1);
            a[k][3] = codes_to_half2((uint16_t)(w1 >> 16));
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (!takes[n]) continue;
#pragma unroll
            for (int k = 0; k < kPart; ++k)
              mma(o[half * kPart + k][n], a[k][0], a[k][1], a[k][2], a[k][3], pt[n][0],
                  pt[n][1]);
          }
        }
      };

      for (int i = 0; i < Smem::kRing - 1; ++i) fetch(i, i);
      int now = 0, behind = Smem::kRing - 1;
      for (int i = 0; i < steps; ++i) {
        copy_wait<Smem::kRing - 2>();
        __syncwarp();
        compute(i, now);
        __syncwarp();
        fetch(i + Smem::kRing - 1, behind);
        behind = now;
        now = now + 1 == Smem::kRing ? 0 : now + 1;
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
        sm.stat[warp][n * 4 + j][lane] = m[n][j];
        sm.stat[warp][n * 4 + 2 + j][lane] = l[n][j];
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float top = -infinity();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.stat[w][n * 4 + j][lane]);
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
          sum += sm.stat[w][n * 4 + 2 + j][lane] * exp2_fast(sm.stat[w][n * 4 + j][lane] - base);
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
    bool write = true;
    const int first_cta = (int)(t.start / part);
    const int last_cta = (int)((t.start + t.units - 1) / part);
    if (first_cta != last_cta) {
      constexpr int64_t kFloats = partial_floats(NT * 8, D);
      // a CTA's first slot holds the tile it continues, its second the tile it starts
      float* const at = a.partial +
                        ((int64_t)blockIdx.x * 2 + (first_cta == (int)blockIdx.x)) * kFloats;
      if (warp == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            at[(n * 4 + j) * 32 + lane] = m[n][j];
            at[(n * 4 + 2 + j) * 32 + lane] = l[n][j];
          }
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            at[NT * 128 + (((warp * kOwn + i) * NT + n) * 4 + k) * 32 + lane] = r[i][n][k];
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int arrived = atomicAdd(a.counters + first_cta, 1);
        sm.last = arrived == last_cta - first_cta;
        if (sm.last) a.counters[first_cta] = 0;
      }
      __syncthreads();
      write = sm.last != 0;
      if (write) {
        __threadfence();
        const auto slot = [&](int cta) {
          return a.partial + ((int64_t)cta * 2 + (cta == first_cta)) * kFloats;
        };
        float top[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[n][j] = -infinity();
            l[n][j] = 0.f;
          }
#pragma unroll 4
        for (int cta = first_cta; cta <= last_cta; ++cta) {
          const float* const p = slot(cta);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              top[n][j] = fmaxf(top[n][j], __ldcg(p + (n * 4 + j) * 32 + lane));
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) r[i][n][k] = 0.f;
#pragma unroll 2
        for (int cta = first_cta; cta <= last_cta; ++cta) {
          const float* const p = slot(cta);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float base = top[n][j] == -infinity() ? 0.f : top[n][j];
              const float by = exp2_fast(__ldcg(p + (n * 4 + j) * 32 + lane) - base);
              l[n][j] += __ldcg(p + (n * 4 + 2 + j) * 32 + lane) * by;
#pragma unroll
              for (int i = 0; i < kOwn; ++i)
#pragma unroll
                for (int k = j; k < 4; k += 2)
                  r[i][n][k] +=
                      __ldcg(p + NT * 128 + (((warp * kOwn + i) * NT + n) * 4 + k) * 32 + lane) *
                      by;
            }
        }
      }
    }

    // ---- write: a lane has 4 * kOwn / 2 neighbouring channels of its columns ----
    if (write) {
      constexpr int kLaneChannels = D / 8;  // channels of lane / 4: 2 of each channel tile
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = n * 8 + q4 * 2 + j;
          if (col >= columns) continue;
          const float by = l[n][j] == 0.f ? 0.f : 1.f / l[n][j];
          uint16_t* const at =
              static_cast<uint16_t*>(a.out.data) +
              (t.row0 + col / t.heads) * a.out.token_stride +
              ((int64_t)t.head * a.group + t.head0 + col % t.heads) * a.out.head_stride +
              g * kLaneChannels + warp * kOwn * 2;
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const float y0 = l[n][j] == 0.f ? 0.f : r[i][n][j] * by;
            const float y1 = l[n][j] == 0.f ? 0.f : r[i][n][2 + j] * by;
            *reinterpret_cast<uint32_t*>(at + i * 2) =
                c.fp16 ? pack2<true>(y0, y1) : pack2<false>(y0, y1);
          }
        }
    }
    u = u_end;
    __syncthreads();  // shared memory is free for the next tile
  }
}

template <int D, int NT>
int launch_tile(const CacheArgs& c, const BatchArgs& b, const AttentionArgs& a,
                cudaStream_t stream) {
  const size_t smem = sizeof(Shared<D, NT>) + sizeof(int64_t) * ((size_t)b.num_seqs + 1) +
                      (a.blocks != nullptr ? ((size_t)b.width + 3) / 4 * 4 : 0);
  // Set on every call: a host-side table entry, cheaper than remembering it per device.
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess) {
    cudaGetLastError();
    return EXACT_TOPK_ERR_CUDA;
  }
  attention_kernel<D, NT><<<a.workers, kThreads, smem, stream>>>(c, b, a);
  return launch_status();
}

}  // namespace

int launch_attention(const CacheArgs& c, const BatchArgs& b, const AttentionArgs& a,
                     cudaStream_t stream) {
  if (c.dim == 128) {
    if (a.columns == 8) return launch_tile<128, 1>(c, b, a, stream);
    if (a.columns == 16) return launch_tile<128, 2>(c, b, a, stream);
    return launch_tile<128, 4>(c, b, a, stream);
  }
  if (a.columns == 8) return launch_tile<64, 1>(c, b, a, stream);
  if (a.columns == 16) return launch_tile<64, 2>(c, b, a, stream);
  return launch_tile<64, 4>(c, b, a, stream);
}

}  // namespace etk
