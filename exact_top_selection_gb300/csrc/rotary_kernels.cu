// Queries and keys turned by their positions (exact_topk_rotary).
//
// Pair i of a head at position p turns by the angle p f_i:
//
//   y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin).
//
// The angle. p f_i in FP32 is off by a quarter of a degree at position 65536 already. Here f_i is given in
// turns as a fraction of 2^64, and p times it, modulo 2^64, is the angle's fraction of a turn: an
// integer product, exact at every position, that needs neither a table nor a reduction.
//
// Bound by HBM: each row is read and written once. A CTA has a few tokens: it works out their
// cosines and sines once, into shared memory, and turns all heads by them.

#include "batch_internal.h"
#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 4;  // of a CTA
constexpr int kMostPairs = EXACT_TOPK_MAX_ROTARY_DIM / 2;
constexpr int kBatch = 4;       // rows' parts on their way in a thread

template <int V>
struct Part {  // V numbers of 16 bits
  uint32_t w[V > 1 ? V / 2 : 1];
};

template <int V>
__device__ __forceinline__ Part<V> load(const uint16_t* at) {
  Part<V> x;
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(at);
    x.w[0] = u.x;
    x.w[1] = u.y;
    x.w[2] = u.z;
    x.w[3] = u.w;
  } else if constexpr (V == 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(at);
    x.w[0] = u.x;
    x.w[1] = u.y;
  } else if constexpr (V == 2) {
    x.w[0] = *reinterpret_cast<const uint32_t*>(at);
  } else {
    x.w[0] = *at;
  }
  return x;
}

template <int V>
__device__ __forceinline__ void store(uint16_t* at, const Part<V>& x) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(at) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  else if constexpr (V == 4)
    *reinterpret_cast<uint2*>(at) = make_uint2(x.w[0], x.w[1]);
  else if constexpr (V == 2)
    *reinterpret_cast<uint32_t*>(at) = x.w[0];
  else
    *at = (uint16_t)x.w[0];
}

// Position of row `token`, or false where it has none.
__device__ __forceinline__ bool position_of(const RotaryArgs& a, const BatchArgs& b, int64_t token,
                                            int* position) {
  if (a.positions != nullptr) {
    *position = a.positions[token];
    return true;
  }
  const int seq = sequence_of_slot(b, token, 1, 0);
  const SeqRows s = sequence_rows(b, 0, seq);
  const int64_t index = token - s.begin;
  if (index < 0 || index >= s.count) return false;
  *position = s.pos0 + (int)index;
  return *position >= 0;
}

// A thread has 2 V channels of a row at a time: V pairs, or, behind the channels that turn, 2 V
// neighbours that are copied. It keeps to its place in the rows and goes from row to row; `lanes`,
// a power of two, are as many threads as stand on a row.
template <bool kFp16, int V, bool kNeighbours>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(RotaryArgs a, BatchArgs b, int tokens_of_cta, int lane_shift) {
  constexpr int kTwo = V > 1 ? 2 : 1;
  __shared__ __align__(16) float2 turn[kMostTokens * kMostPairs];  // cosine and sine, see below
  __shared__ int position[kMostTokens];
  __shared__ int there[kMostTokens];
  const int tid = threadIdx.x;
  const int64_t token0 = (int64_t)blockIdx.x * tokens_of_cta;
  const int64_t left = a.num_tokens - token0;
  const int tokens = left < tokens_of_cta ? (int)left : tokens_of_cta;
  const int turning = a.pairs / V;  // parts of a row that turn
  const int parts = turning + (a.copy_q || a.copy_k ? (a.dim - 2 * a.pairs + 2 * V - 1) / (2 * V) : 0);
  const int heads = a.q_heads + a.k_heads;
  // heads are spread over blockIdx.y where there are few tokens
  const int mine = (heads - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;
  const int rows = tokens * mine, row0 = tid >> lane_shift, row_step = kThreads >> lane_shift;
  const int lane = tid & ((1 << lane_shift) - 1);

  struct Item {
    const uint16_t* from;
    uint16_t* to;
    int token;
    bool copied;  // its rows go elsewhere
  };
  const auto item = [&](int row) {
    const int t = (row >= mine) + (row >= 2 * mine) + (row >= 3 * mine);
    const int head = (row - t * mine) * (int)gridDim.y + (int)blockIdx.y;
    const bool query = head < a.q_heads;
    const RowArgs& in = query ? a.q : a.k;
    const RowArgs& out = query ? a.q_out : a.k_out;
    const int64_t h = query ? head : head - a.q_heads, token = token0 + t;
    return Item{
        static_cast<const uint16_t*>(in.data) + token * in.token_stride + h * in.head_stride,
        static_cast<uint16_t*>(out.data) + token * out.token_stride + h * out.head_stride, t,
        (query ? a.copy_q : a.copy_k) != 0};
  };
  // First channels of a part's two halves; the second one may lie behind the head's last channel.
  const auto first_of = [&](int part) {
    return part < turning ? (kNeighbours ? part * 2 * V : part * V)
                          : 2 * a.pairs + (part - turning) * 2 * V;
  };
  const auto second_of = [&](int part) {
    return part < turning && !kNeighbours ? part * V + a.pairs : first_of(part) + V;
  };
  const auto read = [&](const Item& i, int part, Part<V>* x, Part<V>* y) {
    *x = load<V>(i.from + first_of(part));
    const int second = second_of(part);
    *y = load<V>(i.from + (second < a.dim ? second : first_of(part)));
  };

  // the first rows are on their way while the angles are worked out
  Part<V> x[kBatch], y[kBatch];
  const auto read_batch = [&](int from, int part) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int row = from + n * row_step;
      read(item(row < rows ? row : rows - 1), part, &x[n], &y[n]);
    }
  };
  if (lane < parts) read_batch(row0, lane);

  if (tid < tokens) {
    int p = 0;
    there[tid] = position_of(a, b, token0 + tid, &p);
    position[tid] = p;
  }
  __syncthreads();
  // Pairs of one thread lie `turning` apart in shared memory, two at a time: a warp's reads touch
  // each bank once.
  for (int i = tid; i < tokens * a.pairs; i += kThreads) {
    const int t = i / a.pairs, pair = i - t * a.pairs;
    const uint64_t p = (uint64_t)(int64_t)position[t];
    const uint64_t angle = a.turns[pair] * (a.inverse ? 0ull - p : p);
    float sine, cosine;
    sincospif(__ll2float_rn((int64_t)angle) * 0x1p-63f, &sine, &cosine);
    const int part = pair / V, in = pair % V;
    turn[t * a.pairs + (in / kTwo * turning + part) * kTwo + in % kTwo] =
        make_float2(cosine * a.amplitude, sine * a.amplitude);
  }
  __syncthreads();

  for (int part = lane; part < parts; part += 1 << lane_shift) {
    for (int from = row0; from < rows; from += row_step * kBatch) {
      if (part != lane || from != row0) read_batch(from, part);
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        const int row = from + n * row_step;
        if (row >= rows) break;
        const Item i = item(row);
        if (!there[i.token]) continue;
        if (part < turning) {
          float u[2 * V];  // x's numbers, then y's
#pragma unroll
          for (int k = 0; k < (V > 1 ? V / 2 : 1); ++k) {
            const float2 f = unpack2<kFp16>(x[n].w[k]), g = unpack2<kFp16>(y[n].w[k]);
            u[kTwo * k] = f.x;
            u[V + kTwo * k] = g.x;
            if (V > 1) {
              u[kTwo * k + kTwo - 1] = f.y;
              u[V + kTwo * k + kTwo - 1] = g.y;
            }
          }
          const float2* const at = &turn[i.token * a.pairs + part * kTwo];
#pragma unroll
          for (int k = 0; k < V; k += kTwo) {
            float2 by[kTwo];
            if constexpr (V > 1) {
              const float4 two = *reinterpret_cast<const float4*>(at + k * turning);
              by[0] = make_float2(two.x, two.y);
              by[kTwo - 1] = make_float2(two.z, two.w);
            } else {
              by[0] = at[0];
            }
#pragma unroll
            for (int j = 0; j < kTwo; ++j) {
              float& p = kNeighbours ? u[2 * (k + j)] : u[k + j];
              float& q = kNeighbours ? u[2 * (k + j) + 1] : u[V + k + j];
              const float p0 = p, q0 = q;
              p = p0 * by[j].x - q0 * by[j].y;
              q = q0 * by[j].x + p0 * by[j].y;
            }
          }
#pragma unroll
          for (int k = 0; k < (V > 1 ? V / 2 : 1); ++k) {
            x[n].w[k] = pack2<kFp16>(u[kTwo * k], V > 1 ? u[kTwo * k + kTwo - 1] : 0.f);
            y[n].w[k] = pack2<kFp16>(u[V + kTwo * k], V > 1 ? u[V + kTwo * k + kTwo - 1] : 0.f);
          }
        } else if (!i.copied) {
          continue;
        }
        store<V>(i.to + first_of(part), x[n]);
        const int second = second_of(part);
        if (second < a.dim) store<V>(i.to + second, y[n]);
      }
    }
  }
}

template <bool kFp16, int V, bool kNeighbours>
int launch_parts(const RotaryArgs& a, const BatchArgs& b, dim3 grid, int tokens,
                 cudaStream_t stream) {
  const int parts =
      a.pairs / V + (a.copy_q || a.copy_k ? (a.dim - 2 * a.pairs + 2 * V - 1) / (2 * V) : 0);
  int shift = 0;
  while ((1 << shift) < parts && (1 << shift) < kThreads) ++shift;
  rotary_kernel<kFp16, V, kNeighbours><<<grid, kThreads, 0, stream>>>(a, b, tokens, shift);
  return launch_status();
}

template <bool kFp16, bool kNeighbours>
int launch(const RotaryArgs& a, const BatchArgs& b, cudaStream_t stream) {
  const int heads = a.q_heads + a.k_heads;
  const int64_t waves = 152 * 8;  // eight CTAs for each of GB300's SMs
  // Four tokens a CTA (us for 36 heads of 128 channels, with 1, 2 and 4): 4864 tokens 25.4, 19.4
  // and 18.7, 20000 tokens 98.6, 66.4 and 61.4; 2432 tokens, which get one, 14.1, 11.2 and 11.7,
  // 1000 7.5, 7.9 and 8.0. (Behind a cold L2, as below.)
  const int tokens = a.num_tokens >= waves * kMostTokens ? kMostTokens : 1;
  const int64_t ctas = (a.num_tokens + tokens - 1) / tokens;
  // Heads apart while there are no more CTAs than that. Each works out its token's angles: of 64
  // tokens x 36 heads 1024 CTAs, with rows for 16 or 24 of their 256 threads, take 6.1 us, where up to
  // 152 x 1, 2, 4 and 16 CTAs take 3.2, 3.4, 3.6 and 9.2. 16 tokens 3.9 (3.2, 3.6, 3.6, 4.0), 256
  // tokens 6.0 (3.9, 3.8, 3.8, 9.4), 1000 tokens 7.7 (7.4, 7.7, 7.5, 10.6).
  int split = 1;
  while (split * 2 <= heads && ctas * split * 2 <= waves) split *= 2;
  const dim3 grid((unsigned)ctas, (unsigned)split);
  if (a.pairs % 8 == 0) return launch_parts<kFp16, 8, kNeighbours>(a, b, grid, tokens, stream);
  if (a.pairs % 4 == 0) return launch_parts<kFp16, 4, kNeighbours>(a, b, grid, tokens, stream);
  if (a.pairs % 2 == 0) return launch_parts<kFp16, 2, kNeighbours>(a, b, grid, tokens, stream);
  return launch_parts<kFp16, 1, kNeighbours>(a, b, grid, tokens, stream);
}

}  // namespace

int launch_rotary(const RotaryArgs& a, const BatchArgs& b, cudaStream_t stream) {
  if (a.fp16)
    return a.neighbours ? launch<true, true>(a, b, stream) : launch<true, false>(a, b, stream);
  return a.neighbours ? launch<false, true>(a, b, stream) : launch<false, false>(a, b, stream);
}

}  // namespace etk
