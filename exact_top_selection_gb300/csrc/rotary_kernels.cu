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

// V pairs a thread: V channels and the V of their partners.
template <bool kFp16, int V, bool kNeighbours>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(RotaryArgs a, BatchArgs b, int tokens_of_cta) {
  __shared__ __align__(16) float2 turn[kMostTokens * kMostPairs];  // cosine and sine, see below
  __shared__ int position[kMostTokens];
  __shared__ int there[kMostTokens];
  const int tid = threadIdx.x;
  const int64_t token0 = (int64_t)blockIdx.x * tokens_of_cta;
  const int64_t left = a.num_tokens - token0;
  const int tokens = left < tokens_of_cta ? (int)left : tokens_of_cta;
  if (tid < tokens) {
    int p = 0;
    there[tid] = position_of(a, b, token0 + tid, &p);
    position[tid] = p;
  }
  __syncthreads();
  const int parts = a.pairs / V;  // threads of a row
  // Pairs of one thread lie `parts` apart in shared memory, two at a time: a warp's reads touch
  // each bank once.
  for (int i = tid; i < tokens * a.pairs; i += kThreads) {
    const int t = i / a.pairs, pair = i - t * a.pairs;
    const uint64_t p = (uint64_t)(int64_t)position[t];
    const uint64_t angle = a.turns[pair] * (a.inverse ? 0ull - p : p);
    float sine, cosine;
    sincospif(__ll2float_rn((int64_t)angle) * 0x1p-63f, &sine, &cosine);
    constexpr int kTwo = V > 1 ? 2 : 1;
    const int part = pair / V, in = pair % V;
    turn[t * a.pairs + (in / kTwo * parts + part) * kTwo + in % kTwo] =
        make_float2(cosine * a.amplitude, sine * a.amplitude);
  }
  __syncthreads();

  const int heads = a.q_heads + a.k_heads;
  // heads are spread over blockIdx.y where there are few tokens
  const int mine = (heads - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;
  const int items = tokens * mine * parts;
  const auto place = [&](int item, const uint16_t** from, uint16_t** to, int* t, int* part) {
    const int row = item / parts;
    *part = item - row * parts;
    *t = row / mine;
    const int head = (row - *t * mine) * (int)gridDim.y + (int)blockIdx.y;
    const bool query = head < a.q_heads;
    const RowArgs& in = query ? a.q : a.k;
    const RowArgs& out = query ? a.q_out : a.k_out;
    const int64_t h = query ? head : head - a.q_heads;
    const int64_t token = token0 + *t;
    *from = static_cast<const uint16_t*>(in.data) + token * in.token_stride + h * in.head_stride;
    *to = static_cast<uint16_t*>(out.data) + token * out.token_stride + h * out.head_stride;
  };
  for (int item0 = tid; item0 < items; item0 += kThreads * kBatch) {
    Part<V> x[kBatch], y[kBatch];
    uint16_t* to[kBatch];
    int t[kBatch], part[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int item = item0 + n * kThreads < items ? item0 + n * kThreads : item0;
      const uint16_t* from;
      place(item, &from, &to[n], &t[n], &part[n]);
      const int first = kNeighbours ? part[n] * 2 * V : part[n] * V;
      x[n] = load<V>(from + first);
      y[n] = load<V>(from + first + (kNeighbours ? V : a.pairs));
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (item0 + n * kThreads >= items || !there[t[n]]) continue;
      float u[2 * V];  // x's numbers, then y's
#pragma unroll
      for (int i = 0; i < (V > 1 ? V / 2 : 1); ++i) {
        const float2 f = unpack2<kFp16>(x[n].w[i]), g = unpack2<kFp16>(y[n].w[i]);
        u[2 * i] = f.x;
        if (V > 1) u[2 * i + 1] = f.y;
        u[V + 2 * i] = g.x;
        if (V > 1) u[V + 2 * i + 1] = g.y;
      }
      float2 by_of[V];
      if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float4 two = *reinterpret_cast<const float4*>(
              &turn[t[n] * a.pairs + (i / 2 * parts + part[n]) * 2]);
          by_of[i] = make_float2(two.x, two.y);
          by_of[i + 1] = make_float2(two.z, two.w);
        }
      } else {
        by_of[0] = turn[t[n] * a.pairs + part[n]];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 by = by_of[i];
        float& p = kNeighbours ? u[2 * i] : u[i];
        float& q = kNeighbours ? u[2 * i + 1] : u[V + i];
        const float p0 = p, q0 = q;
        p = p0 * by.x - q0 * by.y;
        q = q0 * by.x + p0 * by.y;
      }
#pragma unroll
      for (int i = 0; i < (V > 1 ? V / 2 : 1); ++i) {
        x[n].w[i] = pack2<kFp16>(u[2 * i], V > 1 ? u[2 * i + 1] : 0.f);
        y[n].w[i] = pack2<kFp16>(u[V + 2 * i], V > 1 ? u[V + 2 * i + 1] : 0.f);
      }
      const int first = kNeighbours ? part[n] * 2 * V : part[n] * V;
      store<V>(to[n] + first, x[n]);
      store<V>(to[n] + first + (kNeighbours ? V : a.pairs), y[n]);
    }
  }

  // ---- channels that do not turn, where the rows go elsewhere ----
  if (!a.copy_q && !a.copy_k) return;
  constexpr int kCopy = V < 4 ? V : 8;  // 2 * pairs and the head's channels are multiples of it
  const int rest = (a.dim - 2 * a.pairs) / kCopy;
  if (rest == 0) return;
  for (int i = tid; i < tokens * mine * rest; i += kThreads) {
    const int row = i / rest, t = row / mine;
    const int head = (row - t * mine) * (int)gridDim.y + (int)blockIdx.y;
    const bool query = head < a.q_heads;
    if (!there[t] || !(query ? a.copy_q : a.copy_k)) continue;
    const RowArgs& in = query ? a.q : a.k;
    const RowArgs& out = query ? a.q_out : a.k_out;
    const int64_t h = query ? head : head - a.q_heads;
    const int first = 2 * a.pairs + (i - row * rest) * kCopy;
    store<kCopy>(static_cast<uint16_t*>(out.data) + (token0 + t) * out.token_stride +
                     h * out.head_stride + first,
                 load<kCopy>(static_cast<const uint16_t*>(in.data) + (token0 + t) * in.token_stride +
                             h * in.head_stride + first));
  }
}

template <bool kFp16, bool kNeighbours>
int launch(const RotaryArgs& a, const BatchArgs& b, cudaStream_t stream) {
  const int heads = a.q_heads + a.k_heads;
  const int64_t waves = 152 * 8;
  const int tokens = a.num_tokens >= waves * kMostTokens ? kMostTokens : 1;
  const int64_t ctas = (a.num_tokens + tokens - 1) / tokens;
  // heads apart until there are some waves of CTAs
  int split = 1;
  while (split * 2 <= heads && ctas * split * 2 <= waves) split *= 2;
  const dim3 grid((unsigned)ctas, (unsigned)split);
  if (a.pairs % 8 == 0)
    rotary_kernel<kFp16, 8, kNeighbours><<<grid, kThreads, 0, stream>>>(a, b, tokens);
  else if (a.pairs % 4 == 0)
    rotary_kernel<kFp16, 4, kNeighbours><<<grid, kThreads, 0, stream>>>(a, b, tokens);
  else if (a.pairs % 2 == 0)
    rotary_kernel<kFp16, 2, kNeighbours><<<grid, kThreads, 0, stream>>>(a, b, tokens);
  else
    rotary_kernel<kFp16, 1, kNeighbours><<<grid, kThreads, 0, stream>>>(a, b, tokens);
  return launch_status();
}

}  // namespace

int launch_rotary(const RotaryArgs& a, const BatchArgs& b, cudaStream_t stream) {
  if (a.fp16)
    return a.neighbours ? launch<true, true>(a, b, stream) : launch<true, false>(a, b, stream);
  return a.neighbours ? launch<false, true>(a, b, stream) : launch<false, false>(a, b, stream);
}

}  // namespace etk
