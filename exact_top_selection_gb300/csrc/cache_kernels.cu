// Writing rows into the paged 8-bit cache and reading them back
// (exact_topk_cache_write, exact_topk_cache_read).
//
// Both move bytes and are bound by HBM.  A CTA takes the part of one page that
// a sequence's rows reach: its codes are contiguous, its rows whole channels of
// one head, so every access is a full line.  The CTAs are laid over the pages
// without any host knowledge of lengths (first_slot).
//
// Writing 108 K tokens of 8 heads x 128 channels takes 103 us (6.4 TB/s, 94% of the rate
// of a copy), reading 262 K tokens of 8 heads x 64 channels back 131 us (6.1 TB/s).  One new token
// of 64 sequences takes 5.6 us: the chain length -> page -> rows -> scale.

#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

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

// 2^e with the smallest e in range for which amax <= 448 * 2^e.  448 = 1.75 * 2^8,
// so a magnitude 1.m * 2^x needs e = x - 8, one more where 1.m > 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < EXACT_TOPK_SCALE_MIN_EXP ? EXACT_TOPK_SCALE_MIN_EXP : e;
  e = e > EXACT_TOPK_SCALE_MAX_EXP ? EXACT_TOPK_SCALE_MAX_EXP : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two numbers as codes.  The conversion saturates; where kSpecial, y + 0 * y, which is NaN for
// an infinity, keeps infinities from becoming 448.
template <bool kSpecial>
__device__ __forceinline__ uint32_t encode2(float x, float y) {
  const float2 v = kSpecial ? make_float2(fmaf(x, 0.f, x), fmaf(y, 0.f, y)) : make_float2(x, y);
  return (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

template <bool kFp16, bool kSpecial>
__device__ __forceinline__ uint2 encode8(const uint4& x, float by) {
  const float2 a = unpack2<kFp16>(x.x), b = unpack2<kFp16>(x.y), c = unpack2<kFp16>(x.z),
               d = unpack2<kFp16>(x.w);
  return make_uint2(
      encode2<kSpecial>(a.x * by, a.y * by) | encode2<kSpecial>(b.x * by, b.y * by) << 16,
      encode2<kSpecial>(c.x * by, c.y * by) | encode2<kSpecial>(d.x * by, d.y * by) << 16);
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

// One pass over the rows: a page's part is held in registers (8 channels a thread
// and row, P * D / 1024 rows of the page), its largest magnitude found across
// the CTA, then coded and stored.  32 warps an SM (64 registers) hide the loads: 103 us for
// 108 K tokens, 24 warps 112; magnitudes and bounds as single floats took 219.  Keys and
// values are separate CTAs (blockIdx.z).
// Scales are powers of two: e4m3 is a floating format, so a finer scale would only
// move the borders of its exponents, and with powers of two every division here and
// every product on reading is exact.
template <bool kFp16, int D, int P>
__global__ void __launch_bounds__(kThreads, P * D >= 16384 ? 5 : 8)
    cache_write_kernel(CacheArgs c, BatchArgs b, RowArgs krows, RowArgs vrows) {
  constexpr int kLanes = D / 8;               // threads on a row
  constexpr int kRows = kThreads / kLanes;    // rows of a pass
  constexpr int kPasses = P / kRows > 0 ? P / kRows : 1;
  constexpr int kShift = P == 16 ? 4 : (P == 32 ? 5 : (P == 64 ? 6 : 7));
  __shared__ float s_max[kWarps];
  __shared__ uint32_t s_hi[kWarps][D / 2], s_lo[kWarps][D / 2];

  PagePart part;
  if (!page_part(b, kShift, blockIdx.x, &part)) return;
  const int page = page_of(c, b, part.seq, part.block);
  if (page < 0) return;
  const bool keys = blockIdx.z == 0;
  const RowArgs src = keys ? krows : vrows;
  uint8_t* const codes = keys ? c.k : c.v;
  float* const scales = keys ? c.k_scale : c.v_scale;
  const bool bounds = keys && c.bounds != nullptr;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = tid % kLanes, row0 = tid / kLanes;
  const int64_t row_base = part.rows.begin + (((int64_t)part.block << kShift) - part.rows.pos0);
  const uint16_t* const rows = static_cast<const uint16_t*>(src.data);

  for (int h = blockIdx.y; h < c.heads; h += gridDim.y) {
    const uint16_t* const from = rows + row_base * src.token_stride +
                                 (int64_t)h * src.head_stride + chunk * 8;
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int o = row0 + i * kRows;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (o >= part.first && o < part.end)
        x[i] = __ldg(reinterpret_cast<const uint4*>(from + o * src.token_stride));
    }
    // Magnitudes compare as integers; an infinity or NaN shows as one at or above infinity's
    // pattern. A page that has one is read again, row by row.
    uint32_t top = 0u, hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = infinities<kFp16>() | 0x80008000u;
      lo[j] = infinities<kFp16>();
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                   __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
      const int o = row0 + i * kRows;
      if (bounds && o >= part.first && o < part.end) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi[j] = larger2<kFp16>(hi[j], w[j]);
          lo[j] = smaller2<kFp16>(lo[j], w[j]);
        }
      }
    }
    const bool special =
        __syncthreads_or((top & 0xFFFFu) >= (infinities<kFp16>() & 0xFFFFu) ||
                         top >= (infinities<kFp16>() & 0xFFFF0000u)) != 0;
    const float2 both = unpack2<kFp16>(top);
    float amax = fmaxf(both.x, both.y);
    if (special) {
      amax = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        hi[j] = infinities<kFp16>() | 0x80008000u;
        lo[j] = infinities<kFp16>();
      }
#pragma unroll 1
      for (int o = row0; o < part.end; o += kRows) {
        if (o < part.first) continue;
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(from + o * src.token_stride));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2<kFp16>(w[j]);
          amax = fmaxf(amax, fmaxf(finite_magnitude(f.x), finite_magnitude(f.y)));
          hi[j] = larger2<kFp16>(hi[j], finite2<kFp16>(w[j]));
          lo[j] = smaller2<kFp16>(lo[j], finite2<kFp16>(w[j]));
        }
      }
    }
    if (bounds) {
#pragma unroll
      for (int o = 16; o >= kLanes; o >>= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          hi[j] = larger2<kFp16>(hi[j], __shfl_xor_sync(~0u, hi[j], o));
          lo[j] = smaller2<kFp16>(lo[j], __shfl_xor_sync(~0u, lo[j], o));
        }
      if (lane < kLanes) {
        *reinterpret_cast<uint4*>(&s_hi[warp][chunk * 4]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(&s_lo[warp][chunk * 4]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    if (lane == 0) s_max[warp] = amax;
    const int64_t tile = (int64_t)page * c.heads + h;
    const float held = part.first > 0 ? scales[tile] : 0.f;  // read before it is replaced
    __syncthreads();
    amax = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const float scale = fmaxf(scale_for(amax), held);
    uint8_t* const out = codes + tile * (P * D);
    const float inverse = 1.f / scale;  // exact: the scale is a power of two
    if (!special) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int o = row0 + i * kRows;
        if (o >= part.first && o < part.end)
          *reinterpret_cast<uint2*>(out + o * D + chunk * 8) =
              encode8<kFp16, false>(x[i], inverse);
      }
    } else {
#pragma unroll 1
      for (int o = row0; o < part.end; o += kRows)
        if (o >= part.first)
          *reinterpret_cast<uint2*>(out + o * D + chunk * 8) = encode8<kFp16, true>(
              __ldg(reinterpret_cast<const uint4*>(from + o * src.token_stride)), inverse);
    }
    if (part.first > 0 && scale != held) {
      const float ratio = held / scale;
      for (int o = row0; o < part.first; o += kRows) {
        uint2* const at = reinterpret_cast<uint2*>(out + o * D + chunk * 8);
        const uint2 was = *at;
        const uint32_t w[2] = {was.x, was.y};
        uint32_t q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f0 = codes_to_float2((uint16_t)w[j]);
          const float2 f1 = codes_to_float2((uint16_t)(w[j] >> 16));
          q[j] = encode2<true>(f0.x * ratio, f0.y * ratio) |
                 encode2<true>(f1.x * ratio, f1.y * ratio) << 16;
        }
        *at = make_uint2(q[0], q[1]);
      }
    }
    if (bounds && tid < D / 2) {
      uint32_t u = larger2<kFp16>(larger2<kFp16>(s_hi[0][tid], s_hi[1][tid]),
                                  larger2<kFp16>(s_hi[2][tid], s_hi[3][tid]));
      uint32_t v = smaller2<kFp16>(smaller2<kFp16>(s_lo[0][tid], s_lo[1][tid]),
                                   smaller2<kFp16>(s_lo[2][tid], s_lo[3][tid]));
      uint32_t* const at = static_cast<uint32_t*>(c.bounds) + tile * D + tid;
      if (part.first > 0) {
        u = larger2<kFp16>(u, at[0]);
        v = smaller2<kFp16>(v, at[D / 2]);
      }
      at[0] = u;
      at[D / 2] = v;
    }
    if (tid == 0) scales[tile] = scale;
    __syncthreads();  // the shared maxima are free for the next head
  }
}

// 16 codes a thread and step: one 16-byte load, two 16-byte stores.
template <bool kFp16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheArgs c, BatchArgs b,
                                                              RowArgs krows, RowArgs vrows) {
  const int P = c.page, D = c.dim;
  PagePart part;
  const bool any = page_part(b, c.page_shift, blockIdx.x, &part);
  const bool keys = blockIdx.z == 0;
  const RowArgs dst = keys ? krows : vrows;
  uint16_t* const rows = static_cast<uint16_t*>(dst.data);
  const int lanes = D / 16, lane_shift = D == 128 ? 3 : 2;
  const int heads = (c.heads - (int)blockIdx.y + (int)gridDim.y - 1) / (int)gridDim.y;

  // rows ahead of the sequence's first token
  if (part.index == 0 && part.rows.pos0 < 0) {
    const int none = part.rows.count < -part.rows.pos0 ? part.rows.count : -part.rows.pos0;
    for (int64_t i = threadIdx.x; i < (int64_t)none * heads * lanes; i += kThreads) {
      const int64_t r = i / lanes;
      uint4* const at = reinterpret_cast<uint4*>(
          rows + (part.rows.begin + r / heads) * dst.token_stride +
          ((int64_t)blockIdx.y + (r % heads) * gridDim.y) * dst.head_stride + (i % lanes) * 16);
      at[0] = at[1] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (!any) return;
  const int page = page_of(c, b, part.seq, part.block);
  const int64_t row_base =
      part.rows.begin + (((int64_t)part.block << c.page_shift) - part.rows.pos0);
  const uint8_t* const codes = keys ? c.k : c.v;
  const float* const scales = keys ? c.k_scale : c.v_scale;
  const int steps = heads << (c.page_shift + lane_shift);
  constexpr int kBatch = 4;  // loads on their way (2: 141 us, 8: 156 us)
  for (int i0 = threadIdx.x; i0 < steps; i0 += kThreads * kBatch) {
    uint4 x[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int i = i0 + n * kThreads;
      const int o = (i >> lane_shift) & (P - 1);
      const int h = (int)blockIdx.y + (i >> (c.page_shift + lane_shift)) * (int)gridDim.y;
      x[n] = make_uint4(0u, 0u, 0u, 0u);
      scale[n] = 0.f;
      if (page >= 0 && i < steps && o >= part.first && o < part.end) {
        const int64_t tile = (int64_t)page * c.heads + h;
        x[n] = __ldg(reinterpret_cast<const uint4*>(codes + (tile * P + o) * D +
                                                    (i & (lanes - 1)) * 16));
        scale[n] = __ldg(scales + tile);
      }
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const int i = i0 + n * kThreads;
      const int o = (i >> lane_shift) & (P - 1);
      const int h = (int)blockIdx.y + (i >> (c.page_shift + lane_shift)) * (int)gridDim.y;
      if (i >= steps || o < part.first || o >= part.end) continue;
      const uint32_t w[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
      uint32_t y[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f0 = codes_to_float2((uint16_t)w[j]);
        const float2 f1 = codes_to_float2((uint16_t)(w[j] >> 16));
        y[2 * j] = pack2<kFp16>(f0.x * scale[n], f0.y * scale[n]);
        y[2 * j + 1] = pack2<kFp16>(f1.x * scale[n], f1.y * scale[n]);
      }
      uint4* const at = reinterpret_cast<uint4*>(rows + (row_base + o) * dst.token_stride +
                                                 h * dst.head_stride + (i & (lanes - 1)) * 16);
      at[0] = make_uint4(y[0], y[1], y[2], y[3]);
      at[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// Heads are spread over CTAs (blockIdx.y) until there are a few waves of them;
// beyond that a CTA takes several, up to 16 KB of codes, so that small pages do not become CTAs
// of a kilobyte each (reading pages of 16 tokens x 64 channels: 131 us, with 4 KB a CTA 182).
dim3 page_grid(const CacheArgs& c, const BatchArgs& b) {
  const int64_t slots = slot_count(b, c.page, 2);
  int y = c.heads;
  while (y > 1 && slots * y > 4096 && c.heads / y * c.page * c.dim < 16384) y = (y + 1) / 2;
  return dim3((unsigned)slots, (unsigned)y, 2u);
}

template <bool kFp16, int D>
void write_page(const CacheArgs& c, const BatchArgs& b, const RowArgs& k, const RowArgs& v,
                cudaStream_t stream) {
  const dim3 grid = page_grid(c, b);
  switch (c.page) {
    case 16:
      cache_write_kernel<kFp16, D, 16><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
    case 32:
      cache_write_kernel<kFp16, D, 32><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
    case 64:
      cache_write_kernel<kFp16, D, 64><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
    default:
      cache_write_kernel<kFp16, D, 128><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
  }
}

}  // namespace

int launch_cache_write(const CacheArgs& c, const BatchArgs& b, const RowArgs& k, const RowArgs& v,
                       cudaStream_t stream) {
  if (c.dim == 128)
    c.fp16 ? write_page<true, 128>(c, b, k, v, stream) : write_page<false, 128>(c, b, k, v, stream);
  else
    c.fp16 ? write_page<true, 64>(c, b, k, v, stream) : write_page<false, 64>(c, b, k, v, stream);
  return launch_status();
}

int launch_cache_read(const CacheArgs& c, const BatchArgs& b, const RowArgs& k, const RowArgs& v,
                      cudaStream_t stream) {
  const dim3 grid = page_grid(c, b);
  if (c.fp16)
    cache_read_kernel<true><<<grid, kThreads, 0, stream>>>(c, b, k, v);
  else
    cache_read_kernel<false><<<grid, kThreads, 0, stream>>>(c, b, k, v);
  return launch_status();
}

}  // namespace etk
