// Writing rows into the paged 4-bit cache and reading them back
// (exact_topk_cache4_write, exact_topk_cache4_read).
//
// 16 channels of a token share a scale s, e4m3; a number is code * s * unit with
//
//   s = e4m3(max |x| / (6 unit)),  code = e2m1(x / (s unit)),  both to nearest even,
//
// so a token depends on no other one, and a page that is continued is not read again, but for
// its key bounds. Both operators move bytes and are bound by HBM; the CTAs are laid over
// the pages as those of the 8-bit cache are.

#include <type_traits>

#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(x)), "l"(reinterpret_cast<const uint64_t&>(y)));
  return r;
}

__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<const uint64_t&>(x)), "l"(reinterpret_cast<const uint64_t&>(y)),
        "l"(reinterpret_cast<const uint64_t&>(z)));
  return r;
}

// 32 bytes in one access, which a group's rows are where their places allow it. In two of 16 bytes, a
// warp's accesses touch every other half of a sector.
__device__ __forceinline__ bool in_one_access(const RowArgs& r) {
  return ((reinterpret_cast<uintptr_t>(r.data) | (uintptr_t)(r.token_stride * 2) |
           (uintptr_t)(r.head_stride * 2)) &
          31u) == 0u;
}

__device__ __forceinline__ void load32(const void* at, uint4& x, uint4& y) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z),
                 "=r"(y.w)
               : "l"(at));
}

__device__ __forceinline__ void store32(void* at, const uint32_t (&x)[4], const uint32_t (&y)[4]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3]), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
               : "memory");
}

// Eight numbers as e2m1 codes, the first in the lowest four bits; nearest even, saturating.
__device__ __forceinline__ uint32_t encode8(const float2 (&y)[4]) {
  uint32_t r;
  asm("{\n.reg .b8 b0, b1, b2, b3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      "mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x),
        "f"(y[3].y));
  return r;
}

// The larger magnitudes of two pairs of the rows' type, NaN where either is; signs are of no meaning.
template <bool kFp16>
__device__ __forceinline__ uint32_t larger_magnitudes2(uint32_t x, uint32_t y) {
  uint32_t r;
  if (kFp16)
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// A group's codes and its scale's code. True where the group has an infinity or a NaN: its scale
// is NaN then.
//
// Rounding. max / 6 and x / (s unit) are rounded twice, to FP32 and to the code. x has at most 11
// significant bits, a border between two codes times the divisor at most 7: the quotient is a border
// exactly or is 2^-12 of itself away from it, and FP32's rounding moves it over none. It has to be
// exact where it is a border: the product with a reciprocal in two parts, which is off by 2^-44 before
// its rounding, is exact for quotients of few bits.
template <bool kFp16>
__device__ __forceinline__ bool encode16(const uint32_t (&w)[8], float unit, float inverse_unit,
                                         uint2* codes, uint32_t* scale) {
  uint32_t top = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = larger_magnitudes2<kFp16>(top, w[i]);
  top &= 0x7FFF7FFFu;
  const bool special = (top & 0xFFFFu) >= (infinities<kFp16>() & 0xFFFFu) ||
                       top >= (infinities<kFp16>() & 0xFFFF0000u);
  const float2 both = unpack2<kFp16>(top);
  const float most = fmaxf(both.x, both.y);
  // a sixth in two parts
  constexpr float kSixth = 1.f / 6.f, kSixthRest = (float)(1. / 6. - (double)kSixth);
  uint32_t code =
      __nv_cvt_float_to_fp8(fmaf(most, kSixth, most * kSixthRest) * inverse_unit, __NV_SATFINITE,
                            __NV_E4M3);
  code = special ? 0x7Fu : (code > 1u ? code : 1u);
  *scale = code;
  const float by = special ? 1.f : codes_to_float2((uint16_t)code).x * unit;
  float inverse;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inverse) : "f"(by));
  float2 y[8];
  if (special || most * inverse > 1e30f) {
    // quotients that overflow saturate, where the correction would make NaN of them
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack2<kFp16>(w[i]);
      y[i] = make_float2(__fdiv_rn(x.x, by), __fdiv_rn(x.y, by));
    }
  } else {
    const float rest = fmaf(-by, inverse, 1.f) * inverse;  // what the reciprocal lacks
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = unpack2<kFp16>(w[i]);
      y[i] = fma2(x, make_float2(inverse, inverse), mul2(x, make_float2(rest, rest)));
    }
  }
  const float2 low[4] = {y[0], y[1], y[2], y[3]}, high[4] = {y[4], y[5], y[6], y[7]};
  *codes = make_uint2(encode8(low), encode8(high));
  return special;
}

// A thread has 16 channels of a row, which need no other thread; the CTA only joins the keys'
// bounds. 108 K tokens of 8 heads x 128 channels in pages of 64 take 92 us (6.2 TB/s); four rows on
// their way in each of 32 warps an SM: with two 123, and 111 before whole pages went without
// predicates and a CTA took several heads. It is near HBM's rate where a page gives each thread
// four rows or more: pages of 32 take 110 us, pages of 16 147, with one row a thread and the join
// of the bounds behind each. Of 64 channels, 216 K tokens: 242, 152, 112 and 99 in pages of 16 to
// 128. Pages of 128 of 128 channels take 109: the bound of 64 registers, made for four rows on
// their way, has eight passes spill (382 bytes a thread, 44 in pages of 64, none in pages of 16).
template <bool kFp16, int D, int P>
__global__ void __launch_bounds__(kThreads, 8)
    cache4_write_kernel(Cache4Args c, BatchArgs b, RowArgs krows, RowArgs vrows) {
  constexpr int kLanes = D / 16;            // threads on a row
  constexpr int kRows = kThreads / kLanes;  // rows of a pass
  constexpr int kPasses = P / kRows > 0 ? P / kRows : 1;
  constexpr int kBatch = kPasses < 4 ? kPasses : 4;  // rows on their way
  constexpr int kShift = P == 16 ? 4 : (P == 32 ? 5 : (P == 64 ? 6 : 7));
  __shared__ uint32_t s_hi[kWarps][D / 2], s_lo[kWarps][D / 2];

  PagePart part;
  if (!page_part(b, kShift, blockIdx.x, &part)) return;
  const int page = page_of(c, b, part.seq, part.block);
  if (page < 0) return;
  const bool keys = blockIdx.z == 0;
  const RowArgs src = keys ? krows : vrows;
  uint8_t* const codes = keys ? c.k : c.v;
  uint8_t* const scales = reinterpret_cast<uint8_t*>(keys ? c.k_scale : c.v_scale);
  const float unit = keys ? c.k_unit : c.v_unit;
  const float inverse_unit = 1.f / unit;  // exact: the unit is a power of two
  const bool bounds = keys && c.bounds != nullptr;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = tid % kLanes, row0 = tid / kLanes;
  const int64_t row_base = part.rows.begin + (((int64_t)part.block << kShift) - part.rows.pos0);
  const uint16_t* const rows = static_cast<const uint16_t*>(src.data);
  const int64_t step = kRows * src.token_stride;
  const bool wide = in_one_access(src);

  for (int h = blockIdx.y; h < c.heads; h += gridDim.y) {
    const uint16_t* const from = rows + row_base * src.token_stride +
                                 (int64_t)h * src.head_stride + chunk * 16;
    const int64_t tile = (int64_t)page * c.heads + h;
    uint8_t* const to = codes + tile * (P * D / 2) + chunk * 8;
    uint8_t* const scale_to = scales + tile * (P * kLanes) + chunk;
    uint32_t hi[8], lo[8];
    const auto no_bounds = [&] {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hi[j] = infinities<kFp16>() | 0x80008000u;
        lo[j] = infinities<kFp16>();
      }
    };
    no_bounds();
    bool special = false;
    // A whole page's rows need no predicates, and are loaded 32 bytes at a time.
    const auto rows_of = [&](auto whole) {
      constexpr bool kWhole = decltype(whole)::value && P >= kRows;
      const uint16_t* at = from + row0 * src.token_stride;
#pragma unroll 1
      for (int i0 = 0; i0 < kPasses; i0 += kBatch) {
        uint4 x[kBatch][2];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int o = row0 + (i0 + i) * kRows;
          x[i][0] = x[i][1] = make_uint4(0u, 0u, 0u, 0u);
          if (kWhole) {
            load32(at, x[i][0], x[i][1]);
          } else if (o >= part.first && o < part.end) {
            x[i][0] = __ldg(reinterpret_cast<const uint4*>(at));
            x[i][1] = __ldg(reinterpret_cast<const uint4*>(at) + 1);
          }
          at += step;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int o = row0 + (i0 + i) * kRows;
          if (!kWhole && (o < part.first || o >= part.end)) continue;
          const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                                 x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
          uint2 code;
          uint32_t scale;
          special |= encode16<kFp16>(w, unit, inverse_unit, &code, &scale);
          *reinterpret_cast<uint2*>(to + o * (D / 2)) = code;
          scale_to[o * kLanes] = (uint8_t)scale;
          if (bounds) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              hi[j] = larger2<kFp16>(hi[j], w[j]);
              lo[j] = smaller2<kFp16>(lo[j], w[j]);
            }
          }
        }
      }
    };
    if (part.first == 0 && part.end == P && wide)
      rows_of(std::true_type());
    else
      rows_of(std::false_type());
    if (!bounds) continue;
    if (__syncthreads_or(special)) {  // the bounds again, of finite numbers
      no_bounds();
#pragma unroll 1
      for (int o = row0; o < part.end; o += kRows) {
        if (o < part.first) continue;
        const uint4* const at = reinterpret_cast<const uint4*>(from + o * src.token_stride);
        const uint4 u = __ldg(at), v = __ldg(at + 1);
        const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hi[j] = larger2<kFp16>(hi[j], finite2<kFp16>(w[j]));
          lo[j] = smaller2<kFp16>(lo[j], finite2<kFp16>(w[j]));
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hi[j] = larger2<kFp16>(hi[j], __shfl_xor_sync(~0u, hi[j], o));
        lo[j] = smaller2<kFp16>(lo[j], __shfl_xor_sync(~0u, lo[j], o));
      }
    if (lane < kLanes) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s_hi[warp][chunk * 8 + j] = hi[j];
        s_lo[warp][chunk * 8 + j] = lo[j];
      }
    }
    __syncthreads();
    if (tid < D / 2) {
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
    __syncthreads();  // the shared bounds are free for the next head
  }
}

// A group a thread and step: its 8 bytes of codes and its scale, two 16-byte stores. A page's heads
// lie one behind the other, so a CTA's groups are one run, and a thread goes through it by steps
// of kThreads; its rows follow by additions. With places worked out for each group by shifts
// and products, 200 instructions a group and 124 us for 262 K tokens of 8 heads x 64 channels; 105 now
// (6.6 TB/s), 119 with two stores of 16 bytes.
template <bool kFp16, int D>
__global__ void __launch_bounds__(kThreads) cache4_read_kernel(Cache4Args c, BatchArgs b,
                                                               RowArgs krows, RowArgs vrows) {
  constexpr int kLanes = D / 16, kRows = kThreads / kLanes;  // rows of a step
  PagePart part;
  const bool any = page_part(b, c.page_shift, blockIdx.x, &part);
  const bool keys = blockIdx.z == 0;
  const RowArgs dst = keys ? krows : vrows;
  uint16_t* const rows = static_cast<uint16_t*>(dst.data);
  // heads [head0, head0 + heads)
  const int each = (c.heads + (int)gridDim.y - 1) / (int)gridDim.y;
  const int head0 = (int)blockIdx.y * each;
  const int heads = c.heads - head0 < each ? c.heads - head0 : each;
  if (heads <= 0) return;

  // rows ahead of the sequence's first token
  if (part.index == 0 && part.rows.pos0 < 0) {
    const int none = part.rows.count < -part.rows.pos0 ? part.rows.count : -part.rows.pos0;
    for (int64_t i = threadIdx.x; i < (int64_t)none * heads * kLanes; i += kThreads) {
      const int64_t r = i / kLanes;
      uint4* const at = reinterpret_cast<uint4*>(
          rows + (part.rows.begin + r / heads) * dst.token_stride +
          (head0 + r % heads) * dst.head_stride + (i % kLanes) * 16);
      at[0] = at[1] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (!any) return;
  const int page = page_of(c, b, part.seq, part.block);
  const int P = 1 << c.page_shift;
  const int64_t row_base =
      part.rows.begin + (((int64_t)part.block << c.page_shift) - part.rows.pos0);
  const int64_t group0 = ((((int64_t)page * c.heads + head0) << c.page_shift) * kLanes);
  const uint8_t* const codes = (keys ? c.k : c.v) + (page < 0 ? 0 : group0 * 8);
  const uint8_t* const scales =
      reinterpret_cast<const uint8_t*>(keys ? c.k_scale : c.v_scale) + (page < 0 ? 0 : group0);
  const float unit = keys ? c.k_unit : c.v_unit;
  const int groups = (heads << c.page_shift) * kLanes;
  // A step is kRows rows further: in the page, or so many heads (a page is a multiple of a step, or
  // a step one of a page).
  const int64_t wrap = kRows < P ? dst.head_stride - (int64_t)(P - kRows) * dst.token_stride
                                 : (int64_t)(kRows / P) * dst.head_stride;
  const int64_t next = (int64_t)kRows * dst.token_stride;
  int o = (int)threadIdx.x / kLanes;
  const int first_head = o >> c.page_shift;
  o &= P - 1;
  uint16_t* at = rows + (row_base + o) * dst.token_stride + (head0 + first_head) * dst.head_stride +
                 (int)threadIdx.x % kLanes * 16;
  constexpr int kBatch = 4;  // loads on their way
  // Steps of a whole page's heads need no predicates, and are stored 32 bytes at a time.
  const auto steps_of = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    for (int i0 = threadIdx.x; i0 < groups; i0 += kThreads * kBatch) {
      uint2 x[kBatch];
      uint32_t scale[kBatch];
      int place = o;
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        const int i = i0 + n * kThreads;
        x[n] = make_uint2(0u, 0u);
        scale[n] = 0u;
        if (kWhole || (page >= 0 && i < groups && place >= part.first && place < part.end)) {
          x[n] = __ldg(reinterpret_cast<const uint2*>(codes) + i);
          scale[n] = __ldg(scales + i);
        }
        place = (place + kRows) & (P - 1);
      }
#pragma unroll
      for (int n = 0; n < kBatch; ++n) {
        if (kWhole || (i0 + n * kThreads < groups && o >= part.first && o < part.end)) {
          const float by = codes_to_float2((uint16_t)scale[n]).x * unit;
          uint32_t y[2][4];
          codes4_to_half2(x[n].x, y[0]);
          codes4_to_half2(x[n].y, y[1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = mul2(unpack2<true>(y[j >> 2][j & 3]), make_float2(by, by));
            y[j >> 2][j & 3] = pack2<kFp16>(f.x, f.y);
          }
          if (kWhole) {
            store32(at, y[0], y[1]);
          } else {
            reinterpret_cast<uint4*>(at)[0] = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
            reinterpret_cast<uint4*>(at)[1] = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
          }
        }
        const bool over = o + kRows >= P;
        at += over ? wrap : next;
        o = (o + kRows) & (P - 1);
      }
    }
  };
  if (page >= 0 && part.first == 0 && part.end == P && groups % (kThreads * kBatch) == 0 &&
      in_one_access(dst))
    steps_of(std::true_type());
  else
    steps_of(std::false_type());
}

// As of the 8-bit cache: heads over CTAs until there are a few waves of them (4096 CTAs), and as
// far as a CTA gets `most` numbers then. 108 K tokens of 8 heads x 128 channels in pages of 16, 32,
// 64 and 128: written in 147, 110, 96 and 109 us with 32768, 160, 125, 105 and 110 with 8192, and
// 257, 156, 105 and 110 with a head a CTA; read in 90, 90, 92 and 90 with 8192, 156, 157, 91 and 90
// with 4096, 286, 157, 91 and 90 with a head a CTA. (A cache of one key head has a head a CTA in
// any case: 258 and 286 us for as many numbers in pages of 16.) Eight sequences of 1000 tokens in
// pages of 16: written in 17.6 us, read in 14.1, from 1024 CTAs on 17.1 and 10.0, from 16384 on
// 21.3 and 22.0. (All behind a cold L2.)
dim3 page_grid(const CacheArgs& c, const BatchArgs& b, int most) {
  const int64_t slots = slot_count(b, c.page, 2);
  int y = c.heads;
  while (y > 1 && slots * y > 4096 && c.heads / y * c.page * c.dim < most) y = (y + 1) / 2;
  return dim3((unsigned)slots, (unsigned)y, 2u);
}

template <bool kFp16, int D>
void write_page(const Cache4Args& c, const BatchArgs& b, const RowArgs& k, const RowArgs& v,
                cudaStream_t stream) {
  const dim3 grid = page_grid(c, b, 32768);
  switch (c.page) {
    case 16:
      cache4_write_kernel<kFp16, D, 16><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
    case 32:
      cache4_write_kernel<kFp16, D, 32><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
    case 64:
      cache4_write_kernel<kFp16, D, 64><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
    default:
      cache4_write_kernel<kFp16, D, 128><<<grid, kThreads, 0, stream>>>(c, b, k, v);
      break;
  }
}

}  // namespace

int launch_cache4_write(const Cache4Args& c, const BatchArgs& b, const RowArgs& k,
                        const RowArgs& v, cudaStream_t stream) {
  if (c.dim == 128)
    c.fp16 ? write_page<true, 128>(c, b, k, v, stream) : write_page<false, 128>(c, b, k, v, stream);
  else
    c.fp16 ? write_page<true, 64>(c, b, k, v, stream) : write_page<false, 64>(c, b, k, v, stream);
  return launch_status();
}

int launch_cache4_read(const Cache4Args& c, const BatchArgs& b, const RowArgs& k, const RowArgs& v,
                       cudaStream_t stream) {
  const dim3 grid = page_grid(c, b, 8192);
  if (c.dim == 128) {
    if (c.fp16)
      cache4_read_kernel<true, 128><<<grid, kThreads, 0, stream>>>(c, b, k, v);
    else
      cache4_read_kernel<false, 128><<<grid, kThreads, 0, stream>>>(c, b, k, v);
  } else {
    if (c.fp16)
      cache4_read_kernel<true, 64><<<grid, kThreads, 0, stream>>>(c, b, k, v);
    else
      cache4_read_kernel<false, 64><<<grid, kThreads, 0, stream>>>(c, b, k, v);
  }
  return launch_status();
}

}  // namespace etk
