// Sequences that grow and shrink on the GPU (exact_topk_update_tables): lengths, row ranges,
// pages from a ring of free ones and back to it, and each new row's slot and position.
//
// Everything a sequence needs to know of the others is four sums over the sequences before it:
// of the pages asked for, of the pages given back, of the rows asked for and of the rows granted.
// One CTA forms them. A page taken is then a place in the ring, or, behind the pages that
// were free, one that another sequence gives back in this call; that sequence's table still
// names it. So all pages and rows can be filled in at once, in any order, and no page is
// counted by an atomic: results do not depend on timing.
//
// Little is moved (4 bytes for a page, 8 for a row): a decoding step is bound by its latency.

#include <climits>

#include "batch_internal.h"
#include "cache_device.cuh"

namespace etk {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kFill = 256;  // threads and units of a CTA that fills in
constexpr int kAloneUnits = 1024;  // one CTA does it all up to here
constexpr int kOwnRows = 4;        // a unit's rows that its own thread writes

__device__ __forceinline__ int pages_of(int length, int shift) {
  return (int)(((int64_t)length + (1 << shift) - 1) >> shift);
}

__device__ __forceinline__ int length_of(const TableArgs& a, int seq) {
  const int64_t most = (int64_t)a.width << a.page_shift;
  const int n = a.kv_len[seq];
  return n < 0 ? 0 : (n > most ? (int)most : n);
}

// Where the sums and the ring's place before the call are kept, and the row ranges: in the workspace,
// or, where one CTA does it all, in its shared memory.
struct Work {
  int32_t *length, *take, *give, *ring, *q_start;
  __device__ Work(int32_t* at, int num_seqs, int32_t* starts)
      : length(at), take(length + num_seqs + 1), give(take + num_seqs + 1),
        ring(give + num_seqs + 1), q_start(starts) {}
};

// Sums over the CTA's threads before each, and over all of them.
template <int N>
__device__ __forceinline__ void sums_before(int64_t (&x)[N], int64_t (&all)[N],
                                            int64_t (*shared)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t own[N], first[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    own[i] = x[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, x[i], o);
      if (lane >= o) x[i] += up;
    }
    if (lane == 31) shared[warp][i] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    first[i] = lane < warps ? shared[lane][i] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(~0u, first[i], o);
      if (lane >= o) first[i] += up;
    }
    all[i] = __shfl_sync(~0u, first[i], 31);
    const int64_t before = __shfl_sync(~0u, first[i], warp > 0 ? warp - 1 : 0);
    x[i] += (warp > 0 ? before : 0) - own[i];
  }
}

// Lengths, row ranges, the ring's new place, and what the filling needs to know.
template <int kEach>
__device__ __forceinline__ void plan(const TableArgs& a, const Work& work) {
  __shared__ int64_t shared3[kMostThreads / 32][3];
  __shared__ int64_t shared2[kMostThreads / 32][2];
  const int tid = threadIdx.x;
  const int64_t most = (int64_t)a.width << a.page_shift;
  int head = a.free_range[0] % a.num_pages;
  if (head < 0) head += a.num_pages;
  int have = a.free_range[1];
  have = have < 0 ? 0 : (have > a.num_pages ? a.num_pages : have);

  int length[kEach], need[kEach], back[kEach];
  int64_t change[kEach];  // what is asked for; 0 where it does not fit the table
  int64_t sum[3] = {0, 0, 0}, all[3];  // pages asked for, pages given back, rows asked for
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int seq = tid * kEach + i;
    length[i] = need[i] = back[i] = 0;
    change[i] = 0;
    if (seq < a.num_seqs) {
      length[i] = length_of(a, seq);
      change[i] = a.negate ? -(int64_t)a.change[seq] : (int64_t)a.change[seq];
      if (change[i] < -(int64_t)length[i]) change[i] = -(int64_t)length[i];
      if (length[i] + change[i] > most) change[i] = 0;
      const int after = pages_of((int)(length[i] + change[i]), a.page_shift);
      const int before = pages_of(length[i], a.page_shift);
      need[i] = after > before ? after - before : 0;
      back[i] = before > after ? before - after : 0;
    }
    sum[0] += need[i];
    sum[1] += back[i];
    sum[2] += change[i] > 0 ? change[i] : 0;
  }
  sums_before<3>(sum, all, shared3);
  const int64_t given = all[1] < a.num_pages ? all[1] : a.num_pages;
  const int64_t there = have + given;
  int64_t take = sum[0], give = sum[1], asked = sum[2];
  int64_t got[2] = {0, 0}, all_got[2];  // rows granted, pages taken
  int64_t first_take[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    first_take[i] = take;
    take += need[i];
    asked += change[i] > 0 ? change[i] : 0;
    if (change[i] > 0 && ((need[i] > 0 && take > there) || asked > a.max_tokens)) change[i] = 0;
    if (change[i] > 0) {
      got[0] += change[i];
      got[1] += need[i];
    }
  }
  sums_before<2>(got, all_got, shared2);
  int64_t row = got[0];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int seq = tid * kEach + i;
    if (seq >= a.num_seqs) continue;
    a.kv_len[seq] = (int)(length[i] + change[i]);
    if (a.applied != nullptr) a.applied[seq] = (int)change[i];
    a.q_start[seq] = work.q_start[seq] = (int)row;
    row += change[i] > 0 ? change[i] : 0;
    work.length[seq] = length[i];
    work.take[seq] = (int)(first_take[i] < a.num_pages ? first_take[i] : a.num_pages);
    work.give[seq] = (int)(give < a.num_pages ? give : a.num_pages);
    give += back[i];
  }
  if (tid == 0) {
    a.q_start[a.num_seqs] = work.q_start[a.num_seqs] = (int)all_got[0];
    work.give[a.num_seqs] = (int)given;
    work.ring[0] = head;
    work.ring[1] = have;
    const int64_t free = have + given - all_got[1];
    a.free_range[0] = (int)((head + all_got[1]) % a.num_pages);
    a.free_range[1] = (int)(free < a.num_pages ? free : a.num_pages);
  }
}

// The sequence that gives back the page at place q, q below the number given back.
__device__ __forceinline__ int giver(const Work& w, int num_seqs, int q) {
  int lo = 0, hi = num_seqs - 1;  // the last one whose first place is at or before q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (w.give[mid] <= q)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int page_given(const TableArgs& a, const Work& w, int q) {
  const int seq = giver(w, a.num_seqs, q);
  const int kept = pages_of(a.kv_len[seq], a.page_shift);
  return a.table[(int64_t)seq * a.pitch + kept + (q - w.give[seq])];
}

// Pages and rows of `units` units from `unit0` on: a unit is the part of a page that a sequence's
// new rows reach, its slots laid out by first_slot. With all threads of the CTA.
__device__ __forceinline__ void fill(const TableArgs& a, const Work& work, int64_t unit0,
                                     int units) {
  __shared__ int s_row[kFill], s_count[kFill], s_slot[kFill], s_position[kFill];
  const int P = 1 << a.page_shift, tid = threadIdx.x;
  const int head = work.ring[0], have = work.ring[1];
  BatchArgs b{};
  b.q_start = work.q_start;
  b.num_tokens = a.max_tokens;
  b.num_seqs = a.num_seqs;
  for (int base = 0; base < units; base += kFill) {
    const int count = units - base < kFill ? units - base : kFill;
    bool many = false;
    if (tid < count) {
      const int64_t unit = unit0 + base + tid;
      const int seq = sequence_of_slot(b, unit, P, 2);
      const int index = (int)(unit - first_slot(b, seq, P, 2));
      const int begin = work.q_start[seq], rows = work.q_start[seq + 1] - begin;
      const int length = work.length[seq];
      const int place = (length >> a.page_shift) + index;  // of the page in the sequence
      const int64_t from = (int64_t)place << a.page_shift;
      const int first = length > from ? length : (int)from;
      const int64_t end = (int64_t)length + rows < from + P ? (int64_t)length + rows : from + P;
      s_count[tid] = 0;
      if (index >= 0 && rows > 0 && end > first) {
        int32_t* const at = a.table + (int64_t)seq * a.pitch + place;
        int page;
        if (first > from) {
          page = *at;  // the page that the sequence had begun
        } else {
          const int i = work.take[seq] + place - pages_of(length, a.page_shift);
          const int64_t in_ring = (int64_t)head + i;
          page = i < have ? a.free_pages[in_ring < a.num_pages ? in_ring : in_ring - a.num_pages]
                          : page_given(a, work, i - have);
          *at = page;
        }
        const int row = begin + (first - length), slot = page * P + (first - (int)from);
        many = (int)end - first > kOwnRows;
        if (many) {
          s_row[tid] = row;
          s_count[tid] = (int)end - first;
          s_slot[tid] = slot;
          s_position[tid] = first;
        } else {
          for (int o = 0; o < (int)end - first; ++o) {
            if (a.slots != nullptr) a.slots[row + o] = slot + o;
            if (a.positions != nullptr) a.positions[row + o] = first + o;
          }
        }
      }
    }
    if (__syncthreads_or(many) && (a.slots != nullptr || a.positions != nullptr))
      for (int i = tid; i < count << a.page_shift; i += blockDim.x) {
        const int u = i >> a.page_shift, o = i & (P - 1);
        if (o >= s_count[u]) continue;
        if (a.slots != nullptr) a.slots[s_row[u] + o] = s_slot[u] + o;
        if (a.positions != nullptr) a.positions[s_row[u] + o] = s_position[u] + o;
      }
    __syncthreads();
  }
}

// Pages given back, behind the free ones. `threads` threads of which this one is `index`.
__device__ __forceinline__ void give_back(const TableArgs& a, const Work& work, int64_t index,
                                          int64_t threads) {
  const int given = work.give[a.num_seqs];
  const int64_t begin = (int64_t)work.ring[0] + work.ring[1];
  for (int64_t q = index; q < given; q += threads)
    a.free_pages[(begin + q) % a.num_pages] = page_given(a, work, (int)q);
}

template <int kEach>
__global__ void __launch_bounds__(kMostThreads) plan_tables_kernel(TableArgs a) {
  plan<kEach>(a, Work(a.work, a.num_seqs, a.q_start));
}

__global__ void __launch_bounds__(kFill) fill_tables_kernel(TableArgs a, int64_t units) {
  const Work work(a.work, a.num_seqs, a.q_start);
  give_back(a, work, (int64_t)blockIdx.x * kFill + threadIdx.x, (int64_t)gridDim.x * kFill);
  const int64_t unit0 = (int64_t)blockIdx.x * kFill;
  const int64_t left = units - unit0;
  if (left > 0) fill(a, work, unit0, left < kFill ? (int)left : kFill);
}

// Both in one CTA, of few units: so of at most kAloneUnits / 2 sequences.
__global__ void __launch_bounds__(kAloneUnits / 2) update_tables_kernel(TableArgs a, int units) {
  constexpr int kSeqs = kAloneUnits / 2 + 1;
  __shared__ int32_t words[3 * kSeqs + 2], starts[kSeqs];
  const Work work(words, a.num_seqs, starts);
  plan<1>(a, work);
  __syncthreads();
  if (work.give[a.num_seqs] > 0) give_back(a, work, threadIdx.x, blockDim.x);
  if (starts[a.num_seqs] > 0) fill(a, work, 0, units);
}

}  // namespace

int launch_update_tables(const TableArgs& a, cudaStream_t stream) {
  // units of the new rows, at most
  const int64_t units = (a.max_tokens >> a.page_shift) + 2 * (int64_t)a.num_seqs;
  const int threads = (a.num_seqs + 31) / 32 * 32;
  if (units <= kAloneUnits) {
    update_tables_kernel<<<1, threads < kFill ? kFill : threads, 0, stream>>>(a, (int)units);
    return launch_status();
  }
  if (threads <= kMostThreads)
    plan_tables_kernel<1><<<1, threads, 0, stream>>>(a);
  else
    plan_tables_kernel<4><<<1, kMostThreads, 0, stream>>>(a);
  int64_t ctas = (units + kFill - 1) / kFill;
  if (ctas < 64) ctas = 64;  // to give pages back
  if (cudaPeekAtLastError() == cudaSuccess)
    fill_tables_kernel<<<(unsigned)ctas, kFill, 0, stream>>>(a, units);
  return launch_status();
}

}  // namespace etk
