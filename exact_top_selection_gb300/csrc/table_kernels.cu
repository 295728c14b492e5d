// Sequences that grow and shrink on the GPU (exact_topk_update_tables): lengths, row ranges,
// pages from a ring of free ones and back to it, and each new row's slot and position.
//
// Everything a sequence needs to know of the others is four sums over the sequences before it:
// of the pages asked for, of the pages given back, of the rows asked for and of the rows granted.
// Every CTA forms them for itself, in shared memory. A page taken is then a place in the ring, or,
// behind the pages that were free, one that another sequence gives back in this call; that
// sequence's table still names it. So all pages and rows can be filled in at once, in any order, and
// no page is counted by an atomic: results do not depend on timing. The last CTA to have read the
// lengths and the ring's place writes the new ones.
//
// Little is moved (4 bytes for a page, 8 for a row): a call is bound by its latency, 3.2 us for a
// decoding step of 64 sequences, 7.4 for 1000 prompts of 1 M tokens in pages of 16. Of those 7.4
// the sums over the sequences are most: 1000 sequences with a token each take 6.6, one sequence
// 4.0, and 4096 15.6. They are five scans of 64 bits, one behind the other's exchange, in every
// CTA. (A CTA that forms them ahead of a second kernel that fills in took 11.4.)

#include <climits>

#include "batch_internal.h"
#include "cache_device.cuh"

namespace etk {
namespace {

// One CTA does it all where there are few units, as many as the call may have: it saves the last
// arrival (64 sequences x 1 token, 129 units, 3.8 us against 4.1), but fills unit by unit what many
// fill at once. Where all units are in use the two cross at about 300: 64 x 8 tokens, 160 units,
// 4.4 and 4.6; 256 x 1 token, 528 units, 6.6 and 5.6; 64 x 128 tokens, 640 units, 7.7 and 6.1;
// beyond the limit 11.6 and 6.2 for 1064 units, 25.8 and 6.9 for 3000. (Device time behind a cold
// L2.)
constexpr int kAloneThreads = 256;
constexpr int kAloneUnits = 1024;
constexpr int kThreads = 512;
// Two CTAs an SM: 66 K units 7.8 us (152 CTAs 7.9, 608 7.8), 250 K units 10.1 (12.0, 12.8), a
// million 25.0 (32.0, 28.1).
constexpr int kMostCtas = 304;
constexpr int kOwnRows = 4;         // a unit's rows that its own thread writes

__device__ __forceinline__ int pages_of(int length, int shift) {
  return (int)(((int64_t)length + (1 << shift) - 1) >> shift);
}

__device__ __forceinline__ int length_of(const TableArgs& a, int seq) {
  const int64_t most = (int64_t)a.width << a.page_shift;
  const int n = a.kv_len[seq];
  return n < 0 ? 0 : (n > most ? (int)most : n);
}

// In shared memory: of each sequence its length before the call, its first place among the pages
// taken and among those given back, and its first row; and where the ring was.
struct Work {
  int32_t *length, *take, *give, *start, *ring;
  __device__ Work(int32_t* at, int num_seqs)
      : length(at), take(length + num_seqs + 1), give(take + num_seqs + 1),
        start(give + num_seqs + 1), ring(start + num_seqs + 1) {}
};

size_t work_bytes(int num_seqs) { return (4 * ((size_t)num_seqs + 1) + 2) * 4; }

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

// What the filling needs to know; then, by the last CTA to come so far, lengths, row ranges and the
// ring's new place.
template <int kEach>
__device__ __forceinline__ void plan(const TableArgs& a, const Work& work) {
  __shared__ int64_t shared3[32][3], shared2[32][2];
  __shared__ int s_last;
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
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int seq = tid * kEach + i;
    const int64_t first = take;
    take += need[i];
    asked += change[i] > 0 ? change[i] : 0;
    if (change[i] > 0 && ((need[i] > 0 && take > there) || asked > a.max_tokens)) change[i] = 0;
    if (change[i] > 0) {
      got[0] += change[i];
      got[1] += need[i];
    }
    if (seq < a.num_seqs) {
      work.length[seq] = length[i];
      work.take[seq] = (int)(first < a.num_pages ? first : a.num_pages);
      work.give[seq] = (int)(give < a.num_pages ? give : a.num_pages);
    }
    give += back[i];
  }
  sums_before<2>(got, all_got, shared2);
  int64_t row = got[0];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int seq = tid * kEach + i;
    if (seq < a.num_seqs) work.start[seq] = (int)row;
    row += change[i] > 0 ? change[i] : 0;
  }
  if (tid == 0) {
    work.start[a.num_seqs] = (int)all_got[0];
    work.give[a.num_seqs] = (int)given;
    work.ring[0] = head;
    work.ring[1] = have;
    // every thread has read what it needs (sums_before waits for all)
    s_last = gridDim.x == 1;
    if (gridDim.x > 1) {
      __threadfence();
      s_last = atomicAdd(a.arrived, 1) == (int)gridDim.x - 1;
      if (s_last) __threadfence();  // nothing is written before all have read
    }
  }
  __syncthreads();
  if (!s_last) return;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int seq = tid * kEach + i;
    if (seq >= a.num_seqs) continue;
    a.kv_len[seq] = (int)(length[i] + change[i]);
    a.q_start[seq] = work.start[seq];
    if (a.applied != nullptr) a.applied[seq] = (int)change[i];
  }
  if (tid == 0) {
    const int64_t free = have + given - all_got[1];
    a.q_start[a.num_seqs] = (int)all_got[0];
    a.free_range[0] = (int)((head + all_got[1]) % a.num_pages);
    a.free_range[1] = (int)(free < a.num_pages ? free : a.num_pages);
    if (gridDim.x > 1) *a.arrived = 0;
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
  const int kept = pages_of(w.length[seq], a.page_shift) - (w.give[seq + 1] - w.give[seq]);
  return a.table[(int64_t)seq * a.pitch + kept + (q - w.give[seq])];
}

// Pages and rows, a CTA's units by its index: a unit is the part of a page that a sequence's new rows
// reach, its slots laid out by first_slot. With all threads of the CTA.
template <int kUnits>
__device__ __forceinline__ void fill(const TableArgs& a, const Work& work, int64_t units) {
  __shared__ int s_row[kUnits], s_count[kUnits], s_slot[kUnits], s_position[kUnits];
  const int P = 1 << a.page_shift, tid = threadIdx.x;
  const int head = work.ring[0], have = work.ring[1];
  BatchArgs b{};
  b.q_start = work.start;
  b.num_tokens = a.max_tokens;
  b.num_seqs = a.num_seqs;
  for (int64_t base = (int64_t)blockIdx.x * kUnits; base < units;
       base += (int64_t)gridDim.x * kUnits) {
    const int count = units - base < kUnits ? (int)(units - base) : kUnits;
    bool many = false;
    if (tid < count) {
      const int64_t unit = base + tid;
      const int seq = sequence_of_slot(b, unit, P, 2);
      const int index = (int)(unit - first_slot(b, seq, P, 2));
      const int begin = work.start[seq], rows = work.start[seq + 1] - begin;
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

template <int kUnits, int kEach>
__global__ void __launch_bounds__(kUnits) update_tables_kernel(TableArgs a, int64_t units) {
  extern __shared__ int32_t words[];
  const Work work(words, a.num_seqs);
  plan<kEach>(a, work);
  if (work.give[a.num_seqs] > 0)
    give_back(a, work, (int64_t)blockIdx.x * kUnits + threadIdx.x, (int64_t)gridDim.x * kUnits);
  if (work.start[a.num_seqs] > 0) fill<kUnits>(a, work, units);
}

template <int kUnits, int kEach>
int launch(const TableArgs& a, int64_t units, int64_t ctas, cudaStream_t stream) {
  constexpr size_t most = (4 * ((size_t)EXACT_TOPK_MAX_SEQS + 1) + 2) * 4;
  const auto kernel = update_tables_kernel<kUnits, kEach>;
  const size_t bytes = work_bytes(a.num_seqs);
  // the largest call's size: the limit is the kernel's, whichever thread launches it
  if (bytes > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                (int)most) != cudaSuccess) {
    cudaGetLastError();
    return EXACT_TOPK_ERR_CUDA;
  }
  kernel<<<(unsigned)ctas, kUnits, bytes, stream>>>(a, units);
  return launch_status();
}

}  // namespace

int launch_update_tables(const TableArgs& a, cudaStream_t stream) {
  // units of the new rows, at most
  const int64_t units = (a.max_tokens >> a.page_shift) + 2 * (int64_t)a.num_seqs;
  if (units <= kAloneUnits) {
    if (a.num_seqs <= kAloneThreads) return launch<kAloneThreads, 1>(a, units, 1, stream);
    return launch<kAloneThreads, 2>(a, units, 1, stream);
  }
  const int64_t ctas = (units + kThreads - 1) / kThreads;
  const int64_t some = ctas < kMostCtas ? ctas : kMostCtas;
  if (a.num_seqs <= kThreads) return launch<kThreads, 1>(a, units, some, stream);
  if (a.num_seqs <= 2 * kThreads) return launch<kThreads, 2>(a, units, some, stream);
  if (a.num_seqs <= 4 * kThreads) return launch<kThreads, 4>(a, units, some, stream);
  return launch<kThreads, 8>(a, units, some, stream);
}

}  // namespace etk
