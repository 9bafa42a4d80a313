// lt_pages.cu -- page tables and slot maps of the paged cache, made on the GPU
// from the requests' lengths (lt_page_release, lt_page_extend).
//
// What has to be known of a request is a prefix sum over the requests before
// it: how many pages were taken, how many tokens placed. The requests are few
// (hundreds) and the tokens and pages many, so every CTA computes the same
// block-wide scan over all requests (8 bytes a request, from L2 after the first
// CTA) in segments of kSegment, and then writes its share of the segment's
// tokens and pages, finding an item's request by a binary search in the
// scanned sums. One launch does the step. No CTA of extend waits for another one; release runs as one
// cluster, whose CTAs exchange how many pages they found.
//
// Bound by latency. In a graph of the same call 20 times, a call: for 64 requests, 4 of them ended, release
// 4.1 us and extend 3.8; for 1000, 50 ended, up to 128 new tokens each (1.6 MB, a quarter of a microsecond at
// HBM's rate), 5.9 and 5.5. Release took 2.7 and 2.9 when it passed on every cell, pages or not.
// When everything ends at once it has eight SMs: 262144 pages of 64 requests 36 us, 512000 of 2000 requests 71.

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/lt_kv4.h"
#include "lt_kv4.cuh"
#include "lt_launch.h"

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;                     // requests a thread scans at a time
constexpr int kSegment = kThreads * kItems;   // requests per scanned segment

struct PageParams {
  const int32_t* lengths;
  const int32_t* new_tokens;
  const uint8_t* finished;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* num_free;
  int64_t* slots;
  int32_t* positions;
  int32_t* starts;
  int32_t* out_lengths;
  int32_t* out_num_free;
  int32_t requests;
  int32_t width;
  int32_t capacity;
  int32_t shift;  // page_size = 1 << shift
  int32_t max_tokens;
};

struct Sums {
  int64_t a, b;
};

// Inclusive scan of one pair per thread over the block; *total gets the block's sums.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* total, Sums* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t a = __shfl_up_sync(~0u, v.a, d), b = __shfl_up_sync(~0u, v.b, d);
    if (lane >= d) {
      v.a += a;
      v.b += b;
    }
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Sums before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const Sums s = warp_sums[w];
    if (w < warp) {
      before.a += s.a;
      before.b += s.b;
    }
    all.a += s.a;
    all.b += s.b;
  }
  *total = all;
  return {v.a + before.a, v.b + before.b};
}

// The first index of ends[0, n) whose value exceeds x (ends ascending).
__device__ __forceinline__ int owner_of(const int64_t* ends, int n, int64_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp_i32(int64_t x, int64_t lo, int64_t hi) {
  return (int32_t)(x < lo ? lo : x > hi ? hi : x);
}

// Item i of all (counted over the whole grid) belongs to the CTA i / kThreads
// mod the grid, so a CTA's threads write neighbouring items. first: the first
// item of this CTA's threads at or after `from`.
__device__ __forceinline__ int64_t first_item(int64_t from) {
  const int64_t block = from / kThreads;
  const int64_t turn = (block % gridDim.x <= blockIdx.x ? 0 : 1) + block / gridDim.x;
  return (turn * gridDim.x + blockIdx.x) * kThreads;
}

// Which cells of the ended requests hold a page is known only by reading them (a page may have been dropped
// behind a window), so a cell's place on the stack hangs on all the cells before it. The CTAs of one cluster
// take equal runs of a segment's cells, count the pages in theirs, exchange the counts over distributed shared
// memory and write; the first tile of a run, the usual run, stays in registers between the two.
constexpr int kMaxRanks = 8;  // CTAs of a portable cluster

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n barrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ int64_t peer_i64(const int64_t* own, int rank) {
  int64_t v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.s64 %0, [a];\n}"
               : "=l"(v) : "r"((uint32_t)__cvta_generic_to_shared(own)), "r"(rank) : "memory");
  return v;
}

constexpr int kReleaseThreads = 1024;                  // a request each
constexpr int kReleaseTile = kReleaseThreads * kItems;  // cells

// Inclusive scan of one number per thread over the block; *total gets the block's sum.
template <class T>
__device__ __forceinline__ T wide_scan(T v, T* total, T* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T u = __shfl_up_sync(~0u, v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  const T own = warp_sums[lane];  // (32 warps)
  T run = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T u = __shfl_up_sync(~0u, run, d);
    if (lane >= d) run += u;
  }
  *total = __shfl_sync(~0u, run, 31);
  return v + __shfl_sync(~0u, run - own, warp);
}

__global__ void __launch_bounds__(kReleaseThreads) release_kernel(PageParams p) {
  __shared__ int64_t request_sums[32];
  __shared__ int page_sums[32];
  __shared__ int64_t ends[kReleaseThreads];
  __shared__ int32_t held_of[kReleaseThreads];
  __shared__ int64_t counts[2];  // pages in this CTA's cells, by turns: a peer may still read the last segment's
  const int rank = blockIdx.x, ranks = gridDim.x;
  lt::kv4::dependency_wait();
  const int64_t low = clamp_i32(*p.num_free, 0, p.capacity);
  int64_t taken = 0;
  int turn = 0;
  bool met = false;
  for (int base = 0; base < p.requests; base += kReleaseThreads) {
    const int r = base + threadIdx.x;
    int64_t held = 0;
    if (r < p.requests) {
      const int32_t len = p.lengths[r];
      const bool ends_now = p.finished[r] != 0;
      if (ends_now) {
        held = ((int64_t)max(len, 0) + ((1 << p.shift) - 1)) >> p.shift;
        if (held > p.width) held = p.width;
      }
      if (base / kReleaseThreads % ranks == rank) p.out_lengths[r] = ends_now ? 0 : len;
    }
    int64_t cells;
    const int64_t end = wide_scan(held, &cells, request_sums);
    if (cells == 0) continue;  // (the same for all CTAs)
    ends[threadIdx.x] = end;
    held_of[threadIdx.x] = (int32_t)held;
    __syncthreads();
    // a single tile in all is the first CTA's, without an exchange
    const bool alone = cells <= kReleaseTile && p.requests <= kReleaseThreads;
    const int64_t share = alone ? cells : (cells + ranks - 1) / ranks;
    const int64_t from = rank * share < cells ? rank * share : cells, to = from + share < cells ? from + share : cells;
    // kItems neighbouring cells a thread, -1 past the run; how many are pages
    auto read = [&](int64_t at, int32_t (&id)[kItems]) {
      const int64_t first = at + threadIdx.x * kItems;
      // the request of a cell: how many ends are at or below it (side by side for the thread's cells)
      int o[kItems] = {}, pages = 0;
#pragma unroll
      for (int step = kReleaseThreads / 2; step > 0; step /= 2)
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (ends[o[i] + step - 1] <= first + i) o[i] += step;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        id[i] = -1;
        if (first + i < to) id[i] = p.table[(int64_t)(base + o[i]) * p.width + (first + i - (ends[o[i]] - held_of[o[i]]))];
      }
#pragma unroll
      for (int i = 0; i < kItems; ++i) pages += id[i] >= 0;
      return pages;
    };
    auto put = [&](int64_t at, const int32_t (&id)[kItems]) {
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (id[i] >= 0) {
          if (at < p.capacity) p.free_pages[at] = id[i];
          ++at;
        }
    };
    int32_t id[kItems];
    int here;
    const int pages = read(from, id);
    const int upto = wide_scan(pages, &here, page_sums);
    int64_t mine = here;
    if (to - from > kReleaseTile) {
      int64_t more = 0;
      int32_t next[kItems];
      for (int64_t at = from + kReleaseTile; at < to; at += kReleaseTile) more += read(at, next);
      int64_t sum;
      wide_scan(more, &sum, request_sums);
      mine += sum;
    }
    int64_t place = low + taken;
    if (alone) {
      taken = mine;  // (of use to the first CTA)
    } else {
      if (threadIdx.x == 0) counts[turn] = mine;
      cluster_sync();
      for (int q = 0; q < ranks; ++q) {
        const int64_t n = peer_i64(&counts[turn], q);
        if (q < rank) place += n;
        taken += n;
      }
      turn ^= 1;
      met = true;
    }
    put(place + upto - pages, id);
    place += here;
    for (int64_t at = from + kReleaseTile; at < to; at += kReleaseTile) {
      const int n = read(at, id), s = wide_scan(n, &here, page_sums);
      put(place + s - n, id);
      place += here;
    }
    __syncthreads();  // (the next segment's sums go where this one's were read)
  }
  if (rank == 0 && threadIdx.x == 0) *p.out_num_free = clamp_i32(low + taken, 0, p.capacity);
  lt::kv4::dependents_launch();
  if (met) cluster_sync();  // (a CTA's counts stay until its peers have read them)
}

__global__ void __launch_bounds__(kThreads) extend_kernel(PageParams p) {
  __shared__ Sums warp_sums[kThreads / 32];
  __shared__ int64_t token_end[kSegment], page_end[kSegment];
  __shared__ int32_t length_of[kSegment], new_of[kSegment];
  __shared__ int first_bad;
  lt::kv4::dependency_wait();
  const int64_t top = clamp_i32(*p.num_free, 0, p.capacity);
  const int64_t page = (int64_t)1 << p.shift;
  int64_t tokens = 0, pages = 0;  // placed by the segments before
  bool stopped = false;
  for (int base = 0; base < p.requests; base += kSegment) {
    const int count = min(kSegment, p.requests - base);
    if (threadIdx.x == 0) first_bad = stopped ? 0 : kSegment;
    int32_t len[kItems], add[kItems];
    int64_t have[kItems], want[kItems];
    Sums mine = {0, 0};
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int r = base + threadIdx.x * kItems + i;
      len[i] = r < p.requests ? p.lengths[r] : 0;
      add[i] = r < p.requests ? max(p.new_tokens[r], 0) : 0;
      const int64_t l = max(len[i], 0);
      have[i] = (l + page - 1) >> p.shift;
      want[i] = (l + add[i] + page - 1) >> p.shift;
      mine.a += add[i];
      mine.b += want[i] - have[i];
    }
    Sums total;
    const Sums scan = block_scan(mine, &total, warp_sums);
    int64_t t = tokens + scan.a - mine.a, g = pages + scan.b - mine.b;
    int bad = kSegment;
#pragma unroll
    for (int i = kItems - 1; i >= 0; --i) {
      // the sums up to and including request i of this thread
      int64_t ti = t, gi = g;
#pragma unroll
      for (int j = 0; j <= i; ++j) {
        ti += add[j];
        gi += want[j] - have[j];
      }
      const int at = threadIdx.x * kItems + i;
      token_end[at] = ti;
      page_end[at] = gi;
      length_of[at] = max(len[i], 0);
      new_of[at] = add[i];
      const int64_t grown = (int64_t)max(len[i], 0) + add[i];
      if (at < count && (gi > top || ti > p.max_tokens || want[i] > p.width || grown > INT32_MAX)) bad = at;
    }
    bad = __reduce_min_sync(~0u, bad);
    if ((threadIdx.x & 31) == 0 && bad < kSegment) atomicMin(&first_bad, bad);
    __syncthreads();
    const int good = min(count, first_bad);  // requests of this segment that are placed
    const int64_t token_stop = good > 0 ? token_end[good - 1] : tokens;
    const int64_t page_stop = good > 0 ? page_end[good - 1] : pages;
    if ((base / kSegment) % gridDim.x == blockIdx.x) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int at = threadIdx.x * kItems + i;
        if (at < count) {
          p.starts[base + at + 1] = (int32_t)(at < good ? token_end[at] : token_stop);
          p.out_lengths[base + at] = at < good ? length_of[at] + new_of[at] : len[i];
        }
      }
    }
    // fresh pages: the nth one taken is the nth from the top of the stack
    for (int64_t b = first_item(pages); b < page_stop; b += (int64_t)gridDim.x * kThreads) {
      const int64_t i = b + threadIdx.x;
      if (i >= pages && i < page_stop) {
        const int o = owner_of(page_end, good, i);
        const int64_t wants = ((int64_t)length_of[o] + new_of[o] + page - 1) >> p.shift;
        const int64_t col = wants - (page_end[o] - i);
        p.table[(int64_t)(base + o) * p.width + col] = p.free_pages[top - 1 - i];
      }
    }
    for (int64_t b = first_item(tokens); b < token_stop; b += (int64_t)gridDim.x * kThreads) {
      const int64_t i = b + threadIdx.x;
      if (i >= tokens && i < token_stop) {
        const int o = owner_of(token_end, good, i);
        const int64_t l = length_of[o];
        const int64_t pos = l + new_of[o] - (token_end[o] - i);
        const int64_t col = pos >> p.shift, had = (l + page - 1) >> p.shift;
        int32_t id;
        if (col < had) {
          id = p.table[(int64_t)(base + o) * p.width + col];  // written by an earlier step
        } else {
          const int64_t wants = (l + new_of[o] + page - 1) >> p.shift;
          id = p.free_pages[top - 1 - (page_end[o] - (wants - col))];
        }
        p.slots[i] = id < 0 ? -1 : (int64_t)id * page + (pos & (page - 1));
        p.positions[i] = (int32_t)pos;
      }
    }
    stopped = stopped || first_bad < kSegment;
    tokens = token_stop;
    pages = page_stop;
    __syncthreads();
  }
  for (int64_t b = first_item(tokens); b < p.max_tokens; b += (int64_t)gridDim.x * kThreads) {
    const int64_t i = b + threadIdx.x;
    if (i >= tokens && i < p.max_tokens) {
      p.slots[i] = -1;
      p.positions[i] = -1;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.starts[0] = 0;
    *p.out_num_free = (int32_t)(top - pages);
  }
  lt::kv4::dependents_launch();
}

}  // namespace

extern "C" {

lt_status lt_page_release(const int32_t* lengths, const uint8_t* finished, int32_t requests,
                          const int32_t* block_table, int32_t table_width, int32_t* free_pages,
                          int32_t free_capacity, const int32_t* num_free, int32_t page_size,
                          int32_t* out_lengths, int32_t* out_num_free, void* stream) {
  const int shift = lt::kv4::page_shift(page_size);
  if (requests < 0 || table_width < 1 || free_capacity < 0 || shift < 0) return LT_ERR_INVALID_ARG;
  if (num_free == nullptr || out_num_free == nullptr || num_free == out_num_free) return LT_ERR_INVALID_ARG;
  if (free_capacity > 0 && free_pages == nullptr) return LT_ERR_INVALID_ARG;
  if (requests > 0 && (lengths == nullptr || finished == nullptr || block_table == nullptr || out_lengths == nullptr ||
                       lengths == out_lengths))
    return LT_ERR_INVALID_ARG;
  PageParams p = {};
  p.lengths = lengths;
  p.finished = finished;
  p.table = const_cast<int32_t*>(block_table);
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.out_lengths = out_lengths;
  p.out_num_free = out_num_free;
  p.requests = requests;
  p.width = table_width;
  p.capacity = free_capacity;
  p.shift = shift;
  // one cluster: a CTA for every tile of the table, up to the portable size
  const int64_t cells = (int64_t)requests * table_width;
  unsigned ranks = 1;
  while (ranks < kMaxRanks && (int64_t)ranks * kReleaseTile < cells) ranks *= 2;
  return lt::kv4::launch(reinterpret_cast<const void*>(&release_kernel), dim3(ranks), kReleaseThreads, 0, &p, stream, ranks);
}

lt_status lt_page_extend(const int32_t* lengths, const int32_t* new_tokens, int32_t requests,
                         int32_t* block_table, int32_t table_width, const int32_t* free_pages,
                         int32_t free_capacity, const int32_t* num_free, int32_t page_size,
                         int32_t max_tokens, int64_t* out_slots, int32_t* out_positions,
                         int32_t* out_starts, int32_t* out_lengths, int32_t* out_num_free,
                         void* stream) {
  const int shift = lt::kv4::page_shift(page_size);
  if (requests < 0 || table_width < 1 || free_capacity < 0 || shift < 0 || max_tokens < 0) return LT_ERR_INVALID_ARG;
  if (num_free == nullptr || out_num_free == nullptr || num_free == out_num_free || out_starts == nullptr)
    return LT_ERR_INVALID_ARG;
  if (free_capacity > 0 && free_pages == nullptr) return LT_ERR_INVALID_ARG;
  if (max_tokens > 0 && (out_slots == nullptr || out_positions == nullptr)) return LT_ERR_INVALID_ARG;
  if (requests > 0 && (lengths == nullptr || new_tokens == nullptr || block_table == nullptr ||
                       out_lengths == nullptr || lengths == out_lengths || new_tokens == out_lengths))
    return LT_ERR_INVALID_ARG;
  PageParams p = {};
  p.lengths = lengths;
  p.new_tokens = new_tokens;
  p.table = block_table;
  p.free_pages = const_cast<int32_t*>(free_pages);
  p.num_free = num_free;
  p.slots = out_slots;
  p.positions = out_positions;
  p.starts = out_starts;
  p.out_lengths = out_lengths;
  p.out_num_free = out_num_free;
  p.requests = requests;
  p.width = table_width;
  p.capacity = free_capacity;
  p.shift = shift;
  p.max_tokens = max_tokens;
  int64_t grid = ((int64_t)max_tokens + 4 * kThreads - 1) / (4 * kThreads);
  grid = grid < 1 ? 1 : grid > 152 ? 152 : grid;
  return lt::kv4::launch(reinterpret_cast<const void*>(&extend_kernel), dim3((unsigned)grid), kThreads, 0, &p, stream);
}

}  // extern "C"
