// lt_kv4_attention.cuh -- what the attention kernels share: their parameters, the
// requests' ranges, query fragments and output stores.
#pragma once

#include <cmath>

#include "lt_async.cuh"
#include "lt_kv4.cuh"

namespace lt {
namespace kv4 {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;  // positions of a tile

struct AttentionParams {
  const void* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;
  const int32_t* positions;
  void* out;
  float* lse;
  int2* plan;       // [requests]: first part, chunks
  float* part_lse;  // [part][kv head][row], in units of log 2; parts: the chunks of requests that have several
  float* part_o;    // [part][kv head][row][D], divided by the part's own sum
  int64_t q_token, q_head;
  int32_t pages, tokens, requests, width, heads, group, shift, list_len, window;
  int32_t parts, target, min_chunk, row_tiles, bf16;
  int32_t max_new;
  int32_t part_rows;  // query rows of a part: max_new * group
  int32_t align;    // positions at which chunks and windows start: multiples of this (32 or 128)
  float scale_log2;
  uint32_t zero;  // 0, which only the host knows (see zero_of)
  // shaped logits: cap tanh(s / cap) where cap > 0, less slope |own position - position|
  const float* slopes;    // [query heads]
  const int32_t* prefix;  // [requests]: positions below it are seen by all of the request's queries
  float cap;              // in units of log 2
  float two_over_cap;     // 2 / cap, of the cap itself
  float one_over_cap;     // 1 / cap, of the cap in units of log 2
  int32_t wide_cap;       // the cap is large against the logits that a hyperbolic tangent by one exponential keeps exact
};

struct Request {
  int length;   // positions in the cache
  int first;    // its first query's row
  int queries;
  int computed;  // the first max_new of them
  int low;      // the first position that any of its queries sees, rounded down to p.align
  int span;     // length - low
};

__device__ __forceinline__ Request request_of(const AttentionParams& p, int r) {
  Request q;
  const int64_t most = min((int64_t)p.width << p.shift, (int64_t)INT32_MAX - 1023);  // (sums of a few tiles stay in 32 bits)
  const int len = max(__ldg(p.lengths + r), 0);
  q.length = (int)(len < most ? len : most);
  int first = r, end = r + 1;
  if (p.starts != nullptr) {
    first = min(max(__ldg(p.starts + r), 0), p.tokens);
    end = min(__ldg(p.starts + r + 1), p.tokens);
  }
  q.first = first;
  q.queries = max(end - first, 0);
  q.computed = min(q.queries, p.max_new);
  q.low = 0;
  if (p.window > 0) q.low = (int)(max((int64_t)q.length - q.queries + 1 - p.window, (int64_t)0) / p.align * p.align);
  if (q.low > q.length) q.low = q.length / p.align * p.align;
  q.span = q.length - q.low;
  return q;
}

// Which request and chunk this CTA has: the requests' positions cut into chunks of one size, flat.
struct Place {
  int request, split, base, count;  // count chunks, the first with flat number base
  int part;                         // where they are several: the number of the first among such chunks
};
// Chunks and, above them, those of requests that have several: one number, so that one scan adds up both.
__device__ __forceinline__ int64_t both_counts(int n) { return n > 1 ? ((int64_t)n << 32) + n : n; }

// The positions of each of a request's chunks: alike, and multiples of p.align.
__device__ __forceinline__ int64_t chunk_of(const AttentionParams& p, const Request& q, int count) {
  return ((int64_t)(q.span + count - 1) / count + p.align - 1) / p.align * p.align;
}

// The requests' spans add up to `total`; with about `target` chunks wanted, a chunk has at most
// total / target positions (a multiple of p.align, min_chunk at least) and request r has
// ceil(span / chunk) of them: ragged requests come out as chunks of like work, which
// the hardware hands to SMs as they fall free. Every CTA computes this from the
// lengths alone.
// For at most 32 requests a warp knows them all: no shared memory, no barrier.
__device__ __forceinline__ bool find_place_in_warp(const AttentionParams& p, int flat, Place* out) {
  const int lane = threadIdx.x & 31;
  Request q = {};
  if (lane < p.requests) q = request_of(p, lane);
  int64_t total = q.span;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
  int64_t chunk = (total + p.target - 1) / p.target;
  chunk = (chunk + p.align - 1) / p.align * p.align;
  if (chunk < p.min_chunk) chunk = p.min_chunk;
  const int n = q.queries > 0 ? max(1, (int)((q.span + chunk - 1) / chunk)) : 0;
  const int64_t own = both_counts(n);
  int64_t sum = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += u;
  }
  const int begin = (int)(sum - own);
  const uint32_t here = __ballot_sync(~0u, flat >= begin && flat < begin + n);
  if (here == 0) return false;
  const int r = __ffs(here) - 1;
  out->request = r;
  out->base = __shfl_sync(~0u, begin, r);
  out->part = __shfl_sync(~0u, (int)((sum - own) >> 32), r);
  out->count = __shfl_sync(~0u, n, r);
  out->split = flat - out->base;
  return true;
}

template <int kCta>
__device__ __forceinline__ bool find_place(const AttentionParams& p, int flat, Place* out, int64_t* sums, Place* found) {
  const int tid = threadIdx.x;
  if (p.requests <= 32) {
    const bool got = find_place_in_warp(p, flat, out);
    __syncthreads();  // (what the caller has set up before is seen by all after this, on both ways)
    return got;
  }
  if (tid == 0) found->request = -1;
  int64_t mine = 0;
  for (int r = tid; r < p.requests; r += kCta) mine += request_of(p, r).span;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(~0u, mine, d);
  if ((tid & 31) == 0) sums[tid >> 5] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll 4
  for (int w = 0; w < kCta / 32; ++w) total += sums[w];
  int64_t chunk = (total + p.target - 1) / p.target;
  chunk = (chunk + p.align - 1) / p.align * p.align;
  if (chunk < p.min_chunk) chunk = p.min_chunk;
  int64_t base = 0;
  for (int first = 0; first < p.requests; first += kCta) {
    const int r = first + tid;
    int n = 0;
    if (r < p.requests) {
      const Request q = request_of(p, r);
      n = q.queries > 0 ? max(1, (int)((q.span + chunk - 1) / chunk)) : 0;
    }
    const int64_t own = both_counts(n);
    int64_t end = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(~0u, end, d);
      if ((tid & 31) >= d) end += u;
    }
    __syncthreads();
    if ((tid & 31) == 31) sums[tid >> 5] = end;
    __syncthreads();
    int64_t all = 0;
#pragma unroll 4
    for (int w = 0; w < kCta / 32; ++w) {
      if (w < (tid >> 5)) end += sums[w];
      all += sums[w];
    }
    const int begin = (int)(base + end - own);
    if (flat >= begin && flat < begin + n) {
      found->request = r;
      found->split = flat - begin;
      found->base = begin;
      found->count = n;
      found->part = (int)((base + end - own) >> 32);
    }
    base += all;
    if ((int)base > flat) break;  // (the same for all threads)
  }
  __syncthreads();
  *out = *found;
  return out->request >= 0;
}

// The request that a query row belongs to; -1 past the last.
__device__ __forceinline__ int owner_of_token(const AttentionParams& p, int token) {
  if (p.starts == nullptr) return token < p.requests ? token : -1;
  if (token < __ldg(p.starts) || token >= __ldg(p.starts + p.requests)) return -1;
  int lo = 0, hi = p.requests - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.starts + mid + 1) > token)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One poll without a time to suspend for: a phase that is complete already, the usual case of a ring that
// runs ahead, is seen at once.
__device__ __forceinline__ bool mbar_ready(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
// A warp waits for a phase, a bounded number of polls; false if it gave up. Every poll ends in a vote, so
// the warp goes on converged.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity) {
  if (__all_sync(~0u, mbar_ready(bar, parity))) return true;
  bool done = false;
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    done = done | mbar_try_wait(bar, parity);
    if (__all_sync(~0u, done)) return true;
  }
  return false;
}

__device__ __forceinline__ void bulk_in(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// 0xFFFF in each half of the word that is no scale of the format: an fp16 NaN, an infinity, or a magnitude above
// 10912 (0x7154), whose product with a code overflows fp16. Weight 0 times such a value would be NaN, so they
// are kept out of the products and put into the rows that see them. (Testing for NaN alone let the others through.)
__device__ __forceinline__ uint32_t unfit_halves(uint32_t h) {
  return ((h & 0x7FFFu) > 0x7154u ? 0xFFFFu : 0u) | ((h & 0x7FFF0000u) > 0x71540000u ? 0xFFFF0000u : 0u);
}

// 0 times each half of the word: zero, or NaN where it is an infinity or a NaN.
__device__ __forceinline__ uint32_t zero_times_halves(uint32_t h) {
  return ((h & 0x7C00u) == 0x7C00u ? 0x7FFFu : 0u) | ((h & 0x7C000000u) == 0x7C000000u ? 0x7FFF0000u : 0u);
}

// bf16 rows become fp16 rows times a power of two: the one that brings the row's largest (magnitude's
// fp32 word `big`) into [2^14, 2^15), so nothing overflows and what lies within 2^-28 of the
// largest stays exact. Rows of zeros, or with an infinity or NaN, are taken as they are.
__device__ __forceinline__ float bf16_row_power(uint32_t big) {
  const int e = (int)(big >> 23);  // biased exponent
  return __uint_as_float((uint32_t)(e == 0 || e == 255 ? 127 : min(268 - e, 253)) << 23);
}
__device__ __forceinline__ uint32_t bf16_pair_to_half(uint32_t w, float mul) {
  const float lo = __uint_as_float(w << 16) * mul, hi = __uint_as_float(w & 0xFFFF0000u) * mul;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
template <int N>
__device__ __forceinline__ uint32_t largest_word(const uint32_t (&w)[N][4]) {
  uint32_t big = 0;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) big = max(big, max(w[j][i] << 16 & 0x7FFF0000u, w[j][i] & 0x7FFF0000u));
  return big;
}
// A row's pieces spread over the four lanes of equal lane / 4; returns the inverse of the power.
template <int N>
__device__ __forceinline__ float bf16_row_to_half(uint32_t (&w)[N][4]) {
  uint32_t big = largest_word<N>(w);
  big = max(big, __shfl_xor_sync(~0u, big, 1));
  big = max(big, __shfl_xor_sync(~0u, big, 2));
  const float mul = bf16_row_power(big);
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][i] = bf16_pair_to_half(w[j][i], mul);
  return 1.0f / mul;
}

// A slope in units of log 2, magnitudes above 2^95 (before the units) as that: its product with a distance, which is below 2^31,
// stays finite, and with a distance of 0 a zero.
__device__ __forceinline__ float bounded_slope(float x) {
  constexpr float kMost = 0x1p95f * 1.4426950408889634f;
  return fminf(fmaxf(x, -kMost), kMost);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) / x for u = x^2 up to 1: the polynomial of degree 6 in u whose largest relative error is least (2^-24, found
// by the exchange method); with its 32-bit steps 3 2^-24.
__host__ __device__ constexpr float tanh_term(int i) {
  return i == 0   ? 0.9999999404f
         : i == 1 ? -0.3333283961f
         : i == 2 ? 0.1332520396f
         : i == 3 ? -0.0534570292f
         : i == 4 ? 0.0202899799f
         : i == 5 ? -0.0062033790f
                  : 0.0010410226f;
}
__device__ __forceinline__ float tanh_over_x(float u) {
  float t = tanh_term(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) t = fmaf(t, u, tanh_term(i));
  return t;
}
// cap tanh(s / cap) in units of log 2, as cap - 2 cap r with r = 1 / (1 + e^2x). In units of 2^-24, absolute: the
// reciprocal is off by 2 of itself and so counts for 4 r, the sum before it for 2 r, the exponential (4 of itself) for 8 r (1 - r),
// its argument's two roundings for 2 x / cosh(x)^2, the last step for |1 - 2 r|: less than 8 together, the most near
// r = 7 / 8. So the capped logit is off by 2^-21 of the cap: for caps to 64 about what 32-bit sums of the products are off
// by. With larger caps, logits up to the cap go by the polynomial. An infinity gives the cap, NaN stays NaN.
__device__ __forceinline__ float capped_by_exp(const AttentionParams& p, float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_fast(s * p.two_over_cap)));
  return fmaf(-2.0f * p.cap, r, p.cap);
}
__device__ __forceinline__ float capped(const AttentionParams& p, float s) {
  float y = capped_by_exp(p, s);
  if (p.wide_cap) {
    const float x = s * p.one_over_cap, u = x * x;
    if (u <= 1.0f) y = s * tanh_over_x(u);
  }
  return y;
}

// Two outputs, rounded once.
__device__ __forceinline__ uint32_t pack_out(const AttentionParams& p, float lo, float hi) {
  uint32_t w;
  if (p.bf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ void store4(const AttentionParams& p, int64_t at, float4 o) {
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_out(p, o.x, o.y), pack_out(p, o.z, o.w));
}

}  // namespace kv4
}  // namespace lt
