// lt_kv4_prefill.cuh -- attention over the 4-bit cache for many query rows a
// request (prefill chunks): tcgen05 with the sums in tensor memory; one translation unit
// without and one with shaped logits (caps, slopes, prefixes).
//
// A CTA takes 256 query rows of one kv head (two tiles of 128, a thread a row) and a
// range of positions in tiles of 128, with one role a warpgroup:
//   warpgroups 0 and 1  softmax of row tile A and B: logits from tensor memory,
//                       weights back into it as fp16, where the second product reads them
//   warpgroup 2         unpacks: a thread turns one position's key or value codes into fp16,
//                       written with the 128-byte swizzle that the tensor core reads
//   warpgroup 3         one warp issues the products, another the bulk copies of packed rows
// in the order  S_A(i) = Q_A K(i)^T,  O_B += P_B(i-1) V(i-1),  S_B(i),  O_A += P_A(i) V(i): while one row
// tile's softmax runs, the tensor core has the other's two products.
//
// Keys are laid out channels inner (K-major), values are the same bytes read as
// the transposed operand (their channels are the product's N). Unpacked tiles live in a
// ring of four; the packed rows' pitch is an odd multiple of 16 bytes (with heads of 256
// twice one), so eight threads reading 16 bytes of eight rows touch all banks (half of them), and the
// swizzle does the same for their stores.
//
// With heads of 256 tensor memory holds one row tile's sums, its queries and two tiles
// of logits of 64 positions: the order is  S(0), S(1), O += P(0) V(0), S(2), O += P(1) V(1), S(3), ... ,
// so that one position tile's softmax runs beside the next one's first product and the last
// one's second, and warpgroup 1 unpacks too.
//
// The running maximum moves only when a row's logits pass it by 2^8 (the sums are
// then rescaled in tensor memory, seldom); weights are held as 2^6 exp(s - max) at
// most 2^14, so fp16 neither overflows nor goes subnormal above 2^-20.
//
// What bounds it: the chain softmax, second product, next first product of a row tile.
// An iteration (both row tiles by 128 positions of D = 128) takes some 3100 clocks, the
// products alone 2048 (64 each, in every operand mode); the softmax's part is some 1700 from the logits'
// arrival to the weights'. What the chain gave up on the way, on a chunk of 2048 tokens
// behind 14336 positions (32 query heads on 8 kv heads): 941 us with one lane issuing, 716
// with the warp issuing and copies in a warp of their own, 650 with short loops and whole-line
// queries and outputs, 511 without cutting requests that fill the SMs, 494 with four
// products a statement, 424 with named barriers, 410 with the longest row tiles first (405 to 416 since
// packed stages are handed back by what was loaded from them): 1.25 PFLOP/s, 65% of cuBLAS's burst; 84% is the most
// that two waves of 256 CTAs on 152 SMs allow. Measured and dropped: a quarter, a third or half of the exponentials on the FMA
// pipes (541, 557, 621 us against 511), two threads a row (541), the first half's weights taken
// before the tile's maximum is known (804 against 716).
//
// Heads of 256, the same chunk: 5063 us with the kernel for few rows; here 1586 with queries
// in shared memory and a key and a value tile, 1238 with the queries in tensor memory and three tiles, 1100 with
// eight warps unpacking, 854 with tiles of 64, logits a tile ahead and five packed stages in place of three
// of 32 positions (1160 with those), 877 since packed stages are handed back by what was loaded from them: 1.18
// PFLOP/s, 61% of cuBLAS's burst, where four waves of 512 CTAs on 152 SMs allow 84%. The unpacked tile's way, read,
// write and fence, is what is left: 748 us without its writes.
//
// Shaped logits (caps, slopes, prefixes) pass once more through tensor memory: shaped, hidden and their maximum taken
// 32 columns at a time. A cap is a polynomial while the logits are below it (12 instructions a logit in all; by
// exponential and reciprocal, which the special function unit has to do for the softmax already, 1066 us against 1031 on the
// chunk below); the chain from a tile's logits to its weights is what bounds it, twice the plain one's: 2048
// tokens behind 14336, 32 query heads on 8 kv heads of 128, cap and slopes, 987 us (411 plain; 975 before stages were handed
// back so, and slopes of each row's own kind). Dropped: no shaping before the
// weights where a bound shows that the maximum stays (1148: with slopes it moves, with a cap alone the two readings cost as
// much), 16 columns at a time (1135).
//
// A value that is NaN, or whose scale is outside the format, is unpacked as zero, and the rows that see it note
// the group: a row's output is NaN there whatever its weight, and rows that do not see it stay clean.

#pragma once

#include "lt_kv4.cuh"
#include "lt_kv4_attention.cuh"
#include "lt_kv4_prefill.h"
#include "lt_kv4_tcgen05.cuh"

namespace {

using namespace lt::kv4;

constexpr int kCta = 512;
constexpr int kSlots = 4;    // unpacked key or value tiles in shared memory
constexpr int kPart = 64;    // positions of a packed stage
constexpr int kMaxRaw = 5;   // packed stages in shared memory or on their way there
// columns of tensor memory: logits and weights first, two tiles
constexpr int kQueryColumn = 128;  // queries, with heads of 256
constexpr int kSumColumn = 256;
constexpr float kShift = 6.0f;
constexpr float kSlack = 8.0f;  // how far logits may pass the maximum (log 2) before it moves

template <int D>
struct Smem {
  static constexpr int kRow = row_bytes(D);
  // Heads of 256 leave room for one row tile. Its queries are in tensor memory, and its position tiles are
  // of 64: two of logits (128 columns), the queries (128) and the sums (256) fit, so that the next
  // tile's logits are there when the softmax of this one ends, and shared memory has room for five packed stages.
  static constexpr bool kOne = D == 256;
  static constexpr int kRowTiles = kOne ? 1 : 2;
  static constexpr int kTok = kOne ? 64 : 128;             // positions of a tile
  static constexpr int kRaw = kOne ? 5 : 3;
  static constexpr int kUnpackers = kOne ? 256 : 128;      // threads that unpack: row tile B's warpgroup is free to
  static constexpr int kParts = kTok / kPart;
  static constexpr int kRing = 512 / kTok;                 // tiles whose notes are kept
  static_assert(kSlots / 2 * kParts + kRaw < kRing * kParts, "notes are read before they are written over");
  static constexpr int kQHalf = 128 * 128;                 // 128 rows by 64 channels, swizzled
  static constexpr int kQTile = kQHalf * (D / 64);
  static constexpr int kHalf = kTok * 128;                 // a tile's positions by 64 channels
  static constexpr int kOperand = kHalf * (D / 64);
  static constexpr int kKv = kOne ? 0 : kRowTiles * kQTile;  // kSlots
  // row tiles; where the queries are in tensor memory, the last slots are what they and the outputs are turned
  // round in, before their first keys and after the last product
  static constexpr int kQ = kOne ? kKv + kSlots * kOperand - kQTile : 0;
  static constexpr int kPacked = kKv + kSlots * kOperand;  // [kRaw][kPart rows]
  static constexpr int kBars = kPacked + kRaw * kPart * kRow;
  static constexpr int kTotal = kBars + 2048 + 1024;     // (slack to align the start to 1024)
};

struct Shared {
  uint64_t packed_full[kMaxRaw], packed_empty[kMaxRaw];
  uint64_t kv_empty[kSlots];
  uint64_t q_full, s_full[2], o_full[2];
  uint64_t o_tile;  // with one row tile: a position tile's second product is done
  // notes of the tiles in work, a ring of 512 positions, eight packed stages. They are made up to seven stages
  // ahead of the softmax (Smem's assertion): while it reads tile i's, tile i's values are not given back, so the
  // unpackers have released at most the first stage of tile i + kSlots / 2, and the copies run kRaw stages on from there
  alignas(16) uint32_t valid[16];     // positions on a page of the cache and in range, as bits
  alignas(16) uint32_t nan_rows[16];  // positions with a value scale that is NaN or outside the format
  uint8_t nan_groups[512];
  int64_t sums[kCta / 32];
  Place found;
  uint32_t tmem;
  int gave_up;
};
static_assert(sizeof(Shared) <= 2048, "shared state");

// A warp waits for a phase, kWaitPolls polls at most; a wait that gives up marks the CTA, whose outputs are NaN
// then, and the warp goes on: the roles keep their steps, so nobody waits for one that has
// left. Every poll ends in a vote, so the warp's control flow is uniform: the callers go on to .aligned
// instructions.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Shared* sh) {
  bool done = mbar_ready(bar, parity);
  if (__all_sync(~0u, done)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < lt::kWaitPolls; ++i) {
    done = done | lt::mbar_try_wait(bar, parity);
    if (__all_sync(~0u, done)) return true;
  }
  *(volatile int*)&sh->gave_up = 1;
  return false;
}

// What the issuing warp waits for comes over the CTA's named barriers: it sees them within some 50 clocks, where
// a look at an mbarrier takes 250 and more while the products keep shared memory busy. A named
// barrier's wait has no limit of its own; it ends because every role keeps its steps, also
// after a wait that gave up.
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("barrier.cta.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ int weights_ready(int which, int half) { return 1 + 2 * which + half; }
constexpr int kWeightsThreads = 128 + 32;
__device__ __forceinline__ int slot_ready(int slot) { return 5 + slot; }
template <int D>
constexpr int kSlotThreads = Smem<D>::kUnpackers / 2 + 32;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 lanes at once
__device__ __forceinline__ void fma2(float& x0, float& x1, float f, float a) {
  asm("{\n .reg .b64 x, f, a;\n mov.b64 x, {%0, %1};\n mov.b64 f, {%2, %2};\n mov.b64 a, {%3, %3};\n"
      " fma.rn.f32x2 x, x, f, a;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1) : "f"(f), "f"(a));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  asm("{\n .reg .b64 x, s;\n mov.b64 s, {%0, %1};\n mov.b64 x, {%2, %3};\n add.rn.f32x2 s, s, x;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(s0), "+f"(s1) : "f"(x0), "f"(x1));
}
__device__ __forceinline__ void mul2(float& x0, float& x1, float f) {
  asm("{\n .reg .b64 x, f;\n mov.b64 x, {%0, %1};\n mov.b64 f, {%2, %2};\n mul.rn.f32x2 x, x, f;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1) : "f"(f));
}
// (d0, d1) = (a0 b0 + c, a1 b1 + c)
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c) {
  asm("{\n .reg .b64 d, a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %6};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c));
}
// What a CTA works on: row0 .. of the request's query rows, positions [from, to).
struct Job {
  Request rq;
  int request, head, row_tile, flat, part, rows, row0, from, to, tiles;
  bool two, final_here;
};

// ---- one row tile's softmax: a thread a row
template <int D, bool kShaped>
__device__ __forceinline__ void softmax_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem, int which) {
  constexpr int kHalf = Smem<D>::kQHalf, kTok = Smem<D>::kTok, kRing = Smem<D>::kRing;
  constexpr int kChunks = D / 8;                          // 16-byte chunks of a row of 16-bit values
  constexpr int kAtOnce = 32 / kChunks;                   // rows of one warp-wide access
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row_in_tile = warp * 32 + lane;
  const int row = job.row0 + which * 128 + row_in_tile;
  const int row_c = min(row, job.rows - 1);
  uint8_t* tile = smem + Smem<D>::kQ + which * Smem<D>::kQTile;
  // chunk c of row r of the tile, where the 128-byte swizzle puts it
  auto chunk_of = [&](int r, int c) { return reinterpret_cast<uint4*>(tile + (c / 8) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };

  // the query rows into shared memory: the warp brings its rows one after the other, then each thread
  // makes its own row fp16, with the power of two that keeps bf16 in range
  float factor = p.scale_log2;
  {
    const int chunk = lane % kChunks;
#pragma unroll 8
    for (int it = 0; it < 32 / kAtOnce; ++it) {
      const int r = warp * 32 + it * kAtOnce + lane / kChunks, of = min(job.row0 + which * 128 + r, job.rows - 1);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)(job.rq.first + of / p.group) * p.q_token +
                          (int64_t)(job.head * p.group + of % p.group) * p.q_head;
      *chunk_of(r, chunk) = __ldg(reinterpret_cast<const uint4*>(q) + chunk);
    }
    __syncwarp();
    float mul = 1.0f;
    if (p.bf16) {
      uint32_t big = 0;
#pragma unroll 4
      for (int c = 0; c < kChunks; ++c) {
        const uint4 v = *chunk_of(row_in_tile, c);
        const uint32_t w[1][4] = {{v.x, v.y, v.z, v.w}};
        big = max(big, largest_word<1>(w));
      }
      mul = bf16_row_power(big);
      factor /= mul;  // (exact: a power of two)
    }
    // logits are compared before they are scaled: a negative scale turns the row round instead, and a scale of
    // zero makes its channels zeros, or NaN where they are not finite
    const uint32_t flip = factor < 0.0f ? 0x80008000u : 0u;
    const bool zero = factor == 0.0f;
    factor = factor == 0.0f ? 1.0f : fabsf(factor);
#pragma unroll 1
    for (int c0 = 0; c0 < kChunks; c0 += 4) {
      uint32_t w[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4* at = chunk_of(row_in_tile, c0 + c);
        const uint4 v = *at;
        w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
#pragma unroll
        for (int e = 4 * c; e < 4 * c + 4; ++e) w[e] = (p.bf16 ? bf16_pair_to_half(w[e], mul) : w[e]) ^ flip;
        if (zero) {
#pragma unroll
          for (int e = 4 * c; e < 4 * c + 4; ++e) w[e] = zero_times_halves(w[e]);
        }
        if (!Smem<D>::kOne) *at = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      }
      if constexpr (Smem<D>::kOne) {
        __syncwarp();  // (`zero` may differ from row to row, and the store is the whole warp's)
        tmem_st16(sh->tmem + ((uint32_t)(warp * 32) << 16) + kQueryColumn + c0 * 4, w);
      }
    }
    if constexpr (Smem<D>::kOne) {
      tmem_wait_st();
      fence_before();
    } else {
      fence_async();
    }
    arrive(&sh->q_full);
    __syncwarp();
  }
  if (which == 1 && !job.two) return;

  const int own = job.rq.length - job.rq.queries + row_c / p.group;  // the row's position
  const int low = p.window > 0 ? max(own + 1 - p.window, 0) : 0;
  int limit = own + 1;
  float slope = 0.0f, shaped_factor = 1.0f;
  if constexpr (kShaped) {
    if (p.prefix != nullptr) limit = max(limit, __ldg(p.prefix + job.request));
    if (p.slopes != nullptr) slope = __ldg(p.slopes + job.head * p.group + row_c % p.group) * 1.4426950408889634f;
    shaped_factor = factor;  // logits are shaped in units of log 2, and stay so
    factor = 1.0f;
  }
  // the polynomial of tanh(x) / x times the logits' factor, and what makes a logit x
  float term[7];
#pragma unroll
  for (int i = 0; i < 7; ++i) term[i] = tanh_term(i) * shaped_factor;
  const float to_cap = shaped_factor * p.one_over_cap;
  // Whether the row's slope goes by each column's distance: where rows see what lies after them, too, and where a slope is
  // so steep that the rounding of its part at a tile's first column (2^-24 of up to 64 slopes beside the row's own position) would show.
  // (then its start_slope is 0, which for a slope of 0 is all the same)
  const bool steep = kShaped && (p.prefix != nullptr || fabsf(slope) > 4.0f);
  const bool by_distance = __any_sync(~0u, steep);  // some row of the warp
  const float start_slope = steep ? 0.0f : -slope;
  slope = steep ? -bounded_slope(slope) : slope;
  const uint32_t lane_base = sh->tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t o_at = lane_base + kSumColumn + which * D;

  // The loop reads a tile's logits twice, once for the maximum and once for the weights: that is little
  // against 128 exponentials a row, and the loops stay short enough for the instruction
  // cache that four kinds of warps share.
  float m = -INFINITY, sum0 = 0.0f, sum1 = 0.0f;  // m in units of log 2
  uint32_t poison = 0;                             // value groups in which this row is NaN
  for (int i = 0; i < job.tiles; ++i) {
    const int buf = Smem<D>::kOne ? i & 1 : which;
    const uint32_t s_at = lane_base + buf * kTok;
    wait_warp(&sh->s_full[buf], (Smem<D>::kOne ? i >> 1 : i) & 1, sh);
    fence_after();
    const int pos0 = job.from + i * kTok;
    const uint32_t* valid = sh->valid + i % kRing * (kTok / 32);
    const uint32_t* nan_rows = sh->nan_rows + i % kRing * (kTok / 32);
    const uint2 valid2 = *reinterpret_cast<const uint2*>(valid), nan2 = *reinterpret_cast<const uint2*>(nan_rows);
    uint32_t all_valid = valid2.x & valid2.y, any_nan = nan2.x | nan2.y;
    if constexpr (kTok == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(valid + 2), n = *reinterpret_cast<const uint2*>(nan_rows + 2);
      all_valid &= v.x & v.y;
      any_nan |= n.x | n.y;
    }
    float top;
    bool hidden = false;
    if constexpr (kShaped) {
      // shaped and hidden in tensor memory, 32 columns at a time, and the maximum taken on the way
      top = -INFINITY;
      const bool plain = __all_sync(~0u, all_valid == ~0u && pos0 + kTok <= limit && pos0 >= low && any_nan == 0);
      float from = (float)(own - pos0);
#pragma unroll 1
      for (int w = 0; w < kTok / 32; ++w, from -= 32.0f) {
        uint32_t y[32];
        tmem_read32(s_at + 32 * w, y);
        float* s = reinterpret_cast<float*>(y);
        // A slope's term rises by the slope from column to column, up to the row's own position; its first column's
        // part comes with the last step before.
        const float start = start_slope * from;
        if (p.cap > 0.0f) {
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
            float u[16], most = 0.0f;
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              u[c] = s[c0 + c], u[c + 1] = s[c0 + c + 1];
              mul2(u[c], u[c + 1], to_cap);
              fma2(u[c], u[c + 1], u[c], u[c + 1], u[c], u[c + 1], 0.0f);
              most = max3(most, u[c], u[c + 1]);
            }
            if (__all_sync(~0u, most <= 1.0f)) {
              // all logits are below the cap: no exponential and no reciprocal, of which the softmax needs one already
              float t[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) t[c] = term[6];
#pragma unroll
              for (int i = 5; i >= 0; --i)
#pragma unroll
                for (int c = 0; c < 16; c += 2) fma2(t[c], t[c + 1], t[c], t[c + 1], u[c], u[c + 1], term[i]);
#pragma unroll
              for (int c = 0; c < 16; c += 2) fma2(s[c0 + c], s[c0 + c + 1], s[c0 + c], s[c0 + c + 1], t[c], t[c + 1], start);
            } else {
              // (the same steps for those below it: a row's results do not go by its neighbours)
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                float t = term[6];
#pragma unroll
                for (int i = 5; i >= 0; --i) t = fmaf(t, u[c], term[i]);
                t = fmaf(s[c0 + c], t, start);
                s[c0 + c] = u[c] <= 1.0f ? t : capped_by_exp(p, s[c0 + c] * shaped_factor) + start;
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; c += 2) fma2(s[c], s[c + 1], shaped_factor, start);
        }
        if (p.slopes != nullptr) {
          if (by_distance) {
            // (rows that do not go by it take the same steps as below: their first column's distance is 0)
            const float first = start_slope == 0.0f ? from : 0.0f;
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = fmaf(slope, fabsf(first - (float)c), s[c]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = fmaf(slope, (float)c, s[c]);
          }
        }
        if (!plain) {
          const int a = low - (pos0 + 32 * w), b = limit - (pos0 + 32 * w);  // (low >= 0: no overflow)
          uint32_t see = valid[w];
          see &= b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
          see &= a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((see >> c) & 1u)) y[c] = 0xFF800000u;
          for (uint32_t left = nan_rows[w] & see; left != 0; left &= left - 1)
            poison |= sh->nan_groups[i % kRing * kTok + 32 * w + __ffs(left) - 1];
          __syncwarp();
        }
        float t0 = top, t1 = s[0];
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          t0 = max3(t0, s[c], s[c + 1]);
          t1 = max3(t1, s[c + 2], s[c + 3]);
        }
        top = fmaxf(t0, t1);
        tmem_st32(s_at + 32 * w, y);
      }
      tmem_wait_st();
    }
#pragma unroll 1
    for (; !kShaped;) {
      float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < kTok / 64; ++h) {
        uint32_t x[64];
        tmem_read64(s_at + 64 * h, x);
        const float* s = reinterpret_cast<const float*>(x);
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          t0 = max3(t0, s[c], s[c + 1]);
          t1 = max3(t1, s[c + 2], s[c + 3]);
          t2 = max3(t2, s[c + 4], s[c + 5]);
          t3 = max3(t3, s[c + 6], s[c + 7]);
        }
      }
      top = fmaxf(max3(t0, t1, t2), t3) * factor;
      // (looked at only now: the words come from shared memory, which the products keep busy)
      const bool plain = all_valid == ~0u && pos0 + kTok <= limit && pos0 >= low && any_nan == 0;
      if (hidden || __all_sync(~0u, plain)) break;
      // hide what this row does not see, in tensor memory, and take the maximum again
      hidden = true;
#pragma unroll 1
      for (int w = 0; w < kTok / 32; ++w) {
        uint32_t y[32];
        tmem_read32(s_at + 32 * w, y);
        const int a = low - (pos0 + 32 * w), b = limit - (pos0 + 32 * w);  // (low >= 0: no overflow)
        uint32_t see = valid[w];
        see &= b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
        see &= a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!((see >> c) & 1u)) y[c] = 0xFF800000u;
        tmem_st32(s_at + 32 * w, y);
        for (uint32_t left = nan_rows[w] & see; left != 0; left &= left - 1)
          poison |= sh->nan_groups[i % kRing * kTok + 32 * w + __ffs(left) - 1];
        __syncwarp();
      }
      tmem_wait_st();
    }
    const bool moves = top > m + kSlack || (m == -INFINITY && top > m);
    if (__any_sync(~0u, moves)) {
      // the product O += P V of tile i - 1 has to be done: with two row tiles S(i) was issued after it; with one
      // S(i) came before it, but after that of tile i - 2, so that this is the phase to wait for
      const float now = moves ? top : m;
      const float a = moves ? exp2_fast(m - now) : 1.0f;
      m = now;
      sum0 *= a;
      sum1 *= a;
      if (i > 0) {
        if constexpr (Smem<D>::kOne) {
          wait_warp(&sh->o_tile, (i - 1) & 1, sh);
          fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tmem_read16(o_at + c, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
          tmem_st16(o_at + c, o);
        }
        tmem_wait_st();
      }
    }
    const float ref = m == -INFINITY ? 0.0f : kShift - m;
#pragma unroll 1
    for (int h = 0; h < kTok / 64; ++h) {
      uint32_t x[64], pk[32];
      tmem_read64(s_at + 64 * h, x);
      float* s = reinterpret_cast<float*>(x);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        fma2(s[2 * e], s[2 * e + 1], factor, ref);
        s[2 * e] = exp2_fast(s[2 * e]);
        s[2 * e + 1] = exp2_fast(s[2 * e + 1]);
        add2(sum0, sum1, s[2 * e], s[2 * e + 1]);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(s[2 * e + 1]), "f"(s[2 * e]));
      }
      tmem_st32(s_at + 32 * h, pk);  // (columns whose logits have been read)
      tmem_wait_st();
      fence_before();
      named_arrive(weights_ready(buf, h), kWeightsThreads);  // the second product starts on the first half
      __syncwarp();
    }
  }
  const bool ok = wait_warp(&sh->o_full[which], 0, sh) && *(volatile int*)&sh->gave_up == 0;
  __syncwarp();
  fence_after();

  // epilogue: divide, turn the rows through the query tile's place into whole lines, write out (or the
  // part and its logarithm)
  const float sum = sum0 + sum1;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float log2_sum = sum == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m - kShift) + __log2f(sum);
  if (!ok) log2_sum = NAN;
  const int64_t part = ((int64_t)job.part * p.heads + job.head) * p.part_rows + job.row0 + which * 128;
  const int per_pass = job.final_here ? D : D / 2;  // columns that fit the tile's rows
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += per_pass) {
#pragma unroll 1
    for (int c = 0; c < per_pass; c += 16) {
      uint32_t o[16];
      if (job.tiles > 0) tmem_read16(o_at + c0 + c, o);
      const bool bad = !ok || ((poison >> ((c0 + c) / 32)) & 1u);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = job.tiles > 0 && sum != 0.0f ? __uint_as_float(o[e]) * inv : 0.0f;
        o[e] = __float_as_uint(bad ? NAN : x);
      }
      if (job.final_here) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = pack_out(p, __uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
        *chunk_of(row_in_tile, c / 8) = make_uint4(h[0], h[1], h[2], h[3]);
        *chunk_of(row_in_tile, c / 8 + 1) = make_uint4(h[4], h[5], h[6], h[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *chunk_of(row_in_tile, c / 4 + e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int it = 0; it < 32 / kAtOnce; ++it) {
      const int r = warp * 32 + it * kAtOnce + lane / kChunks, of = job.row0 + which * 128 + r;
      if (of >= job.rows) continue;
      const uint4 v = *chunk_of(r, lane % kChunks);
      if (job.final_here) {
        const int64_t out_row = (int64_t)(job.rq.first + of / p.group) * p.heads * p.group + job.head * p.group + of % p.group;
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_row * D)[lane % kChunks] = v;
      } else {
        reinterpret_cast<uint4*>(p.part_o + (part + r) * D + c0)[lane % kChunks] = v;
      }
    }
    __syncwarp();
  }
  if (row < job.rows) {
    if (job.final_here) {
      const int64_t out_row = (int64_t)(job.rq.first + row / p.group) * p.heads * p.group + job.head * p.group + row % p.group;
      if (p.lse != nullptr) p.lse[out_row] = log2_sum * 0.6931471805599453f;
    } else {
      p.part_lse[part + row_in_tile] = log2_sum;
    }
  }
}

// ---- packed rows into shared memory: one warp, a bulk copy for each run of positions on a page
template <int D>
__device__ __forceinline__ void copy_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem) {
  constexpr int kRow = row_bytes(D);
  constexpr int kParts = Smem<D>::kParts, kRaw = Smem<D>::kRaw;
  constexpr int kMost = kPart / 32;  // runs of a lane, at pages of one position; words of a stage's valid bits
  const int lane = threadIdx.x & 31;
  const uint32_t packed_at = lt::smem_u32(smem + Smem<D>::kPacked);
  const int run_shift = min(p.shift, 6), runs = kPart >> run_shift;
  const int32_t* table = p.table + (int64_t)job.request * p.width;
  const int stages = kParts * job.tiles;
  int page[kMost];
  auto look_up = [&](int n) {
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int run = lane + 32 * j, at = job.from + n * kPart + (run << run_shift);
      page[j] = n < stages && run < runs && at < job.to ? __ldg(table + (at >> p.shift)) : -1;
    }
  };
  look_up(0);
  int stage = 0;
  uint32_t parity = 1;  // (the first round's stages are free)
  int n = 0;
#pragma unroll 1
  for (; n < stages; ++n) {
    // Where a wait has run out, here or with the unpackers, no place is written any more. (They wait for it in vain once.)
    if (!wait_warp(&sh->packed_empty[stage], parity, sh) || __any_sync(~0u, *(volatile int*)&sh->gave_up)) break;
    uint32_t valid[kMost] = {};
    int count[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int first = (lane + 32 * j) << run_shift, left = job.to - (job.from + n * kPart + first);
      count[j] = page[j] >= 0 && page[j] < p.pages ? min(left, 1 << run_shift) : 0;
#pragma unroll
      for (int w = 0; w < kMost; ++w) {
        const int a = min(max(first - 32 * w, 0), 32), b = min(max(first + count[j] - 32 * w, 0), 32);
        valid[w] |= a < b ? (b == 32 ? ~0u : (1u << b) - 1u) & (~0u << a) : 0u;
      }
    }
    uint32_t there = 0;
#pragma unroll
    for (int w = 0; w < kMost; ++w) {
      valid[w] = __reduce_or_sync(~0u, valid[w]);
      there += __popc(valid[w]);
    }
    if (lane == 0) {
#pragma unroll
      for (int w = 0; w < kMost; ++w) sh->valid[n % (16 / kMost) * kMost + w] = valid[w];
      lt::mbar_arrive_tx(&sh->packed_full[stage], there * kRow);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int first = (lane + 32 * j) << run_shift, at = job.from + n * kPart + first;
      if (count[j] > 0) {
        const uint8_t* src = p.cache + (((((int64_t)page[j] * p.heads + job.head) << p.shift) + (at & ((1 << p.shift) - 1))) * kRow);
        bulk_in(packed_at + (stage * kPart + first) * kRow, src, (uint32_t)count[j] * kRow, &sh->packed_full[stage]);
      }
    }
    look_up(n + 1);
    if (++stage == kRaw) {
      stage = 0;
      parity ^= 1u;
    }
  }
  // nothing is on its way any more when the CTA ends, also where somebody gave up
  for (int i = max(n - kRaw, 0); i < n; ++i) wait_warp(&sh->packed_full[i % kRaw], i / kRaw & 1, sh);
}

// ---- unpacking: a packed stage's positions at a time, a thread the key or the value of a position (with
// D = 256 half of its channels); half of the threads have keys, half values
template <int D>
__device__ __forceinline__ void unpack_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem) {
  constexpr int kRow = row_bytes(D);
  constexpr int kParts = Smem<D>::kParts, kRaw = Smem<D>::kRaw;
  constexpr int kTok = Smem<D>::kTok, kRing = Smem<D>::kRing;
  constexpr int kBlocks = D / 64 * 2 * kPart / Smem<D>::kUnpackers;  // 64-channel blocks of a thread
  const int t = threadIdx.x - (384 - Smem<D>::kUnpackers), lane = t & 31, row = t % kPart, part = t / kPart & 1;
  const int block0 = t / (2 * kPart) * kBlocks;
  // The stage is handed back before this one of the thread's 16-byte chunks is unpacked: early, but when what was loaded
  // last has arrived. us for 2048 tokens behind 14336 with heads of 128, and of 256: before the first chunk 405, 972; the
  // second 410, 906; the last but one 414, 874; the last 411, 887; after all of them 408, 930; before the wait for the slot 410, 978.
  constexpr int kHandBack = Smem<D>::kOne ? 2 * kBlocks - 2 : 0;
  uint32_t chunk_at[8];  // where the row's eight 16-byte chunks lie in a swizzled 128-byte row
#pragma unroll
  for (int c = 0; c < 8; ++c) chunk_at[c] = lt::smem_u32(smem + Smem<D>::kKv) + row * 128 + ((c ^ (row & 7)) << 4);
  // the slots go round: keys of tile i in slot 2 i mod kSlots, values in the next
  int slot = part, stage = 0;
  uint32_t slot_parity = 1, stage_parity = 0;  // (the first round's slots are free)
  bool fed = true;
#pragma unroll 1
  for (int i = 0; i < job.tiles; ++i) {
#pragma unroll 1
    for (int half = 0; half < kParts; ++half) {
      fed = fed && wait_warp(&sh->packed_full[stage], stage_parity, sh);  // (once in vain is enough)
      const int word = i % kRing * (kTok / 32) + half * (kPart / 32) + row / 32;  // (the warp's rows are one word's)
      const uint32_t valid = sh->valid[word];
      const bool there = (valid >> lane) & 1u;
      const uint8_t* from = smem + Smem<D>::kPacked + (stage * kPart + row) * kRow;
      // scales, fp16 pairs; a position that is not there counts as zeros, and so does a NaN value
      uint32_t sc[kBlocks], seen = 0;  // seen: made of every word
#pragma unroll
      for (int g = 0; g < kBlocks; ++g) {
        sc[g] = there ? reinterpret_cast<const uint32_t*>(from + D + part * (D / 16))[block0 + g] : 0u;
        seen ^= sc[g];
        if (part == 1) sc[g] &= ~unfit_halves(sc[g]);
      }
      if (part == 0 && block0 == 0) {
        // the NaN values are noted here, with the keys: the softmax starts when the keys are there
        uint32_t nan = 0;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const uint32_t n = there ? unfit_halves(reinterpret_cast<const uint32_t*>(from + D + D / 16)[g]) : 0u;
          nan |= ((n & 1u) | ((n >> 15) & 2u)) << (2 * g);
        }
        const uint32_t nan_rows = __ballot_sync(~0u, nan != 0);
        if (lane == 0) sh->nan_rows[word] = nan_rows;
        if (nan_rows) sh->nan_groups[i % kRing * kTok + half * kPart + row] = (uint8_t)nan;
        seen ^= nan;
      }
      uint4 codes[2 * kBlocks];
#pragma unroll
      for (int c = 0; c < 2 * kBlocks; ++c) codes[c] = reinterpret_cast<const uint4*>(from + part * (D / 2))[2 * block0 + c];
      if (half == 0) {
        wait_warp(&sh->kv_empty[slot], slot_parity, sh);
        // (until then the queries are in the last slots)
        if (Smem<D>::kOne && i == kSlots / 2 - 1) wait_warp(&sh->q_full, 0, sh);
      }
      const uint32_t to = slot * Smem<D>::kOperand + half * (kPart * 128);
#pragma unroll
      for (int c = 0; c < kBlocks; ++c) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t w[4] = {codes[2 * c + g].x, codes[2 * c + g].y, codes[2 * c + g].z, codes[2 * c + g].w};
          if (2 * c + g < kHandBack) seen ^= w[0] ^ w[1] ^ w[2] ^ w[3];
          if (2 * c + g == kHandBack) {
#pragma unroll
            for (int u = kHandBack; u < 2 * kBlocks; ++u) seen ^= codes[u].x ^ codes[u].y ^ codes[u].z ^ codes[u].w;
            const uint32_t here = zero_of(seen, p.zero);  // every lane has read the stage
            if (lane == 0) arrive(&sh->packed_empty[stage] + here);
          }
          const uint32_t scale = __byte_perm(sc[c], 0, g ? 0x3232 : 0x1010);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            codes_to_half2(w[j], h);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         :: "r"(chunk_at[g * 4 + j] + to + (block0 + c) * Smem<D>::kHalf), "r"(hmul2(h[0], scale)),
                            "r"(hmul2(h[1], scale)), "r"(hmul2(h[2], scale)), "r"(hmul2(h[3], scale)) : "memory");
          }
        }
      }
      if (++stage == kRaw) {
        stage = 0;
        stage_parity ^= 1u;
      }
    }
    fence_async();
    named_arrive(slot_ready(slot), kSlotThreads<D>);
    slot += 2;
    if (slot >= kSlots) {
      slot -= kSlots;
      slot_parity ^= 1u;
    }
  }
}

// ---- the products, issued by one warp
template <int D>
__device__ __forceinline__ void product_role(const Job& job, Shared* sh, uint8_t* smem) {
  constexpr uint32_t kIdescS = instruction(Smem<D>::kTok, false), kIdescO = instruction(D, true);
  const uint32_t q_at = lt::smem_u32(smem + Smem<D>::kQ), kv_at = lt::smem_u32(smem + Smem<D>::kKv);
  const uint32_t tmem = __shfl_sync(~0u, sh->tmem, 0), lead = elect_one();
  wait_warp(&sh->q_full, 0, sh);
  constexpr int kTok = Smem<D>::kTok;
  constexpr bool kOne = Smem<D>::kOne;
  const int tiles = job.tiles;
  if (!kOne && tiles > 0) named_sync(slot_ready(0), kSlotThreads<D>);
  // One place for each product, in a rolled loop: first the weights of a tile by its values, then the logits
  // of a later one, into the columns that the weights were in. With two row tiles even steps
  // are row tile A's, odd ones B's, and the later tile is the next; with one row tile a step
  // is a tile's, and the later tile is the next but one. (Descriptors hold addresses in units of 16 bytes; the steps'
  // offsets are added to them.)
#pragma unroll 1
  for (int step = 0; step < (kOne ? tiles + 2 : 2 * tiles + 2) && tiles > 0; ++step) {
    const int buf = step & 1, which = kOne ? 0 : buf;
    const int i = kOne ? step - 2 : (step >> 1) - 1, next = kOne ? step : i + 1;
    const bool weights = i >= 0 && i < tiles, keys = next < tiles;
    const int value_slot = (uint32_t)(2 * i + 1) % kSlots, key_slot = (uint32_t)(2 * next) % kSlots;
    if (which == 1 && !job.two) continue;
    const bool last = which == 1 || !job.two;  // the product after which a slot is free
    if (weights) {
      if (which == 0) named_sync(slot_ready(value_slot), kSlotThreads<D>);
      const uint64_t value = desc_mn_major(kv_at + value_slot * Smem<D>::kOperand, Smem<D>::kHalf);
#pragma unroll
      for (int half = 0; half < kTok / 64; ++half) {
        named_sync(weights_ready(buf, half), kWeightsThreads);
        fence_after();
        mma_ts4<128>(tmem + kSumColumn + which * D, tmem + buf * kTok + half * 32, value + half * ((64 * 128) >> 4), kIdescO,
                     i > 0 || half > 0, lead);
      }
      if (last) mma_commit(&sh->kv_empty[value_slot], lead);
      if (kOne) mma_commit(&sh->o_tile, lead);
    }
    if (keys) {
      if (which == 0 && (kOne || weights)) named_sync(slot_ready(key_slot), kSlotThreads<D>);
      fence_after();
      const uint64_t q = desc_k_major(q_at + which * Smem<D>::kQTile);
      const uint64_t key = desc_k_major(kv_at + key_slot * Smem<D>::kOperand);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint64_t k = key + c * (Smem<D>::kHalf >> 4);
        if constexpr (kOne)
          mma_ts4<2>(tmem + buf * kTok, tmem + kQueryColumn + c * 32, k, kIdescS, c > 0, lead);
        else
          mma_ss4(tmem + buf * kTok, q + c * (Smem<D>::kQHalf >> 4), k, kIdescS, c > 0, lead);
      }
      mma_commit(&sh->s_full[buf], lead);
      if (last) mma_commit(&sh->kv_empty[key_slot], lead);
    }
  }
  mma_commit(&sh->o_full[0], lead);
  if (job.two) mma_commit(&sh->o_full[1], lead);
}

template <int D, bool kShaped>
__global__ void __launch_bounds__(kCta, 1) prefill_kernel(AttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (lt::smem_u32(smem_raw) & 1023u)) & 1023u);
  Shared* sh = reinterpret_cast<Shared*>(smem + Smem<D>::kBars);
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
  if (tid == 0) {
    for (int s = 0; s < Smem<D>::kRaw; ++s) {
      lt::mbar_init(&sh->packed_full[s], 1);
      lt::mbar_init(&sh->packed_empty[s], Smem<D>::kUnpackers / 32);
    }
    for (int s = 0; s < kSlots; ++s) lt::mbar_init(&sh->kv_empty[s], 1);
    lt::mbar_init(&sh->o_tile, 1);
    lt::mbar_init(&sh->q_full, Smem<D>::kRowTiles * 128);
    for (int t = 0; t < 2; ++t) {
      lt::mbar_init(&sh->s_full[t], 1);
      lt::mbar_init(&sh->o_full[t], 1);
    }
    sh->gave_up = 0;
    lt::mbar_fence_init();
  }
  dependency_wait();

  Job job;
  // A request's last rows see the most positions: every request's last row tile comes first, then their last
  // but one, so the long CTAs start early and the short ones fill in.
  const int units = gridDim.x / p.row_tiles;
  const int nth = blockIdx.x / units, unit = blockIdx.x % units;
  job.head = unit % p.heads;
  job.flat = unit / p.heads;
  Place pl;
  if (!find_place<kCta>(p, job.flat, &pl, sh->sums, &sh->found)) return;
  job.request = pl.request;
  job.rq = request_of(p, pl.request);
  job.rows = job.rq.computed * p.group;
  job.part = pl.part + pl.split;
  constexpr int kRows = Smem<D>::kRowTiles * 128;
  job.row_tile = min((job.rows + kRows - 1) / kRows, p.row_tiles) - 1 - nth;
  if (job.row_tile < 0) return;
  job.final_here = pl.count == 1;
  if (job.flat == pl.base && job.head == 0 && job.row_tile == 0 && tid == 0 && p.plan != nullptr)
    p.plan[pl.request] = make_int2(pl.part, pl.count);
  job.row0 = job.row_tile * kRows;
  job.two = kRows > 128 && job.rows - job.row0 > 128;
  {
    const int64_t at = job.rq.low + pl.split * chunk_of(p, job.rq, pl.count), end = at + chunk_of(p, job.rq, pl.count);
    job.from = (int)(at < job.rq.length ? at : job.rq.length);
    job.to = (int)(end < job.rq.length ? end : job.rq.length);
    const int last = min(job.rows - 1, job.row0 + kRows - 1) / p.group;
    int seen_to = job.rq.length - job.rq.queries + last + 1;
    if (kShaped && p.prefix != nullptr) seen_to = max(seen_to, __ldg(p.prefix + job.request));
    job.to = min(job.to, seen_to);
    if (p.window > 0)
      job.from = max(job.from, (job.rq.length - job.rq.queries + job.row0 / p.group + 1 - p.window) / p.align * p.align);
    job.tiles = job.to > job.from ? (job.to - job.from + Smem<D>::kTok - 1) / Smem<D>::kTok : 0;
  }

  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(lt::smem_u32(&sh->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();

  if (warp < 4 * Smem<D>::kRowTiles)
    softmax_role<D, kShaped>(p, job, sh, smem, warp / 4);
  else if (warp < 12)
    unpack_role<D>(p, job, sh, smem);
  else if (warp == 12)
    product_role<D>(job, sh, smem);
  else if (warp == 13)
    copy_role<D>(p, job, sh, smem);
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  dependents_launch();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(sh->tmem) : "memory");
}

}  // namespace

namespace lt {
namespace kv4 {

template <bool kShaped>
const void* prefill_kernel_ptr(int head_dim, int* smem) {
  if (head_dim == 64) {
    *smem = Smem<64>::kTotal;
    return reinterpret_cast<const void*>(&prefill_kernel<64, kShaped>);
  }
  if (head_dim == 128) {
    *smem = Smem<128>::kTotal;
    return reinterpret_cast<const void*>(&prefill_kernel<128, kShaped>);
  }
  *smem = Smem<256>::kTotal;
  return reinterpret_cast<const void*>(&prefill_kernel<256, kShaped>);
}

}  // namespace kv4
}  // namespace lt
