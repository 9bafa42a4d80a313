// lt_kv4_rows.cuh -- attention over the 4-bit cache for few query rows a request (decode,
// drafted tokens) and for listed positions; one translation unit without and one
// with shaped logits (caps, slopes, prefixes).
//
// Rows. The query heads of one kv head, times a request's new tokens, are the
// query rows that read the same keys and values; a CTA takes 8, 16 or 32 of them
// (NT tiles of 8) and one chunk of the request's positions. Its four warps walk
// the chunk's tiles of 32 positions independently, each with its own ring of
// bulk copies, running maximum and sum, and join once at the end.
//
// Matrix products. At 4.5 bits a value the memory delivers 42 values a clock and
// SM, so the work that counts is that per value: unpacking, scaling, feeding the
// tensor core. Both products take the cache as the 16-row operand straight from
// registers (m16n8k16, fp32 sums): S^T = K Q^T with 16 positions by 8 query rows, and
// O^T = V^T P^T with 16 channels by 8 query rows, so a fragment register of 2
// values serves one 16x8x16 step and the weights go from the first product's
// result to the second's operand with one 8x8 transpose. Two value codes of
// neighbouring positions are brought into one byte before they are converted, so the
// conversion yields the pair that the fragment wants. The accumulator is a few
// registers wide because the rows are few; tcgen05 would want 128 rows, and the
// unpacked values in shared memory.
//
// A product of a code and its scale is an exact fp16 number, so keys and values
// enter the products exactly. The weights are rounded to fp16 (2^-12 relative)
// after a shift by 2^6 that keeps small ones normal; the sums that divide them are
// fp32 and of the unrounded weights.
//
// What bounds it: issue, and the waits between a warp's own instructions. A tile of 32 positions of D = 128
// takes some 725 warp instructions (858 before the maximum became lazy and a CTA's start and end were
// shortened), of which unpacking and scaling are 450; 2.47 are issued a clock and SM, 62% of what its schedulers
// could (2.14, 54%, with heads of 256, whose 168 registers leave 12 warps). More resident warps or deeper rings change
// nothing (5 CTAs an SM with 2 stages 272 us, 4 with 2 or 3 267 to 269, 3 with 4 281, on the 64 ragged
// requests). Measured (4.5-bit rows read once): 64 requests of 2048 to 65536 positions,
// 4 kv heads of 128, 252 us, 4.9 TB/s; one request of 262144 positions, 4 heads of 256,
// 65 us, 4.7 TB/s; the copy rate is 6.8. The widest instances (32 rows; 16 with heads of 256), which serve 17 to
// 64 rows, do not fit the registers: they spill 404 bytes a thread with heads of 128, 308 with 64, 224 with 256.
//
// Shaped logits cost a lane some 5 instructions a logit with a cap and 2 with a slope, of 8 a tile and row tile: 64 ragged requests
// with slopes take 281 us (252 plain), with 128 registers a thread (124 without).
//
// A stage is handed back by the second product's sums; by a word of each load of values it takes 288 and 254.
//
// The running maximum moves for all rows of a tile at once, so a row's roundings go by when its neighbours' logits rise.

#pragma once

#include "lt_kv4.cuh"
#include "lt_kv4_attention.cuh"
#include "lt_kv4_rows.h"

namespace {

using namespace lt::kv4;

constexpr float kShift = 6.0f;  // weights are held as 2^6 exp(s - max)
constexpr float kSlack = 8.0f;  // how far logits may pass the maximum (log 2) before it moves: weights stay below 2^14

template <int D, int NT>
struct Shape {
  static constexpr int kRow = row_bytes(D);
  static constexpr int kTileBytes = kTile * kRow;
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;
  static constexpr int kRing = kWarps * kStages * kTileBytes;
  static constexpr int kJoin = kWarps * NT * 8 * (D + 4) * 4;  // the warps' sums, in the ring's place
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  static constexpr int kPerSm = D == 64 ? (NT == 4 ? 3 : 4) : D == 128 ? (NT == 1 ? 4 : NT == 2 ? 3 : 2) : NT == 1 ? 3 : 2;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds32(a);
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  } else {
    static_assert(N == 4, "1, 2 or 4 words");
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  }
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// This thread's copies so far arrive on the barrier when they are done.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(lt::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n barrier.cluster.wait;" ::: "memory");
}
__device__ __forceinline__ float peer_f32(uint32_t addr, int rank) {
  float v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}"
               : "=f"(v) : "r"(addr), "r"(rank) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t addr, int rank) {
  float4 v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
  return v;
}

template <int D, int NT, bool kList, bool kShaped>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT>::kPerSm)) rows_kernel(AttentionParams p) {
  using Sh = Shape<D, NT>;
  constexpr int kRow = Sh::kRow;
  constexpr int kGroups = D / 32;  // scale groups of a key
  constexpr int kWordsV = D / 64;  // words of value codes a lane takes from a position
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][Sh::kStages];
  __shared__ uint32_t valid_of[kWarps][Sh::kStages];
  __shared__ int pos_of[kList && kShaped ? kWarps : 1][Sh::kStages][kTile];  // listed positions, for their distances
  __shared__ float m_of[kMaxParts][NT * 8];  // a warp's maximum; at the end a part's weight
  __shared__ float l_of[kWarps][NT * 8], part_log2[NT * 8];
  __shared__ int64_t out_of[NT * 8];
  __shared__ int64_t sums[kWarps];
  __shared__ Place found;
  __shared__ int gave_up;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s) lt::mbar_init(&bars[warp][s], kList ? 32 : 1);
    lt::mbar_fence_init();
  }
  if (tid == 0) gave_up = 0;
  dependency_wait();

  // with p.parts > 0 a request (a list) is cut into that many parts, the CTAs of one cluster
  const int rank = p.parts > 0 ? (int)(blockIdx.x % p.parts) : 0;
  const int64_t unit = p.parts > 0 ? blockIdx.x / p.parts : blockIdx.x;
  const int row_tile = (int)(unit % p.row_tiles);
  const int head = (int)(unit / p.row_tiles % p.heads);
  const int flat = (int)(unit / p.row_tiles / p.heads);

  // the request, its rows of this CTA and the range of positions (of list entries)
  Request rq;
  int request, count, token0, rows, from, to, nth_part = 0;
  if constexpr (kList) {
    token0 = flat;  // one query token
    request = owner_of_token(p, token0);
    if (request < 0) return;  // (rows past starts[requests])
    rq = request_of(p, request);
    rows = p.group;
    from = 0;
    to = p.list_len;
    count = 1;
    __syncthreads();
  } else if (p.parts > 0) {
    request = flat;
    rq = request_of(p, request);
    rows = rq.computed * p.group;
    token0 = rq.first;
    from = rq.low;
    to = rq.length;
    count = 1;
    __syncthreads();
  } else {
    Place pl;
    if (!find_place<kThreads>(p, flat, &pl, sums, &found)) return;
    request = pl.request;
    rq = request_of(p, request);
    count = pl.count;
    token0 = rq.first;
    rows = rq.computed * p.group;
    nth_part = pl.part + pl.split;
    if (flat == pl.base && head == 0 && row_tile == 0 && tid == 0 && p.plan != nullptr)
      p.plan[request] = make_int2(pl.part, pl.count);
    // chunks start on tiles: rq.low is a multiple of kTile
    const int64_t at = rq.low + pl.split * chunk_of(p, rq, pl.count), end = at + chunk_of(p, rq, pl.count);
    from = (int)(at < rq.length ? at : rq.length);
    to = (int)(end < rq.length ? end : rq.length);
  }
  const int row0 = row_tile * NT * 8;
  if (row0 >= rows) return;
  if constexpr (!kList) {
    // nothing after the last row's own position, nothing before the first row's window
    const int last = min(rows - 1, row0 + NT * 8 - 1) / p.group;
    int seen_to = rq.length - rq.queries + last + 1;
    if (kShaped && p.prefix != nullptr) seen_to = max(seen_to, __ldg(p.prefix + request));
    to = min(to, seen_to);
    if (p.window > 0) from = max(from, (rq.length - rq.queries + row0 / p.group + 1 - p.window) / kTile * kTile);
  }
  if (p.parts > 1) {
    // the cluster's CTAs take equal runs of tiles
    const int all = to > from ? (to - from + kTile - 1) / kTile : 0, mine = (all + p.parts - 1) / p.parts * kTile;
    const int64_t at = from + (int64_t)rank * mine;
    from = (int)(at < to ? at : to);
    to = (int)(at + mine < to ? at + mine : to);
  }
  const int tiles = to > from ? (to - from + kTile - 1) / kTile : 0;

  // ---- copies: lane i brings the tile's i-th run of positions that lie on one page
  const uint32_t ring = lt::smem_u32(smem) + warp * Sh::kStages * Sh::kTileBytes;
  const int run_shift = kList ? 0 : min(p.shift, 5);
  const int32_t* table = p.table + (int64_t)request * p.width;
  const int32_t* list = kList ? p.positions + (int64_t)token0 * p.list_len : nullptr;
  // The lane's position in a tile (of its run's first one), -1 for none; and the page that a position lies on.
  auto position_of = [&](int tile) {
    const int at = from + tile * kTile + (run_shift == 5 ? 0 : lane << run_shift);
    if (tile >= tiles || at >= to || at >= from + (tile + 1) * kTile) return -1;
    if constexpr (kList) {
      const int pos = __ldg(list + at);
      return pos < rq.length ? pos : -1;
    }
    return at;
  };
  auto page_of = [&](int pos) { return pos >= 0 ? __ldg(table + (pos >> p.shift)) : -1; };
  auto row_at = [&](int page, int pos) { return (((int64_t)page * p.heads + head) << p.shift) + (pos & ((1 << p.shift) - 1)); };
  auto bring = [&](int stage, int pos, int page, uint32_t zero) {
    const bool there = pos >= 0 && page >= 0 && page < p.pages;
    const uint32_t tile_at = ring + stage * Sh::kTileBytes + zero;
    if constexpr (kList) {
      // one row a position: 16-byte copies, the lanes along the rows (a bulk copy a row is no faster: 51 us either
      // way on 1021 lists of 512, then bound by the chain of loads at a CTA's start)
      const uint32_t valid = __ballot_sync(~0u, there);
      if (lane == 0) valid_of[warp][stage] = valid;
      if constexpr (kShaped) {
        pos_of[warp][stage][lane] = pos;
        __syncwarp();
      }
      const int64_t at = there ? row_at(page, pos) : 0;
      constexpr int kChunks = kRow / 16;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int id = k * 32 + lane, of = id / kChunks, chunk = id % kChunks;
        const int64_t row = __shfl_sync(~0u, at, of);
        if ((valid >> of) & 1u) copy16(tile_at + id * 16, p.cache + row * kRow + chunk * 16);
      }
      copies_arrive(&bars[warp][stage]);
    } else if (run_shift == 5) {
      // the tile lies on one page: one copy, and all lanes know its size
      const int count = there ? min(to - pos, kTile) : 0;
      if (lane == 0) {
        valid_of[warp][stage] = count == kTile ? ~0u : (1u << count) - 1u;
        lt::mbar_arrive_tx(&bars[warp][stage], (uint32_t)count * kRow);
        if (count > 0) bulk_in(tile_at, p.cache + row_at(page, pos) * kRow, (uint32_t)count * kRow, &bars[warp][stage]);
      }
      __syncwarp();
    } else {
      const int count = there ? min(to - pos, 1 << run_shift) : 0;
      const uint32_t mine = count > 0 ? ((1u << count) - 1u) << (lane << run_shift) : 0u;
      const uint32_t valid = __reduce_or_sync(~0u, mine);
      if (lane == 0) {
        valid_of[warp][stage] = valid;
        lt::mbar_arrive_tx(&bars[warp][stage], (uint32_t)__popc(valid) * kRow);
      }
      __syncwarp();
      if (count > 0)
        bulk_in(tile_at + (lane << run_shift) * kRow, p.cache + row_at(page, pos) * kRow, (uint32_t)count * kRow, &bars[warp][stage]);
    }
  };

  // Everything that the start waits for from far away is asked for together: the queries, the first tiles'
  // positions, then their pages, then their rows. Later, positions are looked up two tiles and
  // pages one tile before their rows are brought.
  // ---- query fragments: lane (g, c) holds channels 32 j + 8 c .. + 7 of row g of each row tile
  uint32_t qf[NT][kGroups][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = min(row0 + nt * 8 + g, rows - 1);
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)(token0 + row / p.group) * p.q_token +
                        (int64_t)(head * p.group + row % p.group) * p.q_head;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + 32 * j + 8 * c));
      qf[nt][j][0] = v.x, qf[nt][j][1] = v.y, qf[nt][j][2] = v.z, qf[nt][j][3] = v.w;
    }
  }
  int next_pos, next_page, later_pos;
  {
    int pos[Sh::kStages], page[Sh::kStages];
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s) pos[s] = position_of(warp + s * kWarps);
    next_pos = position_of(warp + Sh::kStages * kWarps);
    later_pos = position_of(warp + (Sh::kStages + 1) * kWarps);
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s) page[s] = page_of(pos[s]);
    next_page = page_of(next_pos);
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s)
      if (warp + s * kWarps < tiles) bring(s, pos[s], page[s], 0);
  }
  float factor[NT][2];  // of columns 2c, 2c + 1: logits in units of log 2
  int limit[NT][2], low[NT][2];
  int own[NT][2];  // (shaped) the query's position, and its head's slope in units of log 2
  float slope[NT][2];
  int prefix = 0;
  if constexpr (kShaped) prefix = !kList && p.prefix != nullptr ? __ldg(p.prefix + request) : 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float inv = p.bf16 ? bf16_row_to_half<kGroups>(qf[nt]) : 1.0f;
    factor[nt][0] = __shfl_sync(~0u, inv, 8 * c) * p.scale_log2;
    factor[nt][1] = __shfl_sync(~0u, inv, 8 * c + 4) * p.scale_log2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int token_of = min(row0 + nt * 8 + 2 * c + e, rows - 1) / p.group;
      limit[nt][e] = kList ? INT32_MAX : rq.length - rq.queries + token_of + 1;
      low[nt][e] = !kList && p.window > 0 ? limit[nt][e] - p.window : INT32_MIN;
      if constexpr (kShaped) {
        const int row = min(row0 + nt * 8 + 2 * c + e, rows - 1);
        own[nt][e] = rq.length - rq.queries + (kList ? token0 - rq.first : token_of);
        slope[nt][e] = p.slopes != nullptr ? bounded_slope(__ldg(p.slopes + head * p.group + row % p.group) * 1.4426950408889634f) : 0.0f;
        if (!kList) limit[nt][e] = max(limit[nt][e], prefix);
      }
    }
  }
  // every row sees up to here
  const int safe_to = kList ? INT32_MAX : max(rq.length - rq.queries + row0 / p.group + 1, kShaped ? prefix : INT32_MIN);
  const int safe_from = !kList && p.window > 0
                            ? rq.length - rq.queries + min(rows - 1, row0 + NT * 8 - 1) / p.group + 1 - p.window
                            : INT32_MIN;

  float acc[NT][D / 16][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[nt][t][e] = 0.0f;
  }
  const uint32_t pick = (g >> 2) ? 0x7632u : 0x5410u;  // this lane's value scales: upper or lower halves

  bool ok = true;
  int stage = 0;
  uint32_t parity = 0;
  for (int tile = warp; tile < tiles; tile += kWarps) {
    ok = wait_bounded(&bars[warp][stage], parity);  // (the warp votes: it stays converged)
    if (!ok) break;
    const uint32_t valid = valid_of[warp][stage];
    const uint32_t base = ring + stage * Sh::kTileBytes;
    const int pos0 = from + tile * kTile;
    const bool masked = valid != ~0u || (!kList && (pos0 + kTile > safe_to || pos0 < safe_from));

    // S^T: 32 positions (two 16-row steps) by 8 NT rows
    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.0f;
      const uint32_t ra = base + (mt * 16 + g) * kRow, rb = ra + 8 * kRow;
      uint32_t sa[kGroups / 2], sb[kGroups / 2];
      lds_words(ra + D, sa);
      lds_words(rb + D, sb);
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        uint32_t ha[4], hb[4];
        codes_to_half2(lds32(ra + (j * 4 + c) * 4), ha);
        codes_to_half2(lds32(rb + (j * 4 + c) * 4), hb);
        if constexpr (NT == 1) {
          // with one row tile the scale of the group is cheaper on the product's four results than on eight
          // operand registers
          const __half2 pa = *reinterpret_cast<const __half2*>(&sa[j / 2]), pb = *reinterpret_cast<const __half2*>(&sb[j / 2]);
          const float fa = j & 1 ? __high2float(pa) : __low2float(pa), fb = j & 1 ? __high2float(pb) : __low2float(pb);
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(d, ha[0], hb[0], ha[1], hb[1], qf[0][j][0], qf[0][j][1]);
          mma16816(d, ha[2], hb[2], ha[3], hb[3], qf[0][j][2], qf[0][j][3]);
          s[mt][0][0] = fmaf(d[0], fa, s[mt][0][0]);
          s[mt][0][1] = fmaf(d[1], fa, s[mt][0][1]);
          s[mt][0][2] = fmaf(d[2], fb, s[mt][0][2]);
          s[mt][0][3] = fmaf(d[3], fb, s[mt][0][3]);
        } else {
          const uint32_t ka = __byte_perm(sa[j / 2], 0, j & 1 ? 0x3232 : 0x1010);
          const uint32_t kb = __byte_perm(sb[j / 2], 0, j & 1 ? 0x3232 : 0x1010);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ha[i] = hmul2(ha[i], ka);
            hb[i] = hmul2(hb[i], kb);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(s[mt][nt], ha[0], hb[0], ha[1], hb[1], qf[nt][j][0], qf[nt][j][1]);
            mma16816(s[mt][nt], ha[2], hb[2], ha[3], hb[3], qf[nt][j][2], qf[nt][j][3]);
          }
        }
      }
    }

    // logits, masks, running maximum: it moves only when a logit passes it by 2^kSlack (always at first), so
    // most tiles need neither the maximum over the lanes nor a new scale of the sums
    bool raised = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float away[2];  // how far the tile's first position of this lane is from the queries'
      if constexpr (kShaped && !kList) {
#pragma unroll
        for (int e = 0; e < 2; ++e) away[e] = (float)(own[nt][e] - pos0 - g);
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mt][nt][e] *= factor[nt][e & 1];
          if constexpr (kShaped) {
            if (p.cap > 0.0f) s[mt][nt][e] = capped(p, s[mt][nt][e]);
            // (without slopes they are zeros: a branch around so little costs more)
            const int cell = mt * 16 + (e >> 1) * 8;
            float distance;
            if constexpr (kList)
              distance = (float)(own[nt][e & 1] - pos_of[warp][stage][cell + g]);
            else
              distance = away[e & 1] - (float)cell;
            s[mt][nt][e] = fmaf(-slope[nt][e & 1], fabsf(distance), s[mt][nt][e]);
          }
          if (masked) {
            const int at = mt * 16 + g + (e >> 1) * 8;
            bool sees = (valid >> at) & 1u;
            if constexpr (!kList) sees = sees && pos0 + at < limit[nt][e & 1] && pos0 + at >= low[nt][e & 1];
            if (!sees) s[mt][nt][e] = -INFINITY;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        raised = raised || fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2])) > m[nt][e] + kSlack;
    if (__any_sync(~0u, raised)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
          t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
          t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
          t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
          const float now = fmaxf(m[nt][e], t);
          a[e] = now == m[nt][e] ? 1.0f : exp2_fast(m[nt][e] - now);
          m[nt][e] = now;
          l[nt][e] *= a[e];
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          acc[nt][t][0] *= a[0];
          acc[nt][t][1] *= a[1];
          acc[nt][t][2] *= a[0];
          acc[nt][t][3] *= a[1];
        }
      }
    }

    // weights: fp32 into the sums, fp16 into the second product
    uint32_t pf[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float ref0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0] - kShift;
      const float ref1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1] - kShift;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float w0 = exp2_fast(s[mt][nt][0] - ref0), w1 = exp2_fast(s[mt][nt][1] - ref1);
        const float w2 = exp2_fast(s[mt][nt][2] - ref0), w3 = exp2_fast(s[mt][nt][3] - ref1);
        l[nt][0] += w0 + w2;
        l[nt][1] += w1 + w3;
        pf[mt][nt][0] = transpose8x8(pack_half2(w0, w1));
        pf[mt][nt][1] = transpose8x8(pack_half2(w2, w3));
      }
    }

    // O^T += V^T P^T: channels in 16-row steps; a lane's words of a position are g and g + 8 i
    bool poisoned = false;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const uint32_t r0 = base + (mt * 16 + 2 * c) * kRow;
      const uint32_t rr[4] = {r0, r0 + kRow, r0 + 8 * kRow, r0 + 9 * kRow};
      uint32_t sv[4][kWordsV];
#pragma unroll
      for (int t = 0; t < 4; ++t) lds_words(rr[t] + D + D / 16, sv[t]);
#pragma unroll
      for (int i = 0; i < kWordsV; ++i) {
        uint32_t s01 = __byte_perm(sv[0][i], sv[1][i], pick), s23 = __byte_perm(sv[2][i], sv[3][i], pick);
        if (masked) {
          // what no row sees counts as zero, whatever it holds; a NaN (or a scale that is none) that only some
          // rows see is put into those rows below
          const uint32_t b01 = valid >> (mt * 16 + 2 * c), b23 = b01 >> 8;
          s01 &= ((b01 & 1u) ? 0xFFFFu : 0u) | ((b01 & 2u) ? 0xFFFF0000u : 0u);
          s23 &= ((b23 & 1u) ? 0xFFFFu : 0u) | ((b23 & 2u) ? 0xFFFF0000u : 0u);
          if constexpr (!kList) {
            const uint32_t n01 = unfit_halves(s01), n23 = unfit_halves(s23);
            poisoned = poisoned || (n01 | n23) != 0;
            s01 &= ~n01;
            s23 &= ~n23;
          }
        }
        uint32_t w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = lds32(rr[t] + D / 2 + (g + 8 * i) * 4);
        uint32_t e01[4], o01[4], e23[4], o23[4];
        codes_to_half2((w[0] & 0x0F0F0F0Fu) | ((w[1] << 4) & 0xF0F0F0F0u), e01);
        codes_to_half2(((w[0] >> 4) & 0x0F0F0F0Fu) | (w[1] & 0xF0F0F0F0u), o01);
        codes_to_half2((w[2] & 0x0F0F0F0Fu) | ((w[3] << 4) & 0xF0F0F0F0u), e23);
        codes_to_half2(((w[2] >> 4) & 0x0F0F0F0Fu) | (w[3] & 0xF0F0F0F0u), o23);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t a0 = hmul2(e01[b], s01), a1 = hmul2(o01[b], s01), a2 = hmul2(e23[b], s23), a3 = hmul2(o23[b], s23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][i * 4 + b], a0, a1, a2, a3, pf[mt][nt][0], pf[mt][nt][1]);
        }
      }
    }
    if constexpr (!kList) {
      if (masked && __any_sync(~0u, poisoned)) {
        for (int at = 0; at < kTile; ++at) {
          if (!((valid >> at) & 1u)) continue;
          uint32_t sv[kWordsV];
          lds_words(base + at * kRow + D + D / 16, sv);
#pragma unroll
          for (int i = 0; i < kWordsV; ++i) {
            if (unfit_halves((g >> 2) ? sv[i] >> 16 : sv[i] & 0xFFFFu) == 0) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (pos0 + at < limit[nt][e & 1] && pos0 + at >= low[nt][e & 1])
#pragma unroll
                  for (int b = 0; b < 4; ++b) acc[nt][i * 4 + b][e] = NAN;
          }
        }
      }
    }
    __syncwarp();
    if (tile + Sh::kStages * kWarps < tiles) {
      // Every lane has read the stage: the vote on the maximum went by all keys, and these sums by all values, a word of
      // them each.
      uint32_t seen = 0;
#pragma unroll
      for (int i = 0; i < kWordsV; ++i) seen ^= __float_as_uint(acc[0][i * 4 + 3][0]);
      bring(stage, next_pos, next_page, zero_of(seen, p.zero));
      next_pos = later_pos;
      next_page = page_of(next_pos);
      later_pos = position_of(tile + (Sh::kStages + 2) * kWarps);
    }
    if (++stage == Sh::kStages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  dependents_launch();

  // ---- join the warps
  if (!ok) {
    if (lane == 0) atomicExch(&gave_up, 1);
    // the copies that are still on their way: the one that was waited for and those behind it, if they were asked for
#pragma unroll 1
    for (int s = 0; s < Sh::kStages; ++s) {
      wait_bounded(&bars[warp][stage], parity);
      if (++stage == Sh::kStages) {
        stage = 0;
        parity ^= 1u;
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[nt][e];
      t += __shfl_xor_sync(~0u, t, 4);
      t += __shfl_xor_sync(~0u, t, 8);
      t += __shfl_xor_sync(~0u, t, 16);
      if (g == 0) {
        m_of[warp][nt * 8 + 2 * c + e] = m[nt][e];
        l_of[warp][nt * 8 + 2 * c + e] = t;
      }
    }
  __syncthreads();  // (also: every warp is done with the ring)
  if (tid < NT * 8) {
    // a thread a row: what each warp's sums are to be multiplied by, where the row goes
    float top = m_of[0][tid], sum = 0.0f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, m_of[w][tid]);
    float a[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a[w] = m_of[w][tid] == -INFINITY ? 0.0f : exp2_fast(m_of[w][tid] - top);
      sum += m_of[w][tid] == -INFINITY ? l_of[w][tid] : l_of[w][tid] * a[w];  // (0, or NaN, where a warp saw nothing else)
    }
    const float inv = gave_up ? NAN : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l_of[w][tid] = inv != inv ? inv : a[w] * inv;
    part_log2[tid] = gave_up ? NAN : sum == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top - kShift) + __log2f(sum);
    const int row = min(row0 + tid, rows - 1);
    out_of[tid] = (int64_t)(token0 + row / p.group) * p.heads * p.group + head * p.group + row % p.group;
  }
  __syncthreads();
  float* joined = reinterpret_cast<float*>(smem);
  constexpr int kPitch = D + 4;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = l_of[warp][nt * 8 + 2 * c + e];
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        float* to_row = joined + (warp * NT * 8 + nt * 8 + 2 * c + e) * kPitch + (g + 8 * (t / 4)) * 8 + 2 * (t % 4);
        *reinterpret_cast<float2*>(to_row) = make_float2(acc[nt][t][e] * a, acc[nt][t][e + 2] * a);
      }
    }
  __syncthreads();
  const int here = min(NT * 8, rows - row0) * (D / 4);  // groups of four channels
  const int64_t part = ((int64_t)nth_part * p.heads + head) * p.part_rows + row0;
  for (int u = tid; u < here; u += kThreads) {
    const int row = u / (D / 4), ch = u % (D / 4) * 4;
    float4 o = *reinterpret_cast<const float4*>(joined + row * kPitch + ch);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(joined + (w * NT * 8 + row) * kPitch + ch);
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    if (p.parts > 1)
      // (this thread alone has read the place: the part stays here for the cluster to read)
      *reinterpret_cast<float4*>(joined + row * kPitch + ch) = o;
    else if (count == 1)
      store4(p, out_of[row] * D + ch, o);
    else
      *reinterpret_cast<float4*>(p.part_o + (part + row) * D + ch) = o;
  }
  if (p.parts <= 1) {
    if (tid < NT * 8 && row0 + tid < rows) {
      if (count > 1)
        p.part_lse[part + tid] = part_log2[tid];
      else if (p.lse != nullptr)
        p.lse[out_of[tid]] = part_log2[tid] * 0.6931471805599453f;
    }
    return;
  }
  // ---- join the cluster's parts over distributed shared memory: the weights of the parts by a thread a row,
  // then each CTA a share of the elements
  cluster_sync();
  const uint32_t o_at = lt::smem_u32(joined), l_at = lt::smem_u32(part_log2);
  float(*weight)[NT * 8] = m_of;
  if (tid < NT * 8) {
    float e[kMaxParts], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r) e[r] = r < p.parts ? peer_f32(l_at + tid * 4, r) : -INFINITY;
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r) top = fmaxf(top, e[r]);
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r) {
      const float x = e[r];
      e[r] = x == -INFINITY ? 0.0f : exp2_fast(x - top);  // (NaN stays NaN)
      sum += e[r];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r) weight[r][tid] = inv != inv ? inv : e[r] * inv;
    if (rank == 0 && p.lse != nullptr && row0 + tid < rows)
      p.lse[out_of[tid]] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
  }
  __syncthreads();
  for (int u = rank * kThreads + tid; u < here; u += p.parts * kThreads) {
    const int row = u / (D / 4), ch = u % (D / 4) * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kMaxParts; ++r) {
      if (r >= p.parts) break;
      const float4 x = peer_f32x4(o_at + (row * kPitch + ch) * 4, r);
      const float w = weight[r][row];
      o.x += w * x.x, o.y += w * x.y, o.z += w * x.z, o.w += w * x.w;
    }
    store4(p, out_of[row] * D + ch, o);
  }
  cluster_sync();  // (a CTA's shared memory stays until its peers have read it)
}

template <int D, int NT, bool kShaped>
RowsKernel rows_of(bool list) {
  return {list ? reinterpret_cast<const void*>(&rows_kernel<D, NT, true, kShaped>)
               : reinterpret_cast<const void*>(&rows_kernel<D, NT, false, kShaped>),
          Shape<D, NT>::kSmem, Shape<D, NT>::kPerSm};
}

}  // namespace

namespace lt {
namespace kv4 {

template <bool kShaped>
RowsKernel rows_kernel_of(int d, int nt, bool list) {
  if (d == 64) return nt == 1 ? rows_of<64, 1, kShaped>(list) : nt == 2 ? rows_of<64, 2, kShaped>(list) : rows_of<64, 4, kShaped>(list);
  if (d == 128)
    return nt == 1 ? rows_of<128, 1, kShaped>(list) : nt == 2 ? rows_of<128, 2, kShaped>(list) : rows_of<128, 4, kShaped>(list);
  return nt == 1 ? rows_of<256, 1, kShaped>(list) : rows_of<256, 2, kShaped>(list);
}

}  // namespace kv4
}  // namespace lt
