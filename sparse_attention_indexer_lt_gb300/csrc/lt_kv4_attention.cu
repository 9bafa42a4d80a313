// lt_kv4_attention.cu -- attention over the 4-bit cache for few query rows a
// request (decode, drafted tokens) and for listed positions, and the join of the
// parts of a split request.
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
// shortened), of which unpacking and scaling are 450; 2.50 are issued a clock and SM, 62% of what its schedulers
// could (2.17, 54%, with heads of 256, whose 168 registers leave 12 warps). More resident warps or deeper rings change
// nothing (5 CTAs an SM with 2 stages 272 us, 4 with 2 or 3 267 to 269, 3 with 4 281, on the 64 ragged
// requests). Measured (4.5-bit rows read once): 64 requests of 2048 to 65536 positions,
// 4 kv heads of 128, 253 us, 4.9 TB/s; one request of 262144 positions, 4 heads of 256,
// 65 us, 4.7 TB/s; the copy rate is 6.8. The widest instances (32 rows; 16 with heads of 256), which serve 17 to
// 64 rows, do not fit the registers: they spill 468 bytes a thread with heads of 128, 252 with 64, 232 with 256.

#include <mutex>

#include "lt_kv4.cuh"
#include "lt_kv4_attention.cuh"
#include "lt_kv4_prefill.h"

namespace {

using namespace lt::kv4;

constexpr float kShift = 6.0f;  // weights are held as 2^6 exp(s - max)
constexpr int kMaxParts = 8;    // CTAs of a portable cluster
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
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = lds32(a);
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  } else {
    static_assert(N == 4, "1, 2 or 4 words");
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a));
  }
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

template <int D, int NT, bool kList>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT>::kPerSm)) rows_kernel(AttentionParams p) {
  using Sh = Shape<D, NT>;
  constexpr int kRow = Sh::kRow;
  constexpr int kGroups = D / 32;  // scale groups of a key
  constexpr int kWordsV = D / 64;  // words of value codes a lane takes from a position
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][Sh::kStages];
  __shared__ uint32_t valid_of[kWarps][Sh::kStages];
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
    to = min(to, rq.length - rq.queries + last + 1);
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
  auto bring = [&](int stage, int pos, int page) {
    const bool there = pos >= 0 && page >= 0 && page < p.pages;
    const uint32_t tile_at = ring + stage * Sh::kTileBytes;
    if constexpr (kList) {
      // one row a position: 16-byte copies, the lanes along the rows (a bulk copy a row is no faster: 51 us either
      // way on 1021 lists of 512, then bound by the chain of loads at a CTA's start)
      const uint32_t valid = __ballot_sync(~0u, there);
      if (lane == 0) valid_of[warp][stage] = valid;
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
      if (warp + s * kWarps < tiles) bring(s, pos[s], page[s]);
  }
  float factor[NT][2];  // of columns 2c, 2c + 1: logits in units of log 2
  int limit[NT][2], low[NT][2];
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
    }
  }
  const int safe_to = kList ? INT32_MAX : rq.length - rq.queries + row0 / p.group + 1;  // every row sees up to here
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
    ok = wait_bounded(&bars[warp][stage], parity) && ok;  // (the warp votes: it stays converged)
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
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mt][nt][e] *= factor[nt][e & 1];
          if (masked) {
            const int at = mt * 16 + g + (e >> 1) * 8;
            bool sees = (valid >> at) & 1u;
            if constexpr (!kList) sees = sees && pos0 + at < limit[nt][e & 1] && pos0 + at >= low[nt][e & 1];
            if (!sees) s[mt][nt][e] = -INFINITY;
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
    __syncwarp();  // every lane has read the stage
    if (tile + Sh::kStages * kWarps < tiles) {
      bring(stage, next_pos, next_page);
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
  if (!ok && lane == 0) atomicExch(&gave_up, 1);
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

// Joins the parts of a (query, head): out = sum_i 2^(e_i - top) o_i / sum_i 2^(e_i - top), e_i
// the parts' logarithms. Eight warps share the parts, in one fixed order whatever the timing.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttentionParams p) {
  constexpr int kVec = D / 32;
  __shared__ float o_of[kJoinThreads / 32][D];
  __shared__ float sum_of[kJoinThreads / 32], top_of[kJoinThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  dependency_wait();
  const int q_heads = p.heads * p.group;
  const int64_t token = blockIdx.x / q_heads;
  const int qh = (int)(blockIdx.x % q_heads), head = qh / p.group;
  const int request = owner_of_token(p, (int)token);
  if (request < 0) return;
  const int2 pl = p.plan[request];
  const int n = pl.y;
  const Request rq = request_of(p, request);
  const int64_t nth = token - rq.first;
  if (nth >= rq.computed) return;
  if (n <= 1) return;  // written whole
  const int64_t step = (int64_t)p.heads * p.part_rows;
  const int64_t first = pl.x * step + (int64_t)head * p.part_rows + nth * p.group + qh % p.group;

  float top = -INFINITY;
  bool bad = false;
  for (int i = tid; i < n; i += kJoinThreads) {
    const float e = p.part_lse[first + i * step];
    top = fmaxf(top, e);
    bad = bad || e != e;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) top_of[warp] = top;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, top_of[w]);

  float o[kVec] = {}, sum = 0.0f;
#pragma unroll 4
  for (int i = warp; i < n; i += kJoinThreads / 32) {
    const float e = p.part_lse[first + i * step];
    const float* from = p.part_o + (first + i * step) * D + lane * kVec;
    float x[kVec];
#pragma unroll
    for (int k = 0; k < kVec; k += 2) *reinterpret_cast<float2*>(x + k) = *reinterpret_cast<const float2*>(from + k);
    const float w = e == -INFINITY ? 0.0f : exp2_fast(e - top);
    sum += w;
#pragma unroll
    for (int k = 0; k < kVec; ++k) o[k] += e == -INFINITY ? 0.0f : w * x[k];
  }
#pragma unroll
  for (int k = 0; k < kVec; ++k) o_of[warp][lane * kVec + k] = o[k];
  if (lane == 0) sum_of[warp] = sum;
  __syncthreads();
  dependents_launch();
  float all = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) all += sum_of[w];
  const float inv = all == 0.0f ? 0.0f : 1.0f / all;
  const int64_t out_row = token * q_heads + qh;
  if (tid < D / 4) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(&o_of[w][tid * 4]);
      y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
    }
    y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
    if (bad) y = make_float4(NAN, NAN, NAN, NAN);
    store4(p, out_row * D + tid * 4, y);
  }
  if (p.lse != nullptr && tid == 0)
    p.lse[out_row] = bad ? NAN : all == 0.0f ? -INFINITY : (top + __log2f(all)) * 0.6931471805599453f;
}

// ---- host side

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_smem_set[kMaxDevices][3][4][2];  // by head size, row tiles (3: many rows), listed

struct RowsKernel {
  const void* func;
  int smem, per_sm;
};

template <int D, int NT>
RowsKernel rows_of(bool list) {
  return {list ? reinterpret_cast<const void*>(&rows_kernel<D, NT, true>)
               : reinterpret_cast<const void*>(&rows_kernel<D, NT, false>),
          Shape<D, NT>::kSmem, Shape<D, NT>::kPerSm};
}
RowsKernel rows_kernel_of(int d, int nt, bool list) {
  if (d == 64) return nt == 1 ? rows_of<64, 1>(list) : nt == 2 ? rows_of<64, 2>(list) : rows_of<64, 4>(list);
  if (d == 128) return nt == 1 ? rows_of<128, 1>(list) : nt == 2 ? rows_of<128, 2>(list) : rows_of<128, 4>(list);
  return nt == 1 ? rows_of<256, 1>(list) : rows_of<256, 2>(list);
}

// The launch for these sizes: row tiles, parts and workspace.
struct Plan {
  bool prefill;        // the kernel for many query rows
  int nt, row_tiles;
  int64_t part_rows;   // query rows of a part
  int parts;           // > 0: every request (list) in that many parts, a cluster; 0: chunks of like work
  int target;          // chunks wanted over all requests
  int min_chunk;
  int64_t flats;       // chunks, or requests (lists) at most
  bool join;           // chunks are joined by a second launch
  int64_t plan_bytes, lse_bytes, o_bytes;
  int64_t bytes() const { return join ? plan_bytes + lse_bytes + o_bytes : 0; }
};

constexpr int kMinChunk = 256;
constexpr int kPrefillMinChunk = 512;
// Query rows a kv head from which the kernel for many rows is taken, each side's us with 8 kv heads of D:
//   1 request of 8192 positions, D = 128: 26 there, 25 here with 16 rows, 28 and 37 with 32, 36 and 74 with 256
//   16 requests of 4096, D = 128: 81 and 74 with 32 rows, 87 and 119 with 64; D = 64: 68 and 59, 73 and 57
//   D = 256, 4 kv heads: 1 request of 8192 positions 32 and 35 with 32 rows; 4 of them 48 and 39, with 64 rows 49 and
//   70; 64 requests of 2048 94 and 66 with 20 rows, 101 and 117 with 40
// so from two row tiles of this kernel on (D = 64: from three), and with few CTAs from 17 rows (D = 256, whose
// tiles have fewer rows: with very few). The rows are those of max_new queries, for all requests of the call:
// where one has many queries and others one, these are computed there, too (not measured).
int prefill_from(int d, int64_t units, int sms) {
  return units * (d == 256 ? 16 : 4) <= sms ? 17 : d == 64 ? 65 : 33;
}
constexpr int kPartPositions = 2048;  // positions of a part up to which requests are cut into equal numbers of parts

// rows: the most query rows of a request
Plan finish_plan(Plan a, int heads, int d, int requests, int64_t rows) {
  // A chunk is at least total / target long, so the requests have fewer than target + requests. Parts are kept for
  // the requests that have several chunks alone: each of those is longer than a chunk, so they are fewer than
  // target, and have fewer than 2 target chunks.
  if (a.flats == 0) a.flats = a.target == 1 ? requests : a.target + (int64_t)requests;
  a.join = a.parts == 0 && a.target > 1;
  const int64_t parts = (a.target < requests ? (int64_t)a.target : (int64_t)requests) + a.target - 1;
  a.part_rows = rows;
  a.plan_bytes = ((int64_t)requests * 8 + 15) / 16 * 16;
  a.lse_bytes = (parts * heads * rows * 4 + 15) / 16 * 16;
  a.o_bytes = parts * heads * rows * d * 4;
  return a;
}

// positions: the most that a request can have by its row of the table
Plan make_plan(int sms, int64_t tokens, int heads, int group, int d, int requests, int max_new, int list_len,
               int64_t positions, int window) {
  Plan a = {};
  const int64_t rows = (int64_t)(list_len > 0 ? 1 : max_new) * group;
  const int64_t part_rows = (max_new < tokens ? (int64_t)max_new : tokens) * group;
  a.prefill = list_len == 0 && rows >= prefill_from(d, (int64_t)requests * heads, sms);
  if (a.prefill) {
    a.row_tiles = (int)((rows + prefill_rows(d) - 1) / prefill_rows(d));
    a.min_chunk = kPrefillMinChunk;
    // one CTA an SM: chunks only where one request's row tiles alone do not fill the SMs (their joins cost more
    // than an uneven second wave: 256 row tiles of 16384 positions take 511 us whole, 690 us in halves). With
    // several requests the chunks are cut from all their positions together, so the long ones alone are cut.
    const int64_t units = (int64_t)heads * a.row_tiles;
    a.target = (int)((sms + units - 1) / units);
    return finish_plan(a, heads, d, requests, part_rows);
  }
  const int most = d == 256 ? 2 : 4;
  a.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : most;
  if (a.nt > most) a.nt = most;
  a.row_tiles = (int)((rows + a.nt * 8 - 1) / (a.nt * 8));
  a.min_chunk = kMinChunk;
  const int slots = sms * rows_kernel_of(d, a.nt, list_len > 0).per_sm;
  const int64_t units = (int64_t)heads * a.row_tiles;
  // what one query (a request's queries) can see at most: lengths are known on the device alone, so a table wider
  // than the requests counts as if they filled it
  int64_t seen = list_len > 0 ? list_len : positions;
  if (list_len == 0 && window > 0 && (int64_t)window + max_new + kTile < seen) seen = (int64_t)window + max_new + kTile;
  const int64_t whole = (list_len > 0 ? tokens : (int64_t)requests) * units;
  // parts while the CTAs do not fill the slots and a part is at least a tile for every warp (filling them twice
  // costs the drafted step 55 us instead of 46)
  int parts = 1;
  while (parts < kMaxParts && whole * parts < slots && seen > (int64_t)parts * kTile * kWarps) parts *= 2;
  // Requests stay whole, too, where they are so many that the hardware evens them out and none can be long
  // (us whole against chunks, 8 kv heads of 128: 256 requests to 8192 positions 287 and 303, 1024
  // 956 and 1083; but 128 to 8192 176 and 168, 128 to 32768 638 and 498, 512 of 4 heads 1051 and 998).
  const bool whole_ones = parts == 1 && ((whole >= 3 * slots && seen <= 8192) || (whole >= 8 * slots && seen <= 32768));
  if (list_len > 0 || whole_ones || seen <= (int64_t)parts * kPartPositions) {
    a.parts = parts;
    a.flats = list_len > 0 ? tokens : requests;
    return finish_plan(a, heads, d, requests, part_rows);
  }
  // Several chunks a slot where requests differ in length, so that the last ones to end are short (64 ragged
  // requests: 324, 279, 271, 269 us with 1, 2, 3, 4); one request's chunks are alike, and one
  // wave of them has the fewest starts and joins (262144 positions at D = 256: 82 us, 96 with 2).
  const int64_t target = ((int64_t)slots * (requests == 1 ? 1 : 4) + units - 1) / units;
  a.target = (int)(target < 1 ? 1 : target);
  return finish_plan(a, heads, d, requests, part_rows);
}

lt_status device_of(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return LT_ERR_CUDA;
  if (*dev < 0 || *dev >= kMaxDevices) return LT_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[*dev] == 0 && cudaDeviceGetAttribute(&g_sms[*dev], cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return LT_ERR_CUDA;
  *sms = g_sms[*dev];
  return LT_OK;
}

lt_status check_sizes(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t requests,
                      int32_t max_new, int32_t list_len) {
  if (tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1 || requests < 0 ||
      max_new < 1 || list_len < 0)
    return LT_ERR_INVALID_ARG;
  if (lt_kv4_row_bytes(head_dim) == 0 || tokens > INT32_MAX) return LT_ERR_UNSUPPORTED;
  return LT_OK;
}

}  // namespace

extern "C" {

lt_status lt_kv4_workspace(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                           int32_t requests, int32_t max_new, int32_t list_len, int64_t positions,
                           int32_t window, int64_t* bytes) {
  if (bytes == nullptr) return LT_ERR_INVALID_ARG;
  lt_status st = check_sizes(tokens, q_heads, kv_heads, head_dim, requests, max_new, list_len);
  if (st == LT_OK && (positions < 0 || window < 0)) st = LT_ERR_INVALID_ARG;
  if (st != LT_OK) return st;
  *bytes = 0;
  if (tokens == 0 || requests == 0) return LT_OK;
  int dev = 0, sms = 0;
  st = device_of(&dev, &sms);
  if (st != LT_OK) return st;
  *bytes = make_plan(sms, tokens, kv_heads, q_heads / kv_heads, head_dim, requests, max_new, list_len,
                     positions, window >= positions ? 0 : window).bytes();
  return LT_OK;
}

lt_status lt_kv4_attention(const void* q, int32_t dtype, int64_t tokens, int32_t q_heads,
                           int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                           int64_t q_head_stride, const void* cache, int64_t pages, int32_t page_size,
                           const int32_t* block_table, int32_t table_width, const int32_t* lengths,
                           int32_t requests, const int32_t* starts, int32_t max_new,
                           const int32_t* positions, int32_t list_len, int32_t window, float scale,
                           void* out, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  lt_status st = check_sizes(tokens, q_heads, kv_heads, head_dim, requests, max_new, list_len);
  if (st == LT_ERR_INVALID_ARG) return st;
  const int shift = page_shift(page_size);
  if (dtype != LT_DTYPE_BF16 && dtype != LT_DTYPE_F16) return LT_ERR_INVALID_ARG;
  if (shift < 0 || pages < 0 || table_width < 1 || window < 0 || !(scale == scale) || scale - scale != 0.0f)
    return LT_ERR_INVALID_ARG;
  if (starts == nullptr && (tokens != requests || max_new != 1)) return LT_ERR_INVALID_ARG;
  if (positions != nullptr && window != 0) return LT_ERR_INVALID_ARG;
  if (positions == nullptr && list_len != 0) return LT_ERR_INVALID_ARG;
  if (positions != nullptr && list_len == 0) return LT_ERR_INVALID_ARG;
  if (tokens > 0 && requests > 0) {
    if (q == nullptr || out == nullptr || block_table == nullptr || lengths == nullptr ||
        (cache == nullptr && pages > 0))
      return LT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(q) % 16 || q_token_stride % 8 || q_head_stride % 8 ||
        reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(out) % 16)
      return LT_ERR_INVALID_ARG;
  }
  if (st != LT_OK || pages > INT32_MAX) return LT_ERR_UNSUPPORTED;
  if (tokens == 0 || requests == 0) return LT_OK;
  // a window as wide as the table holds every position; the kernels' sums of
  // positions, queries and window stay within 32 bits
  if (((int64_t)table_width << shift) <= window) window = 0;
  if ((int64_t)window + tokens >= INT32_MAX) return LT_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  st = device_of(&dev, &sms);
  if (st != LT_OK) return st;
  const int group = q_heads / kv_heads;
  const Plan plan = make_plan(sms, tokens, kv_heads, group, head_dim, requests, max_new, list_len,
                              (int64_t)table_width << shift, window);
  if (plan.join && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < plan.bytes()))
    return LT_ERR_INVALID_ARG;
  const int64_t grid = plan.flats * kv_heads * plan.row_tiles * (plan.parts > 1 ? plan.parts : 1), joins = tokens * q_heads;
  if (grid > INT32_MAX || joins > INT32_MAX) return LT_ERR_UNSUPPORTED;

  AttentionParams p = {};
  p.q = q;
  p.cache = static_cast<const uint8_t*>(cache);
  p.table = block_table;
  p.lengths = lengths;
  p.starts = starts;
  p.positions = positions;
  p.out = out;
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (plan.join) {
    p.plan = reinterpret_cast<int2*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + plan.plan_bytes);
    p.part_o = reinterpret_cast<float*>(ws + plan.plan_bytes + plan.lse_bytes);
  }
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.pages = (int32_t)pages;
  p.tokens = (int32_t)tokens;
  p.requests = requests;
  p.width = table_width;
  p.heads = kv_heads;
  p.group = group;
  p.shift = shift;
  p.list_len = list_len;
  p.window = window;
  p.parts = plan.parts;
  p.target = plan.target;
  p.min_chunk = plan.min_chunk;
  p.row_tiles = plan.row_tiles;
  p.max_new = max_new;
  p.part_rows = (int32_t)plan.part_rows;
  p.align = plan.prefill ? 128 : kTile;
  p.bf16 = dtype == LT_DTYPE_BF16;
  p.scale_log2 = scale * 1.4426950408889634f;

  const bool list = list_len > 0;
  RowsKernel k = {};
  if (plan.prefill)
    k.func = prefill_kernel_ptr(head_dim, &k.smem);
  else
    k = rows_kernel_of(head_dim, plan.nt, list);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    bool& set = g_smem_set[dev][head_dim / 128][plan.prefill ? 3 : plan.nt / 2][list];
    if (!set) {
      if (cudaFuncSetAttribute(k.func, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess)
        return LT_ERR_CUDA;
      set = true;
    }
  }
  st = launch(k.func, dim3((unsigned)grid), plan.prefill ? kPrefillThreads : kThreads, (unsigned)k.smem, &p, stream,
              plan.parts > 1 ? plan.parts : 1);
  if (st != LT_OK || !plan.join) return st;
  if (lt::take_injected_failure()) return LT_ERR_CUDA;
  const void* func = head_dim == 64    ? reinterpret_cast<const void*>(&join_kernel<64>)
                     : head_dim == 128 ? reinterpret_cast<const void*>(&join_kernel<128>)
                                       : reinterpret_cast<const void*>(&join_kernel<256>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)joins);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* a[] = {&p};
  return cudaLaunchKernelExC(&cfg, func, a) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

}  // extern "C"
