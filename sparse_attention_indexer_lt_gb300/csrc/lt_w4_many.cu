// lt_w4_many.cu -- products with 4-bit weights for many tokens: tcgen05, the sums in tensor memory.
//
// A CTA takes one or two tiles of 128 outputs and a tile of up to 256 tokens; the weights are the product's
// 128 rows, the tokens its columns, so a tile of few tokens wastes nothing. In steps of 128 inputs,
//   eight warps a tile of outputs   unpack, four of them every other step: a thread the step's inputs of one output, codes
//                 times scale in fp16, into tensor memory, where the product reads its rows: shared memory, which carries
//                 codes and tokens, could not take the unpacked weights' way in and out as well
//   one warp      issues the products
//   two warps     bring the codes, 256 inputs at a time by a tensor map, and the tokens, a bulk copy a step
// The tokens are laid out for that by a launch before: fp16, scaled by a power of two for each token (bf16's
// range does not fit), swizzled, a step's tile contiguous. Where there are few outputs a cluster cuts the inputs, and its
// parts join over distributed shared memory in one order.
//
// What bounds it. Tokens by the hundred: the tokens' way from the L2 cache, which each 128 outputs take again (some 10
// TB/s), and the starts and ends of three waves: 509 tokens through 4096 x 14336 take 49 us, 1.23 PFLOP/s, 63% of
// cuBLAS's burst. Some ten tokens: the start (layout, 4 us to the first product), memory (4.7 TB/s of codes
// while products run) and the cluster's join (4 us): 64 tokens through 8192 x 10240 take 20.6 us, the bytes 7.3.
// On the way, us for those two: the kernel for few tokens, tokens in tiles of 32, 717 and 217; unpacked weights through shared memory,
// 128 outputs, 76 and 67; 256 outputs and the weights asked for before the tokens' layout 62 and 46; codes by a tensor map,
// unpacked weights in tensor memory, 80 and 23.5 (poor tiles); steps of 128 inputs in place of 64 57 and 22; whole lines
// out, parts pushed to their owner, tiles by measured costs 48 and 21.5; two CTAs an SM 48 and 20.4. Dropped: rows
// handed to the products a step late, so that their way to tensor memory is hidden (65 against 57).

#include <cmath>
#include <mutex>

#include "lt_kv4_tcgen05.cuh"
#include "lt_w4_linear.h"

namespace {

using namespace lt::kv4;
using namespace lt::w4;

template <int kTiles>
struct Many {
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kUnpackWarps = 8 * kTiles;
  static constexpr int kCta = kUnpackWarps * 32 + 96;
  static constexpr int kPacked = kRows * 128;  // bytes of the codes of 256 inputs
};
constexpr int kMaxRing = 8;

struct Shared {
  uint64_t codes_full[kMaxRing], codes_empty[kMaxRing];
  uint64_t tokens_full[kMaxRing], tokens_empty[kMaxRing];
  uint64_t rows_full[kMaxRing], rows_empty[kMaxRing];  // unpacked weights in tensor memory
  uint64_t done;
  alignas(16) float inverse[256];
  uint32_t tmem;
  int gave_up;
};

// A warp waits for a phase, kWaitPolls polls at most; a wait that gives up marks the CTA, whose outputs are NaN
// then, and the warp goes on: the roles keep their steps, so nobody waits for one that has left. In a marked CTA nothing more
// is brought, and nobody waits any more (beyond some 64 polls) but for what has to be over before it ends (kOver).
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(lt::smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
template <bool kOver = false>
__device__ __forceinline__ void wait_warp(uint64_t* bar, uint32_t parity, Shared* sh) {
  bool done = ready(bar, parity);
  if (__all_sync(~0u, done)) return;
#pragma unroll 1
  for (uint32_t i = 0; i < lt::kWaitPolls; ++i) {
    done = done | lt::mbar_try_wait(bar, parity);
    if (__all_sync(~0u, done)) return;
    if (!kOver && i % 64 == 63 && __any_sync(~0u, *(volatile int*)&sh->gave_up != 0)) return;
  }
  *(volatile int*)&sh->gave_up = 1;
}

// ---- the tokens as the product reads them: a CTA a token
constexpr int kLayoutThreads = 256;
constexpr int kHeld = 4;  // pieces of 16 bytes that a thread keeps between the two looks at them

__global__ void __launch_bounds__(kLayoutThreads) layout_kernel(ManyParams p) {
  __shared__ uint32_t big_of[kLayoutThreads / 32];
  const int tid = threadIdx.x, token = blockIdx.x;
  dependency_wait();
  // (the product's CTAs may start: everything before this launch is done, so they ask for weights at once)
  dependents_launch();
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + (int64_t)token * p.x_stride);
  const int pieces = p.steps * 16, there = p.k / 8;
  uint4 held[kHeld];
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int q = tid + i * kLayoutThreads;
    held[i] = make_uint4(0u, 0u, 0u, 0u);
    if (q < there) held[i] = __ldg(x + q);
  }
  float mul = 1.0f;
  if (p.bf16) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) big = max(big, largest_of(held[i]));
    for (int q = tid + kHeld * kLayoutThreads; q < there; q += kLayoutThreads) big = max(big, largest_of(__ldg(x + q)));
    big = __reduce_max_sync(~0u, big);
    if ((tid & 31) == 0) big_of[tid >> 5] = big;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLayoutThreads / 32; ++w) big = max(big, big_of[w]);
    mul = token_power(big);
  }
  if (tid == 0) p.inverse[token] = 1.0f / mul;
  uint8_t* to = p.tiles_at + ((int64_t)(token / p.tile) * p.steps * 2 * p.tile + token % p.tile) * 128;
  auto write = [&](int q, const uint4& v) {
    *reinterpret_cast<uint4*>(to + (int64_t)(q / 8) * p.tile * 128 + (((q & 7) ^ (token % p.tile & 7)) << 4)) = p.bf16 ? to_half(v, mul) : v;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kLayoutThreads < pieces) write(tid + i * kLayoutThreads, held[i]);
  for (int q = tid + kHeld * kLayoutThreads; q < pieces; q += kLayoutThreads)
    write(q, q < there ? __ldg(x + q) : make_uint4(0u, 0u, 0u, 0u));
}

// What lane 0 has asked for into a ring is on its way no more, also where somebody gave up.
__device__ __forceinline__ void wait_for_asked(uint64_t* full, int asked, int ring, Shared* sh) {
  asked = __shfl_sync(~0u, asked, 0);
  for (int i = max(asked - ring, 0); i < asked; ++i) wait_warp<true>(&full[i % ring], i / ring & 1, sh);
}

// A place in a ring: its index and the parity of its round.
struct Turn {
  int at = 0;
  uint32_t parity;
  __device__ __forceinline__ explicit Turn(uint32_t first) : parity(first) {}
  __device__ __forceinline__ void next(int ring) {
    if (++at == ring) {
      at = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ void tensor_in(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(lt::smem_u32(bar)) : "memory");
}

// Codes come for two steps at once. A thread has an output, and every other step of it.
template <int kTiles>
__device__ __forceinline__ void unpack_role(const ManyParams& p, Shared* sh, uint32_t packed, int row0, int from, int to) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, odd = warp >> 2 & 1, tile = warp >> 3;
  const int row = tile * 128 + (warp & 3) * 32 + lane;  // (a warp reaches 32 lanes of tensor memory, by its number)
  const int groups = p.k / 32;
  const uint16_t* scales = p.scales + (int64_t)min(row0 + row, p.n - 1) * groups;
  // a row is 64 bytes of the step's box, its four 16-byte pieces turned by the row's second and third bit
  uint32_t piece[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) piece[g] = packed + odd * (Many<kTiles>::kRows * 64) + row * 64 + ((g ^ (row >> 1 & 3)) << 4);
  const uint32_t column = sh->tmem + ((uint32_t)((warp & 3) * 32) << 16) + p.rows_column + tile * 64;
  auto scales_of = [&](uint32_t (&s)[2], int u) {  // of the step's four groups, pairs
    if (u >= to) return;
    if (p.wide_scales) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(scales + u * 8 + odd * 4));
      s[0] = v.x;
      s[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int group = u * 8 + odd * 4 + i * 2;  // (codes past the end are zeros)
        s[i] = __ldg(scales + min(group, groups - 1)) | (uint32_t)__ldg(scales + min(group + 1, groups - 1)) << 16;
      }
    }
  };
  uint32_t s[2] = {}, later[2] = {};
  scales_of(s, from);
  Turn code(0), place(1);
  place.at = odd;
#pragma unroll 1
  for (int u = from; u < to; ++u) {
    if (u * 2 + odd >= p.steps) break;
    scales_of(later, u + 1);
    const bool free = ready(&sh->rows_empty[place.at], place.parity);
    wait_warp(&sh->codes_full[code.at], code.parity, sh);
    uint32_t w[4][4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[g][0]), "=r"(w[g][1]), "=r"(w[g][2]), "=r"(w[g][3]) : "r"(piece[g] + code.at * Many<kTiles>::kPacked) : "memory");
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h[32];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t scale = __byte_perm(s[i], 0, g ? 0x3232 : 0x1010);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t x[4];
          codes_to_half2(w[2 * i + g][j], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[16 * g + 4 * j + e] = hmul2(x[e], scale);
        }
      }
      if (i == 0) {  // (the first half is converted before there has to be a place)
        const uint32_t here = zero_of(w[0][0] ^ w[1][0] ^ w[2][0] ^ w[3][0], p.zero);
        if (lane == 0) arrive(&sh->codes_empty[code.at] + here);
        code.next(p.code_ring);
        if (!__all_sync(~0u, free)) wait_warp(&sh->rows_empty[place.at], place.parity, sh);
        fence_after();
      }
      tmem_st32(column + place.at * (kTiles * 64) + i * 32, h);
    }
    tmem_wait_st();
    fence_before();
    __syncwarp();
    if (lane == 0) arrive(&sh->rows_full[place.at]);
    place.at += 2;
    if (place.at >= p.row_ring) {
      place.at -= p.row_ring;
      place.parity ^= 1u;
    }
    s[0] = later[0];
    s[1] = later[1];
  }
}

template <int kTiles>
__global__ void __launch_bounds__(Many<kTiles>::kCta, 3 - kTiles) many_kernel(ManyParams p, const __grid_constant__ CUtensorMap codes) {
  constexpr int kRows = Many<kTiles>::kRows, kCta = Many<kTiles>::kCta, kUnpackWarps = Many<kTiles>::kUnpackWarps;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (lt::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ Shared shared;
  Shared* sh = &shared;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const uint32_t packed = lt::smem_u32(smem), token_bytes = p.tile * 256;
  const uint32_t tokens_at = packed + p.code_ring * Many<kTiles>::kPacked;
  if (tid == 32) asm volatile("prefetch.tensormap [%0];" :: "l"(&codes) : "memory");
  if (tid == 0) {
    for (int s = 0; s < kMaxRing; ++s) {
      lt::mbar_init(&sh->codes_full[s], 1);
      lt::mbar_init(&sh->codes_empty[s], kUnpackWarps);
      lt::mbar_init(&sh->tokens_full[s], 1);
      lt::mbar_init(&sh->tokens_empty[s], 1);
      lt::mbar_init(&sh->rows_full[s], kUnpackWarps / 2);
      lt::mbar_init(&sh->rows_empty[s], 1);
    }
    lt::mbar_init(&sh->done, 1);
    sh->gave_up = 0;
    lt::mbar_fence_init();
  }
  if (warp == kUnpackWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(lt::smem_u32(&sh->tmem)), "r"(p.columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();

  const int rank = blockIdx.x % p.parts, row0 = (int)(blockIdx.x / p.parts) * kRows;
  const int token0 = blockIdx.y * p.tile, tokens = min(p.tokens - token0, p.tile);
  const int supers = (p.steps + 1) / 2;
  const int from = (int)((int64_t)supers * rank / p.parts), to = (int)((int64_t)supers * (rank + 1) / p.parts);
  const int first = from * 2, last = min(to * 2, p.steps);
  const uint32_t tmem = sh->tmem;

  if (warp < kUnpackWarps) {
    unpack_role<kTiles>(p, sh, packed, row0, from, to);
  } else if (warp == kUnpackWarps) {
    const uint32_t lead = elect_one(), idesc = instruction(p.tile, false), d = __shfl_sync(~0u, tmem, 0);
    Turn token(0), place(0);
#pragma unroll 1
    for (int b = first; b < last; ++b) {
      wait_warp(&sh->tokens_full[token.at], token.parity, sh);
      wait_warp(&sh->rows_full[place.at], place.parity, sh);
      fence_after();
      const uint64_t x = desc_k_major(tokens_at + token.at * token_bytes);
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          mma_ts4<2>(d + m * p.sum_columns, d + p.rows_column + (place.at * kTiles + m) * 64 + i * 32, x + (uint32_t)(i * p.tile * 8), idesc,
                     b > first || i > 0, lead);
      mma_commit(&sh->rows_empty[place.at], lead);
      mma_commit(&sh->tokens_empty[token.at], lead);
      token.next(p.token_ring);
      place.next(p.row_ring);
    }
    mma_commit(&sh->done, lead);
  } else if (warp == kUnpackWarps + 1) {
    Turn code(1);
    int asked = 0;
#pragma unroll 1
    for (int u = from; u < to; ++u) {
      wait_warp(&sh->codes_empty[code.at], code.parity, sh);
      if (lane == 0 && *(volatile int*)&sh->gave_up == 0) {
        uint64_t* bar = &sh->codes_full[code.at];
        const uint32_t at = packed + code.at * Many<kTiles>::kPacked;
        lt::mbar_arrive_tx(bar, Many<kTiles>::kPacked);
        tensor_in(at, &codes, u * 128, row0, bar);
        tensor_in(at + kRows * 64, &codes, u * 128 + 64, row0, bar);
        ++asked;
      }
      __syncwarp();
      code.next(p.code_ring);
    }
    wait_for_asked(sh->codes_full, asked, p.code_ring, sh);
  } else {
    dependency_wait();  // the launch that lays the tokens out
    for (int t = lane; t < tokens; t += 32) sh->inverse[t] = p.inverse[token0 + t];
    const uint8_t* src = p.tiles_at + (int64_t)blockIdx.y * p.steps * token_bytes;
    Turn token(1);
    int asked = 0;
#pragma unroll 1
    for (int b = first; b < last; ++b) {
      wait_warp(&sh->tokens_empty[token.at], token.parity, sh);
      if (lane == 0 && *(volatile int*)&sh->gave_up == 0) {
        lt::mbar_arrive_tx(&sh->tokens_full[token.at], token_bytes);
        lt::bulk_g2s(smem + (tokens_at - packed) + token.at * token_bytes, src + (int64_t)b * token_bytes, token_bytes, &sh->tokens_full[token.at]);
        ++asked;
      }
      __syncwarp();
      token.next(p.token_ring);
    }
    wait_for_asked(sh->tokens_full, asked, p.token_ring, sh);
  }
  __syncwarp();
  wait_warp<true>(&sh->done, 0, sh);  // every product is done: the sums are there, and the rings are free
  fence_after();
  __syncthreads();
  const bool bad = *(volatile int*)&sh->gave_up != 0;

  // A thread a row, 16 tokens at a time; two sets of four warps take turns with a tile's. A cluster's parts: 32 rows, a
  // warp's, belong to one of its CTAs, which all of them write theirs to, [part][its 32 rows][four tokens][row][token].
  constexpr int kGroups = kRows / 32;
  constexpr int kPitch = kRows + 8;  // of a token's outputs in shared memory, 16 bits each
  const int own_groups = (kGroups + p.parts - 1) / p.parts;
  dependency_wait();
  if (bad) {
    // (a wait gave up: everything becomes NaN by the tokens' factors)
    for (int t = tid; t < p.tile; t += kCta) sh->inverse[t] = NAN;
    __syncthreads();
  }
  if (p.parts > 1) cluster_sync();  // the peers' rings are free, too
  if (warp < kUnpackWarps) {
    const int group = (warp >> 3) * 4 + (warp & 3), row = row0 + group * 32 + lane;
    const uint32_t at = tmem + (warp >> 3) * p.sum_columns + ((uint32_t)((warp & 3) * 32) << 16);
    const float bias = p.parts > 1 ? 0.0f : bias_of(p.bias, min(row, p.n - 1), p.bf16);
    const uint32_t to = peer_address(packed + ((rank * own_groups + group / p.parts) * p.tile * 32 + lane * 4) * 4, group % p.parts);
    uint16_t* line = reinterpret_cast<uint16_t*>(smem) + group * 32 + lane;
#pragma unroll 1
    for (int c = (warp >> 2 & 1) * 16; c < tokens; c += 32) {  // (a tile is whole 16s, so there is room past the last token)
      uint32_t y[16];
      tmem_read16(at + c, y);
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&sh->inverse[c + e]);
        v[e] = fmaf(__uint_as_float(y[e]), f.x, bias);
        v[e + 1] = fmaf(__uint_as_float(y[e + 1]), f.y, bias);
        v[e + 2] = fmaf(__uint_as_float(y[e + 2]), f.z, bias);
        v[e + 3] = fmaf(__uint_as_float(y[e + 3]), f.w, bias);
      }
      if (p.parts > 1) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) put_peer(to + (c + e) * 128, make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
      } else if (p.bf16) {
#pragma unroll
        for (int e = 0; e < 16; ++e) line[(c + e) * kPitch] = bits_of(v[e], 1);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) line[(c + e) * kPitch] = bits_of(v[e], 0);
      }
    }
  }
  fence_before();
  if (p.parts == 1) {
    // whole lines out of shared memory: a token's outputs, 16 bytes a thread where they start on that
    __syncthreads();
    const uint16_t* lines = reinterpret_cast<const uint16_t*>(smem);
    for (int u = tid; u < tokens * (kRows / 8); u += kCta) {
      const int t = u / (kRows / 8), at = u % (kRows / 8) * 8;
      const uint4 v = *reinterpret_cast<const uint4*>(lines + t * kPitch + at);
      uint16_t* to = static_cast<uint16_t*>(p.out) + (int64_t)(token0 + t) * p.out_stride + row0 + at;
      if (p.wide_out && row0 + at + 8 <= p.n) {
        *reinterpret_cast<uint4*>(to) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (row0 + at + e < p.n) to[e] = (uint16_t)(e & 1 ? w[e / 2] >> 16 : w[e / 2]);
      }
    }
  } else {
    cluster_sync();
    // the sums in the parts' order, a thread four tokens of a row
    const float4* parts = reinterpret_cast<const float4*>(smem);
    for (int mine = 0; mine * p.parts + rank < kGroups; ++mine) {
      const int row = row0 + (mine * p.parts + rank) * 32 + lane;
      const float bias = bias_of(p.bias, min(row, p.n - 1), p.bf16);
      for (int four = warp; four * 4 < tokens; four += kCta / 32) {
        float4 v = parts[(mine * (p.tile / 4) + four) * 32 + lane];
        for (int r = 1; r < p.parts; ++r) {
          const float4 x = parts[((r * own_groups + mine) * (p.tile / 4) + four) * 32 + lane];
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
        const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row < p.n && four * 4 + e < tokens)
            put(p.out, (int64_t)(token0 + four * 4 + e) * p.out_stride + row, y[e] + bias, p.bf16);
      }
    }
  }
  __syncthreads();
  fence_after();
  dependents_launch();
  if (warp == kUnpackWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(p.columns) : "memory");
}

std::mutex g_mu;
bool g_set[64][2];
constexpr int kSmemMost = 220 * 1024;
constexpr int kSmemBeside = 111 * 1024;       // less than half of an SM's
constexpr int kSmemBesideLeast = 78 * 1024;  // more than a third of it
constexpr int kSmemAlone = 150 * 1024;        // more than what is left beside one of those
static_assert(3 * kSmemBesideLeast >= 228 * 1024 && kSmemAlone + kSmemBesideLeast >= 228 * 1024, "columns for all CTAs of an SM");

// The driver's call that makes a tensor map, by its name: the library is not linked against it.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 found = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return found;
}

// How many clusters of each size the device runs at once, with a CTA on each of their SMs; asked once.
int g_fit[64][kMaxParts + 1];
const int* clusters_that_fit(int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  int* fit = g_fit[dev];
  if (fit[0] != 0) return fit;
  if (lt::take_injected_failure()) return fit;  // (by a test: the device is asked again by the next call)
  const void* func = reinterpret_cast<const void*>(&many_kernel<2>);
  int sms = 0;
  if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fit;  // (no cluster fits: the launch will say why)
  fit[1] = sms;
  for (int parts = 2; parts <= kMaxParts; ++parts) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(parts * sms));
    cfg.blockDim = dim3(Many<2>::kCta);
    cfg.dynamicSmemBytes = kSmemMost;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)parts, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&fit[parts], func, &cfg) != cudaSuccess) fit[parts] = 0;
  }
  fit[0] = 1;
  return fit;
}

}  // namespace

namespace lt {
namespace w4 {

lt_status map_rows(CUtensorMap* map, const void* at, int64_t n, int64_t bytes, int wide, int rows) {
  const auto encode = encoder();
  if (encode == nullptr) return LT_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)n}, strides[1] = {(cuuint64_t)bytes};
  const cuuint32_t box[2] = {(cuuint32_t)wide, (cuuint32_t)rows}, steps[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(at), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE,
                wide == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                : wide == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                             : CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? LT_OK
             : LT_ERR_CUDA;
}

ManyPlan many_plan(int dev, int64_t tokens, int64_t n, int64_t k) {
  const int* fit = clusters_that_fit(dev);
  ManyPlan best = {};
  double least = 0.0;
  const int64_t steps = (k + kManyStep - 1) / kManyStep, supers = (steps + 1) / 2;
  // One or two tiles of outputs a CTA alone on its SM, with all of tensor memory, or (last) one with half of it and another
  // CTA beside it.
  for (int kind = 0; kind < 3; ++kind) {
    const bool half = kind == 2;
    const int row_tiles = kind == 1 ? 2 : 1, columns = half ? 256 : 512, rows = row_tiles * 128;
    // sums and two steps' unpacked weights, at least, in the columns
    const int most = kind == 0 ? 256 : 128, room = (half ? kSmemBeside : kSmemMost) - 1024;
    const int64_t row_ctas = (n + rows - 1) / rows;
    const int64_t fewest = (tokens + most - 1) / most;
    for (int64_t tiles = fewest; tiles < fewest + 6 && tiles <= (tokens + 15) / 16; ++tiles) {
      ManyPlan a = {};
      a.row_tiles = row_tiles;
      a.columns = columns;
      a.tile = (int)((tokens + tiles - 1) / tiles + 15) / 16 * 16;
      a.tiles = (int)((tokens + a.tile - 1) / a.tile);
      // four places for tokens (two, with half the room), then as many for codes as there is room (they are asked for while the
      // tokens are still laid out), the rest for tokens
      a.code_ring = (room - (half ? 2 : 4) * a.tile * 256) / (rows * 128);
      a.code_ring = a.code_ring > 6 ? 6 : a.code_ring < 2 ? 2 : a.code_ring;
      if (half && a.code_ring > 3) a.code_ring = 3;
      a.token_ring = (room - a.code_ring * rows * 128) / (a.tile * 256);
      if (a.token_ring > kMaxRing) a.token_ring = kMaxRing;
      a.sum_columns = (a.tile + 31) / 32 * 32;
      a.row_ring = (columns - row_tiles * a.sum_columns) / (row_tiles * 64);
      if (a.row_ring > kMaxRing) a.row_ring = kMaxRing;
      a.smem = a.code_ring * rows * 128 + a.token_ring * a.tile * 256;
      // Neither more CTAs an SM than that, ever, whatever the sizes, and also where calls of both kinds run at once: each
      // finds its columns of tensor memory free. One that waited for them while its cluster waits for it could be waited
      // for in turn by the cluster that holds them. (A CTA without a cluster may wait, or be waited for: it ends.)
      const int least_smem = half ? kSmemBesideLeast : kSmemAlone;
      if (a.smem < least_smem) a.smem = least_smem;
      for (int parts = 1; parts <= kMaxParts && (parts == 1 || supers >= parts * 2); ++parts) {
        if (fit[parts] < 1) break;
        if (parts > 1 && (rows / 32 + parts - 1) / parts * parts * a.tile * 128 > a.smem) continue;
        // Clocks, as measured: a step's products, unpacking, bytes from memory (all CTAs') and from the L2 cache, whichever is
        // longest; a CTA's start, and its end, longer with a join. Two CTAs beside each other have a step each in the
        // time that their SM takes for both, and hide each other's start and end.
        const int64_t clusters = row_ctas * a.tiles;
        const auto round = [&](int64_t at_once, int beside) {
          const double from_memory = (double)at_once * parts * rows * 72.0 / a.tiles / 2800.0;
          const double products = (row_tiles == 1 ? 4.6 : 10.7) * a.tile;
          const double unpacking = row_tiles == 1 ? 560.0 : 700.0, from_cache = (a.tile * 256.0 + rows * 72.0) / 64.0;
          const double step = beside == 2 ? fmax(fmax(8.6 * a.tile, 720.0), fmax(from_memory, 2.0 * from_cache))
                                          : fmax(fmax(products, unpacking), fmax(from_memory, from_cache));
          return (double)((supers + parts - 1) / parts) * 2 * step + 3000.0 + 18.0 * a.tile * row_tiles +
                 (parts > 1 ? 4000.0 + 400.0 * parts : 500.0);
        };
        double time;
        if (half) {
          const int64_t pairs = clusters / (2 * fit[parts]), left = clusters % (2 * fit[parts]);
          time = (double)pairs * round(2 * fit[parts], 2) + (left == 0 ? 0.0 : round(left, pairs == 0 && left <= fit[parts] ? 1 : 2));
        } else {
          const int64_t waves = (clusters + fit[parts] - 1) / fit[parts];
          time = (double)waves * round(clusters < fit[parts] ? clusters : fit[parts], 1);
        }
        if (best.tile == 0 || time < least) {
          least = time;
          best = a;
          best.parts = parts;
        }
      }
    }
  }
  best.smem += 1024;
  best.steps = steps;
  best.x_bytes = (int64_t)best.tiles * best.tile * steps * 256;
  best.bytes = best.x_bytes + (int64_t)best.tiles * best.tile * 4;
  return best;
}

lt_status launch_many(int dev, ManyParams* p, const ManyPlan& plan, void* stream) {
  const bool two = plan.row_tiles == 2;
  const void* func = two ? reinterpret_cast<const void*>(&many_kernel<2>) : reinterpret_cast<const void*>(&many_kernel<1>);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_set[dev][two]) {
      if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess) return LT_ERR_CUDA;
      g_set[dev][two] = true;
    }
  }
  p->tile = plan.tile;
  p->parts = plan.parts;
  p->steps = (int32_t)plan.steps;
  p->code_ring = plan.code_ring;
  p->token_ring = plan.token_ring;
  p->row_ring = plan.row_ring;
  p->sum_columns = plan.sum_columns;
  p->rows_column = plan.row_tiles * plan.sum_columns;
  p->columns = plan.columns;
  p->wide_scales = p->k % 256 == 0;
  p->wide_out = reinterpret_cast<uintptr_t>(p->out) % 16 == 0 && p->out_stride % 8 == 0;
  CUtensorMap map;
  lt_status st = map_rows(&map, p->codes, p->n, p->k / 2, 64, plan.row_tiles * 128);
  if (st != LT_OK) return st;
  st = kv4::launch(reinterpret_cast<const void*>(&layout_kernel), dim3((unsigned)p->tokens), kLayoutThreads, 0, p, stream);
  if (st != LT_OK) return st;
  if (take_injected_failure()) return LT_ERR_CUDA;
  const int64_t rows = ((int64_t)p->n + plan.row_tiles * 128 - 1) / (plan.row_tiles * 128);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * plan.parts), (unsigned)plan.tiles);
  cfg.blockDim = dim3(two ? Many<2>::kCta : Many<1>::kCta);
  cfg.dynamicSmemBytes = (unsigned)plan.smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim = {(unsigned)plan.parts, 1, 1};
  cfg.attrs = attrs;
  cfg.numAttrs = plan.parts > 1 ? 2 : 1;
  void* args[] = {p, &map};
  return cudaLaunchKernelExC(&cfg, func, args) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

}  // namespace w4
}  // namespace lt
