// lt_w4_many.cu -- products with 4-bit weights for many tokens: tcgen05, the sums in tensor memory.
//
// A CTA takes 128 outputs and a tile of up to 256 tokens; the weights are the product's 128 rows, the tokens its
// columns, so a tile of few tokens wastes nothing. In steps of 64 inputs,
//   warps 0 to 7  unpack the step's weights: a thread a group of 32 of one output, codes times scale in fp16, written with the
//                 128-byte swizzle that the tensor core reads; its codes come straight from memory, four steps ahead
//   warp 8        issues the products
//   warp 9        brings the step's tokens, one bulk copy
// The tokens are laid out for that by a launch before: fp16, scaled by a power of two for each token (bf16's
// range does not fit), swizzled, a step's tile contiguous. Where there are few outputs a cluster cuts the inputs, and its
// parts join over distributed shared memory in one order.

#include <mutex>

#include "lt_kv4_tcgen05.cuh"
#include "lt_w4_linear.h"

namespace {

using namespace lt::kv4;
using namespace lt::w4;

// A CTA has one or two tiles of 128 outputs, two threads an output that unpack.
template <int kTiles>
struct Many {
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kUnpackers = 2 * kRows;
  static constexpr int kCta = kUnpackers + 64;
  static constexpr int kWeights = kRows * 128;  // bytes of a step's unpacked weights
};
constexpr int kMaxStages = 8;
constexpr int kAhead = 6;  // steps whose codes a thread has asked for

struct Shared {
  uint64_t tokens_full[kMaxStages], weights_full[kMaxStages], empty[kMaxStages];
  uint64_t done;
  uint32_t tmem;
  int gave_up;
};

// A warp waits for a phase, kWaitPolls polls at most; a wait that gives up marks the CTA, whose outputs are NaN
// then, and the warp goes on: the roles keep their steps, so nobody waits for one that has left.
__device__ __forceinline__ bool ready(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(lt::smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ void wait_warp(uint64_t* bar, uint32_t parity, Shared* sh) {
  bool done = ready(bar, parity);
  if (__all_sync(~0u, done)) return;
#pragma unroll 1
  for (uint32_t i = 0; i < lt::kWaitPolls; ++i) {
    done = done | lt::mbar_try_wait(bar, parity);
    if (__all_sync(~0u, done)) return;
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
  const int pieces = p.blocks * 8, there = p.k / 8;
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
  uint8_t* to = p.tiles_at + ((int64_t)(token / p.tile) * p.blocks * p.tile + token % p.tile) * 128;
  auto write = [&](int q, const uint4& v) {
    *reinterpret_cast<uint4*>(to + (int64_t)(q / 8) * p.tile * 128 + (((q & 7) ^ (token % p.tile & 7)) << 4)) = p.bf16 ? to_half(v, mul) : v;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kLayoutThreads < pieces) write(tid + i * kLayoutThreads, held[i]);
  for (int q = tid + kHeld * kLayoutThreads; q < pieces; q += kLayoutThreads)
    write(q, q < there ? __ldg(x + q) : make_uint4(0u, 0u, 0u, 0u));
}

__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack_role(const ManyParams& p, Shared* sh, uint32_t ring, uint32_t stage_bytes, int row0, int from, int to) {
  const int tid = threadIdx.x, lane = tid & 31, row = tid / 2, half = tid & 1;
  const int64_t of = min(row0 + row, p.n - 1);
  const int groups = p.k / 32;
  const uint8_t* codes = p.codes + of * (p.k / 2) + half * 16;
  const uint16_t* scales = p.scales + of * groups + half;
  uint32_t piece[4];  // where the group's four 16-byte pieces of fp16 lie
#pragma unroll
  for (int j = 0; j < 4; ++j) piece[j] = ring + row * 128 + (((half * 4 + j) ^ (row & 7)) << 4);
  uint4 code[kAhead];
  uint32_t scale[kAhead];
  auto fetch = [&](int i, int b) {
    code[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0u;
    if (b < to && b * 2 + half < groups) {
      code[i] = load_codes(codes + (int64_t)b * 32);
      scale[i] = __ldg(scales + b * 2);
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i, from + i);
  int stage = 0;
  uint32_t parity = 1;  // (the first round's stages are free)
#pragma unroll 1
  for (int b0 = from; b0 < to; b0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (b0 + i >= to) break;
      const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w}, s = __byte_perm(scale[i], 0, 0x1010);
      fetch(i, b0 + i + kAhead);
      wait_warp(&sh->empty[stage], parity, sh);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h[4];
        codes_to_half2(w[j], h);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                     :: "r"(piece[j] + stage * stage_bytes), "r"(hmul2(h[0], s)), "r"(hmul2(h[1], s)), "r"(hmul2(h[2], s)),
                        "r"(hmul2(h[3], s)) : "memory");
      }
      fence_async();
      __syncwarp();
      if (lane == 0) arrive(&sh->weights_full[stage]);
      if (++stage == p.stages) {
        stage = 0;
        parity ^= 1u;
      }
    }
  }
}

template <int kTiles>
__global__ void __launch_bounds__(Many<kTiles>::kCta) many_kernel(ManyParams p) {
  constexpr int kRows = Many<kTiles>::kRows, kCta = Many<kTiles>::kCta, kWeights = Many<kTiles>::kWeights;
  constexpr int kUnpackWarps = Many<kTiles>::kUnpackers / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (lt::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ Shared shared;
  Shared* sh = &shared;
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;
  const uint32_t ring = lt::smem_u32(smem), stage_bytes = kWeights + p.tile * 128;
  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      lt::mbar_init(&sh->tokens_full[s], 1);
      lt::mbar_init(&sh->weights_full[s], kUnpackWarps);
      lt::mbar_init(&sh->empty[s], 1);
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
  const int from = (int)((int64_t)p.blocks * rank / p.parts), to = (int)((int64_t)p.blocks * (rank + 1) / p.parts);
  const uint32_t tmem = sh->tmem;

  if (warp < kUnpackWarps) {
    unpack_role(p, sh, ring, stage_bytes, row0, from, to);
  } else if (warp == kUnpackWarps) {
    const uint32_t lead = elect_one(), idesc = instruction(p.tile, false), d = __shfl_sync(~0u, tmem, 0);
    int stage = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (int b = from; b < to; ++b) {
      wait_warp(&sh->tokens_full[stage], parity, sh);
      wait_warp(&sh->weights_full[stage], parity, sh);
      fence_after();
      const uint32_t at = ring + stage * stage_bytes;
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
        mma_ss4(d + m * (p.columns / kTiles), desc_k_major(at + m * (128 * 128)), desc_k_major(at + kWeights), idesc, b > from, lead);
      mma_commit(&sh->empty[stage], lead);
      if (++stage == p.stages) {
        stage = 0;
        parity ^= 1u;
      }
    }
    mma_commit(&sh->done, lead);
  } else {
    dependency_wait();  // the launch that lays the tokens out
    const uint8_t* src = p.tiles_at + (int64_t)blockIdx.y * p.blocks * p.tile * 128;
    const uint32_t bytes = p.tile * 128;
    int stage = 0;
    uint32_t parity = 1;
#pragma unroll 1
    for (int b = from; b < to; ++b) {
      wait_warp(&sh->empty[stage], parity, sh);
      if (lane == 0) {
        lt::mbar_arrive_tx(&sh->tokens_full[stage], bytes);
        lt::bulk_g2s(smem + stage * stage_bytes + kWeights, src + (int64_t)b * bytes, bytes, &sh->tokens_full[stage]);
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        parity ^= 1u;
      }
    }
    // nothing is on its way any more, also where the products' warp gave up
    const int last = min(to - from, p.stages);
    for (int i = 0; i < last; ++i) {
      const int nth = to - from - last + i;
      wait_warp(&sh->tokens_full[nth % p.stages], nth / p.stages & 1, sh);
    }
  }
  __syncwarp();
  wait_warp(&sh->done, 0, sh);  // every product is done: the sums are there, and the ring is free
  fence_after();
  __syncthreads();
  const bool bad = *(volatile int*)&sh->gave_up != 0;

  // a thread a row, 16 tokens at a time; two sets of four warps take turns with a tile's
  float* joined = reinterpret_cast<float*>(smem);  // [token][row]
  dependency_wait();
  if (warp < kUnpackWarps) {
    const int tile = warp >> 3, row = tile * 128 + (warp & 3) * 32 + lane;
    const uint32_t at = tmem + tile * (p.columns / kTiles) + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int c = (warp >> 2 & 1) * 16; c < tokens; c += 32) {
      uint32_t y[16];
      tmem_read16(at + c, y);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (c + e >= tokens) break;
        const float v = bad ? NAN : __uint_as_float(y[e]) * p.inverse[token0 + c + e];
        if (p.parts > 1)
          joined[(c + e) * kRows + row] = v;
        else if (row0 + row < p.n)
          put(p.out, (int64_t)(token0 + c + e) * p.out_stride + row0 + row, v, p.bias, row0 + row, p.bf16);
      }
      __syncwarp();
    }
  }
  fence_before();
  if (p.parts > 1) {
    cluster_sync();
    const uint32_t joined_at = lt::smem_u32(joined);
    for (int u = rank * kCta + tid; u < tokens * kRows; u += p.parts * kCta) {
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < kMaxParts; ++r)
        if (r < p.parts) v += peer_f32(joined_at + u * 4, r);
      const int row = row0 + u % kRows;
      if (row < p.n) put(p.out, (int64_t)(token0 + u / kRows) * p.out_stride + row, v, p.bias, row, p.bf16);
    }
    cluster_sync();  // (a CTA's shared memory stays until its peers have read it)
  } else {
    __syncthreads();
  }
  fence_after();
  dependents_launch();
  if (warp == kUnpackWarps) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(p.columns) : "memory");
}

std::mutex g_mu;
bool g_set[64][2];
constexpr int kSmemMost = 220 * 1024;

}  // namespace

namespace lt {
namespace w4 {

ManyPlan many_plan(int sms, int64_t tokens, int64_t n, int64_t k) {
  ManyPlan a = {};
  a.tiles = (int)((tokens + 255) / 256);
  a.tile = (int)((tokens + a.tiles - 1) / a.tiles + 15) / 16 * 16;
  a.tiles = (int)((tokens + a.tile - 1) / a.tile);
  a.blocks = (k + kBlock - 1) / kBlock;
  a.row_tiles = 2;
  const int stage = a.row_tiles * 128 * 128 + a.tile * 128;
  a.stages = (kSmemMost - 2048) / stage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int64_t ctas = (n + a.row_tiles * 128 - 1) / (a.row_tiles * 128) * a.tiles;
  a.parts = 1;
  while (a.parts < kMaxParts && ctas * (a.parts + 1) <= sms && a.blocks >= (a.parts + 1) * 4) ++a.parts;
  a.smem = a.stages * stage;
  const int join = a.tile * a.row_tiles * 128 * 4;
  if (a.parts > 1 && join > a.smem) a.parts = 1;
  a.smem += 1024;
  a.x_bytes = (int64_t)a.tiles * a.tile * a.blocks * 128;
  a.bytes = a.x_bytes + (int64_t)a.tiles * a.tile * 4;
  return a;
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
  p->stages = plan.stages;
  p->blocks = (int32_t)plan.blocks;
  p->columns = 32;
  while (p->columns < plan.tile) p->columns *= 2;
  p->columns *= plan.row_tiles;
  const lt_status st = kv4::launch(reinterpret_cast<const void*>(&layout_kernel), dim3((unsigned)p->tokens), kLayoutThreads, 0, p, stream);
  if (st != LT_OK) return st;
  const int64_t rows = ((int64_t)p->n + plan.row_tiles * 128 - 1) / (plan.row_tiles * 128);
  return kv4::launch(func, dim3((unsigned)(rows * plan.parts), (unsigned)plan.tiles), two ? Many<2>::kCta : Many<1>::kCta,
                     (unsigned)plan.smem, p, stream, plan.parts);
}

}  // namespace w4
}  // namespace lt
