// lt_w4_linear.cu -- products with 4-bit weights (lt_w4_linear) for few tokens, and the
// weights' quantisation (lt_w4_quantise).
//
// Few tokens: the weights are read once and that is the time, so what counts is the work per weight: unpacking,
// scaling, feeding the tensor core. The weights are the 16-row operand straight from registers (m16n8k16,
// fp32 sums), the tokens the eight columns. The order of the inputs within a product is free, so a lane
// takes 16 bytes of codes, a whole group of 32 inputs, of rows g and g + 8: one scale a row, and the
// tokens' fragments are 16 bytes of the same inputs from shared memory. (tcgen05 would want the unpacked
// weights in tensor memory: that is the kernel for many tokens, slower up to two of them.)
//
// Each warp has a ring of its own, of 256 inputs of 16 rows (their codes by a tensor map, their scales by
// another), and asks for the next ones itself. A CTA's eight warps are 1, 2 or 4 row tiles by 8, 4 or 2 parts of the
// inputs; it stays and walks over row blocks with the tokens in shared memory. A cluster cuts the inputs
// further where there are few rows. The parts join in shared memory and over distributed shared memory, in one order
// whatever the timing.
//
// What bounds it: issue and the ALU pipe (67% and 53% of their rates): 16 rows by 128 inputs take some 195 warp
// instructions, 64 of them conversions and scalings. One token through 8192 x 28672 (132 MB): 29 us, 4.5 TB/s, where
// the copy rate allows 19.5. On the way: a CTA for each row block 40 us; CTAs that stay 34; scales of two groups a load
// 33; tensor maps and rings of two stages 30 (with three stages, and a CTA less an SM, 33); fewer steps a join 28 to
// 29. Through 4096 x 4096: 10.0, 6.4, 6.1, 6.0, 6.4 us, most of it the way from launch to
// first weights and the join.

#include <mutex>

#include "lt_async.cuh"
#include "lt_kv4_quantise.cuh"
#include "lt_w4_linear.h"

namespace {

using namespace lt::kv4;
using namespace lt::w4;

constexpr int kStep = 256;  // inputs of a stage
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct LinearParams {
  const void* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const void* bias;
  void* out;
  int64_t x_stride, out_stride;
  int32_t n, k, tokens;
  int32_t row_warps;   // row tiles of a CTA: 1, 2 or 4
  int32_t parts;       // CTAs of a cluster, along the inputs
  int32_t chunk;       // steps whose inputs are in shared memory at a time
  int32_t join_at;     // where the warps' sums are joined, behind the inputs
  int32_t bf16, wide_scales;
  uint32_t stage_bytes, zero;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tensor_in(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(lt::smem_u32(bar)) : "memory");
}
// A warp waits for a phase, a bounded number of polls; false if it gave up. Every poll ends in a vote, so the warp goes
// on converged.
__device__ __forceinline__ bool wait_polls(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(lt::smem_u32(bar)), "r"(parity) : "memory");
  bool done = ok != 0;
  if (__all_sync(~0u, done)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < lt::kWaitPolls; ++i) {
    done = done | lt::mbar_try_wait(bar, parity);
    if (__all_sync(~0u, done)) return true;
  }
  return false;
}

// Where 16-byte piece q of token t lies: pieces of a step (16) by lane group and word, the upper eight's turned
// by one, tokens 32 bytes apart beyond whole 128-byte lines, so that the eight lanes (two tokens, four groups)
// that read 16 bytes together have all banks.
__device__ __forceinline__ int piece_at(int t, int q, int pitch) { return t * pitch + ((q ^ (q >> 3 & 1)) << 4); }

constexpr int kPerSm = 3;   // CTAs
constexpr int kTokens = 8;  // at most: the product's columns
constexpr int kStages = 2;
constexpr int kStageCodes = 16 * 128, kStageBytes = kStageCodes + 1024;  // 256 inputs of 16 rows; scales behind them
constexpr int kRing = kWarps * kStages * kStageBytes;

__global__ void __launch_bounds__(kThreads, kPerSm)
few_kernel(LinearParams p, const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap scales) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (lt::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ uint32_t largest[kTokens];
  __shared__ int gave_up;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int row_shift = p.row_warps >> 1, k_shift = 3 - row_shift;  // (1, 2 or 4 row tiles)
  const int k_warps = kWarps >> row_shift, wr = warp & (p.row_warps - 1), wk = warp >> row_shift;
  const int rank = blockIdx.x % p.parts;
  const int rows = p.row_warps * 16;
  const int tokens = p.tokens;
  const int steps = (p.k + kStep - 1) / kStep, groups = p.k / 32;
  // the CTA's steps of 256 inputs, in chunks whose inputs fit into shared memory; its row blocks are every so many
  const int s_begin = (int)((int64_t)steps * rank / p.parts), s_end = (int)((int64_t)steps * (rank + 1) / p.parts);
  const int chunks = (s_end - s_begin + p.chunk - 1) / p.chunk;
  const int blocks = (p.n + rows - 1) / rows, first = blockIdx.x / p.parts, every = gridDim.x / p.parts;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) lt::mbar_init(&bars[warp][s], 1);
    lt::mbar_fence_init();
  }
  if (tid < kTokens) largest[tid] = 0u;
  if (tid == 0) gave_up = 0;
  dependency_wait();
  __syncthreads();

  // the warp's steps of a chunk
  auto range = [&](int chunk, int* from, int* to) {
    const int c0 = s_begin + chunk * p.chunk, wide = min(p.chunk, s_end - c0);
    *from = c0 + (wide * wk >> k_shift);
    *to = c0 + (wide * (wk + 1) >> k_shift);
  };

  uint8_t* ring = smem + warp * kStages * kStageBytes;
  // What is brought next runs ahead over chunks and row blocks. (Every warp has steps in the first chunk, or none at all.)
  int from0, to0;
  range(0, &from0, &to0);
  int next_chunk = 0, next_s = from0, next_to = to0, next_row = first * rows + wr * 16;
  const int end_row = from0 < to0 ? blocks * rows : 0;
  auto bring = [&](int stage, uint32_t zero) {  // (the whole warp's numbers; lane 0 asks)
    if (next_row >= end_row) return;
    if (lane == 0) {
      uint64_t* bar = &bars[warp][stage];
      const uint32_t at = lt::smem_u32(ring) + stage * kStageBytes + zero;
      lt::mbar_arrive_tx(bar, p.stage_bytes);
      tensor_in(at, &codes, next_s * 128, next_row, bar);
      if (p.wide_scales) tensor_in(at + kStageCodes, &scales, next_s * 16, next_row, bar);
    }
    if (++next_s < next_to) return;
    if (chunks == 1) {
      next_s = from0;
      next_row += every * rows;
      return;
    }
    do {
      if (++next_chunk == chunks) {
        next_chunk = 0;
        next_row += every * rows;
      }
      range(next_chunk, &next_s, &next_to);
    } while (next_s >= next_to);
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) bring(s, 0);

  uint8_t* inputs = smem + kRing;
  const int pitch = p.chunk * kStep * 2 + 32;
  // A chunk's inputs into shared memory; past the last input, zeros. A thread asks for four pieces at a time, of up to four
  // tokens.
  const int side = tokens == 1 ? 0 : tokens == 2 ? 1 : 2;  // log 2 of the tokens beside each other
  auto stage_inputs = [&](int chunk) {
    const int c0 = s_begin + chunk * p.chunk, pieces = min(p.chunk, s_end - c0) * (kStep / 8);
    const int there = min((int64_t)pieces, (int64_t)(p.k / 8) - (int64_t)c0 * (kStep / 8));
#pragma unroll 1
    for (int t0 = 0; t0 < tokens; t0 += 4) {
      const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)t0 * p.x_stride + (int64_t)c0 * kStep;
      uint32_t big[4] = {};
#pragma unroll 1
      for (int q = tid; q < pieces; q += kThreads * 4 >> side) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = i & ((1 << side) - 1), at = q + (i >> side) * kThreads;
          v[i] = make_uint4(0u, 0u, 0u, 0u);
          if (at < there && t0 + t < tokens) v[i] = __ldg(reinterpret_cast<const uint4*>(x + t * p.x_stride) + at);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = i & ((1 << side) - 1), at = q + (i >> side) * kThreads;
          if (at < pieces && t0 + t < tokens) {
            *reinterpret_cast<uint4*>(inputs + piece_at(t0 + t, at, pitch)) = v[i];
            big[i] = max(big[i], largest_of(v[i]));
          }
        }
      }
      if (p.bf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + (i & ((1 << side) - 1));
          big[i] = __reduce_max_sync(~0u, big[i]);
          if (lane == 0 && t < tokens) atomicMax(&largest[t], big[i]);
        }
      }
    }
    __syncthreads();
    if (!p.bf16) return;
#pragma unroll 1
    for (int t = 0; t < tokens; ++t) {
      const float mul = token_power(largest[t]);
#pragma unroll 4
      for (int q = tid; q < pieces; q += kThreads) {
        uint4* at = reinterpret_cast<uint4*>(inputs + piece_at(t, q, pitch));
        *at = to_half(*at, mul);
      }
    }
    __syncthreads();
  };
  float acc[4];
  float power[2] = {1.0f, 1.0f}, inverse[2] = {1.0f, 1.0f};  // of tokens 2c and 2c + 1, whose sums a lane has
  auto powers = [&](bool more) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float now = token_power(largest[min(2 * c + e, tokens - 1)]);
      if (more) {
        // sums so far go over to the new power, which is the largest input's so far and never grows
        const float f = fmaxf(now / power[e], 0x1p-126f);  // (not 0: an infinity stays one)
        acc[e] *= f;
        acc[e + 2] *= f;
      }
      power[e] = now;
      inverse[e] = 1.0f / now;
    }
  };
  if (chunks == 1) {
    stage_inputs(0);
    if (p.bf16) powers(false);
  }
  const uint8_t* xa = inputs + min(g, tokens - 1) * pitch + c * 64;  // the lane's token's inputs
  const int turned = 16 - (c >> 1) * 32;                            // from an even piece to its odd neighbour (see piece_at)
  xa += (c >> 1) * 16;
  // a row's 128 bytes of codes, its 16-byte pieces turned by the row; row g + 8 turns alike
  const uint8_t* lower = ring + g * 128 + ((c ^ g) << 4);
  const int upper = (((4 + c) ^ g) << 4) - ((c ^ g) << 4);
  const uint8_t* scale_at = ring + kStageCodes + g * 16 + c * 2;
  float* joined = reinterpret_cast<float*>(inputs + p.join_at);  // two times [k warp][token][row], in turn
  int place = 0, turns = 0;
  uint32_t parity = 0;
  bool ok = true;
  for (int block = first; block < blocks; block += every, turns ^= 1) {
    acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
    for (int chunk = 0; chunk < chunks; ++chunk) {
      if (chunks > 1) {
        __syncthreads();  // the last chunk's inputs have been read
        stage_inputs(chunk);
      }
      if (chunks > 1 && p.bf16) powers(chunk > 0);
      int from, to;
      range(chunk, &from, &to);
      if (!ok) to = from;
      const uint8_t* x = xa + (from - s_begin - chunk * p.chunk) * (kStep * 2);
#pragma unroll 1
      for (int s = from; s < to; ++s, x += kStep * 2) {
        ok = wait_polls(&bars[warp][place], parity);
        if (!ok) break;  // nothing more is asked for, and nothing waited for before the end
        const uint8_t* code = lower + place * kStageBytes;
        const uint8_t* scale = scale_at + place * kStageBytes;
        uint4 wa[2], wb[2];
        uint32_t ka[2], kb[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          wa[u] = *reinterpret_cast<const uint4*>(code);
          wb[u] = *reinterpret_cast<const uint4*>(code + 1024);
          code += upper;
          if (p.wide_scales) {
            ka[u] = *reinterpret_cast<const uint16_t*>(scale + u * 8);
            kb[u] = *reinterpret_cast<const uint16_t*>(scale + u * 8 + 128);
          } else {
            // (codes past the last input are zeros)
            const int group = min(s * 8 + u * 4 + c, groups - 1), ra = block * rows + wr * 16 + g;
            ka[u] = __ldg(p.scales + (int64_t)min(ra, p.n - 1) * groups + group);
            kb[u] = __ldg(p.scales + (int64_t)min(ra + 8, p.n - 1) * groups + group);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t sa = __byte_perm(ka[u], 0, 0x1010), sb = __byte_perm(kb[u], 0, 0x1010);
          const uint32_t ca[4] = {wa[u].x, wa[u].y, wa[u].z, wa[u].w}, cb[4] = {wb[u].x, wb[u].y, wb[u].z, wb[u].w};
          const uint8_t* odd = x + turned;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t ha[4], hb[4];
            codes_to_half2(ca[j], ha);
            codes_to_half2(cb[j], hb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ha[i] = hmul2(ha[i], sa);
              hb[i] = hmul2(hb[i], sb);
            }
            const uint4 b = *reinterpret_cast<const uint4*>((j & 1 ? odd : x) + u * 256 + (j >> 1) * 32);
            mma16816(acc, ha[0], hb[0], ha[1], hb[1], b.x, b.y);
            mma16816(acc, ha[2], hb[2], ha[3], hb[3], b.z, b.w);
          }
          if (u == 0) {  // (at the start of the step the wait for all loads costs 3%)
            bring(place, zero_of(wa[0].x ^ wa[1].x ^ wb[0].x ^ wb[1].x ^ ka[0] ^ ka[1] ^ kb[0] ^ kb[1], p.zero));
            if (++place == kStages) {
              place = 0;
              parity ^= 1u;
            }
          }
        }
      }
    }
    if (!ok && lane == 0) atomicExch(&gave_up, 1);
    // join the warps, and with a cluster its CTAs
    float* mine = joined + turns * (kWarps * 16 * tokens);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int token = 2 * c + (e & 1), row = wr * 16 + g + (e >> 1) * 8;
      if (token < tokens) mine[(wk * tokens + token) * rows + row] = acc[e] * inverse[e & 1];
    }
    __syncthreads();
    const int all = tokens * rows;
    if (p.parts > 1) {
      for (int u = tid; u < all; u += kThreads) {
        float y = mine[u];
        for (int w = 1; w < k_warps; ++w) y += mine[w * all + u];
        mine[u] = gave_up ? NAN : y;
      }
      cluster_sync();
    }
    for (int u = rank * kThreads + tid; u < all; u += p.parts * kThreads) {
      const int token = u >> (4 + row_shift), row = block * rows + (u & (rows - 1));
      float y = 0.0f;
      if (p.parts > 1) {
#pragma unroll
        for (int r = 0; r < kMaxParts; ++r)
          if (r < p.parts) y += peer_f32(lt::smem_u32(mine) + u * 4, r);
      } else {
        float part[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) part[w] = w < k_warps ? mine[w * all + u] : 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) y += part[w];
        if (gave_up) y = NAN;  // (a wait ran out)
      }
      if (row < p.n) put(p.out, (int64_t)token * p.out_stride + row, y + bias_of(p.bias, row, p.bf16), p.bf16);
    }
    if (p.parts > 1) cluster_sync();  // (a CTA's shared memory stays until its peers have read it)
  }
  if (!ok) {
    // the copies that are still on their way: the one that was waited for and the next, if it was asked for
#pragma unroll 1
    for (int s = 0; s < kStages; ++s) {
      wait_polls(&bars[warp][place], parity);
      if (++place == kStages) {
        place = 0;
        parity ^= 1u;
      }
    }
  }
  dependents_launch();
}

// ---- quantisation: a thread eight inputs, four lanes a group

struct QuantiseParams {
  const void* w;
  uint8_t* codes;
  uint16_t* scales;
  int64_t n, k, stride;
};

template <class S>
__global__ void __launch_bounds__(kThreads) quantise_kernel(QuantiseParams p, bool wide) {
  dependency_wait();
  const int64_t pieces = p.k / 8, whole = (pieces + 31) / 32 * 32;
  for (int64_t row = blockIdx.x; row < p.n; row += gridDim.x) {
    const S* w = static_cast<const S*>(p.w) + row * p.stride;
    for (int64_t q = threadIdx.x + (int64_t)blockIdx.y * kThreads; q < whole; q += (int64_t)gridDim.y * kThreads) {
      Eight<S> x;
      x.clear();
      if (q < pieces) x.load(w + q * 8, wide);
      uint32_t largest = x.largest();
      largest = max(largest, __shfl_xor_sync(~0u, largest, 1));
      largest = max(largest, __shfl_xor_sync(~0u, largest, 2));
      if (q < pieces) {
        const bool bad = !Eight<S>::finite(largest);
        const float s = bad ? 0.0f : Eight<S>::scale(Eight<S>::number(largest));
        reinterpret_cast<uint32_t*>(p.codes + row * (p.k / 2))[q] = bad ? 0u : x.codes(s);
        if ((q & 3) == 0) p.scales[row * (p.k / 32) + q / 4] = bad ? (uint16_t)0x7FFF : __half_as_ushort(__float2half_rn(s));
      }
    }
  }
  dependents_launch();
}

// ---- host side

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_set[kMaxDevices];

lt_status device_of(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return LT_ERR_CUDA;
  if (*dev < 0 || *dev >= kMaxDevices) return LT_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[*dev] == 0 && cudaDeviceGetAttribute(&g_sms[*dev], cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return LT_ERR_CUDA;
  *sms = g_sms[*dev];
  return LT_OK;
}

constexpr int kFewInputs = 96 * 1024;  // bytes of inputs in shared memory at most
constexpr int kFewJoin = 2 * kWarps * 16 * kTokens * 4;  // at most
constexpr int kFewSmem = 1024 + kRing + kFewInputs + kFewJoin;

// Whether a call takes the kernel for few tokens. us there and in the one for many, in a graph:
//   n x k                1 token     2           3           4           6           8
//   64 x 512      bf16   3.2, 4.7    3.4, 4.5    3.6, 4.6    3.8, 4.6    4.9, 4.6    5.4, 4.6
//                 fp16   2.7, 4.6    2.8, 4.5    2.8, 4.6    2.8, 4.6    3.5, 4.6    3.6, 4.6
//   4096 x 4096   bf16   6.7, 8.4    7.3, 8.5    8.1, 8.5    8.5, 8.5    9.5, 8.5    10.0, 8.6
//                 fp16   6.0, 8.4    6.3, 8.4    7.1, 8.4    7.3, 8.5    8.1, 8.5    8.3, 8.5
//   4099 x 5152   bf16   8.1, 10.1   9.0, 10.3   10.1, 10.3  10.4, 10.3  11.0, 10.4  11.5, 10.4
//                 fp16   7.3, 10.1   8.0, 10.2   9.1, 10.2   9.2, 10.3   9.5, 10.4   9.6, 10.4
//   14336 x 4096  bf16   11.9, 14.2  12.7, 14.6  14.6, 14.6  15.1, 14.6  16.6, 14.8  20.1, 14.7
//                 fp16   10.9, 14.3  11.4, 14.4  13.6, 14.6  13.7, 14.6  14.6, 14.6  17.9, 14.7
//   10240 x 8192  bf16   15.8, 17.3  17.7, 17.6  21.6, 17.7  24.9, 17.7  25.2, 17.8  30.2, 17.7
//                 fp16   14.7, 17.4  16.7, 17.6  20.3, 17.5  23.3, 17.4  23.3, 17.7  28.0, 17.7
//   28672 x 8192  bf16   30.8, 36.4  33.6, 36.5  33.8, 36.3  43.1, 36.5  39.8, 36.6  53.5, 36.5
//                 fp16   29.7, 36.2  32.4, 36.4  32.3, 36.4  41.6, 36.2  37.1, 36.4  51.3, 36.2
// Eagerly the second launch of the latter costs the host 6 more, so that this one is taken up to some 12 us, also where it is
// the slower in a graph: bf16 tokens from 5 on (4096 x 4096 with 8: 10.0 against 8.6). Past that the rule is coarse: it takes the
// slower side by 3% at 14336 x 4096 with 4 bf16 tokens and, the other way, by 7 and 12% at 28672 x 8192 with 3.
bool few(int64_t tokens, int64_t n, int64_t k) { return tokens <= 2 || (tokens <= 4 && n * k <= (int64_t)1 << 26) || (tokens <= 8 && n * k <= (int64_t)1 << 25); }

constexpr int64_t kMostSize = (int64_t)1 << 30;

lt_status check_sizes(int64_t tokens, int64_t n, int64_t k) {
  if (tokens < 0 || n < 0 || k < 0) return LT_ERR_INVALID_ARG;
  // (rows and inputs are 32-bit numbers, also those that a CTA would take next)
  if (k == 0 || k % 32 != 0 || k >= kMostSize || n >= kMostSize || tokens > 65535 * 8) return LT_ERR_UNSUPPORTED;
  return LT_OK;
}

}  // namespace

extern "C" {

lt_status lt_w4_quantise(const void* w, int32_t dtype, int64_t n, int64_t k, int64_t row_stride, void* codes, void* scales,
                         void* stream) {
  if (dtype != LT_DTYPE_F32 && dtype != LT_DTYPE_BF16 && dtype != LT_DTYPE_F16) return LT_ERR_INVALID_ARG;
  if (n > 0 && k > 0 && (w == nullptr || codes == nullptr || scales == nullptr)) return LT_ERR_INVALID_ARG;
  const uintptr_t size = dtype == LT_DTYPE_F32 ? 4 : 2;
  if (!aligned(w, size) || !aligned(codes, 16) || !aligned(scales, 16)) return LT_ERR_INVALID_ARG;
  const lt_status st = check_sizes(0, n, k);
  if (st != LT_OK) return st;
  if (n == 0) return LT_OK;
  QuantiseParams p = {w, static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales), n, k, row_stride};
  bool wide = aligned(w, 16) && (row_stride * (int64_t)size) % 16 == 0;
  const void* func = dtype == LT_DTYPE_F32    ? reinterpret_cast<const void*>(&quantise_kernel<float>)
                     : dtype == LT_DTYPE_BF16 ? reinterpret_cast<const void*>(&quantise_kernel<__nv_bfloat16>)
                                              : reinterpret_cast<const void*>(&quantise_kernel<__half>);
  if (lt::take_injected_failure()) return LT_ERR_CUDA;
  const int64_t across = (k / 8 + kThreads - 1) / kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n < 1 << 20 ? n : 1 << 20), (unsigned)(across < 64 ? across : 64));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* a[] = {&p, &wide};
  return cudaLaunchKernelExC(&cfg, func, a) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

lt_status lt_w4_workspace(int64_t tokens, int64_t n, int64_t k, int64_t* bytes) {
  if (bytes == nullptr) return LT_ERR_INVALID_ARG;
  const lt_status st = check_sizes(tokens, n, k);
  if (st != LT_OK) return st;
  *bytes = 0;
  if (few(tokens, n, k) || n == 0) return LT_OK;
  int dev = 0, sms = 0;
  const lt_status found = device_of(&dev, &sms);
  if (found != LT_OK) return found;
  const ManyPlan plan = many_plan(dev, tokens, n, k);
  if (plan.tile == 0) return LT_ERR_CUDA;  // (the device told nothing about itself)
  *bytes = plan.bytes;
  return LT_OK;
}

lt_status lt_w4_linear(const void* x, int32_t dtype, int64_t tokens, int64_t x_stride, const void* codes, const void* scales,
                       int64_t n, int64_t k, const void* bias, void* out, int64_t out_stride, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  if (dtype != LT_DTYPE_BF16 && dtype != LT_DTYPE_F16) return LT_ERR_INVALID_ARG;
  lt_status st = check_sizes(tokens, n, k);
  if (st == LT_ERR_INVALID_ARG) return st;
  if (tokens > 0 && n > 0) {
    if (x == nullptr || codes == nullptr || scales == nullptr || out == nullptr) return LT_ERR_INVALID_ARG;
    if (!aligned(x, 16) || x_stride % 8 || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 2) || !aligned(bias, 2))
      return LT_ERR_INVALID_ARG;
  }
  if (st != LT_OK) return st;
  if (tokens == 0 || n == 0) return LT_OK;
  int dev = 0, sms = 0;
  st = device_of(&dev, &sms);
  if (st != LT_OK) return st;
  if (!few(tokens, n, k)) {
    const ManyPlan plan = many_plan(dev, tokens, n, k);
    if (plan.tile == 0) return LT_ERR_CUDA;  // (the device told nothing about itself)
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < plan.bytes) return LT_ERR_INVALID_ARG;
    ManyParams m = {};
    m.x = x;
    m.codes = static_cast<const uint8_t*>(codes);
    m.scales = static_cast<const uint16_t*>(scales);
    m.bias = bias;
    m.out = out;
    m.tiles_at = static_cast<uint8_t*>(workspace);
    m.inverse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.x_bytes);
    m.x_stride = x_stride;
    m.out_stride = out_stride;
    m.n = (int32_t)n;
    m.k = (int32_t)k;
    m.tokens = (int32_t)tokens;
    m.bf16 = dtype == LT_DTYPE_BF16;
    return launch_many(dev, &m, plan, stream);
  }
  LinearParams p = {};
  p.x = x;
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = static_cast<const uint16_t*>(scales);
  p.bias = bias;
  p.out = out;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.n = (int32_t)n;
  p.k = (int32_t)k;
  p.tokens = (int32_t)tokens;
  p.bf16 = dtype == LT_DTYPE_BF16;
  const int here = (int)tokens;
  const int steps = (int)((k + kStep - 1) / kStep);
  const auto smem_of = [&](int chunk) { return 1024 + kRing + here * (chunk * kStep * 2 + 32 + 2 * kWarps * 16 * 4); };
  p.row_warps = here <= 2 ? 1 : here <= 4 ? 2 : 4;
  const int64_t row_blocks = (n + p.row_warps * 16 - 1) / (p.row_warps * 16);
  // as many steps' inputs in shared memory as fit; the inputs are cut over a cluster where the CTAs do not fill the SMs
  const int k_warps = kWarps / p.row_warps, most = (kFewInputs / here - 32) / (kStep * 2);
  int64_t per_sm = 0;
  for (p.parts = 1;; p.parts *= 2) {
    const int mine = (steps + p.parts - 1) / p.parts;
    p.chunk = mine < most ? mine : most / k_warps * k_warps;
    per_sm = (225 * 1024) / (smem_of(p.chunk) + 1024);
    if (per_sm > kPerSm) per_sm = kPerSm;
    if (p.parts == kMaxParts || steps < p.parts * 2 * k_warps) break;
    if (row_blocks * p.parts * 2 > per_sm * sms && mine <= most) break;
  }
  p.join_at = here * (p.chunk * kStep * 2 + 32);
  const int64_t resident = per_sm * sms / p.parts;
  const int64_t ctas = row_blocks < resident ? row_blocks : resident;
  p.wide_scales = k % 256 == 0;
  p.stage_bytes = kStageCodes + (p.wide_scales ? 256 : 0);
  CUtensorMap code_map, scale_map;
  st = map_rows(&code_map, codes, n, k / 2, 128, 16);
  if (st == LT_OK) st = p.wide_scales ? map_rows(&scale_map, scales, n, k / 16, 16, 16) : st;
  if (st != LT_OK) return st;
  if (!p.wide_scales) scale_map = code_map;  // (not used)
  const void* func = reinterpret_cast<const void*>(&few_kernel);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_set[dev]) {
      if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) != cudaSuccess) return LT_ERR_CUDA;
      g_set[dev] = true;
    }
  }
  if (lt::take_injected_failure()) return LT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas * p.parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (unsigned)smem_of(p.chunk);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim = {(unsigned)p.parts, 1, 1};
  cfg.attrs = attrs;
  cfg.numAttrs = p.parts > 1 ? 2 : 1;
  void* args[] = {&p, &code_map, &scale_map};
  return cudaLaunchKernelExC(&cfg, func, args) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

}  // extern "C"
