// lt_w4_linear.cu -- products with 4-bit weights (lt_w4_linear) for few tokens, and the
// weights' quantisation (lt_w4_quantise).
//
// Few tokens: the weights are read once and that is the time, so what counts is the work per weight: unpacking,
// scaling, feeding the tensor core. The weights are the 16-row operand straight from registers (m16n8k16,
// fp32 sums), the tokens the eight columns. The order of the inputs within a product is free, so a lane
// takes 16 bytes of codes, a whole group of 32 inputs, of rows g and g + 8: four lanes
// read 64 bytes of a row, a lane has one scale a row, and the tokens' fragments are 16 bytes
// of the same inputs from shared memory.
//
// A CTA's eight warps are WR row tiles of 16 by 8 / WR parts of the inputs; a cluster cuts the inputs
// further where there are few rows. The parts join in shared memory and over
// distributed shared memory, in one order whatever the timing.

#include <mutex>

#include "lt_async.cuh"
#include "lt_kv4_quantise.cuh"
#include "lt_w4_linear.h"

namespace {

using namespace lt::kv4;
using namespace lt::w4;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct LinearParams {
  const void* x;
  const uint8_t* codes;
  const __half* scales;
  const void* bias;
  void* out;
  int64_t x_stride, out_stride;
  int32_t n, k, tokens;
  int32_t row_warps;   // row tiles of a CTA: 1 or 2
  int32_t parts;       // CTAs of a cluster, along the inputs
  int32_t chunk;       // steps whose inputs are in shared memory at a time
  int32_t join_at;     // where the warps' sums are joined, behind the inputs
  int32_t bf16;
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// Where 16-byte piece q of token t lies: pieces of a step (16) by lane group and word, the upper eight's turned
// by one, tokens 32 bytes apart beyond whole 128-byte lines, so that the eight lanes (two tokens, four groups)
// that read 16 bytes together have all banks.
__device__ __forceinline__ int piece_at(int t, int q, int pitch) { return t * pitch + ((q ^ (q >> 3 & 1)) << 4); }

constexpr int kPerSm = 3;   // CTAs
constexpr int kTokens = 8;  // columns of the product; a call has at most four tokens

__global__ void __launch_bounds__(kThreads, kPerSm) few_kernel(LinearParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t largest[kTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int row_shift = p.row_warps >> 1, k_shift = 3 - row_shift;  // (one or two row tiles)
  const int k_warps = kWarps >> row_shift, wr = warp & row_shift, wk = warp >> row_shift;
  const int rank = blockIdx.x % p.parts;
  const int rows = p.row_warps * 16;
  const int tokens = p.tokens;
  const int steps = (p.k + kStep - 1) / kStep, groups = p.k / 32;
  // the CTA's steps, in chunks whose inputs fit into shared memory; its row blocks are every so many
  const int s_begin = (int)((int64_t)steps * rank / p.parts), s_end = (int)((int64_t)steps * (rank + 1) / p.parts);
  const int chunks = (s_end - s_begin + p.chunk - 1) / p.chunk;
  const int blocks = (p.n + rows - 1) / rows, first = blockIdx.x / p.parts, every = gridDim.x / p.parts;
  if (tid < kTokens) largest[tid] = 0u;
  dependency_wait();
  __syncthreads();

  // the warp's steps of a chunk
  auto range = [&](int chunk, int* from, int* to) {
    const int c0 = s_begin + chunk * p.chunk, wide = min(p.chunk, s_end - c0);
    *from = c0 + (wide * wk >> k_shift);
    *to = c0 + (wide * (wk + 1) >> k_shift);
  };

  constexpr int U = 2;  // steps of a batch; two batches are on their way
  struct Batch {
    uint4 a[U], b[U];
    uint32_t sa, sb;  // scales of groups 2c and 2c + 1 of the batch's eight
  };
  // where the next batch is fetched from: it runs ahead over chunks and row blocks
  struct Next {
    int block, chunk, s, to;
    const uint8_t *a, *b;
    const uint16_t *sa, *sb;
  } next = {};
  auto aim = [&]() {  // at the rows of next.block
    const int ra = min(next.block * rows + wr * 16 + g, p.n - 1), rb = min(next.block * rows + wr * 16 + g + 8, p.n - 1);
    next.a = p.codes + (int64_t)ra * (p.k / 2);
    next.b = p.codes + (int64_t)rb * (p.k / 2);
    next.sa = reinterpret_cast<const uint16_t*>(p.scales) + (int64_t)ra * groups;
    next.sb = reinterpret_cast<const uint16_t*>(p.scales) + (int64_t)rb * groups;
  };
  auto fetch = [&](Batch& w) {
    if (next.block >= blocks) return;
    const int group = next.s * 4;
    if (group + 4 * U <= groups && groups % 2 == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        w.a[u] = load_once(next.a + (group + c) * 16 + u * 64);
        w.b[u] = load_once(next.b + (group + c) * 16 + u * 64);
      }
      w.sa = __ldg(reinterpret_cast<const uint32_t*>(next.sa + group + 2 * c));
      w.sb = __ldg(reinterpret_cast<const uint32_t*>(next.sb + group + 2 * c));
    } else {
      // past the inputs' end the last group again: its inputs in shared memory are zeros there
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = min(group + 4 * u + c, groups - 1);
        w.a[u] = load_once(next.a + (int64_t)at * 16);
        w.b[u] = load_once(next.b + (int64_t)at * 16);
      }
      const int lower = min(group + 2 * c, groups - 1), upper = min(group + 2 * c + 1, groups - 1);
      w.sa = __ldg(next.sa + lower) | (uint32_t)__ldg(next.sa + upper) << 16;
      w.sb = __ldg(next.sb + lower) | (uint32_t)__ldg(next.sb + upper) << 16;
    }
    next.s += U;
    if (next.s < next.to) return;
    do {
      if (++next.chunk == chunks) {
        next.chunk = 0;
        next.block += every;
        if (next.block >= blocks) return;
        aim();
      }
      range(next.chunk, &next.s, &next.to);
    } while (next.s >= next.to);  // (every warp has steps in the first chunk, or none at all)
  };

  const int pitch = p.chunk * kStep * 2 + 32;
  const uint32_t x_at = lt::smem_u32(smem);
  // a chunk's inputs into shared memory; past the last input, zeros
  auto stage = [&](int chunk) {
    const int c0 = s_begin + chunk * p.chunk, pieces = min(p.chunk, s_end - c0) * 16;
    for (int t = 0; t < tokens; ++t) {
      const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)t * p.x_stride + (int64_t)c0 * kStep;
      uint32_t big = 0;
      for (int q = tid; q < pieces; q += kThreads) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if ((int64_t)c0 * kStep + q * 8 < p.k) v = __ldg(reinterpret_cast<const uint4*>(x) + q);
        *reinterpret_cast<uint4*>(smem + piece_at(t, q, pitch)) = v;
        if (p.bf16) big = max(big, largest_of(v));
      }
      if (p.bf16) {
        big = __reduce_max_sync(~0u, big);
        if (lane == 0) atomicMax(&largest[t], big);
      }
    }
    __syncthreads();
    if (!p.bf16) return;
    for (int t = 0; t < tokens; ++t) {
      const float mul = token_power(largest[t]);
      for (int q = tid; q < pieces; q += kThreads) {
        uint4* at = reinterpret_cast<uint4*>(smem + piece_at(t, q, pitch));
        *at = to_half(*at, mul);
      }
    }
    __syncthreads();
  };

  Batch w0, w1;
  next.block = first;
  next.chunk = 0;
  range(0, &next.s, &next.to);
  const bool works = next.s < next.to && first < blocks;
  if (works) {
    aim();
    fetch(w0);
    fetch(w1);
  }
  if (chunks == 1) stage(0);

  float acc[4];
  float power[2];  // of tokens 2c and 2c + 1, whose sums a lane has
  const uint32_t xa = x_at + min(g, tokens - 1) * pitch;  // the lane's token's inputs
  const int q0 = c * 4, turn = c >> 1;  // (see piece_at)
  const int scale_lane = (lane & ~3) | (c >> 1);
  const uint32_t scale_half = c & 1 ? 0x3232u : 0x1010u;
  auto work = [&](const Batch& w, int at, int count) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= count) break;
      // the scale of group 4 u + c is with lane 2 u + c / 2 of the four
      const uint32_t ka = __byte_perm(__shfl_sync(~0u, w.sa, scale_lane + 2 * u), 0, scale_half);
      const uint32_t kb = __byte_perm(__shfl_sync(~0u, w.sb, scale_lane + 2 * u), 0, scale_half);
      const uint32_t wa[4] = {w.a[u].x, w.a[u].y, w.a[u].z, w.a[u].w};
      const uint32_t wb[4] = {w.b[u].x, w.b[u].y, w.b[u].z, w.b[u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t ha[4], hb[4];
        codes_to_half2(wa[j], ha);
        codes_to_half2(wb[j], hb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ha[i] = hmul2(ha[i], ka);
          hb[i] = hmul2(hb[i], kb);
        }
        uint32_t b0, b1, b2, b3;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3) : "r"(xa + (((at + u) * 16 + q0 + (j ^ turn)) << 4)));
        mma16816(acc, ha[0], hb[0], ha[1], hb[1], b0, b1);
        mma16816(acc, ha[2], hb[2], ha[3], hb[3], b2, b3);
      }
    }
  };

  float* joined = reinterpret_cast<float*>(smem + p.join_at);  // two times [k warp][token][row], in turn
  int phase = 0, turns = 0;
  for (int block = first; block < blocks; block += every, turns ^= 1) {
    acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
    power[0] = power[1] = 1.0f;
    for (int chunk = 0; chunk < chunks; ++chunk) {
      if (chunks > 1) {
        __syncthreads();  // the last chunk's inputs have been read
        stage(chunk);
      }
      if (p.bf16) {
        // sums so far go over to the new power, which is the largest input's so far and never grows
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float now = token_power(largest[min(2 * c + e, tokens - 1)]);
          if (chunk > 0) {
            const float f = fmaxf(now / power[e], 0x1p-126f);  // (not 0: an infinity stays one)
            acc[e] *= f;
            acc[e + 2] *= f;
          }
          power[e] = now;
        }
      }
      int from, to;
      range(chunk, &from, &to);
      const int c0 = s_begin + chunk * p.chunk;
      for (int s = from; s < to; s += U) {
        if (phase == 0) {
          work(w0, s - c0, to - s);
          fetch(w0);
        } else {
          work(w1, s - c0, to - s);
          fetch(w1);
        }
        phase ^= 1;
      }
    }
    // join the warps, and with a cluster its CTAs
    float* mine = joined + turns * (kWarps * 16 * kTokens);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int token = 2 * c + (e & 1), row = wr * 16 + g + (e >> 1) * 8;
      if (token < tokens) mine[(wk * kTokens + token) * rows + row] = p.bf16 ? acc[e] * (1.0f / power[e & 1]) : acc[e];
    }
    __syncthreads();
    const int all = tokens * rows;
    if (p.parts > 1) {
      for (int u = tid; u < all; u += kThreads) {
        float y = mine[u];
        for (int w = 1; w < k_warps; ++w) y += mine[w * kTokens * rows + u];
        mine[u] = y;
      }
      cluster_sync();
    }
    for (int u = rank * kThreads + tid; u < all; u += p.parts * kThreads) {
      const int token = u / rows, row = block * rows + u % rows;
      float y = 0.0f;
      if (p.parts > 1) {
#pragma unroll
        for (int r = 0; r < kMaxParts; ++r)
          if (r < p.parts) y += peer_f32(lt::smem_u32(mine) + u * 4, r);
      } else {
        for (int w = 0; w < k_warps; ++w) y += mine[w * kTokens * rows + u];
      }
      if (row < p.n) put(p.out, (int64_t)token * p.out_stride + row, y + bias_of(p.bias, row, p.bf16), p.bf16);
    }
    if (p.parts > 1) cluster_sync();  // (a CTA's shared memory stays until its peers have read it)
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

constexpr int kFewInputs = 56 * 1024;  // bytes of inputs in shared memory: three CTAs an SM
constexpr int kFewSmem = kFewInputs + 2 * kWarps * 16 * kTokens * 4;
// Whether a call takes the kernel for few tokens. us there and in the one for many (in a graph; eagerly its second
// launch costs the host 6 more):
//   n x k            1 token      2            3            4            6            8
//   1000 x 2048      4.9, 6.0     5.7, 6.1     6.3, 6.1     6.8, 6.1     8.8, 6.2
//   4096 x 4096      6.4, 8.5     7.5, 8.6     8.8, 8.6     9.4, 8.6     10.6, 8.7    11.8, 8.7
//   10240 x 8192     17.6, 19.4   19.7, 19.6   23.2, 19.7   23.2, 19.7   25.8, 19.9   30.4, 19.7
//   28672 x 8192     35.3, 38.1   38.5, 37.8   39.0, 38.0   45.3, 37.8   44.0, 37.9   66.6, 38.1
bool few(int64_t tokens, int64_t n, int64_t k) { return tokens <= 2 || (tokens <= 4 && n * k <= (int64_t)1 << 25); }

lt_status check_sizes(int64_t tokens, int64_t n, int64_t k) {
  if (tokens < 0 || n < 0 || k < 0) return LT_ERR_INVALID_ARG;
  if (k == 0 || k % 32 != 0 || k > INT32_MAX - 1024 || n > INT32_MAX - 1024 || tokens > 65535 * 8) return LT_ERR_UNSUPPORTED;
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
  if (found == LT_OK) *bytes = many_plan(dev, tokens, n, k).bytes;
  return found;
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
  p.scales = static_cast<const __half*>(scales);
  p.bias = bias;
  p.out = out;
  p.x_stride = x_stride;
  p.out_stride = out_stride;
  p.n = (int32_t)n;
  p.k = (int32_t)k;
  p.tokens = (int32_t)tokens;
  p.bf16 = dtype == LT_DTYPE_BF16;
  const int here = (int)tokens;
  p.row_warps = here <= 2 ? 1 : 2;
  const int64_t row_blocks = (n + p.row_warps * 16 - 1) / (p.row_warps * 16);
  const int steps = (int)((k + kStep - 1) / kStep), k_warps = kWarps / p.row_warps;
  const int64_t slots = (int64_t)sms * kPerSm;
  // as many steps' inputs in shared memory as fit; the inputs are cut over a cluster where the CTAs do not fill the SMs
  const int most = (kFewInputs / here - 32) / (kStep * 2);
  p.parts = 1;
  while (p.parts < kMaxParts && steps >= p.parts * 2 * k_warps &&
         (row_blocks * p.parts * 2 <= slots || (steps + p.parts - 1) / p.parts > most))
    p.parts *= 2;
  const int mine = (steps + p.parts - 1) / p.parts;
  p.chunk = mine < most ? mine : most / k_warps * k_warps;
  p.join_at = here * (p.chunk * kStep * 2 + 32);
  const int smem = p.join_at + 2 * kWarps * 16 * kTokens * 4;
  const int64_t resident = slots / p.parts;
  const int64_t ctas = row_blocks < resident ? row_blocks : resident;
  const void* func = reinterpret_cast<const void*>(&few_kernel);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_set[dev]) {
      if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) != cudaSuccess) return LT_ERR_CUDA;
      g_set[dev] = true;
    }
  }
  return launch(func, dim3((unsigned)(ctas * p.parts)), kThreads, (unsigned)smem, &p, stream, p.parts);
}

}  // extern "C"
