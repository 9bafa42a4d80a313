// lt_kv4_cache.cu -- storing rows into the 4-bit cache and loading them back
// (lt_kv4_store, lt_kv4_load).
//
// Store: a lane takes eight channels, four lanes a group of 32 (lt_kv4_quantise.cuh has the
// arithmetic), a warp 256 channels: the key and value of one position and head for
// D = 128, whose row it writes as one run.
//
// HBM would allow 4 bytes read and 9/8 written a channel pair: 6.3 us for 8191 tokens of 8 heads of 128; the store
// takes 16 (168 warp instructions for 256 channels: bound by issue), the load 11, both together 23 to
// 28. What helped the store: no division to find token and head (33 to 28 us), largest magnitudes
// found on packed integers and an approximate reciprocal with an exact remainder (28 to 16).

#include "lt_kv4.cuh"
#include "lt_kv4_quantise.cuh"

namespace {

using lt::kv4::Eight;
using lt::kv4::row_bytes;

constexpr int kThreads = 256;

struct CacheParams {
  const void* k;
  const void* v;
  void* out_k;
  void* out_v;
  const int64_t* slots;
  uint8_t* cache;
  int64_t tokens;
  int64_t slot_end;
  int64_t k_token, k_head, v_token, v_head;
  int32_t heads;
  int32_t shift;
};

// A step of a warp covers 256 channels: lanes walk the 2 * D channels (key, then value) of an item, 16
// (D = 64) or 32 (D = 128) lanes an item; D = 256 takes two warps. A CTA has one head, so no
// index is divided. A thread has kAhead steps in flight: their slots and values are asked
// for before the first is worked on (the values of a token without a slot are read in
// vain, which is rare and in bounds).
constexpr int kAhead = 4;

template <class S, int D>
__global__ void __launch_bounds__(kThreads) store_kernel(CacheParams p, bool wide) {
  constexpr int kLanes = 2 * D / 8;  // lanes of an item
  constexpr int kTokens = kThreads / kLanes;
  constexpr int kRow = row_bytes(D);
  const int part = threadIdx.x % kLanes, head = blockIdx.y;  // part: eight of the item's channels, keys first
  const bool is_v = part >= kLanes / 2;
  const int c = part % (kLanes / 2) * 8;
  const int64_t step = is_v ? p.v_token : p.k_token;
  const S* from = is_v ? static_cast<const S*>(p.v) + head * p.v_head + c : static_cast<const S*>(p.k) + head * p.k_head + c;
  const int64_t stride = (int64_t)gridDim.x * kTokens;
  lt::kv4::dependency_wait();
  for (int64_t base = (int64_t)blockIdx.x * kTokens; base < p.tokens; base += kAhead * stride) {
    Eight<S> x[kAhead];
    int64_t slot[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t t = base + k * stride + threadIdx.x / kLanes;
      slot[k] = -1;
      x[k].clear();
      if (t < p.tokens) {
        slot[k] = __ldg(p.slots + t);
        x[k].load(from + t * step, wide);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (base + k * stride >= p.tokens) break;  // (the same for the whole CTA)
      uint32_t largest = x[k].largest();
      largest = max(largest, __shfl_xor_sync(~0u, largest, 1));
      largest = max(largest, __shfl_xor_sync(~0u, largest, 2));
      const int64_t at = slot[k];
      if (at >= 0 && at < p.slot_end) {
        const bool bad = !Eight<S>::finite(largest);
        const float s = bad ? 0.0f : Eight<S>::scale(Eight<S>::number(largest));
        const uint32_t codes = bad ? 0u : x[k].codes(s);
        uint8_t* row = p.cache + ((((at >> p.shift) * p.heads + head) << p.shift) + (at & ((1 << p.shift) - 1))) * (int64_t)kRow;
        *reinterpret_cast<uint32_t*>(row + part * 4) = codes;
        if ((part & 3) == 0) {
          const uint16_t h = bad ? (uint16_t)0x7FFF : __half_as_ushort(__float2half_rn(s));
          *reinterpret_cast<uint16_t*>(row + D + part / 4 * 2) = h;
        }
        if constexpr (kRow > D + D / 8) {
          if (part == 0) *reinterpret_cast<uint2*>(row + D + D / 8) = make_uint2(0u, 0u);
        }
      }
      __syncwarp();
    }
  }
  lt::kv4::dependents_launch();
}

template <class S>
__device__ __forceinline__ void put8(S* p, const uint32_t (&h)[4]);
template <>
__device__ __forceinline__ void put8<__half>(__half* p, const uint32_t (&h)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
}
template <>
__device__ __forceinline__ void put8<float>(float* p, const uint32_t (&h)[4]) {
  float2 f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
template <>
__device__ __forceinline__ void put8<__nv_bfloat16>(__nv_bfloat16* p, const uint32_t (&h)[4]) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);
    b[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(b[0], b[1], b[2], b[3]);
}

template <class S, int D>
__global__ void __launch_bounds__(kThreads) load_kernel(CacheParams p) {
  constexpr int kLanes = 2 * D / 8;
  constexpr int kTokens = kThreads / kLanes;
  constexpr int kRow = row_bytes(D);
  const int part = threadIdx.x % kLanes, head = blockIdx.y;
  S* to = static_cast<S*>(part >= kLanes / 2 ? p.out_v : p.out_k) + (int64_t)head * D + part % (kLanes / 2) * 8;
  const int64_t stride = (int64_t)gridDim.x * kTokens, step = (int64_t)p.heads * D;
  lt::kv4::dependency_wait();
  for (int64_t base = (int64_t)blockIdx.x * kTokens + threadIdx.x / kLanes; base < p.tokens; base += kAhead * stride) {
    int64_t slot[kAhead];
    uint32_t codes[kAhead], scale[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) slot[k] = base + k * stride < p.tokens ? __ldg(p.slots + base + k * stride) : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      codes[k] = scale[k] = 0u;
      if (slot[k] >= 0 && slot[k] < p.slot_end) {
        const uint8_t* row = p.cache + ((((slot[k] >> p.shift) * p.heads + head) << p.shift) + (slot[k] & ((1 << p.shift) - 1))) * (int64_t)kRow;
        codes[k] = *reinterpret_cast<const uint32_t*>(row + part * 4);
        scale[k] = *reinterpret_cast<const uint16_t*>(row + D + part / 4 * 2);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (base + k * stride >= p.tokens) break;
      uint32_t h[4];
      lt::kv4::codes_to_half2(codes[k], h);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = lt::kv4::hmul2(h[i], scale[k] | (scale[k] << 16));
      put8<S>(to + (base + k * stride) * step, h);
    }
  }
  lt::kv4::dependents_launch();
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A CTA for each head and run of tokens. While there are few, a thread has one step; with more than fill
// the SMs it takes up to kAhead, and beyond a few rounds of CTAs it walks the tokens.
dim3 grid_for(int64_t tokens, int heads, int d) {
  const int64_t per = kThreads / (d / 4), once = (152 * 8 + heads - 1) / heads, most = (152 * 32 + heads - 1) / heads;
  int64_t g = (tokens + per - 1) / per;
  if (g > once) g = (g + kAhead - 1) / kAhead > once ? (g + kAhead - 1) / kAhead : once;
  return dim3((unsigned)(g < 1 ? 1 : g > most ? most : g), (unsigned)heads);
}

template <class S>
const void* store_ptr(int d) {
  return d == 64    ? reinterpret_cast<const void*>(&store_kernel<S, 64>)
         : d == 128 ? reinterpret_cast<const void*>(&store_kernel<S, 128>)
                    : reinterpret_cast<const void*>(&store_kernel<S, 256>);
}
template <class S>
const void* load_ptr(int d) {
  return d == 64    ? reinterpret_cast<const void*>(&load_kernel<S, 64>)
         : d == 128 ? reinterpret_cast<const void*>(&load_kernel<S, 128>)
                    : reinterpret_cast<const void*>(&load_kernel<S, 256>);
}

lt_status check(const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t kv_heads, int32_t head_dim,
                const int64_t* slots, const void* cache, int64_t pages, int32_t page_size) {
  if (tokens < 0 || kv_heads < 1 || pages < 0 || lt::kv4::page_shift(page_size) < 0) return LT_ERR_INVALID_ARG;
  if (dtype != LT_DTYPE_F32 && dtype != LT_DTYPE_BF16 && dtype != LT_DTYPE_F16) return LT_ERR_INVALID_ARG;
  if (tokens > 0 && (k == nullptr || v == nullptr || slots == nullptr || (cache == nullptr && pages > 0)))
    return LT_ERR_INVALID_ARG;
  if (head_dim < 1 || !aligned(cache, 16)) return LT_ERR_INVALID_ARG;
  if (lt_kv4_row_bytes(head_dim) == 0 || kv_heads > 65535) return LT_ERR_UNSUPPORTED;
  return LT_OK;
}

}  // namespace

extern "C" {

int32_t lt_kv4_row_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 || head_dim == 256 ? row_bytes(head_dim) : 0;
}

lt_status lt_kv4_store(const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t kv_heads,
                       int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                       int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                       void* cache, int64_t pages, int32_t page_size, void* stream) {
  const lt_status st = check(k, v, dtype, tokens, kv_heads, head_dim, slots, cache, pages, page_size);
  if (st != LT_OK) return st;
  const uintptr_t size = dtype == LT_DTYPE_F32 ? 4 : 2;
  if (!aligned(k, size) || !aligned(v, size)) return LT_ERR_INVALID_ARG;
  if (tokens == 0 || pages == 0) return LT_OK;
  CacheParams p = {};
  p.k = k;
  p.v = v;
  p.slots = slots;
  p.cache = static_cast<uint8_t*>(cache);
  p.tokens = tokens;
  p.slot_end = pages * page_size;
  p.k_token = k_token_stride;
  p.k_head = k_head_stride;
  p.v_token = v_token_stride;
  p.v_head = v_head_stride;
  p.heads = kv_heads;
  p.shift = lt::kv4::page_shift(page_size);
  // 16-byte loads where every group of eight channels starts on 16 bytes
  const int64_t strides = k_token_stride | k_head_stride | v_token_stride | v_head_stride;
  bool wide = aligned(k, 16) && aligned(v, 16) && (strides * (int64_t)size) % 16 == 0;
  const void* func = dtype == LT_DTYPE_F32    ? store_ptr<float>(head_dim)
                     : dtype == LT_DTYPE_BF16 ? store_ptr<__nv_bfloat16>(head_dim)
                                              : store_ptr<__half>(head_dim);
  if (lt::take_injected_failure()) return LT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid_for(tokens, kv_heads, head_dim);
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

lt_status lt_kv4_load(const void* cache, int64_t pages, int32_t page_size, const int64_t* slots,
                      int64_t tokens, int32_t kv_heads, int32_t head_dim, void* k, void* v,
                      int32_t dtype, void* stream) {
  const lt_status st = check(k, v, dtype, tokens, kv_heads, head_dim, slots, cache, pages, page_size);
  if (st != LT_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return LT_ERR_INVALID_ARG;
  if (tokens == 0) return LT_OK;
  CacheParams p = {};
  p.out_k = k;
  p.out_v = v;
  p.slots = slots;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.tokens = tokens;
  p.slot_end = pages * page_size;
  p.heads = kv_heads;
  p.shift = lt::kv4::page_shift(page_size);
  const void* func = dtype == LT_DTYPE_F32    ? load_ptr<float>(head_dim)
                     : dtype == LT_DTYPE_BF16 ? load_ptr<__nv_bfloat16>(head_dim)
                                              : load_ptr<__half>(head_dim);
  return lt::kv4::launch(func, grid_for(tokens, kv_heads, head_dim), kThreads, 0, &p, stream);
}

}  // extern "C"
