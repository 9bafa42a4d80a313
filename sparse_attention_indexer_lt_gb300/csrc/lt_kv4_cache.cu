// lt_kv4_cache.cu -- storing rows into the 4-bit cache and loading them back
// (lt_kv4_store, lt_kv4_load).
//
// Store: y = x / scale per group of 32 channels, scale the smallest number on a
// grid with 6 * scale >= amax, each y rounded to the nearest of e2m1's levels.
// A lane takes eight channels (one 16-byte load of 16-bit values), four lanes a
// group (two shuffles for amax), a warp 256 channels: the key and value of one
// position and head for D = 128, whose row it writes as one run.
//
// The rounding has to be that of the quotient as a real number, though y itself is
// rounded. For 16-bit inputs that is so: the scale has 9 significant bits and x
// at most 11, so x / scale is a level border exactly or at least 2^-13 of it away,
// and q + r / scale with r = x - q * scale (one exact fused step) is the exact
// quotient where that has at most 24 bits, borders among them. fp32 inputs can lie nearer to
// a border; they are compared with border * scale, which has at most 12 bits.
//
// Bound by HBM: 4 bytes read and 9/8 written per channel pair.

#include <cfloat>
#include <type_traits>

#include "lt_kv4.cuh"

namespace {

using lt::kv4::row_bytes;

constexpr int kThreads = 256;
constexpr float kScaleMax = 10912.0f;

struct CacheParams {
  const void* k;
  const void* v;
  void* out_k;
  void* out_v;
  const int64_t* slots;
  uint8_t* cache;
  int64_t items;  // tokens * kv_heads
  int64_t slot_end;
  int64_t k_token, k_head, v_token, v_head;
  int32_t heads;
  int32_t shift;
};

// The smallest scale >= amax / 6 with 9 significant bits, a multiple of 2^-23 (amax finite).
// The quotient rounded up to fp32 has the same successors on that grid as the exact one,
// since the grid's numbers are fp32 numbers; from 2^-15 on its 9 bits are the word's upper
// ones, below it the multiples of 2^-23.
__device__ __forceinline__ float scale_of(float amax) {
  const float t = __fdiv_ru(amax, 6.0f);
  const float s = t >= 0x1p-15f ? __uint_as_float((__float_as_uint(t) + 0x7FFFu) & ~0x7FFFu) : ceilf(t * 0x1p23f) * 0x1p-23f;
  return fminf(s, kScaleMax);
}

template <class S>
__device__ __forceinline__ void load8(const S* p, bool wide, float (&x)[8]);

template <>
__device__ __forceinline__ void load8<float>(const float* p, bool wide, float (&x)[8]) {
  if (wide) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
  }
}
template <class S>
__device__ __forceinline__ float widen(uint16_t b) {
  if constexpr (std::is_same<S, __nv_bfloat16>::value)
    return __uint_as_float((uint32_t)b << 16);
  else
    return __half2float(__ushort_as_half(b));
}
template <class S>
__device__ __forceinline__ void load8_16(const S* p, bool wide, float (&x)[8]) {
  const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
  if (wide) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = widen<S>((uint16_t)w[i]);
      x[2 * i + 1] = widen<S>((uint16_t)(w[i] >> 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = widen<S>(__ldg(u + i));
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, bool wide, float (&x)[8]) { load8_16(p, wide, x); }
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, bool wide, float (&x)[8]) {
  load8_16(p, wide, x);
}

// The codes of eight channels of a group with this scale (finite inputs).
template <class S>
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], float s) {
  if constexpr (sizeof(S) == 2) {
    const float inv = s > 0.0f ? __frcp_rn(s) : 0.0f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[i] * inv;
      y[i] = fmaf(fmaf(-q, s, x[i]), inv, q);
    }
    return lt::kv4::codes_of(y);
  } else {
    uint32_t w = 0;
    if (s > 0.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        const uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) +
                           (a >= 3.5f * s) + (a > 5.0f * s);
        w |= (c | (x[i] < 0.0f ? 8u : 0u)) << (4 * i);
      }
    }
    return w;
  }
}

// One warp-wide step covers 256 channels: lanes walk the 2 * D channels (key, then value) of an
// item, 16 (D = 64) or 32 (D = 128) lanes an item; D = 256 takes two steps of a warp.
template <class S, int D>
__global__ void __launch_bounds__(kThreads) store_kernel(CacheParams p, bool wide) {
  constexpr int kLanes = 2 * D / 8;  // lanes of an item
  constexpr int kRow = row_bytes(D);
  lt::kv4::dependency_wait();
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < (p.items + 3) / 4 * 4 * kLanes; u += stride) {
    // (items rounded up to four keep whole warps in step for the shuffles)
    const int64_t item = u / kLanes;
    const int part = (int)(u % kLanes);  // of the item's channels: eight each, keys first
    const bool is_v = part >= kLanes / 2;
    const int c = (part % (kLanes / 2)) * 8;
    int64_t slot = -1;
    float x[8] = {};
    const int64_t token = item / p.heads;
    const int head = (int)(item % p.heads);
    if (item < p.items) {
      slot = __ldg(p.slots + token);
      if (slot >= p.slot_end) slot = -1;
    }
    if (slot >= 0) {
      const S* from = is_v ? static_cast<const S*>(p.v) + token * p.v_token + head * p.v_head
                           : static_cast<const S*>(p.k) + token * p.k_token + head * p.k_head;
      load8<S>(from + c, wide, x);
    }
    float amax = 0.0f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(x[i]));
      finite = finite && fabsf(x[i]) <= FLT_MAX;
    }
    if (!finite) amax = INFINITY;  // a NaN is lost in fmaxf: both are carried as infinity
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
    if (slot < 0) continue;  // (only after the shuffles)
    const bool bad = !(amax <= FLT_MAX);
    const float s = bad ? 0.0f : scale_of(amax);
    const uint32_t codes = bad ? 0u : quantise8<S>(x, s);
    uint8_t* row = p.cache + ((((slot >> p.shift) * p.heads + head) << p.shift) + (slot & ((1 << p.shift) - 1))) * (int64_t)kRow;
    *reinterpret_cast<uint32_t*>(row + part * 4) = codes;
    if ((part & 3) == 0) {
      const uint16_t h = bad ? (uint16_t)0x7FFF : __half_as_ushort(__float2half_rn(s));
      *reinterpret_cast<uint16_t*>(row + D + part / 4 * 2) = h;
    }
    if constexpr (kRow > D + D / 8) {
      if (part == 0) *reinterpret_cast<uint2*>(row + D + D / 8) = make_uint2(0u, 0u);
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
  constexpr int kRow = row_bytes(D);
  lt::kv4::dependency_wait();
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < p.items * kLanes; u += stride) {
    const int64_t item = u / kLanes;
    const int part = (int)(u % kLanes);
    const int64_t token = item / p.heads;
    const int head = (int)(item % p.heads);
    const int64_t slot = __ldg(p.slots + token);
    uint32_t h[4] = {};
    if (slot >= 0 && slot < p.slot_end) {
      const uint8_t* row =
          p.cache + ((((slot >> p.shift) * p.heads + head) << p.shift) + (slot & ((1 << p.shift) - 1))) * (int64_t)kRow;
      const uint32_t w = *reinterpret_cast<const uint32_t*>(row + part * 4);
      const uint32_t s = *reinterpret_cast<const uint16_t*>(row + D + part / 4 * 2);
      lt::kv4::codes_to_half2(w, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = lt::kv4::hmul2(h[i], s | (s << 16));
    }
    const bool is_v = part >= kLanes / 2;
    S* to = static_cast<S*>(is_v ? p.out_v : p.out_k) + item * D + (part % (kLanes / 2)) * 8;
    put8<S>(to, h);
  }
  lt::kv4::dependents_launch();
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Enough CTAs for a few rounds of every SM; the kernels walk the items grid-stride.
unsigned grid_for(int64_t threads) {
  int64_t g = (threads + kThreads - 1) / kThreads;
  const int64_t most = 152 * 32;
  return (unsigned)(g < 1 ? 1 : g > most ? most : g);
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
  if (lt_kv4_row_bytes(head_dim) == 0) return LT_ERR_UNSUPPORTED;
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
  p.items = tokens * kv_heads;
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
  cfg.gridDim = dim3(grid_for((p.items + 3) / 4 * 4 * (head_dim / 4)));
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
  p.items = tokens * kv_heads;
  p.slot_end = pages * page_size;
  p.heads = kv_heads;
  p.shift = lt::kv4::page_shift(page_size);
  const void* func = dtype == LT_DTYPE_F32    ? load_ptr<float>(head_dim)
                     : dtype == LT_DTYPE_BF16 ? load_ptr<__nv_bfloat16>(head_dim)
                                              : load_ptr<__half>(head_dim);
  return lt::kv4::launch(func, dim3(grid_for(p.items * (head_dim / 4))), kThreads, 0, &p, stream);
}

}  // extern "C"
