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
// and q - r / scale with r = q * scale - x (one exact fused step) is the exact
// quotient where that has at most 24 bits, borders among them. fp32 inputs can lie nearer to
// a border; they are compared with border * scale, which has at most 12 bits.
//
// HBM would allow 4 bytes read and 9/8 written a channel pair: 6.3 us for 8191 tokens of 8 heads of 128; the store
// takes 16 (168 warp instructions for 256 channels: bound by issue), the load 11, both together 23 to
// 28. What helped the store: no division to find token and head (33 to 28 us), largest magnitudes
// found on packed integers and an approximate reciprocal with an exact remainder (28 to 16).

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
  int64_t tokens;
  int64_t slot_end;
  int64_t k_token, k_head, v_token, v_head;
  int32_t heads;
  int32_t shift;
};

// The smallest scale >= amax / 6 with 9 significant bits, a multiple of 2^-23 (amax finite), from a `t` near
// amax / 6: the next number of the grid at or above t; from 2^-15 on its 9 bits are the word's
// upper ones, below it the grid is the multiples of 2^-23.
__device__ __forceinline__ float scale_above(float t) {
  const float s = t >= 0x1p-15f ? __uint_as_float((__float_as_uint(t) + 0x7FFFu) & ~0x7FFFu) : ceilf(t * 0x1p23f) * 0x1p-23f;
  return fminf(s, kScaleMax);
}

// Eight channels as they lie in memory, and what is asked of them.
template <class S>
struct Eight {  // 16-bit types: pairs in words
  uint32_t w[4];
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load(const S* p, bool wide) {
    if (wide) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
      const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(u + 2 * i) | ((uint32_t)__ldg(u + 2 * i + 1) << 16);
    }
  }
  // The largest magnitude's bits; an infinity's bits or more where one is not finite (they order as integers).
  __device__ __forceinline__ uint32_t largest() const {
    const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
  }
  static __device__ __forceinline__ bool finite(uint32_t bits) { return bits < (std::is_same<S, __half>::value ? 0x7C00u : 0x7F80u); }
  static __device__ __forceinline__ float number(uint32_t bits) {
    if constexpr (std::is_same<S, __half>::value)
      return __half2float(__ushort_as_half((uint16_t)bits));
    else
      return __uint_as_float(bits << 16);
  }
  // t: amax / 6 times 1 - 2^-18 or so. amax has at most 11 bits, so amax / 6 is a number of the grid or at
  // least 2^-13 of itself away from one: the next number above t is the next at or above amax / 6.
  static __device__ __forceinline__ float scale(float amax) { return scale_above(amax * 0x1.55550p-3f); }
  // y = x / s as q - r / s with the exact remainder r = q s - x: exact where the quotient is a level border
  // (inv within 2^-22 of 1 / s will do). A zero keeps its sign, also with s = 0: r is +0 then, and -0 + q is q.
  __device__ __forceinline__ uint32_t codes(float s) const {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = s > 0.0f ? inv : 0.0f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = number(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
      const float q = x * inv;
      y[i] = fmaf(-fmaf(q, s, -x), inv, q);
    }
    return lt::kv4::codes_of(y);
  }
};

template <>
struct Eight<float> {
  float x[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  }
  __device__ __forceinline__ void load(const float* p, bool wide) {
    if (wide) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __ldg(p + i);
    }
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
  }
  static __device__ __forceinline__ bool finite(uint32_t bits) { return bits < 0x7F800000u; }
  static __device__ __forceinline__ float number(uint32_t bits) { return __uint_as_float(bits); }
  // The quotient rounded up to fp32 has the same next number of the grid as the exact one, since the grid's
  // numbers are fp32 numbers.
  static __device__ __forceinline__ float scale(float amax) { return scale_above(__fdiv_ru(amax, 6.0f)); }
  // (fp32 may lie nearer to a border than a rounded quotient tells; border * s has at most 12 bits)
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(x[i]);
      uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) +
                   (a >= 3.5f * s) + (a > 5.0f * s);
      if (s == 0.0f) c = 0;  // (a group of zeros)
      w |= (c | (__float_as_uint(x[i]) >> 31 << 3)) << (4 * i);  // (a zero has a sign, too)
    }
    return w;
  }
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
