// lt_kv4_quantise.cuh -- eight channels into e2m1 codes under the scale of their group of
// 32, for what stores values in 4 bits.
//
// y = x / scale, scale the smallest number on a grid with 6 * scale >= amax, each y
// rounded to the nearest of e2m1's levels. A lane takes eight channels (one 16-byte load of 16-bit
// values), four lanes a group (two shuffles for amax).
//
// The rounding has to be that of the quotient as a real number, though y itself is
// rounded. For 16-bit inputs that is so: the scale has 9 significant bits and x
// at most 11, so x / scale is a level border exactly or at least 2^-13 of it away,
// and q - r / scale with r = q * scale - x (one exact fused step) is the exact
// quotient where that has at most 24 bits, borders among them. fp32 inputs can lie nearer to
// a border, but not nearer than 2^-24 of it, and q - r / scale is off by 2^-45 before its own
// rounding: it is on the right side, or on the border itself. Where it is on a number of three
// bits, the inputs are compared with border * scale, which has at most 12 bits.
#pragma once

#include <cfloat>
#include <type_traits>

#include "lt_kv4.cuh"

namespace lt {
namespace kv4 {

constexpr float kScaleMax = 10912.0f;

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
  __device__ __forceinline__ void take(const uint32_t* words) { w[0] = words[0], w[1] = words[1], w[2] = words[2], w[3] = words[3]; }
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
    return codes_of(y);
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
  __device__ __forceinline__ void take(const uint32_t* words) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(words[i]);
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    return m;
  }
  static __device__ __forceinline__ bool finite(uint32_t bits) { return bits < 0x7F800000u; }
  static __device__ __forceinline__ float number(uint32_t bits) { return __uint_as_float(bits); }
  // As for 16 bits, but amax / 6 may lie nearer to a number of the grid than t is to it: where 6 s (12 bits, exact) does
  // not reach amax, it is the next one.
  static __device__ __forceinline__ float scale(float amax) {
    const float s = scale_above(amax * 0x1.55550p-3f);
    const float next = s >= 0x1p-15f ? __uint_as_float(__float_as_uint(s) + 0x8000u) : s + 0x1p-23f;
    return fminf(6.0f * s < amax ? next : s, kScaleMax);
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = s > 0.0f ? inv : 0.0f;
    float y[8];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[i] * inv;
      y[i] = fmaf(-fmaf(q, s, -x[i]), inv, q);  // (a zero keeps its sign)
      near = near || (__float_as_uint(y[i]) & 0x1FFFFFu) == 0;
    }
    return near ? codes_by_borders(s) : codes_of(y);
  }
  __device__ __forceinline__ uint32_t codes_by_borders(float s) const {
    uint32_t w = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {  // (seldom, but for zeros: a short loop, its input picked out of the registers)
      float v = x[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) v = i == j ? x[j] : v;
      const float a = fabsf(v);
      uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) +
                   (a >= 3.5f * s) + (a > 5.0f * s);
      if (s == 0.0f) c = 0;  // (a group of zeros)
      w |= (c | (__float_as_uint(v) >> 31 << 3)) << (4 * i);  // (a zero has a sign, too)
    }
    return w;
  }
};

}  // namespace kv4
}  // namespace lt
