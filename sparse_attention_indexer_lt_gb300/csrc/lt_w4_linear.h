// lt_w4_linear.h -- internal: what the products with 4-bit weights share.
#pragma once

#include <cudaTypedefs.h>

#include "../../include/lt_w4.h"
#include "lt_kv4.cuh"

namespace lt {
namespace w4 {

constexpr int kMaxParts = 8;  // CTAs of a portable cluster, along the inputs

// bf16 tokens become fp16 ones times a power of two: the one that brings the largest finite magnitude (its fp32
// word) into [2^14, 2^15).
__device__ __forceinline__ float token_power(uint32_t big) {
  const int e = (int)(big >> 23);
  return __uint_as_float((uint32_t)(e == 0 ? 253 : min(268 - e, 253)) << 23);
}
__device__ __forceinline__ uint32_t finite_bf16_pair(uint32_t w) {  // the larger finite magnitude of two, as an fp32 word
  const uint32_t lo = w << 16 & 0x7FFF0000u, hi = w & 0x7FFF0000u;
  return max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u);
}
__device__ __forceinline__ uint32_t largest_of(const uint4& v) {
  return max(max(finite_bf16_pair(v.x), finite_bf16_pair(v.y)), max(finite_bf16_pair(v.z), finite_bf16_pair(v.w)));
}
__device__ __forceinline__ uint32_t pair_to_half(uint32_t w, float mul) {
  const float lo = __uint_as_float(w << 16) * mul, hi = __uint_as_float(w & 0xFFFF0000u) * mul;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ uint4 to_half(const uint4& v, float mul) {
  return make_uint4(pair_to_half(v.x, mul), pair_to_half(v.y, mul), pair_to_half(v.z, mul), pair_to_half(v.w, mul));
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
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void put_peer(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
// An output's bias, and the output, rounded once.
__device__ __forceinline__ float bias_of(const void* bias, int row, int bf16) {
  if (bias == nullptr) return 0.0f;
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(bias)[row]) : __half2float(static_cast<const __half*>(bias)[row]);
}
__device__ __forceinline__ uint16_t bits_of(float y, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
}
__device__ __forceinline__ void put(void* out, int64_t at, float y, int bf16) {
  static_cast<uint16_t*>(out)[at] = bits_of(y, bf16);
}

// ---- many tokens (lt_w4_many.cu)
constexpr int kManyStep = 128;  // inputs of a step

struct ManyPlan {
  int tile, tiles;    // tokens of a tile, a multiple of 16 up to 256; tiles
  int row_tiles;      // tiles of 128 outputs of a CTA: 1 or 2
  int columns;        // of tensor memory that a CTA has: 512 alone on its SM, 256 beside another
  int parts;          // CTAs of a cluster, along the inputs
  int code_ring, token_ring, row_ring;  // places for codes and tokens in shared memory, unpacked weights in tensor memory
  int sum_columns;    // of tensor memory, for the sums of a tile of outputs
  int smem;
  int64_t steps;
  int64_t x_bytes, bytes;  // workspace: the tokens as the tensor core reads them; with their powers
};
// A tensor map of n rows of `bytes` bytes, in boxes of `wide` bytes of `rows` rows. Boxes of 64 and 128 bytes a row have its
// 16-byte pieces turned by the row, so that eight lanes that read a piece of eight rows (of two, four pieces) have all
// banks, or half of them.
lt_status map_rows(CUtensorMap* map, const void* at, int64_t n, int64_t bytes, int wide, int rows);
ManyPlan many_plan(int dev, int64_t tokens, int64_t n, int64_t k);

struct ManyParams {
  const void* x;
  const uint8_t* codes;
  const uint16_t* scales;
  const void* bias;
  void* out;
  uint8_t* tiles_at;  // [tile][64 inputs' block][token][64 inputs], each token's eight 16-byte pieces turned by the token
  float* inverse;     // [token]
  int64_t x_stride, out_stride;
  int32_t n, k, tokens, tile, parts, steps;
  int32_t code_ring, token_ring, row_ring, sum_columns, rows_column, columns;
  int32_t bf16, wide_scales, wide_out;
  uint32_t zero;
};
lt_status launch_many(int dev, ManyParams* p, const ManyPlan& plan, void* stream);

}  // namespace w4
}  // namespace lt
