// lt_kv4.cuh -- the 4-bit cache's row format and what its kernels share.
//
// A row (one position of one kv head, D channels): D/2 bytes of key codes, D/2 of
// value codes, D/32 fp16 key scales, D/32 fp16 value scales, padded to 16 bytes.
// Key, value and scales of a position lie side by side so that a listed position
// is one contiguous read (144 bytes for D = 128) and a run of positions of a page
// one bulk copy. The row's length in words, 4 mod 32 for D = 128 and 20 for D = 64, also
// puts the eight rows that a matrix fragment reads at once on different banks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/lt_kv4.h"
#include "lt_launch.h"

namespace lt {
namespace kv4 {

__host__ __device__ constexpr int row_bytes(int d) { return (d + d / 8 + 15) / 16 * 16; }

inline int page_shift(int32_t page_size) {
  if (page_size < 1 || page_size > LT_KV4_MAX_PAGE || (page_size & (page_size - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

inline lt_status launch(const void* func, dim3 grid, unsigned threads, unsigned smem, void* params, void* stream,
                        unsigned cluster = 1) {
  if (take_injected_failure()) return LT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim = {cluster, 1, 1};
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void* a[] = {params};
  return cudaLaunchKernelExC(&cfg, func, a) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

// The eight e2m1 codes of a word as four fp16 pairs (byte i: channels 2i, 2i + 1).
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Eight numbers rounded to the nearest e2m1 code, ties to even, saturating.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace kv4
}  // namespace lt
