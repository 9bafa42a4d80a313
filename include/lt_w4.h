/*
 * lt_w4.h -- C ABI of products with 4-bit weights (GB300, sm_103a): the
 * projections around a cache that holds 4 bits, too.
 *
 * A weight matrix of n outputs and k inputs is held as the 4-bit cache holds a
 * key (lt_kv4.h): codes in e2m1, one fp16 scale per 32 inputs,
 *
 *   codes   uint8 [n][k / 2], two a byte, the lower input in the low nibble
 *   scales  fp16 [n][k / 32]
 *
 * k is a multiple of 32, n and k are below 2^30, both start on 16 bytes. lt_w4_quantise makes them; codes and
 * scales from elsewhere serve as well, the scales finite, at least 0 and at most 10912 (then
 * code * scale does not overflow). lt_w4_quantise's have 9 significant bits and are multiples of 2^-23, which makes
 * code * scale an exact fp16 number. Products of other scales are rounded to fp16, to the nearest, ties to even: 2^-11
 * of a weight of 2^-14 or more, 2^-25 of smaller ones (half of the scale 2^-24 is 0).
 * What scales outside that range give is not specified, for their own outputs alone.
 *
 * Memory, streams and errors are as in lt_topk.h: DEVICE memory owned by the
 * caller, nothing allocated, nothing kept, the stream never synchronised,
 * programmatic dependent launch, argument errors returned synchronously with
 * nothing launched. Outputs must not overlap inputs.
 */
#ifndef LT_W4_H
#define LT_W4_H

#include "lt_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * lt_w4_quantise -- codes and scales of weights, with the scale and the rounding of
 * lt_kv4_store: a group with a NaN or an infinity has the scale NaN and codes of 0.
 *
 *   w  [n][k] of `dtype` (LT_DTYPE_F32, _BF16 or _F16), inputs contiguous, row_stride
 *      elements from one output to the next
 */
lt_status lt_w4_quantise(const void* w, int32_t dtype, int64_t n, int64_t k, int64_t row_stride,
                         void* codes, void* scales, void* stream);

/*
 * lt_w4_linear -- out[t][i] = sum_j x[t][j] code[i][j] scale[i][j / 32] (+ bias[i]).
 *
 *   x         [tokens][k] of `dtype` (LT_DTYPE_BF16 or _F16), at most 524280 tokens, inputs contiguous, the start
 *             16-byte aligned, x_stride (elements, a multiple of 8) from token to token
 *   bias      [n] of `dtype`, or NULL
 *   out       [tokens][n] of `dtype`, outputs contiguous, out_stride elements from token to token
 *   workspace lt_w4_workspace() bytes, 16-byte aligned (NULL if 0); no contents kept. Calls that
 *             may run at the same time need one each
 *
 * Arithmetic: the products run on the tensor cores in fp16 with fp32 sums. bf16 inputs are
 * scaled by a power of two for each token into fp16's range (exact down to 2^-28 of the
 * token's largest finite input); sums and bias are fp32, rounded once. Two calls with the same sizes give
 * the same bits. Infinities and NaN in a token's inputs reach that token's outputs alone, as in fp32
 * products.
 */
lt_status lt_w4_linear(const void* x, int32_t dtype, int64_t tokens, int64_t x_stride,
                       const void* codes, const void* scales, int64_t n, int64_t k, const void* bias,
                       void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes,
                       void* stream);

/* Bytes of workspace that lt_w4_linear needs for these sizes on the current device. */
lt_status lt_w4_workspace(int64_t tokens, int64_t n, int64_t k, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LT_W4_H */
