/*
 * lt_kv4.h -- C ABI of the 4-bit key/value cache (GB300, sm_103a): page tables
 * and slot maps, storing and loading rows, and attention over the cached
 * positions -- all of a request's, or those that lt_topk listed.
 *
 * The cache. A pool of pages; a page holds page_size consecutive positions of
 * one request for every kv head:
 *
 *   cache  uint8 [pages][kv_heads][page_size][row]
 *
 * page_size is a power of two from 1 to 1024, head_dim D is 64, 128 or 256, and a
 * row of lt_kv4_row_bytes(D) bytes holds one position's key and value:
 *
 *   D/2 bytes   key codes, two a byte, the lower channel in the low nibble
 *   D/2 bytes   value codes
 *   D/32 fp16   key scales, one per 32 channels
 *   D/32 fp16   value scales
 *   padding to a multiple of 16 bytes (8 bytes for D = 64, else none)
 *
 * A code is an e2m1 number (sign bit, then 0, 0.5, 1, 1.5, 2, 3, 4, 6). The scale
 * of a group is the smallest number at least amax / 6 that has 9 significant
 * bits and is a multiple of 2^-23, at most 10912; a channel is stored as its sign
 * (a zero's too) and the code nearest to |x| / scale (ties to the even code), so
 * it is off by at most one scale, and code * scale is an exact fp16 number. Finite
 * values beyond 6 * 10912 saturate. A group that holds a NaN or an infinity is stored as NaN.
 * Other scales (an infinity, a magnitude above 10912) are outside the format;
 * lt_kv4_store writes none.
 *
 * A slot is page * page_size + offset (int64): the place of one position. A
 * block table int32 [requests][table_width] names the pages of each request in
 * order: position p of request r lies on page table[r][p / page_size] at offset
 * p % page_size.
 *
 * Memory, streams and errors are as in lt_topk.h: DEVICE memory owned by the
 * caller, nothing allocated, nothing kept, the stream never synchronised,
 * programmatic dependent launch, argument errors returned synchronously with
 * nothing launched. Outputs must not overlap inputs.
 */
#ifndef LT_KV4_H
#define LT_KV4_H

#include "lt_topk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of 16-bit floats, for the calls of this header. */
#define LT_DTYPE_F16 2

#define LT_KV4_GROUP 32
#define LT_KV4_MAX_PAGE 1024

/* Bytes of a cache row: 80, 144 and 288 for D = 64, 128 and 256; 0 for another D. */
int32_t lt_kv4_row_bytes(int32_t head_dim);

/*
 * lt_page_release -- gives the pages of ended requests back.
 *
 * The pages of every request r with finished[r] != 0, table[r][0 .. ceil(lengths[r] / page_size)), go
 * on top of the stack of free pages, in request and then table order:
 * free_pages[num_free ..]. Cells below 0 hold no page and are passed over (a page
 * dropped behind a window, say, whose cell was set to -1). out_num_free is the
 * new height, out_lengths[r] is 0 for those requests and lengths[r] for the others.
 *
 *   lengths       int32 [requests]; clamped to [0, table_width * page_size]
 *   finished      uint8 [requests]
 *   block_table   int32 [requests][table_width], read only
 *   free_pages    int32 [free_capacity], written from num_free on; pages past
 *                 its capacity are dropped
 *   num_free      int32 [1]
 */
lt_status lt_page_release(const int32_t* lengths, const uint8_t* finished, int32_t requests,
                          const int32_t* block_table, int32_t table_width, int32_t* free_pages,
                          int32_t free_capacity, const int32_t* num_free, int32_t page_size,
                          int32_t* out_lengths, int32_t* out_num_free, void* stream);

/*
 * lt_page_extend -- places the new tokens of a step: pages, slots, positions.
 *
 * Request r grows from lengths[r] by new_tokens[r] positions (negative: none).
 * The pages that it lacks are taken from the top of the stack of free pages,
 * request by request, and written into its row of the block table. The first
 * request that does not fit -- more pages than are free, more tokens than
 * max_tokens in all, or a table row too short -- ends the step: it and every
 * request after it get nothing (out_lengths[r] == lengths[r], no starts of
 * their own), so what was placed is a prefix of the requests.
 *
 *   out_slots      int64 [max_tokens]: the slot of each new token, in request
 *                  order; -1 past the last (or where the table held no page)
 *   out_positions  int32 [max_tokens]: its position in its request; -1 past the last
 *   out_starts     int32 [requests + 1]: the first new token of each request
 *   out_lengths    int32 [requests]
 *   out_num_free   int32 [1]: the height of the stack that is left
 *   block_table    int32 [requests][table_width]; only fresh entries are written
 */
lt_status lt_page_extend(const int32_t* lengths, const int32_t* new_tokens, int32_t requests,
                         int32_t* block_table, int32_t table_width, const int32_t* free_pages,
                         int32_t free_capacity, const int32_t* num_free, int32_t page_size,
                         int32_t max_tokens, int64_t* out_slots, int32_t* out_positions,
                         int32_t* out_starts, int32_t* out_lengths, int32_t* out_num_free,
                         void* stream);

/*
 * lt_kv4_store -- quantises keys and values into their slots.
 *
 *   k, v      [tokens][kv_heads][head_dim] of `dtype` (LT_DTYPE_F32, _BF16 or
 *             _F16), channels contiguous; the strides of tokens and heads are
 *             in elements
 *   slots     int64 [tokens]; a slot outside [0, pages * page_size) is skipped.
 *             Two tokens with the same slot leave either one
 */
lt_status lt_kv4_store(const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t kv_heads,
                       int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride,
                       int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                       void* cache, int64_t pages, int32_t page_size, void* stream);

/*
 * lt_kv4_append -- turns queries and keys by their positions and stores keys and
 * values: the way of a step's new tokens into the cache.
 *
 * Of the first rotary_dim channels of a head, pair i (channels i and i + rotary_dim / 2;
 * 2 i and 2 i + 1 where `interleaved` is not 0) turns by the angle whose cosine and sine the
 * tables hold for the token's position:
 *
 *   a' = a c - b s,   b' = b c + a s
 *
 * each product and each sum rounded to 32 bits. The other channels stay. Queries are
 * rounded to their type; keys are quantised from the 32-bit numbers, values as
 * lt_kv4_store does.
 *
 *   q           [tokens][q_heads][head_dim], or NULL with q_heads 0
 *   k, v        [tokens][kv_heads][head_dim]; all of `dtype` (LT_DTYPE_F32, _BF16 or _F16),
 *               channels contiguous, the strides of tokens and heads in elements
 *   cos_table,  float [max_positions][rotary_dim / 2], 16-byte aligned; rotary_dim is a
 *   sin_table   multiple of 16, at most head_dim
 *   positions   int32 [tokens]: where each token lies in its request. A token whose position is
 *               outside [0, max_positions) (-1, past a step's last token) is passed over:
 *               nothing is stored and its row of out_q stays as it was
 *   slots       int64 [tokens]; a slot outside [0, pages * page_size) stores nothing (its
 *               query is turned all the same). No two tokens have the same slot: what it
 *               holds then is not specified
 *   out_q       like q, strides of its own; it may be q itself (with q's strides), else
 *               it overlaps nothing
 */
lt_status lt_kv4_append(const void* q, const void* k, const void* v, int32_t dtype, int64_t tokens,
                        int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                        int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t v_token_stride, int64_t v_head_stride, const float* cos_table,
                        const float* sin_table, int32_t max_positions, int32_t rotary_dim,
                        int32_t interleaved, const int32_t* positions, const int64_t* slots, void* cache,
                        int64_t pages, int32_t page_size, void* out_q, int64_t out_token_stride,
                        int64_t out_head_stride, void* stream);

/*
 * lt_kv4_load -- the numbers that the slots stand for: k, v
 * [tokens][kv_heads][head_dim] of `dtype`, contiguous; exact in fp16 and fp32,
 * rounded to nearest even in bf16; zeros for a slot outside the cache.
 */
lt_status lt_kv4_load(const void* cache, int64_t pages, int32_t page_size, const int64_t* slots,
                      int64_t tokens, int32_t kv_heads, int32_t head_dim, void* k, void* v,
                      int32_t dtype, void* stream);

/*
 * lt_kv4_attention -- attention of new tokens over the cache.
 *
 * Request r has lengths[r] positions in the cache (at most its table row's, and 2^31 - 1024); its queries are the rows
 * q[starts[r] .. starts[r + 1]), the last of those positions: query i of n lies
 * at position lengths[r] - n + i. Query head h reads kv head
 * h / (q_heads / kv_heads). For each query and head, over its visible positions:
 *
 *   s_p = scale * sum_c q[c] k_p[c],  out = sum_p exp(s_p) v_p / sum_p exp(s_p),
 *   lse = ln sum_p exp(s_p)
 *
 * Visible are the positions up to the query's own (causal); with window > 0 only
 * the last `window` of them. With `positions`, visible are the listed positions
 * inside [0, lengths[r]) instead -- the list says what a query may see; other
 * entries (-1 pads) are ignored, a repeated one counts as often as it stands
 * there -- and window must be 0. A query that sees nothing gets zeros and
 * lse = -inf; so does position data on a page outside [0, pages), which nothing
 * sees. What is not visible has no effect, whatever bytes it holds. Where a query
 * sees a group whose scale is outside the format, its results there (from a key, its
 * whole row) are NaN, infinite or finite: not specified.
 *
 * Arithmetic: the products run on the tensor cores in fp16 with fp32 sums. A
 * stored value is an exact fp16 number; a bf16 query is scaled by a power of two
 * into fp16's range (exact down to 2^-28 of its row's largest); the weights
 * exp(s - max) are rounded to fp16 for the second product; maximum, sums and
 * output are fp32, rounded once.
 *
 *   q          [tokens][q_heads][head_dim], bf16 or fp16 (dtype), channels
 *              contiguous, strides in elements (multiples of 8, the start
 *              16-byte aligned)
 *   starts     int32 [requests + 1], or NULL: one query a request (tokens == requests).
 *              starts[0] is 0; rows at or past starts[requests] are not touched
 *   max_new    at least the largest number of queries of a request (it sizes the
 *              launch; the queries past it are not computed); 1 with starts NULL
 *   positions  int32 [tokens][list_len] or NULL
 *   out        [tokens][q_heads][head_dim] of `dtype`, contiguous
 *   lse        float [tokens][q_heads] or NULL
 *   workspace  lt_kv4_workspace() bytes, 16-byte aligned (NULL if 0); no contents kept
 * q_heads is a multiple of kv_heads; head_dim 64, 128 or 256.
 */
lt_status lt_kv4_attention(const void* q, int32_t dtype, int64_t tokens, int32_t q_heads,
                           int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                           int64_t q_head_stride, const void* cache, int64_t pages, int32_t page_size,
                           const int32_t* block_table, int32_t table_width, const int32_t* lengths,
                           int32_t requests, const int32_t* starts, int32_t max_new,
                           const int32_t* positions, int32_t list_len, int32_t window, float scale,
                           void* out, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream);

/*
 * lt_kv4_attention_ex -- lt_kv4_attention with logits that are capped, lowered with the
 * distance, or seen through a prefix mask. With `own` a query's position and p a cached one,
 *
 *   s_p = scale * sum_c q[c] k_p[c]
 *   s_p = softcap * tanh(s_p / softcap)       with softcap > 0
 *   s_p = s_p - slopes[h] * |own - p|         with slopes
 *
 * and visible are the positions up to the query's own, and those below prefix[r], whichever query of
 * request r looks (a query that lies before the first position sees the prefix alone).
 *
 *   softcap   0 (none), or LT_KV4_MIN_CAP to LT_KV4_MAX_CAP. Beside what the logit before it is off
 *             by, a capped logit is off by at most 2^-21 of caps to 64, 2^-20 of itself with larger ones
 *   slopes    float [q_heads], finite, or NULL; magnitudes above 2^95 count as that (a logit then is finite
 *             whatever the distance); listed positions have distances, too
 *   prefix    int32 [requests] or NULL; below 0 counts as 0, past the request's length as
 *             that; NULL where window > 0 or positions are given
 * All else, the workspace among it, is lt_kv4_attention's.
 */
#define LT_KV4_MIN_CAP 0.0009765625f /* 2^-10 */
#define LT_KV4_MAX_CAP 1048576.0f    /* 2^20 */
lt_status lt_kv4_attention_ex(const void* q, int32_t dtype, int64_t tokens, int32_t q_heads,
                              int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                              int64_t q_head_stride, const void* cache, int64_t pages, int32_t page_size,
                              const int32_t* block_table, int32_t table_width, const int32_t* lengths,
                              int32_t requests, const int32_t* starts, int32_t max_new,
                              const int32_t* positions, int32_t list_len, int32_t window, float scale,
                              float softcap, const float* slopes, const int32_t* prefix,
                              void* out, float* lse, void* workspace, int64_t workspace_bytes,
                              void* stream);

/* Bytes of workspace that lt_kv4_attention needs for these sizes on the current
 * device: 0 where a request's parts are joined within the launch, else room for the
 * parts of the requests that are cut, each with the fp32 outputs of up to max_new
 * queries. How many parts there can be goes by the device's SMs and the query rows,
 * and beyond that not by the requests. list_len 0: without positions (else window
 * is 0); positions = table_width * page_size. */
lt_status lt_kv4_workspace(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                           int32_t requests, int32_t max_new, int32_t list_len, int64_t positions,
                           int32_t window, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LT_KV4_H */
