// lt_kv4_attention.cu -- lt_kv4_attention: the choice of kernel and launch, and the join of the
// parts of a split request. The kernels are in lt_kv4_rows.cuh (few query rows a request, listed
// positions) and lt_kv4_prefill.cuh (many query rows).

#include <mutex>

#include "lt_kv4.cuh"
#include "lt_kv4_attention.cuh"
#include "lt_kv4_prefill.h"
#include "lt_kv4_rows.h"

namespace {

using namespace lt::kv4;

// Joins the parts of a (query, head): out = sum_i 2^(e_i - top) o_i / sum_i 2^(e_i - top), e_i
// the parts' logarithms. Eight warps share the parts, in one fixed order whatever the timing.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttentionParams p) {
  constexpr int kVec = D / 32;
  __shared__ float o_of[kJoinThreads / 32][D];
  __shared__ float sum_of[kJoinThreads / 32], top_of[kJoinThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  dependency_wait();
  const int q_heads = p.heads * p.group;
  const int64_t token = blockIdx.x / q_heads;
  const int qh = (int)(blockIdx.x % q_heads), head = qh / p.group;
  const int request = owner_of_token(p, (int)token);
  if (request < 0) return;
  const int2 pl = p.plan[request];
  const int n = pl.y;
  const Request rq = request_of(p, request);
  const int64_t nth = token - rq.first;
  if (nth >= rq.computed) return;
  if (n <= 1) return;  // written whole
  const int64_t step = (int64_t)p.heads * p.part_rows;
  const int64_t first = pl.x * step + (int64_t)head * p.part_rows + nth * p.group + qh % p.group;

  float top = -INFINITY;
  bool bad = false;
  for (int i = tid; i < n; i += kJoinThreads) {
    const float e = p.part_lse[first + i * step];
    top = fmaxf(top, e);
    bad = bad || e != e;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  if (lane == 0) top_of[warp] = top;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, top_of[w]);

  float o[kVec] = {}, sum = 0.0f;
#pragma unroll 4
  for (int i = warp; i < n; i += kJoinThreads / 32) {
    const float e = p.part_lse[first + i * step];
    const float* from = p.part_o + (first + i * step) * D + lane * kVec;
    float x[kVec];
#pragma unroll
    for (int k = 0; k < kVec; k += 2) *reinterpret_cast<float2*>(x + k) = *reinterpret_cast<const float2*>(from + k);
    const float w = e == -INFINITY ? 0.0f : exp2_fast(e - top);
    sum += w;
#pragma unroll
    for (int k = 0; k < kVec; ++k) o[k] += e == -INFINITY ? 0.0f : w * x[k];
  }
#pragma unroll
  for (int k = 0; k < kVec; ++k) o_of[warp][lane * kVec + k] = o[k];
  if (lane == 0) sum_of[warp] = sum;
  __syncthreads();
  dependents_launch();
  float all = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) all += sum_of[w];
  const float inv = all == 0.0f ? 0.0f : 1.0f / all;
  const int64_t out_row = token * q_heads + qh;
  if (tid < D / 4) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(&o_of[w][tid * 4]);
      y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
    }
    y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
    if (bad) y = make_float4(NAN, NAN, NAN, NAN);
    store4(p, out_row * D + tid * 4, y);
  }
  if (p.lse != nullptr && tid == 0)
    p.lse[out_row] = bad ? NAN : all == 0.0f ? -INFINITY : (top + __log2f(all)) * 0.6931471805599453f;
}

// ---- host side

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_smem_set[kMaxDevices][3][4][2][2];  // by head size, row tiles (3: many rows), listed, shaped

// The launch for these sizes: row tiles, parts and workspace.
struct Plan {
  bool prefill;        // the kernel for many query rows
  int nt, row_tiles;
  int64_t part_rows;   // query rows of a part
  int parts;           // > 0: every request (list) in that many parts, a cluster; 0: chunks of like work
  int target;          // chunks wanted over all requests
  int min_chunk;
  int64_t flats;       // chunks, or requests (lists) at most
  bool join;           // chunks are joined by a second launch
  int64_t plan_bytes, lse_bytes, o_bytes;
  int64_t bytes() const { return join ? plan_bytes + lse_bytes + o_bytes : 0; }
};

constexpr int kMinChunk = 256;
constexpr int kPrefillMinChunk = 512;
// Query rows a kv head from which the kernel for many rows is taken, each side's us with 8 kv heads of D:
//   1 request of 8192 positions, D = 128: 26 there, 25 here with 16 rows, 28 and 37 with 32, 36 and 74 with 256
//   16 requests of 4096, D = 128: 81 and 74 with 32 rows, 87 and 119 with 64; D = 64: 68 and 59, 73 and 57
//   D = 256, 4 kv heads: 1 request of 8192 positions 32 and 35 with 32 rows; 4 of them 48 and 39, with 64 rows 49 and
//   70; 64 requests of 2048 94 and 66 with 20 rows, 101 and 117 with 40
// so from two row tiles of this kernel on (D = 64: from three), and with few CTAs from 17 rows (D = 256, whose
// tiles have fewer rows: with very few). The rows are those of max_new queries, for all requests of the call:
// where one has many queries and others one, these are computed there, too (not measured).
int prefill_from(int d, int64_t units, int sms) {
  return units * (d == 256 ? 16 : 4) <= sms ? 17 : d == 64 ? 65 : 33;
}
constexpr int kPartPositions = 2048;  // positions of a part up to which requests are cut into equal numbers of parts

// rows: the most query rows of a request
Plan finish_plan(Plan a, int heads, int d, int requests, int64_t rows) {
  // A chunk is at least total / target long, so the requests have fewer than target + requests. Parts are kept for
  // the requests that have several chunks alone: each of those is longer than a chunk, so they are fewer than
  // target, and have fewer than 2 target chunks.
  if (a.flats == 0) a.flats = a.target == 1 ? requests : a.target + (int64_t)requests;
  a.join = a.parts == 0 && a.target > 1;
  const int64_t parts = (a.target < requests ? (int64_t)a.target : (int64_t)requests) + a.target - 1;
  a.part_rows = rows;
  a.plan_bytes = ((int64_t)requests * 8 + 15) / 16 * 16;
  a.lse_bytes = (parts * heads * rows * 4 + 15) / 16 * 16;
  a.o_bytes = parts * heads * rows * d * 4;
  return a;
}

// positions: the most that a request can have by its row of the table
Plan make_plan(int sms, int64_t tokens, int heads, int group, int d, int requests, int max_new, int list_len,
               int64_t positions, int window) {
  Plan a = {};
  const int64_t rows = (int64_t)(list_len > 0 ? 1 : max_new) * group;
  const int64_t part_rows = (max_new < tokens ? (int64_t)max_new : tokens) * group;
  a.prefill = list_len == 0 && rows >= prefill_from(d, (int64_t)requests * heads, sms);
  if (a.prefill) {
    a.row_tiles = (int)((rows + prefill_rows(d) - 1) / prefill_rows(d));
    a.min_chunk = kPrefillMinChunk;
    // one CTA an SM: chunks only where one request's row tiles alone do not fill the SMs (their joins cost more
    // than an uneven second wave: 256 row tiles of 16384 positions take 511 us whole, 690 us in halves). With
    // several requests the chunks are cut from all their positions together, so the long ones alone are cut.
    const int64_t units = (int64_t)heads * a.row_tiles;
    a.target = (int)((sms + units - 1) / units);
    return finish_plan(a, heads, d, requests, part_rows);
  }
  const int most = d == 256 ? 2 : 4;
  a.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : most;
  if (a.nt > most) a.nt = most;
  a.row_tiles = (int)((rows + a.nt * 8 - 1) / (a.nt * 8));
  a.min_chunk = kMinChunk;
  const int slots = sms * rows_kernel_of<false>(d, a.nt, list_len > 0).per_sm;
  const int64_t units = (int64_t)heads * a.row_tiles;
  // what one query (a request's queries) can see at most: lengths are known on the device alone, so a table wider
  // than the requests counts as if they filled it
  int64_t seen = list_len > 0 ? list_len : positions;
  if (list_len == 0 && window > 0 && (int64_t)window + max_new + kTile < seen) seen = (int64_t)window + max_new + kTile;
  const int64_t whole = (list_len > 0 ? tokens : (int64_t)requests) * units;
  // parts while the CTAs do not fill the slots and a part is at least a tile for every warp (filling them twice
  // costs the drafted step 55 us instead of 46)
  int parts = 1;
  while (parts < kMaxParts && whole * parts < slots && seen > (int64_t)parts * kTile * kWarps) parts *= 2;
  // Requests stay whole, too, where they are so many that the hardware evens them out and none can be long
  // (us whole against chunks, 8 kv heads of 128: 256 requests to 8192 positions 287 and 303, 1024
  // 956 and 1083; but 128 to 8192 176 and 168, 128 to 32768 638 and 498, 512 of 4 heads 1051 and 998).
  const bool whole_ones = parts == 1 && ((whole >= 3 * slots && seen <= 8192) || (whole >= 8 * slots && seen <= 32768));
  if (list_len > 0 || whole_ones || seen <= (int64_t)parts * kPartPositions) {
    a.parts = parts;
    a.flats = list_len > 0 ? tokens : requests;
    return finish_plan(a, heads, d, requests, part_rows);
  }
  // Several chunks a slot where requests differ in length, so that the last ones to end are short (64 ragged
  // requests: 324, 279, 271, 269 us with 1, 2, 3, 4); one request's chunks are alike, and one
  // wave of them has the fewest starts and joins (262144 positions at D = 256: 82 us, 96 with 2).
  const int64_t target = ((int64_t)slots * (requests == 1 ? 1 : 4) + units - 1) / units;
  a.target = (int)(target < 1 ? 1 : target);
  return finish_plan(a, heads, d, requests, part_rows);
}

lt_status device_of(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return LT_ERR_CUDA;
  if (*dev < 0 || *dev >= kMaxDevices) return LT_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[*dev] == 0 && cudaDeviceGetAttribute(&g_sms[*dev], cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return LT_ERR_CUDA;
  *sms = g_sms[*dev];
  return LT_OK;
}

lt_status check_sizes(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t requests,
                      int32_t max_new, int32_t list_len) {
  if (tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || head_dim < 1 || requests < 0 ||
      max_new < 1 || list_len < 0)
    return LT_ERR_INVALID_ARG;
  if (lt_kv4_row_bytes(head_dim) == 0 || tokens > INT32_MAX) return LT_ERR_UNSUPPORTED;
  return LT_OK;
}

}  // namespace

extern "C" {

lt_status lt_kv4_workspace(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                           int32_t requests, int32_t max_new, int32_t list_len, int64_t positions,
                           int32_t window, int64_t* bytes) {
  if (bytes == nullptr) return LT_ERR_INVALID_ARG;
  lt_status st = check_sizes(tokens, q_heads, kv_heads, head_dim, requests, max_new, list_len);
  if (st == LT_OK && (positions < 0 || window < 0)) st = LT_ERR_INVALID_ARG;
  if (st != LT_OK) return st;
  *bytes = 0;
  if (tokens == 0 || requests == 0) return LT_OK;
  int dev = 0, sms = 0;
  st = device_of(&dev, &sms);
  if (st != LT_OK) return st;
  *bytes = make_plan(sms, tokens, kv_heads, q_heads / kv_heads, head_dim, requests, max_new, list_len,
                     positions, window >= positions ? 0 : window).bytes();
  return LT_OK;
}

lt_status lt_kv4_attention(const void* q, int32_t dtype, int64_t tokens, int32_t q_heads,
                           int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                           int64_t q_head_stride, const void* cache, int64_t pages, int32_t page_size,
                           const int32_t* block_table, int32_t table_width, const int32_t* lengths,
                           int32_t requests, const int32_t* starts, int32_t max_new,
                           const int32_t* positions, int32_t list_len, int32_t window, float scale,
                           void* out, float* lse, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  return lt_kv4_attention_ex(q, dtype, tokens, q_heads, kv_heads, head_dim, q_token_stride, q_head_stride, cache, pages,
                             page_size, block_table, table_width, lengths, requests, starts, max_new, positions, list_len,
                             window, scale, 0.0f, nullptr, nullptr, out, lse, workspace, workspace_bytes, stream);
}

lt_status lt_kv4_attention_ex(const void* q, int32_t dtype, int64_t tokens, int32_t q_heads,
                              int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                              int64_t q_head_stride, const void* cache, int64_t pages, int32_t page_size,
                              const int32_t* block_table, int32_t table_width, const int32_t* lengths,
                              int32_t requests, const int32_t* starts, int32_t max_new,
                              const int32_t* positions, int32_t list_len, int32_t window, float scale,
                              float softcap, const float* slopes, const int32_t* prefix,
                              void* out, float* lse, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  lt_status st = check_sizes(tokens, q_heads, kv_heads, head_dim, requests, max_new, list_len);
  if (st == LT_ERR_INVALID_ARG) return st;
  const int shift = page_shift(page_size);
  if (dtype != LT_DTYPE_BF16 && dtype != LT_DTYPE_F16) return LT_ERR_INVALID_ARG;
  if (shift < 0 || pages < 0 || table_width < 1 || window < 0 || !(scale == scale) || scale - scale != 0.0f)
    return LT_ERR_INVALID_ARG;
  if (starts == nullptr && (tokens != requests || max_new != 1)) return LT_ERR_INVALID_ARG;
  if (positions != nullptr && window != 0) return LT_ERR_INVALID_ARG;
  if (prefix != nullptr && (window != 0 || positions != nullptr)) return LT_ERR_INVALID_ARG;
  if (!(softcap >= 0.0f) || softcap - softcap != 0.0f) return LT_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(slopes) % 4 || reinterpret_cast<uintptr_t>(prefix) % 4) return LT_ERR_INVALID_ARG;
  if (positions == nullptr && list_len != 0) return LT_ERR_INVALID_ARG;
  if (positions != nullptr && list_len == 0) return LT_ERR_INVALID_ARG;
  if (tokens > 0 && requests > 0) {
    if (q == nullptr || out == nullptr || block_table == nullptr || lengths == nullptr ||
        (cache == nullptr && pages > 0))
      return LT_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(q) % 16 || q_token_stride % 8 || q_head_stride % 8 ||
        reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(out) % 16)
      return LT_ERR_INVALID_ARG;
  }
  if (st != LT_OK || pages > INT32_MAX) return LT_ERR_UNSUPPORTED;
  if (softcap != 0.0f && (softcap < LT_KV4_MIN_CAP || softcap > LT_KV4_MAX_CAP)) return LT_ERR_UNSUPPORTED;
  if (tokens == 0 || requests == 0) return LT_OK;
  // a window as wide as the table holds every position; the kernels' sums of
  // positions, queries and window stay within 32 bits
  if (((int64_t)table_width << shift) <= window) window = 0;
  if ((int64_t)window + tokens >= INT32_MAX) return LT_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  st = device_of(&dev, &sms);
  if (st != LT_OK) return st;
  const int group = q_heads / kv_heads;
  const Plan plan = make_plan(sms, tokens, kv_heads, group, head_dim, requests, max_new, list_len,
                              (int64_t)table_width << shift, window);
  if (plan.join && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < plan.bytes()))
    return LT_ERR_INVALID_ARG;
  const int64_t grid = plan.flats * kv_heads * plan.row_tiles * (plan.parts > 1 ? plan.parts : 1), joins = tokens * q_heads;
  if (grid > INT32_MAX || joins > INT32_MAX) return LT_ERR_UNSUPPORTED;

  AttentionParams p = {};
  p.q = q;
  p.cache = static_cast<const uint8_t*>(cache);
  p.table = block_table;
  p.lengths = lengths;
  p.starts = starts;
  p.positions = positions;
  p.out = out;
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (plan.join) {
    p.plan = reinterpret_cast<int2*>(ws);
    p.part_lse = reinterpret_cast<float*>(ws + plan.plan_bytes);
    p.part_o = reinterpret_cast<float*>(ws + plan.plan_bytes + plan.lse_bytes);
  }
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.pages = (int32_t)pages;
  p.tokens = (int32_t)tokens;
  p.requests = requests;
  p.width = table_width;
  p.heads = kv_heads;
  p.group = group;
  p.shift = shift;
  p.list_len = list_len;
  p.window = window;
  p.parts = plan.parts;
  p.target = plan.target;
  p.min_chunk = plan.min_chunk;
  p.row_tiles = plan.row_tiles;
  p.max_new = max_new;
  p.part_rows = (int32_t)plan.part_rows;
  p.align = plan.prefill ? 128 : kTile;
  p.bf16 = dtype == LT_DTYPE_BF16;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.slopes = slopes;
  p.prefix = prefix;
  p.cap = softcap * 1.4426950408889634f;
  p.two_over_cap = softcap > 0.0f ? 2.0f / softcap : 0.0f;
  p.one_over_cap = softcap > 0.0f ? 1.0f / p.cap : 0.0f;
  p.wide_cap = softcap > 64.0f;
  const bool shaped = softcap > 0.0f || slopes != nullptr || prefix != nullptr;

  const bool list = list_len > 0;
  RowsKernel k = {};
  if (plan.prefill)
    k.func = shaped ? prefill_kernel_ptr<true>(head_dim, &k.smem) : prefill_kernel_ptr<false>(head_dim, &k.smem);
  else
    k = shaped ? rows_kernel_of<true>(head_dim, plan.nt, list) : rows_kernel_of<false>(head_dim, plan.nt, list);
  {
    std::lock_guard<std::mutex> lk(g_mu);
    bool& set = g_smem_set[dev][head_dim / 128][plan.prefill ? 3 : plan.nt / 2][list][shaped];
    if (!set) {
      if (cudaFuncSetAttribute(k.func, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) != cudaSuccess)
        return LT_ERR_CUDA;
      set = true;
    }
  }
  st = launch(k.func, dim3((unsigned)grid), plan.prefill ? kPrefillThreads : kThreads, (unsigned)k.smem, &p, stream,
              plan.parts > 1 ? plan.parts : 1);
  if (st != LT_OK || !plan.join) return st;
  if (lt::take_injected_failure()) return LT_ERR_CUDA;
  const void* func = head_dim == 64    ? reinterpret_cast<const void*>(&join_kernel<64>)
                     : head_dim == 128 ? reinterpret_cast<const void*>(&join_kernel<128>)
                                       : reinterpret_cast<const void*>(&join_kernel<256>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)joins);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* a[] = {&p};
  return cudaLaunchKernelExC(&cfg, func, a) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}

}  // extern "C"
