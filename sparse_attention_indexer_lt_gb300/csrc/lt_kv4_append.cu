// lt_kv4_append.cu -- the position rotation of queries and keys on the way into the
// 4-bit cache (lt_kv4_append).
//
// A head's channel pairs (a, b) turn by the angle of (position, pair): a c - b s and
// b c + a s, products and sums each rounded to 32 bits (no fused steps, so that what is
// stored is the same wherever it is computed). Queries are rounded to their type; keys go on
// to the quantiser as they are, in 32 bits; values pass it by unturned.
//
// A thread has eight channels of one token and walks over heads of it, so that its
// cosines and sines stay in registers: for one head they would be four times the bytes of the
// channels. D / 8 threads make a head; a pair's other half lies with a thread R / 16
// lanes on (two shuffled words a channel pair), or in the same thread where neighbours are paired.
// A CTA's heads are of one kind, queries, keys or values (blockIdx.y), so a warp does not diverge.
//
// What bounds it: issue (68% of the schedulers' rate) beside memory: 8191 tokens of 32 query and 8 kv heads of 128
// (177 MB, 26 us at the copy rate) take 34 us, 45 with the load that reads the keys and values back (11). It was
// 46: the channels go by no position, so they are asked for before it, and the next heads' before these are worked on
// (44 to 34 us); products of pairs and a quantiser without comparisons (33 to 27 million warp instructions).

#include "lt_kv4.cuh"
#include "lt_kv4_quantise.cuh"

namespace {

using lt::kv4::Eight;
using lt::kv4::row_bytes;

constexpr int kThreads = 256;
constexpr int kAheadMost = 4;  // heads whose channels a thread asks for before it turns the first; half of it with 32-bit ones

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  void* out_q;
  const float* cos;
  const float* sin;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* cache;
  int64_t tokens, slot_end;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;
  int32_t q_heads, kv_heads, shift, max_pos, half;  // half: channel pairs that turn
  int32_t per;                                      // heads of a CTA
  float minus_zero;
  int32_t q_parts, kv_parts;                        // CTAs that share a token's query heads, its keys
};

// Eight channels: as they came (16-bit types: pairs), and as fp32.
template <class S>
struct Wide {
  uint32_t w[sizeof(S) == 4 ? 8 : 4];
  float x[8];
  // (plain loads: the queries may be turned in place)
  __device__ __forceinline__ void load(const S* p, bool wide) {
    if constexpr (sizeof(S) == 4) {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(p);
      if (wide) {
        const uint4 a = *reinterpret_cast<const uint4*>(u), b = *(reinterpret_cast<const uint4*>(u) + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = u[i];
      }
    } else {
      if (wide) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
      } else {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = u[2 * i] | ((uint32_t)u[2 * i + 1] << 16);
      }
    }
  }
  static __device__ __forceinline__ float number(const uint32_t* w, int i) {
    if constexpr (sizeof(S) == 4)
      return __uint_as_float(w[i]);
    else
      return Eight<S>::number(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
  }
  __device__ __forceinline__ void widen() {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = number(w, i);
  }
  __device__ __forceinline__ void store(S* p, bool wide) const {
    if constexpr (sizeof(S) == 4) {
      if (wide) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i];
      }
    } else {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<S, __half>::value)
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        else
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
      }
      if (wide) {
        *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        uint16_t* u = reinterpret_cast<uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = (uint16_t)(i & 1 ? o[i / 2] >> 16 : o[i / 2]);
      }
    }
  }
};

// (x0, x1) = (x0 c0 + y0 s0, x1 c1 + y1 s1), every product and sum rounded by itself. Products and sums of pairs come
// out of the compiler fused, also where each says how it rounds; so a product adds `zero`, -0.0f, of which only the
// host knows that it leaves it as it is.
__device__ __forceinline__ void turn2(float& x0, float& x1, float c0, float c1, float y0, float y1, float s0, float s1, float zero) {
  asm("{\n .reg .b64 x, c, y, s, z;\n mov.b64 x, {%0, %1};\n mov.b64 c, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 s, {%6, %7};\n mov.b64 z, {%8, %8};\n"
      " fma.rn.f32x2 x, x, c, z;\n fma.rn.f32x2 y, y, s, z;\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1) : "f"(c0), "f"(c1), "f"(y0), "f"(y1), "f"(s0), "f"(s1), "f"(zero));
}

// A thread's cosines and sines, and its channels' turn.
template <bool kPairs>
struct Turn {
  float c[kPairs ? 4 : 8], s[kPairs ? 4 : 8];  // the sines with the sign of the other half's product
  int other;                                   // lane of the other half
  bool turns;
  __device__ __forceinline__ void load(const AppendParams& p, int pos, int first, bool there) {
    const int pairs = kPairs ? first / 2 : first % p.half;
    turns = there && first < 2 * p.half;
    const int lane = threadIdx.x & 31;
    other = lane;
    float sign = 1.0f;
    if constexpr (!kPairs) {
      // (a lane that does not turn is nobody's other half)
      if (first < 2 * p.half) other = first < p.half ? lane + p.half / 8 : lane - p.half / 8;
      if (first < p.half) sign = -1.0f;
    }
    const int64_t at = turns ? (int64_t)pos * p.half + pairs : 0;
#pragma unroll
    for (int i = 0; i < (kPairs ? 4 : 8); i += 4) {
      float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (turns) {
        a = __ldg(reinterpret_cast<const float4*>(p.cos + at + i));
        b = __ldg(reinterpret_cast<const float4*>(p.sin + at + i));
      }
      c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
      s[i] = sign * b.x, s[i + 1] = sign * b.y, s[i + 2] = sign * b.z, s[i + 3] = sign * b.w;
    }
  }
  // All lanes of the warp call this. a c - b s is a c + b (-s), rounded alike; two at a time.
  template <class S>
  __device__ __forceinline__ void apply(Wide<S>& v, float zero) const {
    float(&x)[8] = v.x;
    v.widen();
    if constexpr (kPairs) {
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn2(x[2 * i], x[2 * i + 1], c[i], c[i], x[2 * i + 1], x[2 * i], -s[i], s[i], zero);
      }
    } else {
      constexpr int kWords = sizeof(S) == 4 ? 8 : 4;
      uint32_t w[kWords];
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __shfl_sync(~0u, v.w[i], other);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = Wide<S>::number(w, i);
      if (turns) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) turn2(x[i], x[i + 1], c[i], c[i + 1], y[i], y[i + 1], s[i], s[i + 1], zero);
      }
    }
  }
};

// The codes and, from the first of four lanes, the scale of a group. All lanes of the warp call this.
template <class E>
__device__ __forceinline__ void put_group(const E& x, uint8_t* row, int d, int at_byte, int group, bool there) {
  uint32_t largest = x.largest();
  largest = max(largest, __shfl_xor_sync(~0u, largest, 1));
  largest = max(largest, __shfl_xor_sync(~0u, largest, 2));
  if (!there) return;
  const bool bad = !E::finite(largest);
  const float s = bad ? 0.0f : E::scale(E::number(largest));
  *reinterpret_cast<uint32_t*>(row + at_byte) = bad ? 0u : x.codes(s);
  if ((threadIdx.x & 3) == 0)
    *reinterpret_cast<uint16_t*>(row + d + group * 2) = bad ? (uint16_t)0x7FFF : __half_as_ushort(__float2half_rn(s));
}

template <class S, int D, bool kPairs>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(AppendParams p, int wide) {
  constexpr int kLanes = D / 8;
  constexpr int kRow = row_bytes(D);
  constexpr int kAhead = sizeof(S) == 4 ? kAheadMost / 2 : kAheadMost;
  const int lane = threadIdx.x % kLanes, first = lane * 8;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int part = blockIdx.y;
  const int64_t tc = t < p.tokens ? t : 0;  // (a thread without a token reads the first one's channels in vain)
  const bool is_q = part < p.q_parts, is_v = part >= p.q_parts + p.kv_parts;
  const int from = (part - (is_q ? 0 : p.q_parts) - (is_v ? p.kv_parts : 0)) * p.per, to = min(from + p.per, is_q ? p.q_heads : p.kv_heads);
  const S* src = static_cast<const S*>(is_q ? p.q : is_v ? p.v : p.k) + tc * (is_q ? p.q_token : is_v ? p.v_token : p.k_token) + first;
  const int64_t step = is_q ? p.q_head : is_v ? p.v_head : p.k_head;
  const bool whole = wide >> (is_q ? 0 : is_v ? 3 : 2) & 1;
  lt::kv4::dependency_wait();
  // The channels go by no position: the first heads' are asked for before it, and the next ones' before these are worked on.
  Wide<S> x[kAhead], later[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (from + j < to) x[j].load(src + (from + j) * step, whole);
  int pos = -1;
  int64_t slot = -1;
  if (t < p.tokens) {
    pos = __ldg(p.positions + t);
    slot = __ldg(p.slots + t);
  }
  const bool there = pos >= 0 && pos < p.max_pos, kept = there && slot >= 0 && slot < p.slot_end;
  Turn<kPairs> turn;
  if (!is_v) turn.load(p, pos, first, there);
  uint8_t* page = p.cache + ((((kept ? slot : 0) >> p.shift) * p.kv_heads << p.shift) + ((kept ? slot : 0) & ((1 << p.shift) - 1))) * (int64_t)kRow;
  const int64_t head_bytes = (int64_t)kRow << p.shift;
#pragma unroll 1
  for (int h0 = from; h0 < to; h0 += kAhead) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (h0 + kAhead + j < to) later[j].load(src + (h0 + kAhead + j) * step, whole);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (h0 + j >= to) break;  // (the same for the whole CTA)
      uint8_t* row = page + (h0 + j) * head_bytes;
      if (is_q) {
        turn.apply(x[j], p.minus_zero);
        if (there) x[j].store(static_cast<S*>(p.out_q) + t * p.out_token + (h0 + j) * p.out_head + first, wide & 2);
      } else if (is_v) {
        Eight<S> e;
        e.take(x[j].w);
        put_group(e, row, D, D / 2 + lane * 4, D / 32 + lane / 4, kept);
      } else {
        turn.apply(x[j], p.minus_zero);
        Eight<float> e;
#pragma unroll
        for (int i = 0; i < 8; ++i) e.x[i] = x[j].x[i];
        put_group(e, row, D, lane * 4, lane / 4, kept);
        if constexpr (kRow > D + D / 8) {
          if (lane == 0 && kept) *reinterpret_cast<uint2*>(row + D + D / 8) = make_uint2(0u, 0u);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < (int)(sizeof(x[j].w) / 4); ++i) x[j].w[i] = later[j].w[i];
  }
  lt::kv4::dependents_launch();
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <class S, int D>
const void* append_of(bool pairs) {
  return pairs ? reinterpret_cast<const void*>(&append_kernel<S, D, true>) : reinterpret_cast<const void*>(&append_kernel<S, D, false>);
}
template <class S>
const void* append_ptr(int d, bool pairs) {
  return d == 64 ? append_of<S, 64>(pairs) : d == 128 ? append_of<S, 128>(pairs) : append_of<S, 256>(pairs);
}

}  // namespace

extern "C" lt_status lt_kv4_append(const void* q, const void* k, const void* v, int32_t dtype, int64_t tokens,
                                   int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                                   int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                                   int64_t v_token_stride, int64_t v_head_stride, const float* cos_table,
                                   const float* sin_table, int32_t max_positions, int32_t rotary_dim,
                                   int32_t interleaved, const int32_t* positions, const int64_t* slots, void* cache,
                                   int64_t pages, int32_t page_size, void* out_q, int64_t out_token_stride,
                                   int64_t out_head_stride, void* stream) {
  if (tokens < 0 || q_heads < 0 || kv_heads < 1 || head_dim < 1 || pages < 0 || max_positions < 0 || rotary_dim < 0 ||
      lt::kv4::page_shift(page_size) < 0)
    return LT_ERR_INVALID_ARG;
  if (dtype != LT_DTYPE_F32 && dtype != LT_DTYPE_BF16 && dtype != LT_DTYPE_F16) return LT_ERR_INVALID_ARG;
  if (rotary_dim > head_dim || !aligned(cos_table, 16) || !aligned(sin_table, 16) || !aligned(cache, 16))
    return LT_ERR_INVALID_ARG;
  const uintptr_t size = dtype == LT_DTYPE_F32 ? 4 : 2;
  if (tokens > 0) {
    if (k == nullptr || v == nullptr || positions == nullptr || slots == nullptr || (cache == nullptr && pages > 0) ||
        (q_heads > 0 && (q == nullptr || out_q == nullptr)) ||
        (rotary_dim > 0 && max_positions > 0 && (cos_table == nullptr || sin_table == nullptr)))
      return LT_ERR_INVALID_ARG;
    if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(out_q, size)) return LT_ERR_INVALID_ARG;
    // turned in place, or elsewhere
    if (q_heads > 0 && out_q == q && (out_token_stride != q_token_stride || out_head_stride != q_head_stride))
      return LT_ERR_INVALID_ARG;
  }
  if (lt_kv4_row_bytes(head_dim) == 0 || rotary_dim % 16 != 0 || rotary_dim == 0 || kv_heads > 16384 || q_heads > 32768)
    return LT_ERR_UNSUPPORTED;
  if (tokens == 0 || max_positions == 0) return LT_OK;
  AppendParams p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.out_q = out_q;
  p.cos = cos_table;
  p.sin = sin_table;
  p.positions = positions;
  p.slots = slots;
  p.cache = static_cast<uint8_t*>(cache);
  p.tokens = tokens;
  p.slot_end = pages * page_size;
  p.q_token = q_token_stride;
  p.q_head = q_head_stride;
  p.k_token = k_token_stride;
  p.k_head = k_head_stride;
  p.v_token = v_token_stride;
  p.v_head = v_head_stride;
  p.out_token = out_token_stride;
  p.out_head = out_head_stride;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.shift = lt::kv4::page_shift(page_size);
  p.max_pos = max_positions;
  p.half = rotary_dim / 2;
  p.minus_zero = -0.0f;
  const int per_cta = kThreads / (head_dim / 8);
  const int64_t blocks = (tokens + per_cta - 1) / per_cta;
  if (blocks > INT32_MAX) return LT_ERR_UNSUPPORTED;
  // a head a thread while the CTAs are few, two rounds of kAheadMost from where they fill the GPU's 152 SMs, eight each
  p.per = blocks * (q_heads + 2 * kv_heads) <= 152 * 8 && q_heads + 2 * kv_heads <= 65535 ? 1 : 2 * kAheadMost;
  p.q_parts = (q_heads + p.per - 1) / p.per;
  p.kv_parts = (kv_heads + p.per - 1) / p.per;
  // 16-byte accesses where every group of eight channels starts on 16 bytes: queries, their outputs, keys, values
  auto wide = [&](const void* at, int64_t a, int64_t b) { return aligned(at, 16) && ((a | b) * (int64_t)size) % 16 == 0; };
  int flags = (wide(q, q_token_stride, q_head_stride) ? 1 : 0) | (wide(out_q, out_token_stride, out_head_stride) ? 2 : 0) |
              (wide(k, k_token_stride, k_head_stride) ? 4 : 0) | (wide(v, v_token_stride, v_head_stride) ? 8 : 0);
  const bool pairs = interleaved != 0;
  const void* func = dtype == LT_DTYPE_F32    ? append_ptr<float>(head_dim, pairs)
                     : dtype == LT_DTYPE_BF16 ? append_ptr<__nv_bfloat16>(head_dim, pairs)
                                              : append_ptr<__half>(head_dim, pairs);
  if (lt::take_injected_failure()) return LT_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)(p.q_parts + 2 * p.kv_parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* a[] = {&p, &flags};
  return cudaLaunchKernelExC(&cfg, func, a) == cudaSuccess ? LT_OK : LT_ERR_CUDA;
}
