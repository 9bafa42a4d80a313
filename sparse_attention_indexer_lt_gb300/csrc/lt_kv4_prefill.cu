// lt_kv4_prefill.cu -- attention over the 4-bit cache for many query rows a
// request (prefill chunks): tcgen05 with the sums in tensor memory.
//
// A CTA takes 256 query rows of one kv head (two tiles of 128, one thread a row) and a
// range of positions in tiles of 128, with one role a warpgroup:
//   warpgroups 0 and 1  softmax of row tile A and B: logits from tensor memory,
//                       weights back into it as fp16, where the second product reads them
//   warpgroup 2         unpacks: a thread turns one position's codes into fp16 keys and
//                       values, written with the 128-byte swizzle that the tensor core reads
//   warpgroup 3         one warp issues the products, another the bulk copies of packed rows
// in the order  S_A(i) = Q_A K(i)^T,  O_B += P_B(i-1) V(i-1),  S_B(i),  O_A += P_A(i) V(i): while one row
// tile's softmax runs, the tensor core has the other's two products.
//
// Keys are laid out channels inner (K-major), values are the same bytes read as
// the transposed operand (their channels are the product's N). Unpacked tiles live in a
// ring of four; the packed rows' pitch is an odd multiple of 16 bytes, so eight threads
// reading 16 bytes of eight rows touch all banks, and the swizzle does the same
// for their stores.
//
// The running maximum moves only when a row's logits pass it by 2^8 (the sums are
// then rescaled in tensor memory, seldom); weights are held as 2^6 exp(s - max) at
// most 2^14, so fp16 neither overflows nor goes subnormal above 2^-20.
//
// A value that is NaN is unpacked as zero, and the rows that see it note the group:
// a row's output is NaN there whatever its weight, and rows that do not see it stay clean.

#include <mutex>

#include "lt_kv4.cuh"
#include "lt_kv4_attention.cuh"
#include "lt_kv4_prefill.h"

namespace {

using namespace lt::kv4;

constexpr int kCta = 512;
constexpr int kTok = 128;    // positions of a tile
constexpr int kSlots = 4;    // unpacked key or value tiles in shared memory
constexpr int kRaw = 1;      // packed tiles in shared memory: rows go on to registers, so the next one comes meanwhile
constexpr float kShift = 6.0f;
constexpr float kSlack = 8.0f;  // how far logits may pass the maximum (log 2) before it moves

template <int D>
struct Smem {
  static constexpr int kRow = row_bytes(D);
  static constexpr int kHalf = kTok * 128;               // 128 rows by 64 channels, swizzled
  static constexpr int kOperand = kHalf * (D / 64);
  static constexpr int kQ = 0;                           // two row tiles
  static constexpr int kKv = kQ + 2 * kOperand;          // kSlots
  static constexpr int kPacked = kKv + kSlots * kOperand;  // [kRaw][128 rows]
  static constexpr int kBars = kPacked + kRaw * kTok * kRow;
  static constexpr int kTotal = kBars + 2048 + 1024;     // (slack to align the start to 1024)
};

struct Shared {
  uint64_t packed_full[kRaw], packed_empty[kRaw];
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t q_full, s_full[2], p_full[2][2], o_full[2];
  uint4 valid[4];            // [tile mod 4]: positions on a page of the cache and in range, as bits
  uint4 nan_rows[4];         // positions with a NaN value scale
  uint8_t nan_groups[4][kTok];
  int64_t sums[kCta / 32];
  Place found;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Shared) <= 2048, "shared state");

// ---- tcgen05

__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
  // 128-byte swizzle, eight-row groups 1024 bytes apart
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr, uint32_t next_columns) {
  // 64 columns (128 bytes) inner; the next 64 are next_columns bytes on, the next eight rows 1024
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(next_columns >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// fp16 operands, fp32 sums, M = 128
__device__ __forceinline__ constexpr uint32_t instruction(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// The issuing warp runs these as a whole, so that descriptors stay in uniform registers; `lead` is set in
// one lane, which issues.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t lead) {
  asm volatile("{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
               " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
               :: "r"(lt::smem_u32(bar)), "r"(lead) : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t lead;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(lead));
  return lead;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
         "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
         "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(lt::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for a phase; gives up after kWaitPolls, or as soon as another thread has.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Shared* sh) {
  for (uint32_t i = 0; i < lt::kWaitPolls; ++i) {
    if (i == 0 ? mbar_ready(bar, parity) : lt::mbar_try_wait(bar, parity)) return true;
    if (i > 0 && *(volatile int*)&sh->abort) return false;
  }
  *(volatile int*)&sh->abort = 1;
  return false;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 lanes at once
__device__ __forceinline__ void fma2(float& x0, float& x1, float f, float a) {
  asm("{\n .reg .b64 x, f, a;\n mov.b64 x, {%0, %1};\n mov.b64 f, {%2, %2};\n mov.b64 a, {%3, %3};\n"
      " fma.rn.f32x2 x, x, f, a;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(x0), "+f"(x1) : "f"(f), "f"(a));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  asm("{\n .reg .b64 x, s;\n mov.b64 s, {%0, %1};\n mov.b64 x, {%2, %3};\n add.rn.f32x2 s, s, x;\n mov.b64 {%0, %1}, s;\n}"
      : "+f"(s0), "+f"(s1) : "f"(x0), "f"(x1));
}
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }

// What a CTA works on: row0 .. of the request's query rows, positions [from, to).
struct Job {
  Request rq;
  int request, head, row_tile, flat, rows, row0, from, to, tiles;
  bool two, final_here;
};

// ---- one row tile's softmax: a thread a row
template <int D>
__device__ __forceinline__ void softmax_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem, int which) {
  const int row_in_tile = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int row = job.row0 + which * 128 + row_in_tile;
  const int row_c = min(row, job.rows - 1);
  const int64_t token = job.rq.first + row_c / p.group;
  const int q_head = job.head * p.group + row_c % p.group;

  // the query row as fp16 into shared memory, with the power of two that keeps bf16 in range
  float factor;
  {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + token * p.q_token + (int64_t)q_head * p.q_head);
    uint32_t w[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      const uint4 v = __ldg(q + j);
      w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
    }
    factor = p.scale_log2;
    if (p.bf16) factor *= bf16_words_to_half<D / 8>(w);
    // logits are compared before they are scaled: a negative scale turns the row round instead
    const uint32_t flip = factor < 0.0f ? 0x80008000u : 0u, keep = factor == 0.0f ? 0u : ~0u;
    factor = factor == 0.0f ? 1.0f : fabsf(factor);
    uint8_t* to = smem + Smem<D>::kQ + which * Smem<D>::kOperand + row_in_tile * 128;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) {
      const uint4 v = make_uint4((w[j][0] ^ flip) & keep, (w[j][1] ^ flip) & keep, (w[j][2] ^ flip) & keep, (w[j][3] ^ flip) & keep);
      *reinterpret_cast<uint4*>(to + (j / 8) * Smem<D>::kHalf + (((j & 7) ^ (row_in_tile & 7)) << 4)) = v;
    }
    fence_async();
    arrive(&sh->q_full);
  }
  if (which == 1 && !job.two) return;

  const int limit = job.rq.length - job.rq.queries + row_c / p.group + 1;
  const int low = p.window > 0 ? max(limit - p.window, 0) : 0;
  const uint32_t lane_base = sh->tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t s_at = lane_base + which * kTok, o_at = lane_base + 2 * kTok + which * D;

  float m = -INFINITY, sum0 = 0.0f, sum1 = 0.0f;  // m in units of log 2
  uint32_t poison = 0;                             // value groups in which this row is NaN
  bool ok = true;
  for (int i = 0; i < job.tiles; ++i) {
    ok = wait_or_abort(&sh->s_full[which], i & 1, sh);
    if (!ok) break;
    fence_after();
    uint32_t raw[kTok];
    float* s = reinterpret_cast<float*>(raw);
#pragma unroll
    for (int c = 0; c < kTok; c += 32) tmem_ld32(s_at + c, raw + c);
    const uint4 valid4 = sh->valid[i & 3], nan4 = sh->nan_rows[i & 3];
    const int pos0 = job.from + i * kTok;
    const bool whole = (valid4.x & valid4.y & valid4.z & valid4.w) == ~0u && pos0 + kTok <= limit && pos0 >= low;
    const bool clean = (nan4.x | nan4.y | nan4.z | nan4.w) == 0;
    const bool plain = __all_sync(~0u, whole && clean);
    tmem_wait_ld();

    const uint32_t valid[4] = {valid4.x, valid4.y, valid4.z, valid4.w};
    if (!plain) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // visible: [low, limit) of this row, as bits of the 32 positions
        const int a = low - (pos0 + 32 * w), b = limit - (pos0 + 32 * w);  // (low >= 0: no overflow)
        uint32_t see = valid[w];
        see &= b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
        see &= a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!((see >> c) & 1u)) s[32 * w + c] = -INFINITY;
      }
    }
    if (!clean) {
      const uint32_t nan_rows[4] = {nan4.x, nan4.y, nan4.z, nan4.w};
#pragma unroll
      for (int w = 0; w < 4; ++w)
        for (uint32_t left = nan_rows[w] & valid[w]; left != 0; left &= left - 1) {
          const int t = 32 * w + __ffs(left) - 1;
          if (pos0 + t < limit && pos0 + t >= low) poison |= sh->nan_groups[i & 3][t];
        }
    }

    float top = s[0], top2 = s[1], top3 = s[2], top4 = s[3];
#pragma unroll
    for (int c = 4; c < kTok - 4; c += 8) {
      top = max3(top, s[c], s[c + 1]);
      top2 = max3(top2, s[c + 2], s[c + 3]);
      top3 = max3(top3, s[c + 4], s[c + 5]);
      top4 = max3(top4, s[c + 6], s[c + 7]);
    }
    top = max3(top, s[kTok - 4], s[kTok - 3]);
    top2 = max3(top2, s[kTok - 2], s[kTok - 1]);
    top = fmaxf(max3(top, top2, top3), top4) * factor;

    const bool moves = top > m + kSlack || (m == -INFINITY && top > m);
    if (__any_sync(~0u, moves)) {
      // S(i) is there, so the product O += P V of tile i - 1, issued before it, is done
      const float now = moves ? top : m;
      const float a = moves ? exp2_fast(m - now) : 1.0f;
      m = now;
      sum0 *= a;
      sum1 *= a;
      if (i > 0) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tmem_ld16(o_at + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
          tmem_st16(o_at + c, o);
        }
        tmem_wait_st();
      }
    }
    const float ref = m == -INFINITY ? 0.0f : kShift - m;
    uint32_t pk[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float& x0 = s[64 * h + 2 * e];
        float& x1 = s[64 * h + 2 * e + 1];
        fma2(x0, x1, factor, ref);
        x0 = exp2_fast(x0);
        x1 = exp2_fast(x1);
        add2(sum0, sum1, x0, x1);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(x1), "f"(x0));
      }
      tmem_st32(s_at + 32 * h, pk);
      tmem_wait_st();
      fence_before();
      arrive(&sh->p_full[which][h]);  // the second product starts on the first half
    }
  }
  ok = wait_or_abort(&sh->o_full[which], 0, sh) && ok;
  fence_after();

  // epilogue: divide, write out (or the part and its logarithm)
  const float sum = sum0 + sum1;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float log2_sum = sum == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m - kShift) + __log2f(sum);
  if (!ok) log2_sum = NAN;
  const bool mine = row < job.rows;
  const int64_t part = (((int64_t)job.flat * p.heads + job.head) * p.row_tiles + job.row_tile) * 256 + which * 128 + row_in_tile;
  const int64_t out_row = token * p.heads * p.group + q_head;
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    uint32_t o[32];
    if (job.tiles > 0) {
      tmem_ld32(o_at + c, o);
      tmem_wait_ld();
    }
    const bool bad = !ok || ((poison >> (c / 32)) & 1u);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (job.tiles > 0 && sum != 0.0f)
        x = make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv, __uint_as_float(o[e + 2]) * inv,
                        __uint_as_float(o[e + 3]) * inv);
      if (bad) x = make_float4(NAN, NAN, NAN, NAN);
      if (mine) {
        if (job.final_here)
          store4(p, out_row * D + c + e, x);
        else
          *reinterpret_cast<float4*>(p.part_o + part * D + c + e) = x;
      }
    }
  }
  if (mine) {
    if (job.final_here) {
      if (p.lse != nullptr) p.lse[out_row] = log2_sum * 0.6931471805599453f;
    } else {
      p.part_lse[part] = log2_sum;
    }
  }
}

// ---- packed rows into shared memory: one warp, a bulk copy for each run of positions on a page
template <int D>
__device__ __forceinline__ void copy_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem) {
  constexpr int kRow = row_bytes(D);
  constexpr int kMost = kTok / 32;  // runs of a lane, at pages of one position
  const int lane = threadIdx.x & 31;
  const uint32_t packed_at = lt::smem_u32(smem + Smem<D>::kPacked);
  const int run_shift = min(p.shift, 7), runs = kTok >> run_shift;
  const int32_t* table = p.table + (int64_t)job.request * p.width;
  int page[kMost];
  auto look_up = [&](int tile) {
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int run = lane + 32 * j, at = job.from + tile * kTok + (run << run_shift);
      page[j] = tile < job.tiles && run < runs && at < job.to ? __ldg(table + (at >> p.shift)) : -1;
    }
  };
  look_up(0);
  int stage = 0;
  uint32_t parity = 1;  // (the first round's stages are free)
  for (int i = 0; i < job.tiles; ++i) {
    if (!wait_or_abort(&sh->packed_empty[stage], parity, sh)) break;
    uint32_t valid[4] = {0u, 0u, 0u, 0u};
    int count[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int first = (lane + 32 * j) << run_shift, left = job.to - (job.from + i * kTok + first);
      count[j] = page[j] >= 0 && page[j] < p.pages ? min(left, 1 << run_shift) : 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int a = min(max(first - 32 * w, 0), 32), b = min(max(first + count[j] - 32 * w, 0), 32);
        valid[w] |= a < b ? (b == 32 ? ~0u : (1u << b) - 1u) & (~0u << a) : 0u;
      }
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) valid[w] = __reduce_or_sync(~0u, valid[w]);
    if (lane == 0) {
      sh->valid[i & 3] = make_uint4(valid[0], valid[1], valid[2], valid[3]);
      lt::mbar_arrive_tx(&sh->packed_full[stage],
                         (uint32_t)(__popc(valid[0]) + __popc(valid[1]) + __popc(valid[2]) + __popc(valid[3])) * kRow);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int first = (lane + 32 * j) << run_shift, at = job.from + i * kTok + first;
      if (count[j] > 0) {
        const uint8_t* src = p.cache + (((((int64_t)page[j] * p.heads + job.head) << p.shift) + (at & ((1 << p.shift) - 1))) * kRow);
        bulk_in(packed_at + (stage * kTok + first) * kRow, src, (uint32_t)count[j] * kRow, &sh->packed_full[stage]);
      }
    }
    look_up(i + 1);
    if (++stage == kRaw) {
      stage = 0;
      parity ^= 1u;
    }
  }
}

// ---- unpacking: a thread a position
template <int D>
__device__ __forceinline__ void unpack_role(const Job& job, Shared* sh, uint8_t* smem) {
  constexpr int kRow = row_bytes(D);
  constexpr int kGroups = D / 32;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, row = warp * 32 + lane;
  uint32_t chunk_at[8];  // where the row's eight 16-byte chunks lie in a swizzled 128-byte row
#pragma unroll
  for (int c = 0; c < 8; ++c) chunk_at[c] = lt::smem_u32(smem + Smem<D>::kKv) + row * 128 + ((c ^ (row & 7)) << 4);
  int slot = 0;
  uint32_t slot_parity = 1;  // (the first round's slots are free)
  bool ok = true;
  for (int i = 0; i < job.tiles && ok; ++i) {
    const int stage = i % kRaw;
    ok = wait_or_abort(&sh->packed_full[stage], (i / kRaw) & 1, sh);
    if (!ok) break;
    const uint4 valid4 = sh->valid[i & 3];
    const uint32_t valid = warp == 0 ? valid4.x : warp == 1 ? valid4.y : warp == 2 ? valid4.z : valid4.w;
    const bool there = (valid >> lane) & 1u;
    const uint8_t* from = smem + Smem<D>::kPacked + (stage * kTok + row) * kRow;
    // the row's codes and scales (fp16 pairs: keys, then values; a position that is not there counts as zeros)
    uint4 codes[D / 16];
    uint32_t sc[kGroups];
#pragma unroll
    for (int g = 0; g < D / 16; ++g) codes[g] = reinterpret_cast<const uint4*>(from)[g];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sc[g] = there ? reinterpret_cast<const uint32_t*>(from + D)[g] : 0u;
    __syncwarp();  // every lane has read the stage
    if (lane == 0) arrive(&sh->packed_empty[stage]);
    uint32_t nan = 0;
#pragma unroll
    for (int g = 0; g < kGroups / 2; ++g) {
      const uint32_t n = nan_halves(sc[kGroups / 2 + g]);
      sc[kGroups / 2 + g] &= ~n;
      nan |= ((n & 1u) | ((n >> 15) & 2u)) << (2 * g);
    }
    const uint32_t nan_rows = __ballot_sync(~0u, nan != 0);
    if (lane == 0) reinterpret_cast<uint32_t*>(&sh->nan_rows[i & 3])[warp] = nan_rows;
    if (nan_rows) sh->nan_groups[i & 3][row] = (uint8_t)nan;
#pragma unroll
    for (int part = 0; part < 2; ++part) {  // keys, then values
      ok = ok && wait_or_abort(&sh->kv_empty[slot], slot_parity, sh);
      if (!ok) break;
      const uint32_t to = slot * Smem<D>::kOperand;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const uint4 v = codes[part * kGroups + g];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const uint32_t pair = sc[part * (kGroups / 2) + g / 2];
        const uint32_t scale = __byte_perm(pair, 0, g & 1 ? 0x3232 : 0x1010);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h[4];
          codes_to_half2(w[j], h);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                       :: "r"(chunk_at[(g & 1) * 4 + j] + to + (g / 2) * Smem<D>::kHalf), "r"(hmul2(h[0], scale)),
                          "r"(hmul2(h[1], scale)), "r"(hmul2(h[2], scale)), "r"(hmul2(h[3], scale)) : "memory");
        }
      }
      fence_async();
      arrive(&sh->kv_full[slot]);
      if (++slot == kSlots) {
        slot = 0;
        slot_parity ^= 1u;
      }
    }
  }
}

// ---- the products, issued by one warp
template <int D>
__device__ __forceinline__ void product_role(const Job& job, Shared* sh, uint8_t* smem) {
  constexpr uint32_t kIdescS = instruction(kTok, false), kIdescO = instruction(D, true);
  const uint32_t q_at = lt::smem_u32(smem + Smem<D>::kQ), kv_at = lt::smem_u32(smem + Smem<D>::kKv);
  const uint32_t tmem = __shfl_sync(~0u, sh->tmem, 0), lead = elect_one();
  bool ok = wait_or_abort(&sh->q_full, 0, sh);
  int slot = 0;
  uint32_t parity = 0;
  auto next_slot = [&] {
    if (++slot == kSlots) {
      slot = 0;
      parity ^= 1u;
    }
  };
  // (descriptors hold addresses in units of 16 bytes; the steps' offsets are added to them, and the
  // loops stay rolled: this warpgroup runs on few registers, and a product takes 64 clocks)
  // (descriptors hold addresses in units of 16 bytes; the steps' offsets are added to them)
  auto logits = [&](int which, int key_slot) {
    const uint64_t q = desc_k_major(q_at + which * Smem<D>::kOperand), key = desc_k_major(kv_at + key_slot * Smem<D>::kOperand);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t at = ((k / 4) * Smem<D>::kHalf + (k % 4) * 32) >> 4;
      mma_ss(tmem + which * kTok, q + at, key + at, kIdescS, k > 0, lead);
    }
    mma_commit(&sh->s_full[which], lead);
  };
  auto outputs = [&](int which, int value_slot, bool first, int half) {
    const uint64_t value = desc_mn_major(kv_at + value_slot * Smem<D>::kOperand, Smem<D>::kHalf);
#pragma unroll
    for (int k = half * (kTok / 32); k < (half + 1) * (kTok / 32); ++k)
      mma_ts(tmem + 2 * kTok + which * D, tmem + which * kTok + k * 8, value + k * (2048 >> 4), kIdescO, !first || k > 0, lead);
  };
  // both halves of a row tile's second product
  auto weigh = [&](int which, int value_slot, int i) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (!wait_or_abort(&sh->p_full[which][half], i & 1, sh)) return false;
      fence_after();
      outputs(which, value_slot, i == 0, half);
    }
    return true;
  };
  // K(i + 1) and V(i) are waited for while a product runs, so that the tensor core waits for weights only
  auto wait_slot = [&] {
    ok = ok && wait_or_abort(&sh->kv_full[slot], parity, sh);
    const int at = slot;
    next_slot();
    return at;
  };
  int key = job.tiles > 0 ? wait_slot() : 0, value = 0;
  fence_after();
  if (job.tiles > 0 && ok) logits(0, key);
  for (int i = 0; i < job.tiles && ok; ++i) {
    // here S_A(i) is issued
    if (job.two) {
      if (i > 0) {
        ok = weigh(1, value, i - 1);
        if (!ok) break;
        mma_commit(&sh->kv_empty[value], lead);
      }
      logits(1, key);
    }
    mma_commit(&sh->kv_empty[key], lead);
    value = wait_slot();
    if (i + 1 < job.tiles) key = wait_slot();
    if (!ok) break;
    fence_after();
    ok = weigh(0, value, i);
    if (!ok) break;
    if (!job.two) mma_commit(&sh->kv_empty[value], lead);
    if (i + 1 < job.tiles) logits(0, key);
  }
  if (ok && job.two && job.tiles > 0) weigh(1, value, job.tiles - 1);
  mma_commit(&sh->o_full[0], lead);
  mma_commit(&sh->o_full[1], lead);
}

template <int D>
__global__ void __launch_bounds__(kCta, 1) prefill_kernel(AttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (lt::smem_u32(smem_raw) & 1023u)) & 1023u);
  Shared* sh = reinterpret_cast<Shared*>(smem + Smem<D>::kBars);
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
  if (tid == 0) {
    for (int s = 0; s < kRaw; ++s) {
      lt::mbar_init(&sh->packed_full[s], 1);
      lt::mbar_init(&sh->packed_empty[s], 4);
    }
    for (int s = 0; s < kSlots; ++s) {
      lt::mbar_init(&sh->kv_full[s], 128);
      lt::mbar_init(&sh->kv_empty[s], 1);
    }
    lt::mbar_init(&sh->q_full, 256);
    for (int t = 0; t < 2; ++t) {
      lt::mbar_init(&sh->s_full[t], 1);
      lt::mbar_init(&sh->p_full[t][0], 128);
      lt::mbar_init(&sh->p_full[t][1], 128);
      lt::mbar_init(&sh->o_full[t], 1);
    }
    sh->abort = 0;
    lt::mbar_fence_init();
  }
  dependency_wait();

  Job job;
  const int64_t unit = blockIdx.x;
  // the last rows see the most positions: they start first
  job.row_tile = p.row_tiles - 1 - (int)(unit % p.row_tiles);
  job.head = (int)(unit / p.row_tiles % p.heads);
  job.flat = (int)(unit / p.row_tiles / p.heads);
  Place pl;
  if (!find_place<kCta>(p, job.flat, &pl, sh->sums, &sh->found)) return;
  job.request = pl.request;
  job.rq = request_of(p, pl.request);
  job.rows = job.rq.queries * p.group;
  job.final_here = pl.count == 1;
  if (job.flat == pl.base && job.head == 0 && job.row_tile == 0 && tid == 0 && p.plan != nullptr)
    p.plan[pl.request] = make_int2(pl.base, pl.count);
  job.row0 = job.row_tile * 256;
  if (job.row0 >= job.rows) return;
  job.two = job.rows - job.row0 > 128;
  {
    const int64_t at = job.rq.low + (int64_t)pl.split * pl.chunk;
    job.from = (int)(at < job.rq.length ? at : job.rq.length);
    job.to = (int)(at + pl.chunk < job.rq.length ? at + pl.chunk : job.rq.length);
    const int last = min(job.rows - 1, job.row0 + 255) / p.group;
    job.to = min(job.to, job.rq.length - job.rq.queries + last + 1);
    if (p.window > 0)
      job.from = max(job.from, (job.rq.length - job.rq.queries + job.row0 / p.group + 1 - p.window) / kTile * kTile);
    job.tiles = job.to > job.from ? (job.to - job.from + kTok - 1) / kTok : 0;
  }

  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(lt::smem_u32(&sh->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();

  // 512 threads of 128 registers are split as 2 x 184 + 80 + 64 a thread of the four warpgroups
  if (warp < 8) {
    regs_up<184>();
    softmax_role<D>(p, job, sh, smem, warp / 4);
  } else if (warp < 12) {
    regs_down<80>();
    unpack_role<D>(job, sh, smem);
  } else {
    regs_down<64>();
    if (warp == 12) product_role<D>(job, sh, smem);
    if (warp == 13) copy_role<D>(p, job, sh, smem);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  dependents_launch();
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(sh->tmem) : "memory");
}

}  // namespace

namespace lt {
namespace kv4 {

const void* prefill_kernel_ptr(int head_dim, int* smem) {
  if (head_dim == 64) {
    *smem = Smem<64>::kTotal;
    return reinterpret_cast<const void*>(&prefill_kernel<64>);
  }
  if (head_dim == 128) {
    *smem = Smem<128>::kTotal;
    return reinterpret_cast<const void*>(&prefill_kernel<128>);
  }
  return nullptr;
}

}  // namespace kv4
}  // namespace lt
