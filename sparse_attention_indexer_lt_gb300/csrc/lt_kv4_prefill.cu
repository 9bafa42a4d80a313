// lt_kv4_prefill.cu -- attention over the 4-bit cache for many query rows a
// request (prefill chunks): tcgen05 with the sums in tensor memory.
//
// A CTA takes 256 query rows of one kv head (two tiles of 128, a thread a row) and a
// range of positions in tiles of 128, with one role a warpgroup:
//   warpgroups 0 and 1  softmax of row tile A and B: logits from tensor memory,
//                       weights back into it as fp16, where the second product reads them
//   warpgroup 2         unpacks: a thread turns one position's key or value codes into fp16,
//                       written with the 128-byte swizzle that the tensor core reads
//   warpgroup 3         one warp issues the products, another the bulk copies of packed rows
// in the order  S_A(i) = Q_A K(i)^T,  O_B += P_B(i-1) V(i-1),  S_B(i),  O_A += P_A(i) V(i): while one row
// tile's softmax runs, the tensor core has the other's two products.
//
// Keys are laid out channels inner (K-major), values are the same bytes read as
// the transposed operand (their channels are the product's N). Unpacked tiles live in a
// ring of four; the packed rows' pitch is an odd multiple of 16 bytes (with heads of 256
// twice one), so eight threads reading 16 bytes of eight rows touch all banks (half of them), and the
// swizzle does the same for their stores.
//
// With heads of 256 tensor memory holds one row tile's sums, its queries and two tiles
// of logits of 64 positions: the order is  S(0), S(1), O += P(0) V(0), S(2), O += P(1) V(1), S(3), ... ,
// so that one position tile's softmax runs beside the next one's first product and the last
// one's second, and warpgroup 1 unpacks too.
//
// The running maximum moves only when a row's logits pass it by 2^8 (the sums are
// then rescaled in tensor memory, seldom); weights are held as 2^6 exp(s - max) at
// most 2^14, so fp16 neither overflows nor goes subnormal above 2^-20.
//
// What bounds it: the chain softmax, second product, next first product of a row tile.
// An iteration (both row tiles by 128 positions of D = 128) takes some 3100 clocks, the
// products alone 2048 (64 each, in every operand mode); the softmax's part is some 1700 from the logits'
// arrival to the weights'. What the chain gave up on the way, on a chunk of 2048 tokens
// behind 14336 positions (32 query heads on 8 kv heads): 941 us with one lane issuing, 716
// with the warp issuing and copies in a warp of their own, 650 with short loops and whole-line
// queries and outputs, 511 without cutting requests that fill the SMs, 494 with four
// products a statement, 424 with named barriers, 410 with the longest row tiles first: 1.26
// PFLOP/s, 65% of cuBLAS's burst; 84% is the most that two waves of 256 CTAs on 152 SMs
// allow. Measured and dropped: a quarter, a third or half of the exponentials on the FMA
// pipes (541, 557, 621 us against 511), two threads a row (541), the first half's weights taken
// before the tile's maximum is known (804 against 716).
//
// Heads of 256, the same chunk: 5063 us with the kernel for few rows; here 1586 with queries
// in shared memory and a key and a value tile, 1238 with the queries in tensor memory and three tiles, 1100 with
// eight warps unpacking, 854 with tiles of 64, logits a tile ahead and five packed stages in place of three
// of 32 positions (1160 with those): 1.21 PFLOP/s, 63% of cuBLAS's burst, where four waves of 512 CTAs on 152
// SMs allow 84%. The unpacked tile's way, read, write and fence, is what is left: 748 us without its writes.
//
// A value that is NaN, or whose scale is outside the format, is unpacked as zero, and the rows that see it note
// the group: a row's output is NaN there whatever its weight, and rows that do not see it stay clean.

#include <mutex>

#include "lt_kv4.cuh"
#include "lt_kv4_attention.cuh"
#include "lt_kv4_prefill.h"

namespace {

using namespace lt::kv4;

constexpr int kCta = 512;
constexpr int kSlots = 4;    // unpacked key or value tiles in shared memory
constexpr int kPart = 64;    // positions of a packed stage
constexpr int kMaxRaw = 5;   // packed stages in shared memory or on their way there
// columns of tensor memory: logits and weights first, two tiles
constexpr int kQueryColumn = 128;  // queries, with heads of 256
constexpr int kSumColumn = 256;
constexpr float kShift = 6.0f;
constexpr float kSlack = 8.0f;  // how far logits may pass the maximum (log 2) before it moves

template <int D>
struct Smem {
  static constexpr int kRow = row_bytes(D);
  // Heads of 256 leave room for one row tile. Its queries are in tensor memory, and its position tiles are
  // of 64: two of logits (128 columns), the queries (128) and the sums (256) fit, so that the next
  // tile's logits are there when the softmax of this one ends, and shared memory has room for five packed stages.
  static constexpr bool kOne = D == 256;
  static constexpr int kRowTiles = kOne ? 1 : 2;
  static constexpr int kTok = kOne ? 64 : 128;             // positions of a tile
  static constexpr int kRaw = kOne ? 5 : 3;
  static constexpr int kUnpackers = kOne ? 256 : 128;      // threads that unpack: row tile B's warpgroup is free to
  static constexpr int kParts = kTok / kPart;
  static constexpr int kRing = 512 / kTok;                 // tiles whose notes are kept
  static_assert(kSlots / 2 * kParts + kRaw < kRing * kParts, "notes are read before they are written over");
  static constexpr int kQHalf = 128 * 128;                 // 128 rows by 64 channels, swizzled
  static constexpr int kQTile = kQHalf * (D / 64);
  static constexpr int kHalf = kTok * 128;                 // a tile's positions by 64 channels
  static constexpr int kOperand = kHalf * (D / 64);
  static constexpr int kKv = kOne ? 0 : kRowTiles * kQTile;  // kSlots
  // row tiles; where the queries are in tensor memory, the last slots are what they and the outputs are turned
  // round in, before their first keys and after the last product
  static constexpr int kQ = kOne ? kKv + kSlots * kOperand - kQTile : 0;
  static constexpr int kPacked = kKv + kSlots * kOperand;  // [kRaw][kPart rows]
  static constexpr int kBars = kPacked + kRaw * kPart * kRow;
  static constexpr int kTotal = kBars + 2048 + 1024;     // (slack to align the start to 1024)
};

struct Shared {
  uint64_t packed_full[kMaxRaw], packed_empty[kMaxRaw];
  uint64_t kv_empty[kSlots];
  uint64_t q_full, s_full[2], o_full[2];
  uint64_t o_tile;  // with one row tile: a position tile's second product is done
  // notes of the tiles in work, a ring of 512 positions, eight packed stages. They are made up to seven stages
  // ahead of the softmax (Smem's assertion): while it reads tile i's, tile i's values are not given back, so the
  // unpackers have released at most the first stage of tile i + kSlots / 2, and the copies run kRaw stages on from there
  alignas(16) uint32_t valid[16];     // positions on a page of the cache and in range, as bits
  alignas(16) uint32_t nan_rows[16];  // positions with a value scale that is NaN or outside the format
  uint8_t nan_groups[512];
  int64_t sums[kCta / 32];
  Place found;
  uint32_t tmem;
  int gave_up;
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
// Four products in a row, 16 of the inner dimension each; only the first may start a new sum.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
  asm volatile("{\n .reg .pred p, q, t;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
               " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
               " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
               " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead) : "memory");
}
// (kStep: from one 16 of the inner dimension to the next in B, in units of 16 bytes)
template <int kStep>
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t lead) {
  asm volatile("{\n .reg .pred p, q, t;\n .reg .b32 a;\n .reg .b64 b;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n setp.eq.u32 t, 0, 0;\n"
               " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
               " add.s32 a, %1, 8;\n add.s64 b, %2, %6;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
               " add.s32 a, %1, 16;\n add.s64 b, %2, %7;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
               " add.s32 a, %1, 24;\n add.s64 b, %2, %8;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n}"
               :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep)
               : "memory");
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

// Loads from tensor memory, each with its wait in one statement: registers that are still to be written
// must not be seen by the compiler, which would copy and reuse them.
__device__ __forceinline__ void tmem_read16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      :
        "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_read32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      :
        "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_read64(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, "
      "%24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, "
      "%46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      :
        "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr)
      : "memory");
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
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(lt::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A warp waits for a phase, kWaitPolls polls at most; a wait that gives up marks the CTA, whose outputs are NaN
// then, and the warp goes on: the roles keep their steps, so nobody waits for one that has
// left. Every poll ends in a vote, so the warp's control flow is uniform: the callers go on to .aligned
// instructions.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Shared* sh) {
  bool done = mbar_ready(bar, parity);
  if (__all_sync(~0u, done)) return true;
#pragma unroll 1
  for (uint32_t i = 0; i < lt::kWaitPolls; ++i) {
    done = done | lt::mbar_try_wait(bar, parity);
    if (__all_sync(~0u, done)) return true;
  }
  *(volatile int*)&sh->gave_up = 1;
  return false;
}

// What the issuing warp waits for comes over the CTA's named barriers: it sees them within some 50 clocks, where
// a look at an mbarrier takes 250 and more while the products keep shared memory busy. A named
// barrier's wait has no limit of its own; it ends because every role keeps its steps, also
// after a wait that gave up.
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("barrier.cta.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ int weights_ready(int which, int half) { return 1 + 2 * which + half; }
constexpr int kWeightsThreads = 128 + 32;
__device__ __forceinline__ int slot_ready(int slot) { return 5 + slot; }
template <int D>
constexpr int kSlotThreads = Smem<D>::kUnpackers / 2 + 32;

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
// What a CTA works on: row0 .. of the request's query rows, positions [from, to).
struct Job {
  Request rq;
  int request, head, row_tile, flat, part, rows, row0, from, to, tiles;
  bool two, final_here;
};

// ---- one row tile's softmax: a thread a row
template <int D>
__device__ __forceinline__ void softmax_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem, int which) {
  constexpr int kHalf = Smem<D>::kQHalf, kTok = Smem<D>::kTok, kRing = Smem<D>::kRing;
  constexpr int kChunks = D / 8;                          // 16-byte chunks of a row of 16-bit values
  constexpr int kAtOnce = 32 / kChunks;                   // rows of one warp-wide access
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, row_in_tile = warp * 32 + lane;
  const int row = job.row0 + which * 128 + row_in_tile;
  const int row_c = min(row, job.rows - 1);
  uint8_t* tile = smem + Smem<D>::kQ + which * Smem<D>::kQTile;
  // chunk c of row r of the tile, where the 128-byte swizzle puts it
  auto chunk_of = [&](int r, int c) { return reinterpret_cast<uint4*>(tile + (c / 8) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)); };

  // the query rows into shared memory: the warp brings its rows one after the other, then each thread
  // makes its own row fp16, with the power of two that keeps bf16 in range
  float factor = p.scale_log2;
  {
    const int chunk = lane % kChunks;
#pragma unroll 8
    for (int it = 0; it < 32 / kAtOnce; ++it) {
      const int r = warp * 32 + it * kAtOnce + lane / kChunks, of = min(job.row0 + which * 128 + r, job.rows - 1);
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + (int64_t)(job.rq.first + of / p.group) * p.q_token +
                          (int64_t)(job.head * p.group + of % p.group) * p.q_head;
      *chunk_of(r, chunk) = __ldg(reinterpret_cast<const uint4*>(q) + chunk);
    }
    __syncwarp();
    float mul = 1.0f;
    if (p.bf16) {
      uint32_t big = 0;
#pragma unroll 4
      for (int c = 0; c < kChunks; ++c) {
        const uint4 v = *chunk_of(row_in_tile, c);
        const uint32_t w[1][4] = {{v.x, v.y, v.z, v.w}};
        big = max(big, largest_word<1>(w));
      }
      mul = bf16_row_power(big);
      factor /= mul;  // (exact: a power of two)
    }
    // logits are compared before they are scaled: a negative scale turns the row round instead, and a scale of
    // zero makes its channels zeros, or NaN where they are not finite
    const uint32_t flip = factor < 0.0f ? 0x80008000u : 0u;
    const bool zero = factor == 0.0f;
    factor = factor == 0.0f ? 1.0f : fabsf(factor);
#pragma unroll 1
    for (int c0 = 0; c0 < kChunks; c0 += 4) {
      uint32_t w[16];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint4* at = chunk_of(row_in_tile, c0 + c);
        const uint4 v = *at;
        w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
#pragma unroll
        for (int e = 4 * c; e < 4 * c + 4; ++e) w[e] = (p.bf16 ? bf16_pair_to_half(w[e], mul) : w[e]) ^ flip;
        if (zero) {
#pragma unroll
          for (int e = 4 * c; e < 4 * c + 4; ++e) w[e] = zero_times_halves(w[e]);
        }
        if (!Smem<D>::kOne) *at = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      }
      if constexpr (Smem<D>::kOne) {
        __syncwarp();  // (`zero` may differ from row to row, and the store is the whole warp's)
        tmem_st16(sh->tmem + ((uint32_t)(warp * 32) << 16) + kQueryColumn + c0 * 4, w);
      }
    }
    if constexpr (Smem<D>::kOne) {
      tmem_wait_st();
      fence_before();
    } else {
      fence_async();
    }
    arrive(&sh->q_full);
    __syncwarp();
  }
  if (which == 1 && !job.two) return;

  const int limit = job.rq.length - job.rq.queries + row_c / p.group + 1;
  const int low = p.window > 0 ? max(limit - p.window, 0) : 0;
  const uint32_t lane_base = sh->tmem + ((uint32_t)(warp * 32) << 16);
  const uint32_t o_at = lane_base + kSumColumn + which * D;

  // The loop reads a tile's logits twice, once for the maximum and once for the weights: that is little
  // against 128 exponentials a row, and the loops stay short enough for the instruction
  // cache that four kinds of warps share.
  float m = -INFINITY, sum0 = 0.0f, sum1 = 0.0f;  // m in units of log 2
  uint32_t poison = 0;                             // value groups in which this row is NaN
  for (int i = 0; i < job.tiles; ++i) {
    const int buf = Smem<D>::kOne ? i & 1 : which;
    const uint32_t s_at = lane_base + buf * kTok;
    wait_warp(&sh->s_full[buf], (Smem<D>::kOne ? i >> 1 : i) & 1, sh);
    fence_after();
    const int pos0 = job.from + i * kTok;
    const uint32_t* valid = sh->valid + i % kRing * (kTok / 32);
    const uint32_t* nan_rows = sh->nan_rows + i % kRing * (kTok / 32);
    const uint2 valid2 = *reinterpret_cast<const uint2*>(valid), nan2 = *reinterpret_cast<const uint2*>(nan_rows);
    uint32_t all_valid = valid2.x & valid2.y, any_nan = nan2.x | nan2.y;
    if constexpr (kTok == 128) {
      const uint2 v = *reinterpret_cast<const uint2*>(valid + 2), n = *reinterpret_cast<const uint2*>(nan_rows + 2);
      all_valid &= v.x & v.y;
      any_nan |= n.x | n.y;
    }
    float top;
    bool hidden = false;
#pragma unroll 1
    for (;;) {
      float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < kTok / 64; ++h) {
        uint32_t x[64];
        tmem_read64(s_at + 64 * h, x);
        const float* s = reinterpret_cast<const float*>(x);
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
          t0 = max3(t0, s[c], s[c + 1]);
          t1 = max3(t1, s[c + 2], s[c + 3]);
          t2 = max3(t2, s[c + 4], s[c + 5]);
          t3 = max3(t3, s[c + 6], s[c + 7]);
        }
      }
      top = fmaxf(max3(t0, t1, t2), t3) * factor;
      // (looked at only now: the words come from shared memory, which the products keep busy)
      const bool plain = all_valid == ~0u && pos0 + kTok <= limit && pos0 >= low && any_nan == 0;
      if (hidden || __all_sync(~0u, plain)) break;
      // hide what this row does not see, in tensor memory, and take the maximum again
      hidden = true;
#pragma unroll 1
      for (int w = 0; w < kTok / 32; ++w) {
        uint32_t y[32];
        tmem_read32(s_at + 32 * w, y);
        const int a = low - (pos0 + 32 * w), b = limit - (pos0 + 32 * w);  // (low >= 0: no overflow)
        uint32_t see = valid[w];
        see &= b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
        see &= a <= 0 ? ~0u : a >= 32 ? 0u : ~0u << a;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!((see >> c) & 1u)) y[c] = 0xFF800000u;
        tmem_st32(s_at + 32 * w, y);
        for (uint32_t left = nan_rows[w] & see; left != 0; left &= left - 1)
          poison |= sh->nan_groups[i % kRing * kTok + 32 * w + __ffs(left) - 1];
        __syncwarp();
      }
      tmem_wait_st();
    }
    const bool moves = top > m + kSlack || (m == -INFINITY && top > m);
    if (__any_sync(~0u, moves)) {
      // the product O += P V of tile i - 1 has to be done: with two row tiles S(i) was issued after it; with one
      // S(i) came before it, but after that of tile i - 2, so that this is the phase to wait for
      const float now = moves ? top : m;
      const float a = moves ? exp2_fast(m - now) : 1.0f;
      m = now;
      sum0 *= a;
      sum1 *= a;
      if (i > 0) {
        if constexpr (Smem<D>::kOne) {
          wait_warp(&sh->o_tile, (i - 1) & 1, sh);
          fence_after();
        }
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tmem_read16(o_at + c, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
          tmem_st16(o_at + c, o);
        }
        tmem_wait_st();
      }
    }
    const float ref = m == -INFINITY ? 0.0f : kShift - m;
#pragma unroll 1
    for (int h = 0; h < kTok / 64; ++h) {
      uint32_t x[64], pk[32];
      tmem_read64(s_at + 64 * h, x);
      float* s = reinterpret_cast<float*>(x);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        fma2(s[2 * e], s[2 * e + 1], factor, ref);
        s[2 * e] = exp2_fast(s[2 * e]);
        s[2 * e + 1] = exp2_fast(s[2 * e + 1]);
        add2(sum0, sum1, s[2 * e], s[2 * e + 1]);
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[e]) : "f"(s[2 * e + 1]), "f"(s[2 * e]));
      }
      tmem_st32(s_at + 32 * h, pk);  // (columns whose logits have been read)
      tmem_wait_st();
      fence_before();
      named_arrive(weights_ready(buf, h), kWeightsThreads);  // the second product starts on the first half
      __syncwarp();
    }
  }
  const bool ok = wait_warp(&sh->o_full[which], 0, sh) && *(volatile int*)&sh->gave_up == 0;
  __syncwarp();
  fence_after();

  // epilogue: divide, turn the rows through the query tile's place into whole lines, write out (or the
  // part and its logarithm)
  const float sum = sum0 + sum1;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float log2_sum = sum == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m - kShift) + __log2f(sum);
  if (!ok) log2_sum = NAN;
  const int64_t part = ((int64_t)job.part * p.heads + job.head) * p.part_rows + job.row0 + which * 128;
  const int per_pass = job.final_here ? D : D / 2;  // columns that fit the tile's rows
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += per_pass) {
#pragma unroll 1
    for (int c = 0; c < per_pass; c += 16) {
      uint32_t o[16];
      if (job.tiles > 0) tmem_read16(o_at + c0 + c, o);
      const bool bad = !ok || ((poison >> ((c0 + c) / 32)) & 1u);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = job.tiles > 0 && sum != 0.0f ? __uint_as_float(o[e]) * inv : 0.0f;
        o[e] = __float_as_uint(bad ? NAN : x);
      }
      if (job.final_here) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = pack_out(p, __uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
        *chunk_of(row_in_tile, c / 8) = make_uint4(h[0], h[1], h[2], h[3]);
        *chunk_of(row_in_tile, c / 8 + 1) = make_uint4(h[4], h[5], h[6], h[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *chunk_of(row_in_tile, c / 4 + e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
    __syncwarp();
#pragma unroll 4
    for (int it = 0; it < 32 / kAtOnce; ++it) {
      const int r = warp * 32 + it * kAtOnce + lane / kChunks, of = job.row0 + which * 128 + r;
      if (of >= job.rows) continue;
      const uint4 v = *chunk_of(r, lane % kChunks);
      if (job.final_here) {
        const int64_t out_row = (int64_t)(job.rq.first + of / p.group) * p.heads * p.group + job.head * p.group + of % p.group;
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out_row * D)[lane % kChunks] = v;
      } else {
        reinterpret_cast<uint4*>(p.part_o + (part + r) * D + c0)[lane % kChunks] = v;
      }
    }
    __syncwarp();
  }
  if (row < job.rows) {
    if (job.final_here) {
      const int64_t out_row = (int64_t)(job.rq.first + row / p.group) * p.heads * p.group + job.head * p.group + row % p.group;
      if (p.lse != nullptr) p.lse[out_row] = log2_sum * 0.6931471805599453f;
    } else {
      p.part_lse[part + row_in_tile] = log2_sum;
    }
  }
}

// ---- packed rows into shared memory: one warp, a bulk copy for each run of positions on a page
template <int D>
__device__ __forceinline__ void copy_role(const AttentionParams& p, const Job& job, Shared* sh, uint8_t* smem) {
  constexpr int kRow = row_bytes(D);
  constexpr int kParts = Smem<D>::kParts, kRaw = Smem<D>::kRaw;
  constexpr int kMost = kPart / 32;  // runs of a lane, at pages of one position; words of a stage's valid bits
  const int lane = threadIdx.x & 31;
  const uint32_t packed_at = lt::smem_u32(smem + Smem<D>::kPacked);
  const int run_shift = min(p.shift, 6), runs = kPart >> run_shift;
  const int32_t* table = p.table + (int64_t)job.request * p.width;
  const int stages = kParts * job.tiles;
  int page[kMost];
  auto look_up = [&](int n) {
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int run = lane + 32 * j, at = job.from + n * kPart + (run << run_shift);
      page[j] = n < stages && run < runs && at < job.to ? __ldg(table + (at >> p.shift)) : -1;
    }
  };
  look_up(0);
  int stage = 0;
  uint32_t parity = 1;  // (the first round's stages are free)
#pragma unroll 1
  for (int n = 0; n < stages; ++n) {
    wait_warp(&sh->packed_empty[stage], parity, sh);
    uint32_t valid[kMost] = {};
    int count[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int first = (lane + 32 * j) << run_shift, left = job.to - (job.from + n * kPart + first);
      count[j] = page[j] >= 0 && page[j] < p.pages ? min(left, 1 << run_shift) : 0;
#pragma unroll
      for (int w = 0; w < kMost; ++w) {
        const int a = min(max(first - 32 * w, 0), 32), b = min(max(first + count[j] - 32 * w, 0), 32);
        valid[w] |= a < b ? (b == 32 ? ~0u : (1u << b) - 1u) & (~0u << a) : 0u;
      }
    }
    uint32_t there = 0;
#pragma unroll
    for (int w = 0; w < kMost; ++w) {
      valid[w] = __reduce_or_sync(~0u, valid[w]);
      there += __popc(valid[w]);
    }
    if (lane == 0) {
#pragma unroll
      for (int w = 0; w < kMost; ++w) sh->valid[n % (16 / kMost) * kMost + w] = valid[w];
      lt::mbar_arrive_tx(&sh->packed_full[stage], there * kRow);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      const int first = (lane + 32 * j) << run_shift, at = job.from + n * kPart + first;
      if (count[j] > 0) {
        const uint8_t* src = p.cache + (((((int64_t)page[j] * p.heads + job.head) << p.shift) + (at & ((1 << p.shift) - 1))) * kRow);
        bulk_in(packed_at + (stage * kPart + first) * kRow, src, (uint32_t)count[j] * kRow, &sh->packed_full[stage]);
      }
    }
    look_up(n + 1);
    if (++stage == kRaw) {
      stage = 0;
      parity ^= 1u;
    }
  }
}

// ---- unpacking: a packed stage's positions at a time, a thread the key or the value of a position (with
// D = 256 half of its channels); half of the threads have keys, half values
template <int D>
__device__ __forceinline__ void unpack_role(const Job& job, Shared* sh, uint8_t* smem) {
  constexpr int kRow = row_bytes(D);
  constexpr int kParts = Smem<D>::kParts, kRaw = Smem<D>::kRaw;
  constexpr int kTok = Smem<D>::kTok, kRing = Smem<D>::kRing;
  constexpr int kBlocks = D / 64 * 2 * kPart / Smem<D>::kUnpackers;  // 64-channel blocks of a thread
  const int t = threadIdx.x - (384 - Smem<D>::kUnpackers), lane = t & 31, row = t % kPart, part = t / kPart & 1;
  const int block0 = t / (2 * kPart) * kBlocks;
  uint32_t chunk_at[8];  // where the row's eight 16-byte chunks lie in a swizzled 128-byte row
#pragma unroll
  for (int c = 0; c < 8; ++c) chunk_at[c] = lt::smem_u32(smem + Smem<D>::kKv) + row * 128 + ((c ^ (row & 7)) << 4);
  // the slots go round: keys of tile i in slot 2 i mod kSlots, values in the next
  int slot = part, stage = 0;
  uint32_t slot_parity = 1, stage_parity = 0;  // (the first round's slots are free)
  bool fed = true;
#pragma unroll 1
  for (int i = 0; i < job.tiles; ++i) {
#pragma unroll 1
    for (int half = 0; half < kParts; ++half) {
      fed = fed && wait_warp(&sh->packed_full[stage], stage_parity, sh);  // (once in vain is enough)
      const int word = i % kRing * (kTok / 32) + half * (kPart / 32) + row / 32;  // (the warp's rows are one word's)
      const uint32_t valid = sh->valid[word];
      const bool there = (valid >> lane) & 1u;
      const uint8_t* from = smem + Smem<D>::kPacked + (stage * kPart + row) * kRow;
      // scales, fp16 pairs; a position that is not there counts as zeros, and so does a NaN value
      uint32_t sc[kBlocks];
#pragma unroll
      for (int g = 0; g < kBlocks; ++g) {
        sc[g] = there ? reinterpret_cast<const uint32_t*>(from + D + part * (D / 16))[block0 + g] : 0u;
        if (part == 1) sc[g] &= ~unfit_halves(sc[g]);
      }
      if (part == 0 && block0 == 0) {
        // the NaN values are noted here, with the keys: the softmax starts when the keys are there
        uint32_t nan = 0;
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          const uint32_t n = there ? unfit_halves(reinterpret_cast<const uint32_t*>(from + D + D / 16)[g]) : 0u;
          nan |= ((n & 1u) | ((n >> 15) & 2u)) << (2 * g);
        }
        const uint32_t nan_rows = __ballot_sync(~0u, nan != 0);
        if (lane == 0) sh->nan_rows[word] = nan_rows;
        if (nan_rows) sh->nan_groups[i % kRing * kTok + half * kPart + row] = (uint8_t)nan;
      }
      uint4 codes[2 * kBlocks];
#pragma unroll
      for (int c = 0; c < 2 * kBlocks; ++c) codes[c] = reinterpret_cast<const uint4*>(from + part * (D / 2))[2 * block0 + c];
      __syncwarp();  // every lane has read the stage
      if (lane == 0) arrive(&sh->packed_empty[stage]);
      if (half == 0) {
        wait_warp(&sh->kv_empty[slot], slot_parity, sh);
        // (until then the queries are in the last slots)
        if (Smem<D>::kOne && i == kSlots / 2 - 1) wait_warp(&sh->q_full, 0, sh);
      }
      const uint32_t to = slot * Smem<D>::kOperand + half * (kPart * 128);
#pragma unroll
      for (int c = 0; c < kBlocks; ++c) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const uint32_t w[4] = {codes[2 * c + g].x, codes[2 * c + g].y, codes[2 * c + g].z, codes[2 * c + g].w};
          const uint32_t scale = __byte_perm(sc[c], 0, g ? 0x3232 : 0x1010);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
            codes_to_half2(w[j], h);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         :: "r"(chunk_at[g * 4 + j] + to + (block0 + c) * Smem<D>::kHalf), "r"(hmul2(h[0], scale)),
                            "r"(hmul2(h[1], scale)), "r"(hmul2(h[2], scale)), "r"(hmul2(h[3], scale)) : "memory");
          }
        }
      }
      if (++stage == kRaw) {
        stage = 0;
        stage_parity ^= 1u;
      }
    }
    fence_async();
    named_arrive(slot_ready(slot), kSlotThreads<D>);
    slot += 2;
    if (slot >= kSlots) {
      slot -= kSlots;
      slot_parity ^= 1u;
    }
  }
}

// ---- the products, issued by one warp
template <int D>
__device__ __forceinline__ void product_role(const Job& job, Shared* sh, uint8_t* smem) {
  constexpr uint32_t kIdescS = instruction(Smem<D>::kTok, false), kIdescO = instruction(D, true);
  const uint32_t q_at = lt::smem_u32(smem + Smem<D>::kQ), kv_at = lt::smem_u32(smem + Smem<D>::kKv);
  const uint32_t tmem = __shfl_sync(~0u, sh->tmem, 0), lead = elect_one();
  wait_warp(&sh->q_full, 0, sh);
  constexpr int kTok = Smem<D>::kTok;
  constexpr bool kOne = Smem<D>::kOne;
  const int tiles = job.tiles;
  if (!kOne && tiles > 0) named_sync(slot_ready(0), kSlotThreads<D>);
  // One place for each product, in a rolled loop: first the weights of a tile by its values, then the logits
  // of a later one, into the columns that the weights were in. With two row tiles even steps
  // are row tile A's, odd ones B's, and the later tile is the next; with one row tile a step
  // is a tile's, and the later tile is the next but one. (Descriptors hold addresses in units of 16 bytes; the steps'
  // offsets are added to them.)
#pragma unroll 1
  for (int step = 0; step < (kOne ? tiles + 2 : 2 * tiles + 2) && tiles > 0; ++step) {
    const int buf = step & 1, which = kOne ? 0 : buf;
    const int i = kOne ? step - 2 : (step >> 1) - 1, next = kOne ? step : i + 1;
    const bool weights = i >= 0 && i < tiles, keys = next < tiles;
    const int value_slot = (uint32_t)(2 * i + 1) % kSlots, key_slot = (uint32_t)(2 * next) % kSlots;
    if (which == 1 && !job.two) continue;
    const bool last = which == 1 || !job.two;  // the product after which a slot is free
    if (weights) {
      if (which == 0) named_sync(slot_ready(value_slot), kSlotThreads<D>);
      const uint64_t value = desc_mn_major(kv_at + value_slot * Smem<D>::kOperand, Smem<D>::kHalf);
#pragma unroll
      for (int half = 0; half < kTok / 64; ++half) {
        named_sync(weights_ready(buf, half), kWeightsThreads);
        fence_after();
        mma_ts4<128>(tmem + kSumColumn + which * D, tmem + buf * kTok + half * 32, value + half * ((64 * 128) >> 4), kIdescO,
                     i > 0 || half > 0, lead);
      }
      if (last) mma_commit(&sh->kv_empty[value_slot], lead);
      if (kOne) mma_commit(&sh->o_tile, lead);
    }
    if (keys) {
      if (which == 0 && (kOne || weights)) named_sync(slot_ready(key_slot), kSlotThreads<D>);
      fence_after();
      const uint64_t q = desc_k_major(q_at + which * Smem<D>::kQTile);
      const uint64_t key = desc_k_major(kv_at + key_slot * Smem<D>::kOperand);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint64_t k = key + c * (Smem<D>::kHalf >> 4);
        if constexpr (kOne)
          mma_ts4<2>(tmem + buf * kTok, tmem + kQueryColumn + c * 32, k, kIdescS, c > 0, lead);
        else
          mma_ss4(tmem + buf * kTok, q + c * (Smem<D>::kQHalf >> 4), k, kIdescS, c > 0, lead);
      }
      mma_commit(&sh->s_full[buf], lead);
      if (last) mma_commit(&sh->kv_empty[key_slot], lead);
    }
  }
  mma_commit(&sh->o_full[0], lead);
  if (job.two) mma_commit(&sh->o_full[1], lead);
}

template <int D>
__global__ void __launch_bounds__(kCta, 1) prefill_kernel(AttentionParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (lt::smem_u32(smem_raw) & 1023u)) & 1023u);
  Shared* sh = reinterpret_cast<Shared*>(smem + Smem<D>::kBars);
  const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0);
  if (tid == 0) {
    for (int s = 0; s < Smem<D>::kRaw; ++s) {
      lt::mbar_init(&sh->packed_full[s], 1);
      lt::mbar_init(&sh->packed_empty[s], Smem<D>::kUnpackers / 32);
    }
    for (int s = 0; s < kSlots; ++s) lt::mbar_init(&sh->kv_empty[s], 1);
    lt::mbar_init(&sh->o_tile, 1);
    lt::mbar_init(&sh->q_full, Smem<D>::kRowTiles * 128);
    for (int t = 0; t < 2; ++t) {
      lt::mbar_init(&sh->s_full[t], 1);
      lt::mbar_init(&sh->o_full[t], 1);
    }
    sh->gave_up = 0;
    lt::mbar_fence_init();
  }
  dependency_wait();

  Job job;
  // A request's last rows see the most positions: every request's last row tile comes first, then their last
  // but one, so the long CTAs start early and the short ones fill in.
  const int units = gridDim.x / p.row_tiles;
  const int nth = blockIdx.x / units, unit = blockIdx.x % units;
  job.head = unit % p.heads;
  job.flat = unit / p.heads;
  Place pl;
  if (!find_place<kCta>(p, job.flat, &pl, sh->sums, &sh->found)) return;
  job.request = pl.request;
  job.rq = request_of(p, pl.request);
  job.rows = job.rq.computed * p.group;
  job.part = pl.part + pl.split;
  constexpr int kRows = Smem<D>::kRowTiles * 128;
  job.row_tile = min((job.rows + kRows - 1) / kRows, p.row_tiles) - 1 - nth;
  if (job.row_tile < 0) return;
  job.final_here = pl.count == 1;
  if (job.flat == pl.base && job.head == 0 && job.row_tile == 0 && tid == 0 && p.plan != nullptr)
    p.plan[pl.request] = make_int2(pl.part, pl.count);
  job.row0 = job.row_tile * kRows;
  job.two = kRows > 128 && job.rows - job.row0 > 128;
  {
    const int64_t at = job.rq.low + pl.split * chunk_of(p, job.rq, pl.count), end = at + chunk_of(p, job.rq, pl.count);
    job.from = (int)(at < job.rq.length ? at : job.rq.length);
    job.to = (int)(end < job.rq.length ? end : job.rq.length);
    const int last = min(job.rows - 1, job.row0 + kRows - 1) / p.group;
    job.to = min(job.to, job.rq.length - job.rq.queries + last + 1);
    if (p.window > 0)
      job.from = max(job.from, (job.rq.length - job.rq.queries + job.row0 / p.group + 1 - p.window) / p.align * p.align);
    job.tiles = job.to > job.from ? (job.to - job.from + Smem<D>::kTok - 1) / Smem<D>::kTok : 0;
  }

  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(lt::smem_u32(&sh->tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();

  if (warp < 4 * Smem<D>::kRowTiles)
    softmax_role<D>(p, job, sh, smem, warp / 4);
  else if (warp < 12)
    unpack_role<D>(job, sh, smem);
  else if (warp == 12)
    product_role<D>(job, sh, smem);
  else if (warp == 13)
    copy_role<D>(p, job, sh, smem);
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
  *smem = Smem<256>::kTotal;
  return reinterpret_cast<const void*>(&prefill_kernel<256>);
}

}  // namespace kv4
}  // namespace lt
