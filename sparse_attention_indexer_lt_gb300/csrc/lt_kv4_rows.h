// lt_kv4_rows.h -- internal: the attention kernel for few query rows a request.
#pragma once

namespace lt {
namespace kv4 {

constexpr int kMaxParts = 8;  // CTAs of a portable cluster

struct RowsKernel {
  const void* func;
  int smem, per_sm;
};

// head_dim 64, 128 or 256, nt tiles of 8 query rows: 1, 2 or (not with 256) 4; kShaped: logits with a cap, a
// slope or a prefix
template <bool kShaped>
RowsKernel rows_kernel_of(int head_dim, int nt, bool list);
extern template RowsKernel rows_kernel_of<false>(int, int, bool);
extern template RowsKernel rows_kernel_of<true>(int, int, bool);

}  // namespace kv4
}  // namespace lt
