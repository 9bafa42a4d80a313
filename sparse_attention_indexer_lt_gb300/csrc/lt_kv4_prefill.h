// lt_kv4_prefill.h -- internal: the attention kernel for many query rows a request.
#pragma once

namespace lt {
namespace kv4 {

constexpr int kPrefillThreads = 512;
// query rows of a CTA
inline int prefill_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }

// head_dim 64, 128 or 256; *smem: its dynamic shared memory; kShaped: logits with a cap, a slope or a prefix.
template <bool kShaped>
const void* prefill_kernel_ptr(int head_dim, int* smem);
extern template const void* prefill_kernel_ptr<false>(int, int*);
extern template const void* prefill_kernel_ptr<true>(int, int*);

}  // namespace kv4
}  // namespace lt
