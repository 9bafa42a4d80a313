// lt_kv4_prefill.h -- internal: the attention kernel for many query rows a request.
#pragma once

namespace lt {
namespace kv4 {

constexpr int kPrefillThreads = 512;
// query rows of a CTA
inline int prefill_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }

// head_dim 64, 128 or 256; *smem: its dynamic shared memory.
const void* prefill_kernel_ptr(int head_dim, int* smem);

}  // namespace kv4
}  // namespace lt
