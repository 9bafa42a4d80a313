// lt_kv4_prefill.h -- internal: the attention kernel for many query rows a request.
#pragma once

namespace lt {
namespace kv4 {

constexpr int kPrefillThreads = 512;
constexpr int kPrefillRows = 256;  // query rows of a CTA

// nullptr for a head size that it does not take; *smem: its dynamic shared memory.
const void* prefill_kernel_ptr(int head_dim, int* smem);

}  // namespace kv4
}  // namespace lt
