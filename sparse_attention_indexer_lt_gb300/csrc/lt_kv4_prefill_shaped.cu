// lt_kv4_prefill_shaped.cu -- the attention kernels for many query rows, logits with a cap, a slope or a prefix.
#include "lt_kv4_prefill.cuh"

namespace lt {
namespace kv4 {
template const void* prefill_kernel_ptr<true>(int, int*);
}  // namespace kv4
}  // namespace lt
