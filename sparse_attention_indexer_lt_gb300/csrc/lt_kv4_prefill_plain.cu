// lt_kv4_prefill_plain.cu -- the attention kernels for many query rows, plain logits.
#include "lt_kv4_prefill.cuh"

namespace lt {
namespace kv4 {
template const void* prefill_kernel_ptr<false>(int, int*);
}  // namespace kv4
}  // namespace lt
