// lt_kv4_rows_shaped.cu -- the attention kernels for few query rows, logits with a cap, a slope or a prefix.
#include "lt_kv4_rows.cuh"

namespace lt {
namespace kv4 {
template RowsKernel rows_kernel_of<true>(int, int, bool);
}  // namespace kv4
}  // namespace lt
