// lt_kv4_rows_plain.cu -- the attention kernels for few query rows, plain logits.
#include "lt_kv4_rows.cuh"

namespace lt {
namespace kv4 {
template RowsKernel rows_kernel_of<false>(int, int, bool);
}  // namespace kv4
}  // namespace lt
