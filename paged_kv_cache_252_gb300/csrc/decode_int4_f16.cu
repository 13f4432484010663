// Instantiations of the INT4 decode kernel for fp16 queries.
#include "decode_int4_kernel.cuh"

namespace pkv {

DecodeInt4Kernel decode_int4_kernel_f16(int d, int rows) { return int4_kernel_for<false>(d, rows); }

}  // namespace pkv
