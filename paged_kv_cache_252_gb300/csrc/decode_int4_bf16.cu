// Instantiations of the INT4 decode kernel for bf16 queries.
#include "decode_int4_kernel.cuh"

namespace pkv {

DecodeInt4Kernel decode_int4_kernel_bf16(int d, int rows) { return int4_kernel_for<true>(d, rows); }

}  // namespace pkv
