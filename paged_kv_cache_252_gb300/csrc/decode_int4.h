// The INT4 decode kernels as their host code sees them.
#pragma once

#include <cstddef>
#include <cstdint>

#include "pkv_internal.h"

namespace pkv {

struct DecodeInt4Args : DecodeArgs {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* meta;         // [block][KV head][K, V][16][D / 64] words: s, z
};

struct DecodeInt4Kernel {
  const void* fn;
  int threads;
  size_t smem;                 // for units of the given rows
};
DecodeInt4Kernel decode_int4_kernel_f16(int d, int rows);
DecodeInt4Kernel decode_int4_kernel_bf16(int d, int rows);
inline DecodeInt4Kernel decode_int4_kernel_of(int d, int rows, bool bf16) {
  return bf16 ? decode_int4_kernel_bf16(d, rows) : decode_int4_kernel_f16(d, rows);
}

}  // namespace pkv
