// Element codecs of the KV cache writers: E5M2 bytes and INT8 row scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

// fp16 bit pattern -> E5M2 byte. E5M2 keeps fp16's sign, exponent field and
// bias and the top two mantissa bits, so rounding the 16-bit magnitude at bit 8
// (round half to even: add 0x7F plus the bit that will become the last kept
// mantissa bit) yields the E5M2 magnitude directly; a carry moves into the
// exponent as it should. Results beyond the largest finite code 0x7B (57344),
// including infinities, saturate to it; NaN becomes 0x7E; the sign is kept.
__device__ __forceinline__ uint32_t e5m2_of_fp16(uint32_t h) {
  const uint32_t mag = h & 0x7FFFu;
  uint32_t r = (mag + 0x7Fu + ((mag >> 8) & 1u)) >> 8;
  r = r > 0x7Bu ? 0x7Bu : r;
  r = mag > 0x7C00u ? 0x7Eu : r;
  return ((h >> 8) & 0x80u) | r;
}

__device__ __forceinline__ uint32_t e5m2x4(uint32_t lo_pair, uint32_t hi_pair) {
  return e5m2_of_fp16(lo_pair & 0xFFFFu) | (e5m2_of_fp16(lo_pair >> 16) << 8) |
         (e5m2_of_fp16(hi_pair & 0xFFFFu) << 16) | (e5m2_of_fp16(hi_pair >> 16) << 24);
}

// Two fp32 values -> two E5M2 bytes (lo in bits 0..7), each rounded once (nearest, ties to
// even; |x| > 57344 and infinities saturate). The conversion instruction's NaN code is
// 0x7F; the cache's is 0x7E.
__device__ __forceinline__ uint32_t e5m2x2_of_f32(float lo, float hi) {
  uint16_t pair;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(hi), "f"(lo));
  uint32_t b = pair;
  if (lo != lo) b = (b & 0xFF00u) | 0x7Eu;
  if (hi != hi) b = (b & 0x00FFu) | 0x7E00u;
  return b;
}

// Scale of an INT8 row from its largest magnitude: max|x| / 127 rounded up to the nearest
// fp16 value (so that the decode can fold it into an fp16 weight exactly). IEEE
// division (__fdiv_rn), so codes do not depend on compiler flags.
__device__ __forceinline__ float int8_row_scale(float amax) {
  return __half2float(__float2half_ru(__fdiv_rn(amax, 127.0f)));
}

// round-half-even(x / scale) clamped to [-127, 127] (0 for an all-zero row), in
// offset binary (code + 128), which the decode kernel widens with one byte permute.
__device__ __forceinline__ uint32_t int8_byte(float x, float scale) {
  float qv = 0.f;
  if (scale != 0.f) {
    qv = rintf(__fdiv_rn(x, scale));
    qv = fmaxf(qv, -127.0f);
    qv = fminf(qv, 127.0f);
  }
  return static_cast<uint32_t>(static_cast<int>(qv) + 128);
}

}  // namespace pkv
