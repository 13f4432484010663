// The INT4 cache: its layout and the arithmetic of its codes.
//
// A row (token, KV head) of D dimensions is G = D / 64 groups of 64. A group holds z, the
// largest fp16 number not above its least value, s, the smallest fp16 number not below
// (its largest value - z) / 15, and 64 codes c in 0..15: dimension d stands for z + s c_d, c_d
// being the nearest of the sixteen (halfway: the even one). c never passes 15, as
// 15 s >= largest - z. Both numbers are fp16, so that z + s c is within half a step of any
// value of the group and s enters a product of fp16 operands unrounded. Values beyond
// +-65504 (a bf16 source's) count as +-65504; a group that holds an infinity or NaN has
// s = NaN and reads back as NaN.
//
// A row's codes are D / 8 32-bit words. Word i * G + g holds dimensions 64 g + 8 i + e,
// e = 0..7: e = 2 m at bits 4 m, e = 2 m + 1 at bits 16 + 4 m, so that (w >> 4 m) & 0x000F000F
// is a pair of neighbouring dimensions in the two halves of a register. The groups
// alternate by word: a thread that takes neighbouring words holds the same dimensions of
// every group. A block's [s, z] pairs lie as 32-bit words [K, V][16 tokens][G], s in the low half.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

constexpr int kInt4Group = 64;

// Bit position of dimension e (0..7) of a word.
__host__ __device__ constexpr int int4_bit(int e) { return (e & 1) * 16 + (e >> 1) * 4; }

// x + y as (d, err): d the rounded sum, d + err the exact one.
__device__ __forceinline__ float two_sum(float x, float y, float& err) {
  const float d = __fadd_rn(x, y), yy = __fsub_rn(d, x);
  err = __fadd_rn(__fsub_rn(x, __fsub_rn(d, yy)), __fsub_rn(y, yy));
  return d;
}

struct Int4Group {
  float z, s, inv;   // inv: 1 / s, 0 for s = 0
};

// z and s of a group from its least and largest value (within +-65504): exactly as defined, in fp32.
__device__ __forceinline__ Int4Group int4_group(float lo, float hi) {
  Int4Group q;
  q.z = __half2float(__float2half_rd(lo));
  float err;
  const float d = two_sum(hi, -q.z, err);
  __half s = __float2half_ru(__fdiv_rn(d, 15.f));
  // Rounding is monotonic, so s is not above the exact answer; it is below only where 15 s is
  // the rounded difference and the exact one is larger.
  if (__fmul_rn(15.f, __half2float(s)) == d && err > 0.f) s = __ushort_as_half(__half_as_ushort(s) + 1);
  q.s = __half2float(s);
  q.inv = q.s > 0.f ? __frcp_rn(q.s) : 0.f;
  q.z += 0.f;        // (-0 is 0)
  return q;
}

// The code of x where its quotient lies close to a border between two codes: the sign of
// x - z - border s, which fp32 gives exactly (border s has 16 bits, the difference of two close
// numbers is exact, and the sum of that with the first difference's rounding error keeps its sign).
static __device__ __noinline__ float int4_code_exact(float x, float z, float s, float below) {
  float err;
  const float d = two_sum(x, -z, err);
  const float t = __fadd_rn(__fsub_rn(d, __fmul_rn(below + 0.5f, s)), err);
  if (t != 0.f) return t > 0.f ? below + 1.f : below;
  return below * 0.5f == floorf(below * 0.5f) ? below : below + 1.f;   // halfway: the even code
}

// A quotient in fp32 is off by less than 16 * 3 * 2^-24 < 3e-6: codes of quotients nearer than 1e-5 to
// a border are settled exactly.
__device__ __forceinline__ uint32_t int4_code(float x, const Int4Group& q) {
  const float v = (x - q.z) * q.inv;
  float c = rintf(v);
  if (fabsf(v - c) > 0.5f - 1e-5f) c = int4_code_exact(x, q.z, q.s, floorf(v));
  return static_cast<uint32_t>(__float2int_rn(c));
}

// Pair m (dimensions 2 m and 2 m + 1) of a word as fp16 numbers 0..15.
__device__ __forceinline__ __half2 int4_pair(uint32_t w, int m) {
  const uint32_t u = ((w >> (4 * m)) & 0x000F000Fu) | 0x64006400u;   // 1024 + c
  return __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6400)));
}

}  // namespace pkv
