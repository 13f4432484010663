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
  float z, s, inv;   // inv: 1 / s to a bit, 0 for s = 0
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
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.inv) : "f"(q.s));   // (s is 0 or normal in fp32)
  if (q.s == 0.f) q.inv = 0.f;
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

// Two fp32 operations an instruction, each rounded by itself.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 halves_of(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The code of x, its quotient v: settled exactly where v lies near a border.
__device__ __forceinline__ uint32_t int4_code(float x, float v, const Int4Group& q) {
  float c = rintf(v);
  if (fabsf(v - c) > 0.5f - 1e-5f) c = int4_code_exact(x, q.z, q.s, floorf(v));
  return static_cast<uint32_t>(__float2int_rn(c));
}

// The codes of a word's dimensions, x[m] = dimensions 2 m and 2 m + 1. Adding 1.5 * 2^23 to a quotient rounds it
// to the nearest code (halfway: the even one). A quotient in fp32 is off by less than 16 * 4 * 2^-24 < 4e-6: words with one
// nearer than 1e-5 to a border are settled exactly (one word in 5 of a warp's on 8-bit mantissas).
__device__ __forceinline__ uint32_t int4_word(const float2 (&x)[4], const Int4Group& q) {
  const uint64_t minus_z = f32x2(-q.z, -q.z), inv = f32x2(q.inv, q.inv), minus_inv = f32x2(-q.inv, -q.inv);
  const uint64_t magic = f32x2(12582912.f, 12582912.f), minus_magic = f32x2(-12582912.f, -12582912.f);
  uint64_t c[4];
  float off = 0.f;
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const uint64_t d = add2(f32x2(x[m].x, x[m].y), minus_z);
    c[m] = add2(fma2(d, inv, magic), minus_magic);
    const float2 o = halves_of(fma2(d, minus_inv, c[m]));
    off = fmaxf(off, fmaxf(fabsf(o.x), fabsf(o.y)));
  }
  if (off > 0.5f - 1e-5f) {
    uint32_t w = 0;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      w |= int4_code(x[m].x, (x[m].x - q.z) * q.inv, q) << int4_bit(2 * m);
      w |= int4_code(x[m].y, (x[m].y - q.z) * q.inv, q) << int4_bit(2 * m + 1);
    }
    return w;
  }
  // Four codes of 4 bits in a float's integer: the even dimensions' and the odd ones'.
  const uint64_t k16 = f32x2(16.f, 16.f);
  const float2 h = halves_of(add2(fma2(fma2(fma2(c[3], k16, c[2]), k16, c[1]), k16, c[0]), f32x2(8388608.f, 8388608.f)));
  return __byte_perm(__float_as_uint(h.x), __float_as_uint(h.y), 0x5410);
}

// Pair m (dimensions 2 m and 2 m + 1) of a word as fp16 numbers 0..15.
__device__ __forceinline__ __half2 int4_pair(uint32_t w, int m) {
  const uint32_t u = ((w >> (4 * m)) & 0x000F000Fu) | 0x64006400u;   // 1024 + c
  return __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6400)));
}

}  // namespace pkv
