// Attention of a chunk of new tokens over the paged cache on the 5th-generation tensor
// core (tcgen05). For every unit (256 query rows of one sequence and KV head, see
// prefill_plan.cuh) and KV tile of 128 positions, per row tile i of 128 rows:
//   S_i (128 rows x 128 positions, fp32) = Q_i K^T          Q, K from shared memory
//   P_i = 2^(S_i c - m_i + shift)                            softmax warps, one row a thread
//   O_i (128 rows x D, fp32)  += P_i V                        P from tensor memory, V from shared
// with one pass over the positions, running maxima m and sums l in fp32. The two row tiles
// take turns: while one's scores are exponentiated the other's products run.
//
// Tensor memory (512 columns): O_0, O_1, S_0, S_1 at 0, 128, 256, 384. P_i (16-bit, 64
// columns) takes the place of the first half of S_i, which its own threads have read; the
// next S_i is issued behind the P V product that reads P_i (products execute in issue order).
//
// Warps: 0..3 and 4..7 the softmax of row tiles 0 and 1; warps 8 and 11 issue their products;
// warps 12..15 bring the K and V tiles: of a 16-bit cache as copies of 16-token boxes through the
// block table into the swizzled operand layout (and the queries; warp 10 clears V rows behind
// the context), of a one-byte cache from a ring of raw parts, widened to fp16 (warp 10 copies the
// parts and the queries). Warp 9 works out the pieces.
//
// Masks. Only tiles that reach past some row's last position compare positions; a masked
// score is -inf, its weight 0. V rows behind the context are zeroed (a stale NaN times
// weight 0 would be NaN). A later token of the chunk that holds an infinity or NaN still
// meets weight 0 of the rows before it: an output row with a non-finite element is
// computed again by prefill_row, which reads only what the row sees, unless what it sees accounts for
// all of them (accounted_for). A row whose weights have no sum is NaN.
//
// The running maximum moves only when a score exceeds it by more than kSlack (base 2) and a
// tile's weights so sum to more than kMostSum = 2^(kSlack + kShift): O is rescaled a few times a
// row, not every tile. fp16 weights carry a shift of 2^7: they stay at or below 2^15, and weights
// down to 2^-21 of the largest keep full precision. An INT8 cache's K scale multiplies the scores,
// its V scale the weight, and the product is what is rounded to fp16. So that these products keep full
// precision down to 2^-18 of the largest whatever the scales' size, m there is the largest sum of a
// score and its V scale's exponent, and l and O carry that factor. (Under the largest score alone, with
// a shift for the largest scale an fp16 row gives, 516, values of at most 0.0025 left weights of 2^-12
// of the largest no bits at all. The exponents cost an 8192-token prompt 1 %.) Their shift is 2^5: m has
// no slack there, so products may come to 65504 before it moves. The weights' rounding to 16 bits is the
// products' operand type; scores, sums and O stay fp32.
//
// Measured (32 query heads on 8 KV heads of 128 dimensions; a large library product of bf16
// reaches 1895 TFLOP/s). A KV tile against two row tiles is 2050 cycles of products; it takes
// 2500 to 2600 where only the softmax's instructions compete.
//   8192-token prompt    bf16 358 us, 1537 TFLOP/s: the products' operands and the softmax's
//                        chain from scores to weights share the SM (tensor pipe busy 66 %), and
//                        25 us are the ends of pieces; 16384 tokens 1320 us, 1665 TFLOP/s.
//                        E5M2 428 us: the stores of the widening pass are 20 us of the difference; the
//                        rest has no cause found (a ring of four stages, as here, costs bf16 nothing).
//                        INT8 513 us: its row scales, two 16-byte reads a thread for every four scores
//                        (the LSU's data pipe is busy 54 %, so not at its limit).
//   prompts of 512 / 1024 / 2048 tokens (bf16)   17 / 26 / 48 us: the start, some 8000 cycles from plan to
//                        first weights, and the ends of pieces, of 4000 to 10000, over few tiles.
//   head size 64         8192 tokens 312 us bf16, 327 E5M2, 406 INT8: half of the products, and the
//                        same chain from scores to weights, which is what a tile takes there.
//   100 tokens over a context of 130972 (bf16)   193 us, 537 MB read once: 80 us of memory time,
//                        113 of products; rows fill 400 of 512.
//   one token            10 us: five of launch and planning, five of one chain through the CTA.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <cstdint>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_tc.cuh"
#include "prefill_plan.cuh"
#include "prefill_row.cuh"

namespace pkv {

constexpr int kPfRing = 4;   // pieces worked out ahead

template <int KV, int D>
struct PfShape {
  static constexpr bool kWiden = KV == kKvE5m2 || KV == kKvInt8;
  static constexpr bool kBf16 = KV == kKvBf16;
  static constexpr int kHalves = D / 64;
  static constexpr int kThreads = 512;
  // Warps that read the pieces: eight softmax, two issuing, four loading, one more (warp 10).
  static constexpr int kReaders = 15;
  // Register budgets (per thread of a warpgroup); twice the first and the others make the
  // launch's 512 x 128. What spills decides: an 8192-token E5M2 prompt takes 422 us with 64 for the
  // issuing warps and 433 with 56, an INT8 one 511 with 184 / 64 / 80 and 527 with 192 / 48 / 80, of
  // head size 64 426 and 405.
  static constexpr int kLaunchRegs = 128;
  static constexpr bool kInt8Wide = KV == kKvInt8 && D == 128, kInt8Narrow = KV == kKvInt8 && D == 64;
  static constexpr int kSoftmaxRegs = kInt8Wide ? 184 : 192;
  static constexpr int kIssueRegs = kInt8Narrow ? 48 : (kWiden ? 64 : 72);
  static constexpr int kLoadRegs = KV == kKvInt8 ? 80 : (kWiden ? 64 : 56);
  static_assert(2 * kSoftmaxRegs + kIssueRegs + kLoadRegs == 4 * kLaunchRegs, "register split");
  static constexpr int kStages = kWiden ? (D == 128 ? 4 : 8) : (D == 128 ? 5 : 10);
  static constexpr uint32_t kHalfBytes = kPfTile * 128;             // 64 dimensions of a KV tile
  static constexpr uint32_t kStageBytes = kHalves * kHalfBytes;
  // V as the products read it: by block for 16-bit caches (a block's halves adjacent, as one
  // copy writes them), by half for widened tiles.
  static constexpr uint32_t kVBlockBytes = kWiden ? kBlockSize * 128 : kHalves * kBlockSize * 128;
  static constexpr uint32_t kVHalfStep = kWiden ? kHalfBytes : kBlockSize * 128;
  static constexpr uint32_t kQHalfBytes = kPfRows * 128;
  static constexpr uint32_t kQBytes = kHalves * kQHalfBytes;
  static constexpr float kSlack = KV == kKvInt8 ? 0.f : 8.f;
  static constexpr float kShift = KV == kKvBf16 ? 0.f : (KV == kKvInt8 ? 5.f : 7.f);
  // 2^(slack + shift); over INT8 the most the products may come to.
  static constexpr float kMostSum = KV == kKvBf16 ? 256.f : (KV == kKvInt8 ? 65504.f : 32768.f);
  // Row scales of an INT8 cache's tiles: tile t + kScaleRing is written once the K stage of
  // tile t + kScaleRing - kStages / 2 is released, which is after the softmax of the tile before
  // that one, so tile t's are no longer read when kScaleRing > kStages / 2.
  static constexpr int kScaleRing = kStages;
  static constexpr int kScaleSlot = 2 * kPfTile + 4;   // K, V, and the loading warps' largest V scales
  // Shared memory from a 1024-aligned base.
  static constexpr uint32_t kRing = kQBytes;
  static constexpr int kRawRing = 3;                                   // one-byte caches: parts of 8 KB as they lie
  static constexpr uint32_t kRaw = kRing + kStages * kStageBytes;
  static constexpr uint32_t kScales = kRaw + (kWiden ? kRawRing * 8192 : 0);   // INT8: [kScaleRing][kScaleSlot] floats
  static constexpr uint32_t kBars = kScales + (KV == kKvInt8 ? kScaleRing * kScaleSlot * 4 : 0);
  static constexpr uint32_t kMisc = kBars + (4 * kStages + 11 + 2 * kPfRing + kScaleRing + 2 * kRawRing) * 8;
  static constexpr uint32_t kPieces = kMisc + 256 + sizeof(PfStart);   // ring of kPfRing
  static constexpr uint32_t kSmem = kPieces + kPfRing * sizeof(PfPiece) + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

// One slot row tile: m[128], l[128], O[D / 8][128][8].
__host__ __device__ constexpr int pf_slot_floats(int d) { return 256 + d * 128; }

constexpr uint32_t kPfOCol = 0, kPfSCol = 256;

// Bounded wait: gives up after kWaitLimitNs or once another warp has given up. Rows being
// computed again (busy) take their time without counting.
struct PfCtl {
  volatile int abort;
  volatile int busy;
};
__device__ __forceinline__ bool pf_wait_sleeping(uint32_t bar, uint32_t parity, PfCtl* ctl) {
  uint64_t t0 = global_timer_ns();
  for (;;) {
    if (mbar_try_wait_sleep(bar, parity, kTcSleepNs)) return true;
    if (ctl->abort) return false;
    if (ctl->busy) t0 = global_timer_ns();
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
}
__device__ __forceinline__ bool pf_wait(uint32_t bar, uint32_t parity, PfCtl* ctl) {
  if (mbar_try_wait(bar, parity)) return true;
  return pf_wait_sleeping(bar, parity, ctl);
}

// A warp's flagged rows again, reading only what they see. Rows whose values account for what is not finite
// in them stand: with one such value early in a 4096-token prompt, to compute all rows behind it again took
// 40 ms instead of 0.05.
template <int KV, int D>
__device__ __forceinline__ void pf_redo(const PrefillArgs& a, unsigned mask, int s, int qb, int past, int j0, int first,
                                     int h, PfCtl* ctl) {
  if ((threadIdx.x & 31) == 0) atomicAdd(const_cast<int*>(&ctl->busy), 1);
  __syncwarp();
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  NonFinite out;
  int end = 0;
  for (unsigned rest = mask; rest; rest &= rest - 1) {
    const int r = first + __ffs(rest) - 1, j = j0 + r / a.group;
    out.add<KV == kKvBf16 ? kKvBf16 : kKvF16, E>(
        static_cast<const uint16_t*>(a.out) +
        (static_cast<size_t>(qb + j) * a.num_q_heads + h * a.group + r % a.group) * D + lane * E);
    end = max(end, past + j + 1);
  }
  const int upto = accounted_for<KV, D>(a, s, h, out, end);
  while (mask) {
    const int r = first + __ffs(mask) - 1;
    mask &= mask - 1;
    const int j = j0 + r / a.group;
    if (past + j + 1 >= upto) continue;
    prefill_row<KV, D>(a, s, qb + j, h * a.group + r % a.group, max(past + j + 1, 0));
  }
  if ((threadIdx.x & 31) == 0) atomicSub(const_cast<int*>(&ctl->busy), 1);
}

// 16 one-byte elements -> 16 fp16 in two 16-byte chunks, exact.
template <int KV>
__device__ __forceinline__ void widen16(const uint4& v, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KV == kKvE5m2) {
      o[2 * i] = __byte_perm(w[i], 0, 0x1404);
      o[2 * i + 1] = __byte_perm(w[i], 0, 0x3424);
    } else {
      // byte = code + 128: 0x64|byte is the fp16 value 1152 + code
      const uint32_t a = __byte_perm(w[i], 0x64646464u, 0x4140), b = __byte_perm(w[i], 0x64646464u, 0x4342);
      const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
      const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
      const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
      o[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
      o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

// Scores of positions vis and up: -inf.
__device__ __forceinline__ void pf_mask(uint32_t (&sv)[4][32], int vis) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll
    for (int e = 0; e < 32; ++e) sv[g][e] = 32 * g + e < vis ? sv[g][e] : 0xFF800000u;
  }
}

// The exponent e of a V scale below 2^e (as a number of 2^23 plus its field); -31 at least: 127 times a
// smaller one is half of the least step of an fp16 output.
__device__ __forceinline__ float scale_exponent(float v) {
  return __uint_as_float((__float_as_uint(fmaxf(fabsf(v), 0x1p-32f)) >> 23) | 0x4B000000u) - (8388608.f + 126.f);
}

// The largest of 128 scores times c (an INT8 cache's: times their K scales, which hold c, plus their V
// scales' exponents): eight chains.
template <int KV>
__device__ __forceinline__ float pf_max(const uint32_t (&sv)[4][32], float c, const float4* k_scales) {
  float mx[8];
  if constexpr (KV == kKvInt8) {
#pragma unroll
    for (int x = 0; x < 8; ++x) mx[x] = -INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 f = k_scales[8 * g + e / 4], v = k_scales[kPfTile / 4 + 8 * g + e / 4];
        const float x = fmaf(__uint_as_float(sv[g][e]), f.x, scale_exponent(v.x));
        const float y = fmaf(__uint_as_float(sv[g][e + 1]), f.y, scale_exponent(v.y));
        const float z = fmaf(__uint_as_float(sv[g][e + 2]), f.z, scale_exponent(v.z));
        const float w = fmaf(__uint_as_float(sv[g][e + 3]), f.w, scale_exponent(v.w));
        mx[2 * g] = max3(mx[2 * g], x, y);
        mx[2 * g + 1] = max3(mx[2 * g + 1], z, w);
      }
    }
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      mx[2 * g] = __uint_as_float(sv[g][0]);
      mx[2 * g + 1] = __uint_as_float(sv[g][1]);
    }
#pragma unroll
    for (int e = 2; e < 30; e += 4) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        mx[2 * g] = max3(mx[2 * g], __uint_as_float(sv[g][e]), __uint_as_float(sv[g][e + 1]));
        mx[2 * g + 1] = max3(mx[2 * g + 1], __uint_as_float(sv[g][e + 2]), __uint_as_float(sv[g][e + 3]));
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) mx[2 * g] = max3(mx[2 * g], __uint_as_float(sv[g][30]), __uint_as_float(sv[g][31]));
  }
  const float m = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
  return KV == kKvInt8 ? m : m * c;
}

// Weights 2^(s c + sub) of 128 scores, packed in pairs, and their sum; an INT8 cache's are packed
// times its V scales (its K scales, which hold c, multiply the scores). FMAs and sums go two to an instruction: alone on its scheduler
// a warp is quicker with scalar ones (787 against 963 cycles a tile), but every instruction
// saved beside the products counts (16384-token prompt 1511 us against 1620, with either in
// pairs 1544 and 1563).
template <int KV>
__device__ __forceinline__ void pf_weights(const uint32_t (&sv)[4][32], uint32_t (&pw)[4][16], float c, float sub,
                                           const float4* k_scales, const float4* v_scales, float& sum) {
  float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int g = 0; g < 4; ++g) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float4 kc = make_float4(c, c, c, c);
      // (read where they are used: hoisted, the scales' registers spill)
      if constexpr (KV == kKvInt8) kc = lds_f4_early(smem_addr(k_scales + 8 * g + e / 4));
      float q[4];
      fma_pair(q[0], q[1], __uint_as_float(sv[g][e]), __uint_as_float(sv[g][e + 1]), kc.x, kc.y, sub);
      fma_pair(q[2], q[3], __uint_as_float(sv[g][e + 2]), __uint_as_float(sv[g][e + 3]), kc.z, kc.w, sub);
#pragma unroll
      for (int x = 0; x < 4; ++x) q[x] = fast_exp2(q[x]);
      add_pair(l[0], l[1], q[0], q[1]);
      add_pair(l[2], l[3], q[2], q[3]);
      if constexpr (KV == kKvInt8) {
        const float4 f = lds_f4_early(smem_addr(v_scales + 8 * g + e / 4));
        mul_pair(q[0], q[1], f.x, f.y);
        mul_pair(q[2], q[3], f.z, f.w);
      }
      pw[g][e / 2] = pack2<KV == kKvBf16>(q[0], q[1]);
      pw[g][e / 2 + 1] = pack2<KV == kKvBf16>(q[2], q[3]);
    }
  }
  sum = (l[0] + l[1]) + (l[2] + l[3]);
}

// Boxes first, first + step, ... of a unit's query rows, one thread: box b holds tokens
// b * box_tokens .. of the unit; each 64-dimension half goes to its own half of the buffer.
template <int D>
__device__ __forceinline__ void pf_load_q(const PrefillArgs& a, const CUtensorMap* tm, uint32_t dst, uint32_t bar,
                                          int head, int token, int boxes, int first, int step) {
  const int rows = a.box_tokens * a.group;
  const int mine = boxes > first ? (boxes - first + step - 1) / step : 0;
  mbar_arrive_expect_tx(bar, mine * (D / 64) * rows * 128);
#pragma unroll 1
  for (int b = first; b < boxes; b += step) {
#pragma unroll
    for (int hf = 0; hf < D / 64; ++hf)
      tma_load_3d_keep(dst + hf * (kPfRows * 128) + b * rows * 128, tm, 64 * hf, head, token + b * a.box_tokens, bar);
  }
}

template <int KV, int D>
__global__ void __launch_bounds__(PfShape<KV, D>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k0,
                   const __grid_constant__ CUtensorMap tm_k1, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ PrefillArgs a) {
  using Sh = PfShape<KV, D>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_addr(smem);
  const uint32_t full = base + Sh::kBars, empty = full + 8 * NS;
  const uint32_t q_full = empty + 8 * NS, q_empty = q_full + 8;
  const uint32_t s_full = q_empty + 8;      // [2] scores of row tile i written
  const uint32_t p_ready = s_full + 16;     // [2] weights of row tile i written, O_i rescaled
  const uint32_t o_done = p_ready + 16;     // [2] last P V product of a piece's row tile i complete
  const uint32_t turn = o_done + 16;        // [2] row tile i's products may be issued
  const uint32_t final_bar = turn + 16;
  // Per stage, so that a use is never more than one phase ahead of its waiter:
  const uint32_t v_tail = final_bar + 8;    // [NS] V rows behind the context zeroed
  const uint32_t v_sent = v_tail + 8 * NS;  // [NS] copies of such a tile issued
  const uint32_t pc_full = v_sent + 8 * NS; // [kPfRing] piece worked out
  const uint32_t pc_empty = pc_full + 8 * kPfRing;   // [kPfRing] piece no longer read
  const uint32_t sc_full = pc_empty + 8 * kPfRing;   // [kScaleRing] row scales of a tile written (INT8)
  const uint32_t raw_full = sc_full + 8 * Sh::kScaleRing;   // [kRawRing] part landed (one-byte caches)
  const uint32_t raw_empty = raw_full + 8 * Sh::kRawRing;  // [kRawRing] part read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sh::kMisc);
  PfCtl* ctl = reinterpret_cast<PfCtl*>(smem + Sh::kMisc + 8);
  volatile int* last_piece = reinterpret_cast<volatile int*>(smem + Sh::kMisc + 16);   // [2]
  volatile unsigned* row_bad = reinterpret_cast<volatile unsigned*>(smem + Sh::kMisc + 160);   // [8] merged rows
  long long* scratch = reinterpret_cast<long long*>(smem + Sh::kMisc + 32);            // [16]
  PfStart* start = reinterpret_cast<PfStart*>(smem + Sh::kMisc + 256);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) {   // a lane for each index (one thread for all: 10.2 us a tiny call against 9.7)
    if (lane < NS) {
      mbar_init(full + 8 * lane, 4);
      mbar_init(empty + 8 * lane, 2);
      mbar_init(v_tail + 8 * lane, 1);
      mbar_init(v_sent + 8 * lane, 1);
    }
    if (lane < 2) {
      mbar_init(s_full + 8 * lane, 1);
      mbar_init(p_ready + 8 * lane, 4);
      mbar_init(o_done + 8 * lane, 1);
      mbar_init(turn + 8 * lane, 1);
    }
    if (lane < Sh::kScaleRing) mbar_init(sc_full + 8 * lane, 4);
    if (lane < Sh::kRawRing) {
      mbar_init(raw_full + 8 * lane, 1);
      mbar_init(raw_empty + 8 * lane, 4);
    }
    if (lane < kPfRing) {
      mbar_init(pc_full + 8 * lane, 1);
      mbar_init(pc_empty + 8 * lane, Sh::kReaders);
    }
    if (lane == 0) {
      mbar_init(q_full, Sh::kWiden ? 1 : 4);
      mbar_init(q_empty, 2);
      mbar_init(final_bar, 2);
      ctl->abort = 0;
      ctl->busy = 0;
    }
    fence_barrier_init();
    __syncwarp();
    if (lane == 0) mbar_arrive(turn);   // row tile 0 begins
  }
  if (warp == 8) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k0);
    prefetch_tensormap(&tm_v);
  }
  tc_fence_before_sync();
  pdl_wait_prior_grid();
  pf_plan(a, scratch, start);   // its barriers also publish the set-up above
  tc_fence_after_sync();
  pdl_launch_dependents();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  volatile PfPiece* ring = reinterpret_cast<volatile PfPiece*>(smem + Sh::kPieces);
  auto piece_ready = [&](uint32_t n) { return pf_wait(pc_full + 8 * (n % kPfRing), (n / kPfRing) & 1, ctl); };
  auto piece_done = [&](uint32_t n) { mbar_arrive(pc_empty + 8 * (n % kPfRing)); };

  if (start->any) {
    if (warp < 8) {
      // ------------------------------- softmax --------------------------------------
      regs_grow<Sh::kSoftmaxRegs>();
      const int i = warp >> 2;                      // row tile
      const int r = tid & 127;                      // row of the tile, TMEM lane
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
      const uint32_t s_col = lanes + kPfSCol + 128 * i, o_col = lanes + kPfOCol + 128 * i;
      const uint32_t bar_s = s_full + 8 * i, bar_p = p_ready + 8 * i, bar_o = o_done + 8 * i;
      const float c = a.scale_log2;
      bool alive = true;
      uint32_t cnt = 0, done = 0;                   // tiles and pieces of this row tile so far
      uint32_t seen = 0;                            // KV tiles of the CTA so far (INT8 scale ring)
      auto give_up = [&] {
        alive = false;
        ctl->abort = 1;
        if (lane == 0 && a.status) atomicOr(a.status, kDevTimeout);
      };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!alive) return;
        const bool ok = pf_wait(bar, parity, ctl);
        if (!__all_sync(0xffffffffu, ok)) give_up();
      };
      // The unit's row is fixed: query token tok behind the unit's first, query head hd of the group.
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
      const int ru = 128 * i + r, tok = ru / a.group, hd = ru - tok * a.group, tok0 = 128 * i / a.group;
      for (uint32_t np = 0;; ++np) {
        // All four warps go on or stop together (they meet at barriers).
        bool none = !alive || !piece_ready(np);
        if (bar_red_or(1 + i, 128, none)) break;
        const volatile PfPiece* pc = ring + np % kPfRing;
        if (pc->end) break;
        uint32_t nth = seen;                        // KV tile of the CTA
        const int ka = pc->ka, span = (pc->klast - ka) * kPfTile, pend = pc->klast * kPfTile;
        int left = pc->kb[i] - ka, p0 = PfPiece::at(ka, pc->rot, ka, pc->klast) * kPfTile;
        seen += pc->klast - ka;
        if (left <= 0) {
          __syncwarp();
          if (lane == 0) piece_done(np);
          continue;
        }
        // visible positions of this row and of the tile's first (<= 0: none)
        const int limit = ru < pc->rows ? pc->past + pc->j0 + tok + 1 : 0;
        const int limit0 = pc->past + pc->j0 + tok0 + 1;
        float m = -INFINITY, l = 0.f;
        int fresh = 1;   // 1 in the piece's first tile; opaque, or the loop body is compiled twice
        for (; left > 0; --left, ++cnt, ++nth, fresh = 0, p0 = p0 + kPfTile == pend ? pend - span : p0 + kPfTile) {
          asm volatile("" : "+r"(fresh));
          const bool first = fresh != 0;
          wait(bar_s, cnt & 1);
          const uint32_t slot = nth % Sh::kScaleRing;
          if constexpr (KV == kKvInt8) wait(sc_full + 8 * slot, (nth / Sh::kScaleRing) & 1);
          if (!alive) continue;
          tc_fence_after_sync();
          // Weights against the running maximum as it stands. Whether it may stand is seen from
          // their sum: a score over it by more than the slack shows as a sum over 2^slack (a tile's
          // 128 weights of at most 1 never do; of an INT8 cache the sum times the largest V scale, as the
          // packed products must stay in fp16's range), and a row with no maximum yet is known. Then, in a second round from the
          // same scores, the maximum is found and moves. (Finding it first in every tile cost 300
          // to 400 of the 1350 cycles between a tile's scores and weights.)
          const float4* k_scales = reinterpret_cast<const float4*>(smem + Sh::kScales) + slot * (Sh::kScaleSlot / 4);
          const bool masked = p0 + kPfTile > limit0;
          uint32_t pw[4][16];
          float ls, most = 1.f;   // a tile's sum of weights; its largest V scale
          if constexpr (KV == kKvInt8) {
            const float4 f = k_scales[kPfTile / 2];
            most = __uint_as_float(max(max(__float_as_uint(f.x), __float_as_uint(f.y)),
                                       max(__float_as_uint(f.z), __float_as_uint(f.w))));
          }
          auto round = [&](bool settle) {
            uint32_t sv[4][32];   // 32 scores each
            tmem_ld128(s_col, sv[0], sv[1], sv[2], sv[3]);
            if (__builtin_expect(masked, 0)) {
              __syncwarp();   // keeps this a branch: as predicated selects it would run in every tile
              pf_mask(sv, limit - p0);
            }
            if (__builtin_expect(settle, 0)) {
              const float mx = pf_max<KV>(sv, c, k_scales);
              const bool need = mx > m + Sh::kSlack;
              if (__any_sync(0xffffffffu, need)) {
                const float mn = need ? mx : m;
                const float alpha = need ? fast_exp2(m - mn) : 1.f;   // 0 from -inf
                m = mn;
                l *= alpha;
                if (!first) {
                  // Products complete in issue order: these scores were issued behind the last P V.
#pragma unroll 1
                  for (int e = 0; e < D; e += 16) {
                    uint32_t ov[16];
                    tmem_ld16(o_col + e, ov);
#pragma unroll
                    for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * alpha);
                    tmem_st16(o_col + e, ov);
                  }
                }
              }
            }
            pf_weights<KV>(sv, pw, c, Sh::kShift - (m == -INFINITY ? 0.f : m), k_scales, k_scales + 32, ls);
          };
          // (only rows that see positions of this tile ask for a second round)
          auto moves = [&] {
            return __any_sync(0xffffffffu, limit > p0 && (!(ls * most <= Sh::kMostSum) || m == -INFINITY)) != 0;
          };
          bool settle = true;
          if (!first) {
            round(false);
            settle = moves();
          }
          if (__builtin_expect(settle, 0)) round(true);
          l += ls;
#pragma unroll
          for (int g = 0; g < 4; ++g) tmem_st16_async(s_col + 16 * g, pw[g]);
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_p);
        }

        // ---- end of the piece ----
#ifdef PKV_GIVE_UP
        // (the build that tests this path: status[1] names softmax warps whose wait here runs out)
        if (a.status && (a.status[1] >> warp & 1)) give_up();
#endif
        wait(bar_o, done++ & 1);
        const int pieces = pc->pieces[i], first_cta = pc->first[i], own = pieces > 1 ? blockIdx.x - first_cta : 0;
        // A wait may have given up in one warp and not in its neighbour. Over a cut unit's piece they go
        // on as one: the join meets at barriers, and a piece that is counted must have been stored whole.
        if (pieces > 1 ? bar_red_or(1 + i, 128, !alive) : !alive) {
          alive = false;
          continue;   // to the barrier that ends it for all four
        }
        tc_fence_after_sync();
        const bool real = ru < pc->rows;
        uint16_t* dst = static_cast<uint16_t*>(a.out) +
                        (static_cast<size_t>(pc->qb + pc->j0 + tok) * a.num_q_heads + pc->h * a.group + hd) * D;
        bool odd = false;   // a real row whose result is not finite
        // The row's result is the sum over its unit's pieces p of w_p O_p, in their order, over that
        // of w_p l_p: this piece's O from tensor memory, others' (of a cut unit, for the last
        // to finish) from their slots.
        const size_t slot_sz = pf_slot_floats(D);
        auto slot_of = [&](int p) {
          return a.partials + (static_cast<size_t>(2 * (first_cta + p) + (p == 0 ? 1 : 0)) * a.slot_tiles + i) * slot_sz;
        };
        const int rows = min(pc->rows - 128 * i, 128);
        const bool few = rows <= 32;
        // One CTA adds up the pieces lo + step y, y < n, of which its own is the me-th: all of them,
        // or, of more than kPfJoin, first those of every group of g neighbours, then the groups' sums.
        int lo = 0, step = 1, n = pieces, me = own, g = 0;
        if (pieces > kPfJoin && !few) {
          for (g = 3; g * g < pieces;) ++g;
          lo = own / g * g;
          n = min(g, pieces - lo);
          me = own - lo;
        }
#pragma unroll 1
        for (;;) {
          bool write = true, last = true;
          float M = m, mu = m == -INFINITY ? 0.f : m, L = l;   // w_p = 2^(m_p - mu)
          if (n > 1) {
            // (A group's count is at its first CTA, the first group's at the next one: no other unit
            // begins at either.)
            unsigned long long* ctr = a.piece_counts + 2 * (first_cta + (g && lo == 0 ? 1 : lo)) + i;
            unsigned long long old = 0;   // (thread 0's) the counter as last seen
            if (r == 0) {
              // If every other piece is counted, this one is the last and need not be published (the
              // first piece of a unit, at the end of its CTA's stretch, usually is).
              const unsigned long long all = (static_cast<unsigned long long>(a.epoch) << 32) | (n - 1);
              old = *reinterpret_cast<volatile unsigned long long*>(ctr);
              last_piece[i] = !few && old == all && atomicCAS(ctr, all, 0ull) == all;   // 0: clear for a replay
              if (last_piece[i]) fence_acq_rel_gpu();   // the others' slots, for the threads behind the barrier
            }
            named_bar_sync(1 + i, 128);
            last = last_piece[i] != 0;
            if (!last) {
              float* sl = slot_of(lo + step * me);
              if (real) {
                sl[r] = m;
                sl[128 + r] = l;
              }
#pragma unroll 1
              for (int e = 0; e < D; e += 32) {
                uint32_t ov[32];
                tmem_ld32(o_col + e, ov);
                if (real) {
#pragma unroll
                  for (int x = 0; x < 32; x += 8) st_global_v8(sl + 256 + ((e + x) / 8 * 128 + r) * 8, ov + x);
                }
              }
              named_bar_sync(1 + i, 128);
              if (r == 0) {
                fence_acq_rel_gpu();   // releases what the barrier ordered before it
                const unsigned long long tag = static_cast<unsigned long long>(a.epoch) << 32;
                unsigned long long want;
                for (;;) {
                  const unsigned counted = (old >> 32) == a.epoch ? static_cast<unsigned>(old) : 0u;
                  want = static_cast<int>(counted + 1) == n ? 0ull : tag | (counted + 1);
                  const unsigned long long got = atomicCAS(ctr, old, want);
                  if (got == old) break;
                  old = got;
                }
                last_piece[i] = want == 0ull;
                if (want == 0ull) fence_acq_rel_gpu();
              }
              named_bar_sync(1 + i, 128);
              last = last_piece[i] != 0;
            }
            named_bar_sync(1 + i, 128);   // read before the next piece's flag
            write = last && !few;
            if (write && real) {
#pragma unroll 4
              for (int y = 0; y < n; ++y) M = fmaxf(M, y == me ? m : slot_of(lo + step * y)[r]);
              mu = M == -INFINITY ? 0.f : M;
              L = 0.f;
#pragma unroll 4
              for (int y = 0; y < n; ++y) {
                const float* sl = slot_of(lo + step * y);
                L = y == me ? fmaf(l, fast_exp2(m - mu), L) : fmaf(sl[128 + r], fast_exp2(sl[r] - mu), L);
              }
            }
            if (last && few) {
              // Few rows (single decode rows over a long context): items of 8 dimensions of one row,
              // spread over the 128 threads, all pieces from their slots.
              if (r < 4) row_bad[4 * i + r] = 0;
              named_bar_sync(1 + i, 128);
              const int items = rows * (D / 8);
#pragma unroll 1
              for (int it = r; it < items; it += 128) {
                const int ch = it / rows, rr = it - ch * rows;
                float M = -INFINITY;
#pragma unroll 4
                for (int p = 0; p < pieces; ++p) M = fmaxf(M, slot_of(p)[rr]);
                const float mr = M == -INFINITY ? 0.f : M;
                float Lr = 0.f, o[8] = {};
#pragma unroll 2
                for (int p = 0; p < pieces; ++p) {
                  const float* sl = slot_of(p);
                  const float wp = fast_exp2(sl[rr] - mr);
                  const float4* src = reinterpret_cast<const float4*>(sl + 256 + (ch * 128 + rr) * 8);
                  const float4 f0 = src[0], f1 = src[1];
                  Lr = fmaf(sl[128 + rr], wp, Lr);
                  o[0] = fmaf(wp, f0.x, o[0]);
                  o[1] = fmaf(wp, f0.y, o[1]);
                  o[2] = fmaf(wp, f0.z, o[2]);
                  o[3] = fmaf(wp, f0.w, o[3]);
                  o[4] = fmaf(wp, f1.x, o[4]);
                  o[5] = fmaf(wp, f1.y, o[5]);
                  o[6] = fmaf(wp, f1.z, o[6]);
                  o[7] = fmaf(wp, f1.w, o[7]);
                }
                const int u = 128 * i + rr, j = u / a.group;
                // (a row that sees nothing is 0; one whose visible scores are all -inf, or not all numbers, NaN)
                const bool blind = pc->past + pc->j0 + j < 0;
                const float inv = Lr > 0.f ? 1.f / Lr : (Lr == 0.f && blind ? 0.f : NAN);
                // (an unseen NaN scale of an INT8 cache spoils the sum, nothing else does)
                float bad = KV == kKvInt8 ? Lr - Lr : 0.f;
                uint32_t y[4];
#pragma unroll
                for (int x = 0; x < 8; x += 2) {
                  bad = fmaf(o[x], 0.f, fmaf(o[x + 1], 0.f, bad));
                  y[x / 2] = pack2<Sh::kBf16>(o[x] * inv, o[x + 1] * inv);
                }
                if (bad != 0.f && (KV == kKvInt8 || Lr > 0.f || blind)) atomicOr(const_cast<unsigned*>(row_bad) + 4 * i + (rr >> 5), 1u << (rr & 31));
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                          (static_cast<size_t>(pc->qb + pc->j0 + j) * a.num_q_heads + pc->h * a.group + u -
                                           j * a.group) * D + 8 * ch) = make_uint4(y[0], y[1], y[2], y[3]);
              }
              __threadfence_block();
              named_bar_sync(1 + i, 128);
              odd = (row_bad[4 * i + (warp & 3)] >> lane) & 1u;
            }
          }
          if (write && !(g && n == 1)) {
            // (as above)
            const float inv = L > 0.f ? 1.f / L : (L == 0.f && limit <= 0 ? 0.f : NAN), w_own = n > 1 ? fast_exp2(m - mu) : 1.f;
            float bad = 0.f;
#pragma unroll 1
            for (int e = 0; e < D; e += 32) {
              uint32_t ov[32];
              tmem_ld32(o_col + e, ov);
              if (real) {
                if (n > 1) {
                  float acc[32];
#pragma unroll
                  for (int x = 0; x < 32; ++x) acc[x] = 0.f;
#pragma unroll 1
                  for (int y = 0; y < n; ++y) {
                    if (y == me) {
#pragma unroll
                      for (int x = 0; x < 32; ++x) acc[x] = fmaf(w_own, __uint_as_float(ov[x]), acc[x]);
                    } else {
                      const float* sl = slot_of(lo + step * y);
                      const float wp = fast_exp2(sl[r] - mu);
                      uint32_t f[32];
#pragma unroll
                      for (int x = 0; x < 32; x += 8) ld_global_v8(sl + 256 + ((e + x) / 8 * 128 + r) * 8, f + x);
#pragma unroll
                      for (int x = 0; x < 32; ++x) acc[x] = fmaf(wp, __uint_as_float(f[x]), acc[x]);
                    }
                  }
#pragma unroll
                  for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(acc[x]);
                }
              }
              if (g) {
                tmem_st32(o_col + e, ov);
              } else if (real) {
                uint32_t y[16];
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                  const float u = __uint_as_float(ov[x]), v = __uint_as_float(ov[x + 1]);
                  bad = fmaf(u, 0.f, fmaf(v, 0.f, bad));
                  y[x / 2] = pack2<Sh::kBf16>(u * inv, v * inv);
                }
                // whole 32-byte sectors where the output's alignment allows: neighbouring threads
                // write different rows
                if (wide) {
                  st_global_v8(dst + e, y);
                  st_global_v8(dst + e + 16, y + 8);
                } else {
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    *reinterpret_cast<uint4*>(dst + e + 8 * x) = make_uint4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]);
                }
              }
            }
            odd = real && g == 0 && (KV == kKvInt8 ? !(bad == 0.f && L < INFINITY) : bad != 0.f && (L > 0.f || limit <= 0));
            if (g) {
              m = M;
              l = L;
            }
          }
          if (!last || g == 0) break;
          me = lo / g;
          n = (pieces + g - 1) / g;
          step = g;
          lo = g = 0;
        }
        __syncwarp();
        const unsigned again = __ballot_sync(0xffffffffu, odd);
        if (again) pf_redo<KV, D>(a, again, pc->s, pc->qb, pc->past, pc->j0, 128 * i + 32 * (warp & 3), pc->h, ctl);
        tc_fence_before_sync();   // O_i is read before the next piece's product overwrites it
        __syncwarp();
        if (lane == 0) piece_done(np);
      }
    } else if (warp >= 12) {
      regs_shrink<Sh::kLoadRegs>();
      if constexpr (!Sh::kWiden) {
        // -------------------- copies of queries and tiles (16-bit caches) ----------------
        // Four warps, one issuing lane each: a lane takes some 75 cycles over a copy, and a
        // 128-position K and V tile is 24 of them (one lane alone bounded the kernel). Warp x
        // copies blocks 2x and 2x + 1 of a tile: two 2 KB boxes (64 dimensions each) of K,
        // and for V, whose layout lets a block's halves lie together, one 4 KB box.
        const int x = warp - 12;
        const int total_rows = a.num_blocks * a.num_kv_heads * kBlockSize;   // host guarantees < 2^31
        uint32_t st = 0, stage = 0, round = 0, piece = 0, queries = 0;   // queries: pieces whose queries were asked for
        bool ok = true;
        for (;; ++piece) {
          ok = __all_sync(0xffffffffu, piece_ready(piece));
          const volatile PfPiece* pc = ring + piece % kPfRing;
          if (!ok || pc->end) break;
          const int32_t* bt = a.block_tables + static_cast<size_t>(pc->s) * a.max_blocks_per_seq;
          const int ctx = pc->ctx, h = pc->h, ka = pc->ka, klast = pc->klast, rot = pc->rot, tail = pc->tail;
          const int boxes = (pc->rows + a.box_tokens * a.group - 1) / (a.box_tokens * a.group);
          const int token = pc->qb + pc->j0;
          __syncwarp();
          if (lane == 0) piece_done(piece);
#pragma unroll 1
          for (int k = ka; k < klast; ++k) {
            // Rows of both blocks: lanes 0 and 1 look them up.
            int mine = total_rows;   // wholly past the end: the copy fills zeros
            if (lane < 2) {
              const int p = PfPiece::at(k, rot, ka, klast) * kPfTile + (2 * x + lane) * kBlockSize;
              if (p < ctx) {
                const int id = bt[p >> 4];
                if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
                  mine = (id * a.num_kv_heads + h) * kBlockSize;
                else if (a.status) atomicOr(a.status, kDevBadBlock);
              }
            }
            const int row0 = __shfl_sync(0xffffffffu, mine, 0), row1 = __shfl_sync(0xffffffffu, mine, 1);
            if (elect_one()) {
              if (k == ka) {
                ok = piece == 0 || pf_wait(q_empty, (piece - 1) & 1, ctl);
                if (ok) {
                  pf_load_q<D>(a, &tm_q, base, q_full, h * a.group, token, boxes, x, 4);
                  ++queries;
                }
              }
#pragma unroll 1
              for (int v = 0; v < 2 && ok; ++v) {
                if (st >= NS && !pf_wait(empty + 8 * stage, round ^ 1, ctl)) {
                  ok = false;
                  break;
                }
                const uint32_t bar = full + 8 * stage;
                const uint32_t dst = base + Sh::kRing + stage * Sh::kStageBytes;
                mbar_arrive_expect_tx(bar, Sh::kStageBytes / 4);
                if (v == 0) {
                  const uint32_t d = dst + 2 * x * (kBlockSize * 128);
                  tma_load_2d_keep(d, &tm_k0, 0, row0, bar);
                  tma_load_2d_keep(d + kBlockSize * 128, &tm_k0, 0, row1, bar);
                  if constexpr (Sh::kHalves == 2) {
                    tma_load_2d_keep(d + Sh::kHalfBytes, &tm_k1, 0, row0, bar);
                    tma_load_2d_keep(d + Sh::kHalfBytes + kBlockSize * 128, &tm_k1, 0, row1, bar);
                  }
                } else {
                  const uint32_t d = dst + 2 * x * Sh::kVBlockBytes;
                  tma_load_3d_keep(d, &tm_v, 0, row0, 0, bar);
                  tma_load_3d_keep(d + Sh::kVBlockBytes, &tm_v, 0, row1, 0, bar);
                  if (x == 0 && k == tail) mbar_arrive(v_sent + 8 * stage);
                }
                ++st;
                if (++stage == NS) {
                  stage = 0;
                  round ^= 1;
                }
              }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          if (!ok) break;
        }
        st = __reduce_max_sync(0xffffffffu, st);   // of the lane that counted
        queries = __reduce_max_sync(0xffffffffu, queries);
        if (lane == 0) {
          if (!ok) {
            ctl->abort = 1;
            if (a.status) atomicOr(a.status, kDevTimeout);
          }
          // Drain: every copy issued into this CTA's shared memory lands before exit. (Where a role
          // gave up a barrier may stay incomplete; the first such wait outlasts any copy.)
          bool landed = queries == 0 || mbar_wait(q_full, (queries - 1) & 1);
#pragma unroll 1
          for (uint32_t k = st > NS ? st - NS : 0; k < st && landed; ++k)
            landed = mbar_wait(full + 8 * (k % NS), (k / NS) & 1);
        }
        __syncwarp();
      } else {
        // ------------------------- widening loader (one-byte caches) --------------------
        // Warp 10 copies parts of 8 KB (half a tile of head size 128, a tile of 64) into a ring of raw
        // buffers; these four warps widen them into the stages the products read. A thread's rows
        // are the same in every block, so its addresses are constants beside the part's.
        constexpr int LPR = D / 16;               // lanes of a row (16 bytes each)
        constexpr int RPW = 32 / LPR;             // rows of a warp's 16-byte reads
        constexpr int NL = 4;                     // reads of a thread per part
        constexpr int kParts = D / 64;            // parts of a tile's K or V
        const int wi = warp - 12, wt = tid - 384;
        const int cc = lane % LPR, rw = wi * RPW + lane / LPR;
        const uint8_t* raw = smem + Sh::kRaw + rw * D + ((cc ^ (D == 128 ? rw & 7 : (rw >> 1) & 3)) << 4);
        // Elements 16 cc .. 16 cc + 15: chunks 2 (cc % 4), + 1 of half cc / 4. The upper half's
        // lanes write their second chunk first, so that a row's eight lanes cover eight chunks
        // (all banks) in each store.
        const bool upper = (cc >> 2) != 0;
        const int c0 = 2 * (cc & 3) + (cc >> 2), c1 = 2 * (cc & 3) + 1 - (cc >> 2);
        uint8_t* out0 = smem + Sh::kRing + (cc >> 2) * Sh::kHalfBytes + rw * 128;
        const int o0 = (c0 ^ (rw & 7)) << 4, o1 = (c1 ^ (rw & 7)) << 4;
        uint32_t stage = 0, round = 0, uses = 0, tiles = 0, slot = 0, raw_round = 0;
        bool alive = true;
        for (uint32_t np = 0; alive; ++np) {
          alive = __all_sync(0xffffffffu, piece_ready(np));
          const volatile PfPiece* pc = ring + np % kPfRing;
          if (!alive || pc->end) break;
          const int32_t* bt = a.block_tables + static_cast<size_t>(pc->s) * a.max_blocks_per_seq;
          const int ctx = pc->ctx, h = pc->h, ka = pc->ka, klast = pc->klast;
          int t = PfPiece::at(ka, pc->rot, ka, klast);
          __syncwarp();
          if (lane == 0) piece_done(np);
          auto next = [&](int x) { return x + 1 == klast ? ka : x + 1; };   // (behind the last step: unused)
          // Row scales of an INT8 cache, a tile ahead; their blocks' ids another tile.
          auto id_of = [&](int x) {
            const int pos = x * kPfTile + wt;
            return pos < ctx ? bt[pos >> 4] : -1;
          };
          auto scales_of = [&](int id, float& k, float& v) {
            k = v = 0.f;
            if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.num_blocks)) return;
            const float* from = a.scales + (static_cast<size_t>(id) * a.num_kv_heads + h) * 32 + (wt & 15);
            k = from[0] * a.scale_log2;
            v = from[16];
          };
          int id = -1;
          float next_k = 0.f, next_v = 0.f;
          if constexpr (KV == kKvInt8) {
            scales_of(id_of(t), next_k, next_v);
            id = id_of(next(t));
          }
#pragma unroll 1
          for (int k = ka; k < klast; ++k, t = next(t)) {
            const float scale_k = next_k, scale_v = next_v;
            if constexpr (KV == kKvInt8) {
              scales_of(id, next_k, next_v);
              id = id_of(next(next(t)));
            }
#pragma unroll 1
            for (int n = 0; n < 2 * kParts; ++n) {
              const int part = n & (kParts - 1), v = n / kParts;
              bool ok = part != 0 || uses < NS || pf_wait(empty + 8 * stage, round ^ 1, ctl);
              ok = ok && pf_wait(raw_full + 8 * slot, raw_round, ctl);
              if (!__all_sync(0xffffffffu, ok)) {
                alive = false;
                ctl->abort = 1;
                if (lane == 0 && a.status) atomicOr(a.status, kDevTimeout);
                break;
              }
              const uint8_t* src = raw + slot * 8192;
              uint8_t* dst = out0 + stage * Sh::kStageBytes + part * (kPfTile / kParts) * 128;
              uint4 x[NL];
#pragma unroll
              for (int q = 0; q < NL; ++q) x[q] = *reinterpret_cast<const uint4*>(src + q * 2048);
              __syncwarp();
              if (lane == 0) mbar_arrive(raw_empty + 8 * slot);
              if (++slot == Sh::kRawRing) {
                slot = 0;
                raw_round ^= 1;
              }
              if (t * kPfTile + kPfTile > ctx) {   // rows behind the context: whatever the block holds
                const int row = t * kPfTile + part * (kPfTile / kParts) + rw;
#pragma unroll
                for (int q = 0; q < NL; ++q)
                  if (row + q * (4 * RPW) >= ctx) x[q] = make_uint4(0u, 0u, 0u, 0u);
              }
#pragma unroll
              for (int q = 0; q < NL; ++q) {
                uint4 lo, hi;
                widen16<KV>(upper ? make_uint4(x[q].z, x[q].w, x[q].x, x[q].y) : x[q], lo, hi);
                *reinterpret_cast<uint4*>(dst + q * (4 * RPW * 128) + o0) = lo;
                *reinterpret_cast<uint4*>(dst + q * (4 * RPW * 128) + o1) = hi;
              }
              if (part == kParts - 1) {
                if constexpr (KV == kKvInt8) {
                  // a masked score, -inf, must stay that times an all-zero row's K scale
                  const float f = v ? scale_v : (scale_k == 0.f ? 1e-30f : scale_k);
                  float* to = reinterpret_cast<float*>(smem + Sh::kScales) + tiles % Sh::kScaleRing * Sh::kScaleSlot;
                  to[v * kPfTile + wt] = f;
                  // (bits of positive floats are in their order, a NaN's above all)
                  const unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(f)));
                  if (v && lane == 0) to[2 * kPfTile + wi] = __uint_as_float(most);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                  mbar_arrive(full + 8 * stage);
                  if (KV == kKvInt8 && v == 1) mbar_arrive(sc_full + 8 * (tiles % Sh::kScaleRing));
                }
                tiles += v;
                ++uses;
                if (++stage == NS) {
                  stage = 0;
                  round ^= 1;
                }
              }
            }
            if (!alive) break;
          }
        }
      }
    } else {
      regs_shrink<Sh::kIssueRegs>();
      if (warp == 8 || warp == 11) {
        // ----------------------------- product issue ----------------------------------
        // One thread for each row tile. The tensor pipe accepts a product only when the one
        // before has nearly run, so a single thread's waits, commits and bookkeeping (some 700
        // cycles of a KV tile's 3550) were idle time there; with two, one thread's fall into the
        // other's products. They take strict turns, a row tile's products of one KV tile each:
        // left to themselves both row tiles fall into step and their softmax leaves the pipe idle
        // (8192-token prompt: 577 us). The turn passes before a thread's last product.
        if (elect_one()) {
          const int i = warp == 8 ? 0 : 1;
          constexpr uint32_t id_s = idesc_kind_f16(128, 128, Sh::kBf16, 0, 0);   // Q (K-major) x K^T (K-major)
          constexpr uint32_t id_o = idesc_kind_f16(128, D, Sh::kBf16, 0, 1);     // P (TMEM) x V (dimensions contiguous)
          // An operand's later atoms: its first descriptor with the address field advanced
          // (16-byte units; shared-memory addresses stay below 2^18, so it never carries).
          const uint64_t dq = smem_desc_sw128(base + i * 128 * 128, 0, 1024);
          const uint64_t dk = smem_desc_sw128(base + Sh::kRing, 0, 1024);
          const uint64_t dv = smem_desc_sw128(base + Sh::kRing, Sh::kVHalfStep, 1024);
          const uint32_t t_s = tmem + kPfSCol + 128 * i, t_o = tmem + kPfOCol + 128 * i;
          uint32_t stage = 0, round = 0, cnt = 0, piece = 0, tails = 0;
          bool ok = true;
          auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!pf_wait(bar, parity, ctl)) ok = false;
            return ok;
          };
          auto next_stage = [&] {
            if (++stage == NS) {
              stage = 0;
              round ^= 1;
            }
          };
          const uint32_t my_turn = turn + 8 * i, other_turn = turn + 8 * (1 - i);
          uint32_t turns = 0;
          auto issue_s = [&](uint32_t at) {
            const uint64_t kb = dk + ((at * Sh::kStageBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              if (kk == D / 16 - 1) mbar_arrive(other_turn);
              tc_mma_f16_ss(t_s, dq + (((kk >> 2) * Sh::kQHalfBytes + (kk & 3) * 32) >> 4),
                            kb + (((kk >> 2) * Sh::kHalfBytes + (kk & 3) * 32) >> 4), id_s, kk > 0);
            }
            tc_commit(s_full + 8 * i);
          };
          // Stages (and the queries) are released by both threads: behind the products that
          // read them, or at once where this row tile has none.
          for (;; ++piece) {
            if (!piece_ready(piece)) {
              ok = false;
              break;
            }
            const volatile PfPiece* pc = ring + piece % kPfRing;
            if (pc->end) break;
            const int tail = Sh::kWiden ? -1 : pc->tail;   // see warp 10
            const int kb = pc->kb[i], klast = pc->klast;
            int k = pc->ka;
            piece_done(piece);
            if (!wait(q_full, piece & 1)) break;
            if (!wait(full + 8 * stage, round)) break;
            if (!wait(my_turn, turns++ & 1)) break;
            if (k < kb) {
              tc_fence_after_sync();
              issue_s(stage);
              tc_commit(empty + 8 * stage);
              if (k + 1 == kb) tc_commit(q_empty);
            } else {
              mbar_arrive(other_turn);
              mbar_arrive(empty + 8 * stage);
              mbar_arrive(q_empty);
            }
            next_stage();
            int fresh = 1;   // 1 at the piece's first tile; opaque, or the loop body is compiled twice
#pragma unroll 1
            for (; k < klast; ++k, fresh = 0) {
              asm volatile("" : "+r"(fresh));
              const bool first = fresh != 0;
              const uint32_t vs = stage;
              if (!wait(full + 8 * vs, round)) break;
              next_stage();
              const uint32_t ks = stage;
              if (k + 1 < klast) {
                if (!wait(full + 8 * ks, round)) break;
                next_stage();
              }
              if (k == tail) {
                if (k < kb && !wait(v_tail + 8 * vs, (tails >> vs) & 1)) break;
                tails ^= 1u << vs;
              }
              if (k < kb) {
                const uint64_t vb = dv + ((vs * Sh::kStageBytes) >> 4);
                if (!wait(p_ready + 8 * i, cnt & 1) || !wait(my_turn, turns++ & 1)) break;
                ++cnt;
                tc_fence_after_sync();
                const bool more = k + 1 < kb;
#pragma unroll
                for (int kk = 0; kk < kPfTile / 16; ++kk) {
                  if (kk == kPfTile / 16 - 1 && !more) mbar_arrive(other_turn);
                  tc_mma_f16_ts(t_o, t_s + kk * 8, vb + ((kk * Sh::kVBlockBytes) >> 4), id_o, kk > 0 || !first);
                }
                if (more) {
                  issue_s(ks);
                  tc_commit(empty + 8 * ks);
                  if (k + 2 == kb) tc_commit(q_empty);   // the last scores are issued
                } else {
                  tc_commit(o_done + 8 * i);   // else the next scores' barrier tells of it
                  if (k + 1 < klast) mbar_arrive(empty + 8 * ks);
                }
                tc_commit(empty + 8 * vs);
              } else {
                if (!wait(my_turn, turns++ & 1)) break;
                mbar_arrive(other_turn);
                mbar_arrive(empty + 8 * vs);
                if (k + 1 < klast) mbar_arrive(empty + 8 * ks);
              }
            }
            if (!ok) break;
          }
          if (!ok) {
            ctl->abort = 1;
            if (a.status) atomicOr(a.status, kDevTimeout);
          }
          // Every product issued completes before the tensor memory is released.
          tc_commit(final_bar);
          mbar_wait(final_bar, 0);
        }
        __syncwarp();
      } else if (warp == 10 && !Sh::kWiden) {
        // ---------------- V rows behind the context in its last block: zeros --------------
        // (Whole blocks behind it are copied as zeros.) A piece that ends in such a block has the
        // product wait for this warp once.
        uint32_t st = 0, sent = 0;
        bool ok = true;
        for (uint32_t np = 0;; ++np) {
          ok = __all_sync(0xffffffffu, piece_ready(np));
          const volatile PfPiece* pc = ring + np % kPfRing;
          if (!ok || pc->end) break;
          const int ctx = pc->ctx, ka = pc->ka, klast = pc->klast, tail = pc->tail;
          __syncwarp();
          if (lane == 0) piece_done(np);
          if (tail >= ka && tail < klast) {
            const uint32_t vst = st + 2 * (tail - ka) + 1, vs = vst % NS;
            // Once this use's copies are issued, the stage's barrier is in this use's phase.
            ok = pf_wait(v_sent + 8 * vs, (sent >> vs) & 1, ctl) && pf_wait(full + 8 * vs, (vst / NS) & 1, ctl);
            sent ^= 1u << vs;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int r0 = ctx & (kPfTile - 1), r1 = (r0 + 15) & ~15;
            uint8_t* vt = smem + Sh::kRing + vs * Sh::kStageBytes;
#pragma unroll 1
            for (int x = lane; x < (r1 - r0) * Sh::kHalves * 8; x += 32) {
              const int row = r0 + x / (Sh::kHalves * 8), ch = x % (Sh::kHalves * 8);
              *reinterpret_cast<uint4*>(vt + (row >> 4) * Sh::kVBlockBytes + (ch >> 3) * Sh::kVHalfStep +
                                        (row & 15) * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_tail + 8 * vs);
          }
          st += 2 * (klast - ka);
        }
        if (!ok && lane == 0) {
          ctl->abort = 1;
          if (a.status) atomicOr(a.status, kDevTimeout);
        }
        __syncwarp();
      } else if (warp == 10) {
        // ----------------- copies of queries and raw parts (one-byte caches) -----------------
        // Lane b copies block b of a tile; its row is looked up a tile ahead. A piece's queries go
        // behind its first K and V parts, which need not wait for the piece before to end.
        constexpr int kParts = D / 64, kPer = kPfTile / kBlockSize / kParts;   // blocks of a part
        const int total_rows = a.num_blocks * a.num_kv_heads * kBlockSize;   // host guarantees < 2^31
        uint32_t parts = 0, slot = 0, round = 0, piece = 0, queries = 0;
        bool ok = true;
        for (;; ++piece) {
          ok = __all_sync(0xffffffffu, piece_ready(piece));
          const volatile PfPiece* pc = ring + piece % kPfRing;
          if (!ok || pc->end) break;
          const int32_t* bt = a.block_tables + static_cast<size_t>(pc->s) * a.max_blocks_per_seq;
          const int ctx = pc->ctx, h = pc->h, ka = pc->ka, klast = pc->klast;
          const int boxes = (pc->rows + a.box_tokens * a.group - 1) / (a.box_tokens * a.group);
          const int token = pc->qb + pc->j0;
          int t = PfPiece::at(ka, pc->rot, ka, klast);
          __syncwarp();
          if (lane == 0) piece_done(piece);
          auto id_of = [&](int x) {
            const int pos = x * kPfTile + lane * kBlockSize;
            return lane < kPfTile / kBlockSize && pos < ctx ? bt[pos >> 4] : -1;
          };
          int id = id_of(t);
          bool asked = false;
#pragma unroll 1
          for (int k = ka; k < klast && ok; ++k) {
            int row = total_rows;   // wholly past the end: the copy fills zeros
            if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_blocks))
              row = (id * a.num_kv_heads + h) * kBlockSize;
            else if (lane < kPfTile / kBlockSize && t * kPfTile + lane * kBlockSize < ctx && a.status)
              atomicOr(a.status, kDevBadBlock);
            t = t + 1 == klast ? ka : t + 1;
            id = id_of(t);
#pragma unroll 1
            for (int n = 0; n < 2 * kParts; ++n) {
              const int at = lane - (n & (kParts - 1)) * kPer;
              ok = parts < Sh::kRawRing || pf_wait(raw_empty + 8 * slot, round ^ 1, ctl);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              if (lane == 0) mbar_arrive_expect_tx(raw_full + 8 * slot, 8192);
              __syncwarp();
              if (at >= 0 && at < kPer)
                tma_load_2d_keep(base + Sh::kRaw + slot * 8192 + at * (kBlockSize * D), n < kParts ? &tm_k0 : &tm_v, 0, row,
                                 raw_full + 8 * slot);
              ++parts;
              if (++slot == Sh::kRawRing) {
                slot = 0;
                round ^= 1;
              }
              if (!asked && n == 1) {
                asked = true;
                ok = piece == 0 || pf_wait(q_empty, (piece - 1) & 1, ctl);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) pf_load_q<D>(a, &tm_q, base, q_full, h * a.group, token, boxes, 0, 1);
                ++queries;
                __syncwarp();
              }
            }
          }
          if (!ok) break;
        }
        if (lane == 0) {
          if (!ok) {
            ctl->abort = 1;
            if (a.status) atomicOr(a.status, kDevTimeout);
          }
          // Every copy issued lands before exit (where a role gave up: within these bounded waits).
          bool landed = queries == 0 || mbar_wait(q_full, (queries - 1) & 1);
#pragma unroll 1
          for (uint32_t n = parts > Sh::kRawRing ? parts - Sh::kRawRing : 0; n < parts && landed; ++n)
            landed = mbar_wait(raw_full + 8 * (n % Sh::kRawRing), (n / Sh::kRawRing) & 1);
        }
        __syncwarp();
      } else if (warp == 9) {
        // ------------------------------- pieces ---------------------------------------------
        if (lane == 0) {
          uint32_t np = 0;
          auto room = [&] { return np < kPfRing || pf_wait(pc_empty + 8 * (np % kPfRing), (np / kPfRing - 1) & 1, ctl); };
          bool ok = true;
          for (PfWalk w(a, *start); !w.done(); w.advance()) {
            if (!(ok = room())) break;
            if (!pf_piece(w, ring + np % kPfRing)) continue;
            mbar_arrive(pc_full + 8 * (np % kPfRing));
            ++np;
          }
          if (ok && (ok = room())) {
            ring[np % kPfRing].end = 1;
            mbar_arrive(pc_full + 8 * (np % kPfRing));
          }
          if (!ok) {
            ctl->abort = 1;
            if (a.status) atomicOr(a.status, kDevTimeout);
          }
        }
        __syncwarp();
      }
    }
  }

  // Teardown: every role is done with the tensor memory.
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace pkv
