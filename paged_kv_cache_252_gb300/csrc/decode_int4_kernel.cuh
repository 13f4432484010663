// Paged decode attention over an INT4 cache (layout and codec: pkv_int4.cuh). The work line, the
// pieces and their combination are those of decode_common.cuh; this file is what a CTA does
// with its share.
//
// Mathematics. With a group's codes c, scale s and least value z (K: per token and 64 dimensions):
//   score(t, r) = sum over groups  s_tg (q_rg . c_tg) + z_tg sum(q_rg)
//   out(r, d)   = sum over t  p_tr (z_tg + s_tg c_td) / sum over t p_tr
//               = [ sum_t P_tr (c_td - 8)  +  sum_t p_tr (z_tg + 8 s_tg) ] / sum_t p_tr,   P = p s
// so both products run on the codes themselves (mma.sync m16n8k16, fp16 operands, fp32
// accumulators) and the scales touch only scores and weights. A code enters without any
// conversion: four bits in the lowest bits of a 16-bit half are the fp16 number c 2^-24, four
// bits above them c 2^-20, so one AND makes a pair of operands. The 2^-24 is exact and comes off in
// fp32; where a pair is 16 times too large, q is stored 16 times smaller (K) or the output
// row is scaled at the end (V). The 8 is taken off by a product with a constant operand, over the same
// rounded P, every few steps.
//
// Precision. q is scaled by a power of two per row so that its largest element lies in [2^11, 2^12) (every other pair of
// dimensions 16 times lower): fp16 then holds the 11 bits of an fp16 query exactly down to 2^-21 of the largest, a bf16
// query's 8 down to 2^-24. The running reference m of a row is of the score plus the exponent of the token's V scale, so
// that P, rounded to fp16, is at most 2^15 and keeps all its bits down to 2^-25 of the largest contribution
// whatever the scales' size. m starts from and moves on exact maxima, but only when a P (or a p beside a
// zero scale) passes the limit: a rare, warp-wide event.
//
// Structure of a CTA: WR x WB warps. Row warp wr has 8 NT of the unit's rows; stream wb takes every
// WB-th step of STEP blocks of the share through a ring of its own of RING steps, filled by cp.async of the
// stream's own warps (no producer warp: at 2.3 KB a block one issuing thread would bound the CTA).
// A lane's K words of a token (neighbouring 16 bytes) are the A operand of S^T = K Q^T as they
// lie; V words of two tokens are paired by byte permutes for O^T = V^T P^T. The tokens of a
// block take the 16 product slots in an order in which both reads hit all banks.
//
// What bounds it. One query token of 4 heads a KV head: instructions, 248 a warp and block (64 of them the ANDs that
// unpack), issued on 52 % of the cycles with three warps a scheduler, most stalls on fixed latencies: 4 sequences of 131072
// tokens take 95 us, 5.4 TB/s, 80 % of the copy rate, where the bytes alone take 77 and fetching them without computing 86.
// 32 rows: 727 instructions a block over its two row warps, each of which unpacks every word for itself (128 ANDs where 64 would
// do), two warps a scheduler, issued on 49 % of the cycles: 347 us (128 sequences to 8192 tokens)
// where the bytes take 95, the products 37 and fetching with the pieces' ends 156. A tcgen05 form for more
// than 16 rows (a token a thread, codes unpacked to tensor memory, a product a group and exact scales on the scores) took as
// many instructions, 777, and 408 us; so did sixteen warps in place of eight.
//
// (Figures of forms that were not taken, here and below, stand beside what this one measured at the time: scores are rounded since,
// two an instruction, at 247 -> 248 and 743 -> 727 instructions, 96 -> 95 and 343 -> 347 us.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "decode_common.cuh"
#include "decode_int4.h"
#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

template <int D>
struct Int4Tile {
  static constexpr int G = D / kInt4Group;
  static constexpr int RB = D / 2;               // bytes of a row
  static constexpr int TILE = kBlockSize * RB;   // bytes of a block's K (or V)
  static constexpr int META = 2 * kBlockSize * G * 4;
  static constexpr int STAGE = 2 * TILE + META;
};

// Warps, ring (in steps), CTAs an SM and blocks a step of the kernel for a row count.
template <int NT_, int WR_, int WB_, int RING_, int CTAS_, int STEP_, bool PAIR_ = false>
struct Int4Shape {
  // PAIR: units of at most 4 rows of two groups. A row takes two of the products' eight columns, r for the first group and
  // r + 4 for the second, so that a lane holds scores, scales and weights of one group where it would hold those of two, half of
  // them of padding rows: 247 instructions a block in place of 272, 4 x 131072 tokens 96 us in place of 101.
  static constexpr bool PAIR = PAIR_;
  static_assert(!PAIR_ || (NT_ == 1 && WR_ == 1 && WB_ > 2), "pair");
  static constexpr int NT = NT_, WR = WR_, WB = WB_, RING = RING_, CTAS = CTAS_, STEP = STEP_;
  static_assert(RING >= 2 && (STEP == 1 || STEP == 2), "ring");
  static constexpr int ROWS = 8 * NT * WR, THREADS = 32 * WR * WB;
  // A piece's queries: prepared once a row and shared by the streams, or by every warp for its own rows. Four streams save
  // more by sharing than the barrier costs (64 sequences 30.5 us against 32.0), two do not (32 rows: 348 against 336).
  static constexpr bool kShareQ = WB > 2;
};
// Two blocks a step against one: 4 rows 30.0 against 31.3 us (64 sequences), 8 rows 76 against 85, 16 rows 116 against 122, 32
// rows 343 against 409. A row count takes the smallest shape that holds it (on the next one: 8 rows 107 us, 16 rows 145,
// 32 rows 648). Rings and CTAs an SM: as many CTAs as the registers allow, and the deepest ring beside them. 16 rows: two
// streams a CTA and four CTAs 113 us, four and two 115, one and eight 147. 64 rows of 64 dimensions leave registers for
// four n-tiles a warp, so that half as many warps unpack the same words: 126 us against 135 (64 sequences to 8192 tokens); for 32 such
// rows it is the other way round (73 against 68).
using Int4Rows4 = Int4Shape<1, 1, 4, 3, 3, 2, true>;
using Int4Rows8 = Int4Shape<1, 1, 4, 3, 3, 2>;
using Int4Rows16 = Int4Shape<2, 1, 2, 4, 4, 2>;
using Int4Rows32 = Int4Shape<2, 2, 2, 5, 2, 2>;
using Int4Rows64 = Int4Shape<2, 4, 1, 5, 2, 2>;
using Int4Rows64Narrow = Int4Shape<4, 2, 2, 5, 2, 1>;   // head size 64

// The walk of a stream's fetching, kept in shared memory: read once for up to 32 blocks.
struct Int4Walk {
  long long ub;
  int s, h, nb, lb, take, k;
};

struct Int4Smem {
  int qs, rf, qsum, vis, walk, mrg_o, mrg_ml, fin_ml, fac, misc, total;
};
constexpr int kInt4FanLog = 3, kInt4Fan = 1 << kInt4FanLog;   // children of a node of the join

template <int D, class Sh>
__host__ __device__ constexpr Int4Smem int4_smem(int rows) {
  Int4Smem s{};
  s.qs = Sh::WB * Sh::RING * Sh::STEP * Int4Tile<D>::STAGE;
  s.rf = s.qs + (Sh::kShareQ ? Sh::ROWS * (D * 2 + 16) : 0);
  s.qsum = s.rf + (Sh::kShareQ ? Sh::ROWS * 4 : 0);
  s.vis = s.qsum + (Sh::kShareQ ? Sh::ROWS * Int4Tile<D>::G * 4 : 0);
  s.walk = s.vis + Sh::WB * Sh::ROWS * 8;
  s.mrg_o = s.walk + Sh::WR * Sh::WB * static_cast<int>(sizeof(Int4Walk));
  s.mrg_ml = s.mrg_o + Sh::WB * rows * (D + 4) * 4;
  s.fin_ml = s.mrg_ml + (Sh::WB * rows * 8 + 15) / 16 * 16;
  s.fac = s.fin_ml + (rows * 8 + 15) / 16 * 16;
  s.misc = s.fac + (kInt4Fan * rows * 4 + 15) / 16 * 16;
  s.total = s.misc + 256;
  return s;
}

template <int N>
__device__ __forceinline__ void cp_async_wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void cp_async_16_full(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void sts_zero_16(uint32_t dst) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  } else {
    const uint4 v = lds_v4(addr);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

// Steps after which the 8s come off the accumulators. The tensor core's accumulation cuts off what lies below its sum's last
// bit, half of it a product on average; a result of n similar weights is some sqrt(n) times smaller than the sums of 8 P and c P,
// so that many steps lose its bits (4 sequences of 131072 tokens: 6e-4 of the result, with 8 steps of two blocks less than 1e-4).
// Costs 2 % (99 -> 101 us).
constexpr int kInt4Flush = 8;
// The reference m of a row before any visible score: low enough to be left by any score.
constexpr float kInt4Unset = -1e37f;
constexpr float kInt4Shift = 11.f;     // P of the reference's own token: below 2^11
constexpr float kInt4Limit = 32768.f;  // P that moves the reference
constexpr float kInt4FarP = 1.0995116e12f;   // 2^40: a sum of two p that moves it (their scales may be 0)

// e with |s| < 2^e, at least -25 (a scale of 0); a NaN scale counts as 0, or it would push the row's other group out of range.
__device__ __forceinline__ float int4_scale_exponent(float s) {
  return s == s ? fmaxf(static_cast<float>(static_cast<int>(__float_as_uint(fabsf(s)) >> 23) - 126), -25.f) : -25.f;
}

// ex of a row of queries, 2^ex <= its largest element < 2^(ex + 1), from -116 (rows below are scaled by 2^127, the most
// there is) to 127 (an infinity or NaN counts as that and stays what it is); and the factor that undoes the row's scaling by
// 2^(11 - ex) and the codes' by 2^-24.
__device__ __forceinline__ int int4_q_exponent(float mx) {
  return max(-116, min(127, static_cast<int>(__float_as_uint(mx) >> 23) - 127));
}
__device__ __forceinline__ float int4_q_factor(float scale_log2, int ex) {
  const int e = min(13 + ex, 127);   // (2^(13 + ex) may pass fp32's range)
  return scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * static_cast<float>(1 << (13 + ex - e));
}

// As mma_f16 and movmatrix_t, for the compiler to move between others.
__device__ __forceinline__ void mma_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Joins the pieces of a unit that several CTAs share (the split-softmax rule of decode_common.cuh) in a tree: a
// node is merged by the last of its kInt4Fan children to arrive, which goes on as that node. A child's (m, l, o) lie in slot (unit +
// its first CTA); a node's arrivals are counted in a byte a level of that slot's counter, tagged with the call. The first
// child, usually the last to arrive, first tries to count itself as the completing one, unpublished. One CTA that joins all pieces reads
// 38 of 64 rows in some 80 us (1 sequence of 262144 tokens: 401 us instead of 320).
// FEW (at most 8 rows, an item or two a thread): an item's weights and values in one round trip; else the rows' weights first.
// The piece: o[r] at o + r * (D + 4), m and l at ml[r], ml[R + r], complete before the call. Returns true in the
// CTA that holds the whole unit there. Every thread of the CTA calls it.
template <int D, int NTHR, bool FEW>
__device__ __forceinline__ bool int4_join(const DecodeArgs& a, int u, int c_first, int c_last, int Rs, float* o, float* ml, float* fac,
                                          volatile int* fin) {
  const int tid = threadIdx.x, R = a.rows, ooff = partial_o_offset(R);
  const long long slot0 = static_cast<long long>(u) + c_first;
  const int items = Rs * (D / 4);
  int idx = static_cast<int>(blockIdx.x) - c_first, cnt = c_last - c_first + 1;
#pragma unroll 1
  for (int lv = 0; cnt > 1; ++lv, idx >>= kInt4FanLog, cnt = (cnt + kInt4Fan - 1) >> kInt4FanLog) {
    const int kid0 = idx & ~(kInt4Fan - 1), kids = min(kInt4Fan, cnt - kid0), sh = kInt4FanLog * lv;
    if (kids == 1) continue;
    const unsigned long long one = 1ull << (8 * lv), tag = static_cast<unsigned long long>(a.epoch) << 32;
    unsigned long long* ctr = a.piece_counts + slot0 + (static_cast<long long>(kid0) << sh);
    unsigned long long cur = 0ull;   // (thread 0's guess of the counter)
    __syncthreads();
    if (tid == 0) {
      bool done = false;
      if (idx == kid0) {
        const unsigned long long others = tag | one * (kids - 1);
        cur = atomicCAS(ctr, others, others + one);
        done = cur == others;
        if (done) fence_acq_rel_gpu();   // acquire: the other children's slots are read next
      }
      fin[0] = done;
    }
    __syncthreads();
    if (!fin[0]) {
      float* P = a.partials + static_cast<size_t>(slot0 + (static_cast<long long>(idx) << sh)) * a.slot_floats;
      for (int x = tid; x < items; x += NTHR) {
        const int r = x / (D / 4), d4 = x % (D / 4);
        *reinterpret_cast<float4*>(P + ooff + r * D + d4 * 4) = *reinterpret_cast<const float4*>(o + r * (D + 4) + d4 * 4);
      }
      for (int r = tid; r < Rs; r += NTHR) {
        P[r] = ml[r];
        P[R + r] = ml[R + r];
      }
      __syncthreads();   // every thread's stores before thread 0's release fence
      if (tid == 0) {
        fence_acq_rel_gpu();
        unsigned long long want;
        for (;;) {   // (a counter of another call reads as clear)
          want = (cur >> 32) == a.epoch ? cur + one : tag | one;
          const unsigned long long prev = atomicCAS(ctr, cur, want);
          if (prev == cur) break;
          cur = prev;
        }
        const bool done = static_cast<int>((want >> (8 * lv)) & 0xFFull) == kids;
        if (done) fence_acq_rel_gpu();
        fin[1] = done;
      }
      __syncthreads();
      if (!fin[1]) return false;
    }
    // M = max m, L = sum l 2^(m - M), o = sum o 2^(m - M) over the children in order (the bits do not depend on who joins them).
    const float* base = a.partials + static_cast<size_t>(slot0 + (static_cast<long long>(kid0) << sh)) * a.slot_floats;
    const size_t step = static_cast<size_t>(a.slot_floats) << sh;
    const int own = idx - kid0;
    if constexpr (FEW) {
      float M[8 * (D / 4) / NTHR + 1], L[8 * (D / 4) / NTHR + 1];
#pragma unroll
      for (int e = 0; e < 8 * (D / 4) / NTHR; ++e) {
        const int x = tid + e * NTHR, r = x / (D / 4), d4 = x % (D / 4);
        if (x >= items) break;
        float mc[kInt4Fan], lc[kInt4Fan];
        float4 v[kInt4Fan];
        M[e] = -INFINITY;
#pragma unroll
        for (int k = 0; k < kInt4Fan; ++k) {
          const bool far = k < kids && k != own;
          mc[k] = far ? __ldcg(base + k * step + r) : -INFINITY;
          lc[k] = far ? __ldcg(base + k * step + R + r) : 0.f;
          v[k] = far ? __ldcg(reinterpret_cast<const float4*>(base + k * step + ooff + r * D + d4 * 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
          if (k == own) {
            mc[k] = ml[r];
            lc[k] = ml[R + r];
            v[k] = *reinterpret_cast<const float4*>(o + r * (D + 4) + d4 * 4);
          }
        }
#pragma unroll
        for (int k = 0; k < kInt4Fan; ++k) M[e] = fmaxf(M[e], mc[k]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        L[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kInt4Fan; ++k) {
          const float f = fast_exp2(mc[k] - M[e]);   // (M is finite)
          L[e] += f * lc[k];
          acc.x += f * v[k].x;
          acc.y += f * v[k].y;
          acc.z += f * v[k].z;
          acc.w += f * v[k].w;
        }
        *reinterpret_cast<float4*>(o + r * (D + 4) + d4 * 4) = acc;
      }
      __syncthreads();   // ml is read
#pragma unroll
      for (int e = 0; e < 8 * (D / 4) / NTHR; ++e) {
        const int x = tid + e * NTHR, r = x / (D / 4);
        if (x < items && x % (D / 4) == 0) {
          ml[r] = M[e];
          ml[R + r] = L[e];
        }
      }
    } else {
      for (int r = tid; r < Rs; r += NTHR) {
        float mc[kInt4Fan], lc[kInt4Fan], M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < kInt4Fan; ++k) {
          const bool far = k < kids && k != own;
          mc[k] = far ? __ldcg(base + k * step + r) : (k == own ? ml[r] : -INFINITY);
          lc[k] = far ? __ldcg(base + k * step + R + r) : (k == own ? ml[R + r] : 0.f);
          M = fmaxf(M, mc[k]);
        }
#pragma unroll
        for (int k = 0; k < kInt4Fan; ++k) {
          const float f = fast_exp2(mc[k] - M);   // (M is finite)
          L += f * lc[k];
          fac[k * R + r] = f;
        }
        ml[r] = M;
        ml[R + r] = L;
      }
      __syncthreads();
      // Four items of a thread at a time, a child's four loads in flight with the next child's.
#pragma unroll 1
      for (int x0 = tid; x0 < items; x0 += 4 * NTHR) {
        float4 acc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k = 0; k < kids; k += 2) {
          float4 v[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = x0 + e * NTHR, r = x / (D / 4), d4 = x % (D / 4);
              v[j][e] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (x < items && k + j < kids)
                v[j][e] = k + j == own ? *reinterpret_cast<const float4*>(o + r * (D + 4) + d4 * 4)
                                       : __ldcg(reinterpret_cast<const float4*>(base + (k + j) * step + ooff + r * D + d4 * 4));
            }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int x = x0 + e * NTHR;
              if (x < items && k + j < kids) {
                const float f = fac[(k + j) * R + x / (D / 4)];
                acc[e].x += f * v[j][e].x;
                acc[e].y += f * v[j][e].y;
                acc[e].z += f * v[j][e].z;
                acc[e].w += f * v[j][e].w;
              }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = x0 + e * NTHR, r = x / (D / 4), d4 = x % (D / 4);
          if (x < items) *reinterpret_cast<float4*>(o + r * (D + 4) + d4 * 4) = acc[e];
        }
      }
    }
    if (tid == 0) atomicAdd(ctr, 0ull - one * kids);   // clear for a replay
  }
  __syncthreads();
  return true;
}

template <int D, class Sh, bool BF16>
__global__ void __launch_bounds__(Sh::THREADS, Sh::CTAS) decode_int4_kernel(const __grid_constant__ DecodeInt4Args a) {
  using T = Int4Tile<D>;
  constexpr int G = T::G, NT = Sh::NT, WR = Sh::WR, WB = Sh::WB, RING = Sh::RING, STEP = Sh::STEP, UNIT = STEP * T::STAGE,
                NTHR = Sh::THREADS;
  constexpr bool PAIR = Sh::PAIR;
  constexpr int GS = PAIR ? 1 : G;   // groups whose scales and weights a lane holds
  constexpr float kNegInf = -INFINITY;
  extern __shared__ __align__(128) uint8_t smem[];
  const int R = a.rows;
  const Int4Smem lay = int4_smem<D, Sh>(R);
  float* mrg_o = reinterpret_cast<float*>(smem + lay.mrg_o);
  float* mrg_m = reinterpret_cast<float*>(smem + lay.mrg_ml);
  float* mrg_l = mrg_m + WB * R;
  float* fin_ml = reinterpret_cast<float*>(smem + lay.fin_ml);
  long long* red = reinterpret_cast<long long*>(smem + lay.misc);
  long long* plan = red + 10;
  volatile int* fin = reinterpret_cast<volatile int*>(plan + 5);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wr = warp % WR, wb = warp / WR;
  const int i8 = lane >> 2, c4 = lane & 3;
  const int row_base = wr * 8 * NT;
  const int row2 = PAIR ? 2 * (c4 & 1) : 2 * c4;   // first of the two rows of a lane's columns of n-tile 0
  const int own_g = PAIR ? c4 >> 1 : 0;            // PAIR: the columns' group
  constexpr int QS = D * 2 + 16;
  uint8_t* qs = smem + lay.qs;
  float* rf_s = reinterpret_cast<float*>(smem + lay.rf);
  float* qsum_s = reinterpret_cast<float*>(smem + lay.qsum);
  unsigned long long* vis_s = reinterpret_cast<unsigned long long*>(smem + lay.vis) + warp * 8 * NT;

  if constexpr (Sh::kShareQ) {   // padding rows: zero queries and factors
    for (int idx = tid; idx < Sh::ROWS * (QS / 16); idx += NTHR) reinterpret_cast<uint4*>(qs)[idx] = make_uint4(0, 0, 0, 0);
    for (int idx = tid; idx < Sh::ROWS * (1 + G); idx += NTHR) rf_s[idx] = 0.f;
  }

  prefetch_plan_inputs(a.context_lens, a.block_tables, a.num_seqs, a.max_blocks_per_seq);
  // Everything below reads inputs a previous kernel in the stream may write.
  pdl_wait_prior_grid();
  const int Hkv = a.num_kv_heads, mbs = a.max_blocks_per_seq;
  const int n = a.q_per_seq, Gq = a.group, Hq = a.num_q_heads;
  const long long ncta = gridDim.x;
  plan_cta_share(a, red, plan);
  pdl_launch_dependents();
  const long long total = plan[0], b0 = plan[1], b1 = plan[2];
  if (b0 >= b1 || plan[3] < 0) return;

  // Walk state: the unit (s, h), its first block's position ub on the work line, the first block
  // lb this CTA takes of it.
  const int pc0 = a.piece_cost;
  int s = static_cast<int>(plan[3]);
  int ctx = a.context_lens[s];
  int nb = unit_blocks(ctx, mbs);
  int h, lb;
  long long ub;
  {
    const long long off = b0 - static_cast<long long>(Hkv) * plan[4];
    h = static_cast<int>(off / (nb + pc0));
    const int o = static_cast<int>(off % (nb + pc0));
    lb = o > pc0 ? o - pc0 : 0;
    ub = b0 - o + pc0;
  }

  // ---- the stream's fetching: the same walk, up to RING - 1 of its steps ahead ----
  const uint32_t ring = smem_addr(smem) + wb * (RING * UNIT), ring_end = ring + RING * UNIT;
  Int4Walk* walk = reinterpret_cast<Int4Walk*>(smem + lay.walk) + warp;
  if (lane == 0) *walk = {ub, s, h, nb, lb, static_cast<int>(min(static_cast<long long>(nb), b1 - ub)) - lb, wb};
  __syncwarp();
  int f_id = 0, f_pos = 0, f_left = 0, f_h = 0;   // the stream's next block ids, one a lane; the next one's lane; how many
  bool f_more = true;
  // The next up to 32 blocks of the stream in the piece at hand, or in the next one that has any.
  auto next_ids = [&]() {
    long long w_ub = walk->ub;
    int w_s = walk->s, w_h = walk->h, w_nb = walk->nb, w_lb = walk->lb, w_take = walk->take, w_k = walk->k;
    int steps = (w_take + STEP - 1) / STEP;
    while (w_k >= steps) {
      w_k -= steps;
      if (w_lb + w_take < w_nb || w_ub + w_nb + pc0 >= b1) {   // the share ends in this piece
        f_more = false;
        return;
      }
      w_ub += w_nb + pc0;
      w_lb = 0;
      if (++w_h == Hkv) {
        w_h = 0;
        ++w_s;
        w_nb = unit_blocks(a.context_lens[w_s], mbs);
      }
      w_take = static_cast<int>(min(static_cast<long long>(w_nb), b1 - w_ub));
      steps = (w_take + STEP - 1) / STEP;
    }
    const int mine = min(32 / STEP, (steps - w_k + WB - 1) / WB);
    const int at = (w_k + lane / STEP * WB) * STEP + lane % STEP;
    const bool there = lane / STEP < mine && at < w_take;
    f_left = __popc(__ballot_sync(0xffffffffu, there));
    f_pos = 0;
    f_h = w_h;
    f_id = there ? a.block_tables[static_cast<size_t>(w_s) * mbs + w_lb + at] : 0;
    __syncwarp();
    if (lane == 0) *walk = {w_ub, w_s, w_h, w_nb, w_lb, w_take, w_k + mine * WB};
    __syncwarp();
  };
  constexpr int KC = T::TILE / 16, MC = T::META / 16, ALL = 2 * KC + MC;
  // This thread's 16-byte chunk of every 32 WR. Head size 128: tokens 2 and 3 (mod 4) have their halves
  // exchanged, so that V words of four tokens lie in different banks.
  const int chunk = 32 * wr + lane;
  const uint32_t chunk_at = 16u * (D == 128 ? chunk ^ ((chunk >> 2) & 2) : chunk);
  const uint8_t* const k_base = a.k_cache + 16 * chunk;
  const uint8_t* const v_base = a.v_cache + 16 * chunk;
  const uint8_t* const m_base = a.meta + 16 * chunk;
  auto fetch_block = [&](uint32_t dst, int blk) {
    const uint32_t tile = static_cast<uint32_t>(blk) * Hkv + f_h;   // (the host keeps rows below 2^31)
    const uint8_t* k_src = k_base + static_cast<size_t>(tile) * T::TILE;
    const uint8_t* v_src = v_base + static_cast<size_t>(tile) * T::TILE;
    const uint8_t* m_src = m_base + static_cast<size_t>(tile) * T::META;
#pragma unroll
    for (int x = 0; x < (ALL + 32 * WR - 1) / (32 * WR); ++x) {
      const int base = 32 * WR * x;   // a part's chunks come in multiples of 32
      if (base + (WR == 1 ? 0 : 32 * wr) < KC) {
        cp_async_16_full(dst + 16 * base + chunk_at, k_src + 16 * base);
      } else if (base + (WR == 1 ? 0 : 32 * wr) < 2 * KC) {
        cp_async_16_full(dst + 16 * base + chunk_at, v_src + 16 * (base - KC));
      } else if (base + chunk < ALL) {
        cp_async_16_full(dst + 16 * (base + chunk), m_src + 16 * (base - 2 * KC));
      }
    }
  };
  auto block_ok = [&](int blk) { return static_cast<unsigned>(blk) < static_cast<unsigned>(a.num_blocks); };
  // The next step's blocks (one, where no second is left in the piece) to dst; nothing behind the share's end.
  auto fetch = [&](uint32_t dst) {
    if (f_left == 0 && f_more) next_ids();
    const int blk0 = __shfl_sync(0xffffffffu, f_id, f_pos), blk1 = STEP == 2 ? __shfl_sync(0xffffffffu, f_id, f_pos + 1) : blk0;
    if (f_left >= STEP && block_ok(blk0) && block_ok(blk1)) {
      fetch_block(dst, blk0);
      if constexpr (STEP == 2) fetch_block(dst + T::STAGE, blk1);
      f_left -= STEP;
    } else if (f_left > 0) {
#pragma unroll 1
      for (int y = 0; y < STEP && f_left > 0; ++y, --f_left) {
        const int blk = y ? blk1 : blk0;
        if (block_ok(blk)) {
          fetch_block(dst + y * T::STAGE, blk);
        } else {   // a bad block id reads zeros
          if (lane == 0 && wr == 0 && a.status) atomicOr(a.status, kDevBadBlock);
          for (int x = chunk; x < ALL; x += 32 * WR) sts_zero_16(dst + y * T::STAGE + 16 * x);
        }
      }
    }
    f_pos += STEP;
    cp_async_commit();
  };
  auto stream_sync = [&]() {
    if constexpr (WR == 1) __syncwarp();
    else named_bar_sync(4 + wb, 32 * WR);
  };
#pragma unroll 1
  for (int x = 0; x < RING - 1; ++x) fetch(ring + x * UNIT);

  // Token of product slot i8 (and of i8 + 8: 8 more): slots 2 j, 2 j + 1 hold tokens j, (j ^ 1) + 4.
  const int tok = (i8 & 1) ? ((i8 >> 1) ^ 1) + 4 : i8 >> 1;
  const int tv0 = c4, tv1 = (c4 ^ 1) + 4;
  const uint32_t k_off = D == 128 ? tok * 64 + ((c4 ^ (tok & 2)) << 4) : tok * 32 + c4 * 8;
  auto v_off = [&](int t) -> uint32_t {
    return T::TILE + (D == 128 ? t * 64 + (((i8 >> 1) ^ (t & 2)) << 4) + 8 * (i8 & 1) : t * 32 + 4 * i8);
  };
  const uint32_t v_off0 = v_off(tv0), v_off1 = v_off(tv1);
  const uint32_t m_off = 2 * T::TILE + tok * 4 * G + 4 * own_g;

  // The stream's next step: where its blocks lie and where the last one's lay; its index in the piece.
  uint32_t st = ring, st_last = ring_end - UNIT;
  int kk = wb;
  while (ub < b1) {
    const int take = static_cast<int>(min(static_cast<long long>(nb), b1 - ub)) - lb;
    const bool first = (lb == 0), last = (lb + take == nb);
    const bool split = !(first && last);
    const int u = s * Hkv + h;
    const int cap = mbs * kBlockSize;
    const int ctx_eff = ctx < cap ? ctx : cap;
    // Query rows as in the other decode kernels: a count outside [1, q_per_seq], or rows past the
    // end of q, is flagged and the sequence gets no rows.
    int n_s = n, qb = s * n;
    if (a.cu_q_lens) {
      qb = a.cu_q_lens[s];
      n_s = a.cu_q_lens[s + 1] - qb;
    }
    const bool rows_ok = n_s >= 1 && n_s <= n && qb >= 0 && qb <= a.q_rows - n_s;
    const int Rs = rows_ok ? Gq * n_s : 0;
    if (!rows_ok) {
      n_s = 1;
      qb = 0;
    }
    if (first && tid == 0 && (!rows_ok || ctx < n_s || ctx > cap) && a.status) atomicOr(a.status, kDevBadCtx);

    const int cb = ctx_eff - n_s;
    // Element offset of a row of q and out: row r is query token r / Gq, query head h Gq + r % Gq.
    auto row_at = [&](int r) {
      const int j = r / Gq;
      return (static_cast<size_t>(qb + j) * Hq + h * Gq + (r - j * Gq)) * D;
    };

    // Queries: lane (i8, c4) holds row i8's words 2 c4 and 2 c4 + 1 of every group, the B operand of S^T as they
    // lie, scaled to the row's largest element in [2^11, 2^12), the odd pairs of a word by 2^-4 more.
    uint32_t qf[NT][2 * G][4];   // word 2 c4 + x / G of group x % G
    float rf[NT][2], qz[NT][GS][2];   // rows row2, row2 + 1: the factor that undoes all scaling; sums by group
    if constexpr (Sh::kShareQ) {
      // One row a warp; the last piece's were read before its streams merged.
#pragma unroll 2
      for (int r = warp; r < Rs; r += WR * WB) {
        const int j = r / Gq, gi = r - j * Gq;
        constexpr int E = D / 32;   // elements of a lane
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (static_cast<size_t>(qb + j) * Hq + h * Gq + gi) * D + E * lane;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(src + e);
          if constexpr (BF16) {
            x[e] = __uint_as_float(w << 16);
            x[e + 1] = __uint_as_float(w & 0xFFFF0000u);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
            x[e] = f.x;
            x[e + 1] = f.y;
          }
        }
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const int ex = int4_q_exponent(mx);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 11 - ex) << 23);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x[e] *= up;
          sum += x[e];
        }
#pragma unroll
        for (int o = 16 / G; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float f = ((E * lane + e) >> 1) & 1 ? 0.0625f : 1.f;
          *reinterpret_cast<uint32_t*>(qs + r * QS + (E * lane + e) * 2) = pack_f16x2(x[e] * f, x[e + 1] * f);
        }
        if (lane % (32 / G) == 0) qsum_s[r * G + lane / (32 / G)] = sum * 0x1p-24f;
        if (lane == 0) rf_s[r] = int4_q_factor(a.scale_log2, ex);
      }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2 * G; ++x) {
          const int r = PAIR ? i8 & 3 : row_base + nt * 8 + i8;
          uint4 v = *reinterpret_cast<const uint4*>(qs + r * QS + (kInt4Group * (x % G) + 8 * (2 * c4 + x / G)) * 2);
          if (PAIR && (i8 >> 2) != x % G) v = make_uint4(0, 0, 0, 0);
          qf[nt][x][0] = v.x;
          qf[nt][x][1] = v.y;
          qf[nt][x][2] = v.z;
          qf[nt][x][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = row_base + nt * 8 + row2 + e;
          rf[nt][e] = rf_s[r];
#pragma unroll
          for (int g = 0; g < GS; ++g) qz[nt][g][e] = qsum_s[r * G + (PAIR ? own_g : g)];
        }
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row_base + nt * 8 + i8;
        float x[2 * G][8];
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * G; ++k) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < Rs)
            v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + row_at(r) + kInt4Group * (k % G) + 8 * (2 * c4 + k / G));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            if constexpr (BF16) {
              x[k][2 * m] = __uint_as_float(w[m] << 16);
              x[k][2 * m + 1] = __uint_as_float(w[m] & 0xFFFF0000u);
            } else {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[m]));
              x[k][2 * m] = f.x;
              x[k][2 * m + 1] = f.y;
            }
            mx = fmaxf(mx, fmaxf(fabsf(x[k][2 * m]), fabsf(x[k][2 * m + 1])));
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = int4_q_exponent(mx);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 11 - ex) << 23);
        float sum[G];
#pragma unroll
        for (int g = 0; g < G; ++g) sum[g] = 0.f;
#pragma unroll
        for (int k = 0; k < 2 * G; ++k)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float x0 = x[k][2 * m] * up, x1 = x[k][2 * m + 1] * up, f = m & 1 ? 0.0625f : 1.f;
            sum[k % G] += x0 + x1;
            qf[nt][k][m] = pack_f16x2(x0 * f, x1 * f);
          }
        const float back = r < Rs ? int4_q_factor(a.scale_log2, ex) : 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
          sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int from = 4 * (2 * c4 + e);
          rf[nt][e] = __shfl_sync(0xffffffffu, back, from);
#pragma unroll
          for (int g = 0; g < G; ++g) qz[nt][g][e] = __shfl_sync(0xffffffffu, sum[g], from) * 0x1p-24f;
        }
      }
    }
    __syncwarp();
    if (lane < 8 * NT) {   // the drafts that a row sees
      const int r = row_base + lane, j = r / Gq;
      vis_s[lane] = (a.tree_masks && r < Rs) ? a.tree_masks[qb + j] : ((j >= 63) ? ~0ull : ((2ull << j) - 1ull));
    }
    __syncwarp();

    float m_run[NT][2], l_run[NT][2];
    float o_acc[NT][G][4][4], o_bias[NT][GS][4], o_z[NT][GS][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_run[nt][e] = kInt4Unset;
        l_run[nt][e] = 0.f;
#pragma unroll
        for (int g = 0; g < GS; ++g) o_z[nt][g][e] = 0.f;
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (g < GS) o_bias[nt][g][x] = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) o_acc[nt][g][x][e] = 0.f;
        }
      }
    }

    // STEP blocks, at st; the first one's first token's position is tok0. Masked: any of their
    // tokens may be hidden, and the second block may be absent.
    auto step = [&](auto masked, const int tok0, const bool absent) {
      constexpr int NB = STEP;
      constexpr bool kMasked = decltype(masked)::value;
      const uint32_t at[2] = {st, st + T::STAGE};
      // ---- S^T (16 tokens x 8 NT rows a block), one accumulator a group ----
      float sa[NB][NT][GS][4];
      uint32_t mk[NB][2][GS], mv[NB][2][GS];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t ka[2 * G], kb[2 * G];
        lds_words<2 * G>(at[b] + k_off, ka);
        lds_words<2 * G>(at[b] + k_off + 8 * T::RB, kb);
        lds_words<GS>(at[b] + m_off, mk[b][0]);
        lds_words<GS>(at[b] + m_off + 32 * G, mk[b][1]);
        lds_words<GS>(at[b] + m_off + 64 * G, mv[b][0]);
        lds_words<GS>(at[b] + m_off + 96 * G, mv[b][1]);
#pragma unroll
        for (int x = 0; x < 2 * G; ++x) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t wa = ka[x] >> (8 * hf), wb2 = kb[x] >> (8 * hf);
            const uint32_t a0 = wa & 0x000F000Fu, a1 = wb2 & 0x000F000Fu, a2 = wa & 0x00F000F0u, a3 = wb2 & 0x00F000F0u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float(&acc)[4] = sa[b][nt][PAIR ? 0 : x % G];
              if (x < (PAIR ? 1 : G) && hf == 0) mma_new(acc, a0, a1, a2, a3, qf[nt][x][2 * hf], qf[nt][x][2 * hf + 1]);
              else mma_acc(acc, a0, a1, a2, a3, qf[nt][x][2 * hf], qf[nt][x][2 * hf + 1]);
            }
          }
        }
      }
      // (the V words, ahead of the scores' arithmetic)
      uint32_t w[NB][4][G];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        lds_words<G>(at[b] + v_off0, w[b][0]);
        lds_words<G>(at[b] + v_off1, w[b][1]);
        lds_words<G>(at[b] + v_off0 + 8 * T::RB, w[b][2]);
        lds_words<G>(at[b] + v_off1 + 8 * T::RB, w[b][3]);
      }

      // ---- scales; scores ----
      float sv[NB][2][GS], zv[NB][2][GS];
      // [2 x + e]: token tok + 8 x, row 2 c4 + e. Rounded: a product that m were taken off unrounded would differ from the rounded one
      // in m by half its last place, which for scores beyond 2^26 passes the range of p.
      float sc[NB][NT][4];
      bool hid[NB][NT][4];   // (all false without a mask)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sk[GS], zk[GS];
#pragma unroll
          for (int g = 0; g < GS; ++g) {
            const float2 fk = __half22float2(*reinterpret_cast<const __half2*>(&mk[b][x][g]));
            const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&mv[b][x][g]));
            sk[g] = fk.x;
            zk[g] = fk.y;
            sv[b][x][g] = fv.x;
            zv[b][x][g] = fmaf(8.f, fv.x, fv.y);
          }
          const int d = tok0 + 16 * b + tok + 8 * x - cb;   // (ctx_eff is cb + n_s)
          const bool there = !kMasked || (d < n_s && !(b == 1 && absent));
          if (!there) {   // behind the context: whatever lies there
#pragma unroll
            for (int g = 0; g < GS; ++g) sv[b][x][g] = zv[b][x][g] = 0.f;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = zk[0] * qz[nt][0][e];
              if constexpr (GS == 2) v = fmaf(zk[1], qz[nt][1][e], v);
#pragma unroll
              for (int g = 0; g < GS; ++g) v = fmaf(sa[b][nt][g][2 * x + e], sk[g], v);
              if constexpr (PAIR) v += __shfl_xor_sync(0xffffffffu, v, 2);   // the other group's part
              sc[b][nt][2 * x + e] = v;
              hid[b][nt][2 * x + e] = kMasked && !(there && (d < 0 || (d < 64 && ((vis_s[nt * 8 + row2 + e] >> d) & 1ull))));
            }
            const float2 f = halves_of(mul2(f32x2(sc[b][nt][2 * x], sc[b][nt][2 * x + 1]), f32x2(rf[nt][0], rf[nt][1])));
            sc[b][nt][2 * x] = f.x;
            sc[b][nt][2 * x + 1] = f.y;
          }
        }

      // ---- weights p = 2^(score - m) and P = p s; the reference moved where one is too large ----
      float p[NB][NT][4], p2[NB][NT][2];   // and p of a row's two tokens together
      uint32_t ph[NB][NT][GS][2];   // P of a token's two rows
      auto weights = [&]() {
        float far = 0.f;
        __half2 top = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 d = halves_of(add2(f32x2(sc[b][nt][2 * x], sc[b][nt][2 * x + 1]), f32x2(-m_run[nt][0], -m_run[nt][1])));
              p[b][nt][2 * x] = fast_exp2(d.x);
              p[b][nt][2 * x + 1] = fast_exp2(d.y);
              if (kMasked && hid[b][nt][2 * x]) p[b][nt][2 * x] = 0.f;
              if (kMasked && hid[b][nt][2 * x + 1]) p[b][nt][2 * x + 1] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) p2[b][nt][e] = p[b][nt][e] + p[b][nt][2 + e];
            far = fmaxf(far, fmaxf(p2[b][nt][0], p2[b][nt][1]));
#pragma unroll
            for (int g = 0; g < GS; ++g)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                float P0 = p[b][nt][2 * x] * sv[b][x][g], P1 = p[b][nt][2 * x + 1] * sv[b][x][g];
                if (kMasked && hid[b][nt][2 * x]) P0 = 0.f;   // (beside a NaN scale too)
                if (kMasked && hid[b][nt][2 * x + 1]) P1 = 0.f;
                ph[b][nt][g][x] = pack_f16x2(P0, P1);
                top = __hmax2(top, __habs2(*reinterpret_cast<const __half2*>(&ph[b][nt][g][x])));
              }
          }
        return !__hble2(top, __half2half2(__float2half(kInt4Limit))) || far > kInt4FarP;
      };
      if (__any_sync(0xffffffffu, weights())) {
        float ve[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ve[b][x] = int4_scale_exponent(sv[b][x][0]);
            if constexpr (GS == 2) ve[b][x] = fmaxf(ve[b][x], int4_scale_exponent(sv[b][x][1]));
            if constexpr (PAIR) ve[b][x] = fmaxf(ve[b][x], __shfl_xor_sync(0xffffffffu, ve[b][x], 2));
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = kNegInf;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (!hid[b][nt][2 * x + e]) mx = fmaxf(mx, __fadd_ru(sc[b][nt][2 * x + e], ve[b][x] - kInt4Shift));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float m_new = fmaxf(m_run[nt][e], mx);   // (rounded up: no P above 2^11)
            const float alpha = fast_exp2(m_run[nt][e] - m_new);
            m_run[nt][e] = m_new;
            l_run[nt][e] *= alpha;
#pragma unroll
            for (int g = 0; g < G; ++g) {
              if (g < GS) {
                o_z[nt][g][e] *= alpha;
                o_bias[nt][g][e] *= alpha;
                o_bias[nt][g][2 + e] *= alpha;
              }
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                o_acc[nt][g][x][e] *= alpha;
                o_acc[nt][g][x][2 + e] *= alpha;
              }
            }
          }
        weights();
      }

      // ---- O^T (dimensions x rows) += V^T P^T ----
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t pb[NT][GS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) l_run[nt][e] += p2[b][nt][e];
#pragma unroll
          for (int g = 0; g < GS; ++g) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              if (kMasked && hid[b][nt][v]) continue;
              o_z[nt][g][v & 1] = fmaf(p[b][nt][v], zv[b][v >> 1][g], o_z[nt][g][v & 1]);
            }
            // The S^T layout (token, rows 2 c4, 2 c4 + 1) transposed: (row i8, slots 2 c4, 2 c4 + 1).
            pb[nt][g][0] = transposed(ph[b][nt][g][0]);
            pb[nt][g][1] = transposed(ph[b][nt][g][1]);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          // Even and odd dimensions of the two tokens of a slot pair.
          const uint32_t x01 = __byte_perm(w[b][0][g], w[b][1][g], 0x5410), y01 = __byte_perm(w[b][0][g], w[b][1][g], 0x7632);
          const uint32_t x23 = __byte_perm(w[b][2][g], w[b][3][g], 0x5410), y23 = __byte_perm(w[b][2][g], w[b][3][g], 0x7632);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t keep = x & 1 ? 0x00F000F0u : 0x000F000Fu;
            const int sh = 8 * (x >> 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_acc(o_acc[nt][g][x], (x01 >> sh) & keep, (y01 >> sh) & keep, (x23 >> sh) & keep, (y23 >> sh) & keep,
                      pb[nt][PAIR ? 0 : g][0], pb[nt][PAIR ? 0 : g][1]);
          }
          if (g >= GS) continue;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)   // 8 in every element
            mma_acc(o_bias[nt][g], 0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u, pb[nt][g][0], pb[nt][g][1]);
        }
      }
    };

    // The steps whose tokens every row sees come first.
    const int steps = (take + STEP - 1) / STEP;
    const int clear = min(take, max(cb, 0) / kBlockSize - lb) / STEP;
    int since = 0;
#pragma unroll 1
    for (; kk < steps; kk += WB) {
      cp_async_wait_groups<RING - 2>();
      stream_sync();   // the step's blocks are there for all of the stream's warps, and the last step's are read
      fetch(st_last);
      if (row_base < Rs) {
        const int tok0 = (lb + kk * STEP) * kBlockSize;
        if (kk < clear) step(std::false_type{}, tok0, false);
        else step(std::true_type{}, tok0, kk * STEP + 1 == take);
        if (++since == kInt4Flush) {
          since = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
#pragma unroll
              for (int g = 0; g < G; ++g)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  o_acc[nt][g][x][e] = fmaf(o_bias[nt][PAIR ? 0 : g][e], x & 1 ? -16.f : -1.f, o_acc[nt][g][x][e]);
#pragma unroll
              for (int g = 0; g < GS; ++g) o_bias[nt][g][e] = 0.f;
            }
        }
      }
      st_last = st;
      st = st + UNIT == ring_end ? ring : st + UNIT;
    }
    kk -= steps;

    // ---- merge the streams of this piece ----
    if constexpr (!Sh::kShareQ) __syncthreads();   // every warp has left the last merge
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row_base + nt * 8 + row2 + e;
        float lsum = l_run[nt][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
        if (i8 == 0 && own_g == 0 && r < R) {
          mrg_m[wb * R + r] = m_run[nt][e];
          mrg_l[wb * R + r] = lsum;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float z = o_z[nt][PAIR ? 0 : g][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
          float y[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float f = x & 1 ? 0.0625f : 1.f;
            y[2 * x] = fmaf(fmaf(o_acc[nt][g][x][e], f, -o_bias[nt][PAIR ? 0 : g][e]), 0x1p24f, z);
            y[2 * x + 1] = fmaf(fmaf(o_acc[nt][g][x][2 + e], f, -o_bias[nt][PAIR ? 0 : g][e]), 0x1p24f, z);
          }
          if (r < R && (!PAIR || g == own_g)) {
            float4* mo = reinterpret_cast<float4*>(mrg_o + static_cast<size_t>(wb * R + r) * (D + 4) + kInt4Group * g + 8 * i8);
            mo[0] = make_float4(y[0], y[1], y[2], y[3]);
            mo[1] = make_float4(y[4], y[5], y[6], y[7]);
          }
        }
      }
    __syncthreads();
    auto store_row = [&](int r, int d4, const float4& v, float l) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int j = r / Gq, gi = r - j * Gq;
      uint2 pk;
      pk.x = pack_p<BF16 ? kKvBf16 : kKvF16>(v.x * inv, v.y * inv);
      pk.y = pack_p<BF16 ? kKvBf16 : kKvF16>(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + (static_cast<size_t>(qb + j) * Hq + h * Gq + gi) * D + d4 * 4) = pk;
    };
    for (int idx = tid; idx < Rs * (D / 4); idx += NTHR) {
      const int r = idx / (D / 4), d4 = idx % (D / 4);
      float M = kNegInf;
#pragma unroll
      for (int w = 0; w < WB; ++w) M = fmaxf(M, mrg_m[w * R + r]);
      float lsum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WB; ++w) {
        const float f = fast_exp2(mrg_m[w * R + r] - M);
        lsum += f * mrg_l[w * R + r];
        const float4 v = *reinterpret_cast<const float4*>(mrg_o + static_cast<size_t>(w * R + r) * (D + 4) + d4 * 4);
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      if (!split) {
        store_row(r, d4, acc, lsum);
      } else {
        // (in place of stream 0's: only this thread reads or writes these four values)
        *reinterpret_cast<float4*>(mrg_o + static_cast<size_t>(r) * (D + 4) + d4 * 4) = acc;
        if (d4 == 0) {
          fin_ml[r] = M;
          fin_ml[R + r] = lsum;
        }
      }
    }
    if (split) {
      int c_first, c_last;
      unit_owners(a, ub, nb, total, ncta, &c_first, &c_last);
      if (int4_join<D, NTHR, (Sh::ROWS <= 8)>(a, u, c_first, c_last, Rs, mrg_o, fin_ml, reinterpret_cast<float*>(smem + lay.fac), fin)) {
        for (int idx = tid; idx < Rs * (D / 4); idx += NTHR) {
          const int r = idx / (D / 4), d4 = idx % (D / 4);
          store_row(r, d4, *reinterpret_cast<const float4*>(mrg_o + r * (D + 4) + d4 * 4), fin_ml[R + r]);
        }
      }
    }

    // ---- the next unit (a piece that stops before the unit's end ended the share) ----
    if (lb + take < nb) break;
    ub += nb + pc0;
    lb = 0;
    if (++h == Hkv) {
      h = 0;
      ++s;
      if (ub < b1) {
        ctx = a.context_lens[s];
        nb = unit_blocks(ctx, mbs);
      }
    }
  }
  cp_async_wait_all();
}

template <int D, class Sh, bool BF16>
DecodeInt4Kernel int4_kernel(int rows) {
  return {reinterpret_cast<const void*>(&decode_int4_kernel<D, Sh, BF16>), Sh::THREADS,
          static_cast<size_t>(int4_smem<D, Sh>(rows).total)};
}
template <bool BF16, class Sh, class Sh64 = Sh>
DecodeInt4Kernel int4_kernel(int d, int rows) {
  return d == 128 ? int4_kernel<128, Sh, BF16>(rows) : int4_kernel<64, Sh64, BF16>(rows);
}
template <bool BF16>
DecodeInt4Kernel int4_kernel_for(int d, int rows) {
  if (rows <= 4 && d == 128) return int4_kernel<128, Int4Rows4, BF16>(rows);
  if (rows <= 8) return int4_kernel<BF16, Int4Rows8>(d, rows);
  if (rows <= 16) return int4_kernel<BF16, Int4Rows16>(d, rows);
  if (rows <= 32) return int4_kernel<BF16, Int4Rows32>(d, rows);
  return int4_kernel<BF16, Int4Rows64, Int4Rows64Narrow>(d, rows);
}

}  // namespace pkv
