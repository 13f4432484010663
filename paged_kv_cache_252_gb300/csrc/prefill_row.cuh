// One query row of causal attention over a sequence's blocks, by one warp in fp32
// on the CUDA cores: out = sum_p softmax_p(scale * q . K_p) V_p over the visible
// positions p < limit, with a running maximum and sum. Positions past the limit
// are never read, so whatever they hold (stale rows, infinities, NaN) cannot reach the row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include <cstdint>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

// Arguments of the prefill kernels (passed by value).
struct PrefillArgs {
  void* out;                   // [q_rows][Hq][D] fp16/bf16
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* scales;         // INT8 cache: [num_blocks][Hkv][2][16] K then V row scales, else null
  const int32_t* block_tables; // [S][max_blocks_per_seq]
  const int32_t* context_lens; // [S]
  const int32_t* cu_q_lens;    // [S+1]
  int32_t* status;
  int32_t q_rows, num_seqs, num_q_heads, num_kv_heads, group;
  int32_t max_blocks_per_seq, num_blocks;
  float scale_log2;            // softmax scale * log2(e)
  int32_t box_tokens, unit_tokens;     // query tokens of a TMA box and of a unit (prefill_plan.cuh)
  unsigned long long* piece_counts;    // [2 grid]: (call epoch << 32) | pieces of a cut row tile finished
  float* partials;                     // [2 grid][row tiles] slots of pf_slot_floats
  int32_t slot_tiles;                  // row tiles of a slot (1 or 2)
  uint32_t epoch;                      // distinct for every call (tags the piece counters)
};

// A sequence's query rows and lengths, with everything out of range made harmless:
// no rows where the row range is bad, the context clamped to [0, capacity].
struct PrefillSeq {
  int n, qb, ctx;
  bool bad;
  __device__ int past() const { return ctx - n; }   // positions before the first query token (may be < 0)
};
__device__ __forceinline__ PrefillSeq prefill_seq(const PrefillArgs& a, int s) {
  PrefillSeq p;
  p.qb = a.cu_q_lens[s];
  const long long n = static_cast<long long>(a.cu_q_lens[s + 1]) - p.qb;
  const bool rows_ok = n >= 0 && p.qb >= 0 && p.qb + n <= a.q_rows;
  p.n = rows_ok ? static_cast<int>(n) : 0;
  const int ctx = a.context_lens[s], cap = a.max_blocks_per_seq * kBlockSize;
  p.ctx = ctx < 0 ? 0 : (ctx < cap ? ctx : cap);
  p.bad = !rows_ok || (p.n > 0 && (ctx < p.n || ctx > cap));
  return p;
}

// 8 consecutive elements at element offset e of a cache, in fp32 (INT8 codes unscaled).
template <int KV>
__device__ __forceinline__ void load8(const void* cache, size_t e, float (&x)[8]) {
  if constexpr (KV == kKvF16 || KV == kKvBf16) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + e);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (KV == kKvBf16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + e);
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xFFu;
      x[i] = KV == kKvE5m2 ? __half2float(__ushort_as_half(static_cast<uint16_t>(b << 8)))
                           : static_cast<float>(static_cast<int>(b) - 128);
    }
  }
}

template <int KV>
__device__ __forceinline__ float load1(const void* cache, size_t e) {
  if constexpr (KV == kKvF16) return __half2float(static_cast<const __half*>(cache)[e]);
  else if constexpr (KV == kKvBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(cache)[e]);
  else if constexpr (KV == kKvE5m2)
    return __half2float(__ushort_as_half(static_cast<uint16_t>(static_cast<const uint8_t*>(cache)[e]) << 8));
  else return static_cast<float>(static_cast<int>(static_cast<const uint8_t*>(cache)[e]) - 128);
}

// Which of E neighbouring elements are (or hold, of several rows) NaN or an infinity, a bit each.
struct NonFinite {
  unsigned nan = 0, pos = 0, neg = 0;
  template <int KV, int E>
  __device__ __forceinline__ void add(const void* p) {
    constexpr unsigned kInf = KV == kKvBf16 ? 0x7F80u : (KV == kKvE5m2 ? 0x7Cu : 0x7C00u);
    constexpr unsigned kSign = KV == kKvE5m2 ? 0x80u : 0x8000u;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const unsigned x = KV == kKvE5m2 ? static_cast<const uint8_t*>(p)[e] : static_cast<const uint16_t*>(p)[e];
      nan |= static_cast<unsigned>((x & (kSign - 1u)) > kInf) << e;
      pos |= static_cast<unsigned>(x == kInf) << e;
      neg |= static_cast<unsigned>(x == (kInf | kSign)) << e;
    }
  }
};

// The position (whole blocks, exclusive; INT_MAX: none below `end`) up to which a sequence's value rows of KV
// head h account for what is not finite in outputs, by one warp: a NaN by a NaN or by infinities of
// both signs in its dimension, an infinity by any of them. `out` has the lane's E = D / 32 dimensions. A value
// of an INT8 cache is its code times its scale; a NaN K scale makes the whole row NaN.
template <int KV, int D>
__device__ __forceinline__ int accounted_for(const PrefillArgs& a, int s, int h, const NonFinite& out, int end) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int32_t* bt = a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq;
  NonFinite seen;
#pragma unroll 1
  for (int p = 0; p < end; p += kBlockSize) {
    const int b = bt[p >> 4];
    if (static_cast<unsigned>(b) < static_cast<unsigned>(a.num_blocks)) {
      const size_t tile = static_cast<size_t>(b) * a.num_kv_heads + h;
      constexpr int kBytes = KV == kKvE5m2 || KV == kKvInt8 ? 1 : 2;
      const uint8_t* from = static_cast<const uint8_t*>(a.v_cache) + (tile * kBlockSize * D + lane * E) * kBytes;
      if constexpr (KV == kKvInt8) {
        const float f = a.scales[tile * 32 + lane];   // K scales, then V scales
        if (__any_sync(0xffffffffu, f != f)) seen.nan = (1u << E) - 1u;
        for (unsigned inf = __ballot_sync(0xffffffffu, fabsf(f) == INFINITY) >> 16; inf; inf &= inf - 1) {
          const int t = __ffs(inf) - 1;
          const bool minus = __shfl_sync(0xffffffffu, f, 16 + t) < 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int code = static_cast<int>(from[t * D + e]) - 128;
            seen.nan |= static_cast<unsigned>(code == 0) << e;
            seen.pos |= static_cast<unsigned>(code != 0 && (code < 0) == minus) << e;
            seen.neg |= static_cast<unsigned>(code != 0 && (code < 0) != minus) << e;
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < kBlockSize; ++t) seen.add<KV, E>(from + t * D * kBytes);
      }
    }
    const unsigned any = seen.nan | seen.pos | seen.neg, none = seen.nan | (seen.pos & seen.neg);
    if (!__any_sync(0xffffffffu, (out.nan & ~none) | ((out.pos | out.neg) & ~any))) return p + kBlockSize;
  }
  return INT_MAX;
}

// Row `row` (token qb + j) of query head hq of sequence s; limit = visible positions. The
// warp's lanes take 32 positions at a time for the scores, then D/32 dimensions each
// for the sum.
template <int KV, int D>
__device__ __forceinline__ void prefill_row(const PrefillArgs& a, int s, int row, int hq, int limit) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int h = hq / a.group;
  const size_t qo = (static_cast<size_t>(row) * a.num_q_heads + hq) * D;
  constexpr int Q = KV == kKvBf16 ? kKvBf16 : kKvF16;
  const int32_t* bt = a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int p0 = 0; p0 < limit; p0 += 32) {
    const int p = p0 + lane;
    float x = -INFINITY, sv = 1.f;
    long long crow = -1;   // cache row of position p; -1: beyond the limit or a bad block (reads as zeros)
    if (p < limit) {
      const int b = bt[p >> 4];
      float dot = 0.f;
      if (static_cast<unsigned>(b) < static_cast<unsigned>(a.num_blocks)) {
        crow = (static_cast<long long>(b) * a.num_kv_heads + h) * kBlockSize + (p & 15);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          float q[8], k[8];
          load8<Q>(a.q, qo + 8 * c, q);   // the same for every lane
          load8<KV>(a.k_cache, static_cast<size_t>(crow) * D + 8 * c, k);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(q[i], k[i], dot);
        }
        if constexpr (KV == kKvInt8) {
          dot *= a.scales[(crow >> 4) * 32 + (crow & 15)];
          sv = a.scales[(crow >> 4) * 32 + 16 + (crow & 15)];
        }
      } else if (a.status) {
        atomicOr(a.status, kDevBadBlock);
      }
      x = dot * a.scale_log2;
    }
    float mx = x;
    bool nan = x != x;
#pragma unroll 1
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    nan = __any_sync(0xffffffffu, nan);
    const float mn = fmaxf(m, mx);
    const float mu = mn == -INFINITY ? 0.f : mn;   // nothing but -inf so far: every weight is 0
    const float alpha = exp2f(m - mu), w = p < limit ? exp2f(x - mu) : 0.f;
    m = mn;
    float sum = w;
#pragma unroll 1
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    l = l * alpha + sum;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
    const float wv = w * sv;
    const int cnt = limit - p0 < 32 ? limit - p0 : 32;
#pragma unroll 1
    for (int t0 = 0; t0 < cnt; t0 += 8) {   // eight rows' loads under way at once
      float v[8][E];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const long long rt = __shfl_sync(0xffffffffu, crow, t0 + t);   // (-1 behind the limit)
#pragma unroll
        for (int e = 0; e < E; ++e)
          v[t][e] = rt >= 0 ? load1<KV>(a.v_cache, static_cast<size_t>(rt) * D + lane * E + e) : 0.f;
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const float wt = __shfl_sync(0xffffffffu, wv, t0 + t);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(wt, v[t][e], o[e]);
      }
    }
    if (nan || l != l) break;   // every element is NaN from here on
  }
  // No visible position: zeros. Visible ones that all scored -inf: 0/0, as the formula gives.
  const float inv = limit > 0 ? 1.f / l : 0.f;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + qo + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float y = limit > 0 ? o[e] * inv : 0.f;
    if constexpr (KV == kKvBf16) dst[e] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    else dst[e] = __half_as_ushort(__float2half_rn(y));
  }
}

}  // namespace pkv
