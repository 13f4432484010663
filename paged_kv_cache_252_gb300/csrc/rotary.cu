// Rotary position embedding of query and key rows, and its fusion with the cache write
// (declared in include/pagedkv.h; "kernel1" of the KVCache Quant section of
// "AI大模型推理速度翻倍，Colossal-Inference开源发布" is the writer it extends).
//
// A row's first rotary_dim dimensions form rotary_dim / 2 pairs (dimensions i and
// i + rotary_dim/2, or 2i and 2i + 1 when interleaved). Pair i of a token at position p
// turns by the angle a = p * inv_freq[i]:
//   y_re = f (x_re cos a - x_im sin a),   y_im = f (x_re sin a + x_im cos a),
// in fp32, rounded once to the output's type (a query's 16 bits, the key's cache type).
//
// Angles. p * inv_freq reaches 10^6 rad, where an fp32 product is off by 0.03 rad. One
// turn is 2^64 here: each CTA converts inv_freq / 2 pi once to a 64-bit fraction of a turn
// per position (in whole numbers: an fp64 product's error, 2^-53 of the angle, came to 0.003 rad at
// position 2^45), and p times that step modulo 2^64 is the angle, the whole turns gone exactly;
// quarter turns taken off, the rest as two fp32 numbers goes to sincospif. No angle needs the fp64 unit.
//
// Work. A row of D dimensions is D/16 items: an item is one pair of 16-byte chunks, eight
// (re, im) pairs of the rotated part or sixteen plain dimensions (the unrotated tail, and
// the whole of a value row), so every thread moves two 16-byte loads and two stores
// whatever the layout. A CTA takes tiles of a few tokens: their cosines and sines go
// through shared memory once, and the tile's items (all heads of q, key and value) are
// spread over its threads. The D/16 lanes of one row are neighbours in a warp, which
// gives the INT8 writer its row maximum by shuffles. The next tile's angles are worked out while
// this tile's rows are under way (8192 tokens 42 us without, 37 with).
//
// Bound by memory, a step of few tokens by its launch. Measured, 32 query and 8 KV heads of 128:
// 8192 bf16 tokens 37 us, 5.4 TB/s (a copy reaches 6.77); 64 tokens 3 us. 2001 fp16 tokens of
// 16 + 4 heads of 64, half of each rotated: 5 us. 512 tokens of 64 + 8 heads to an E5M2 cache: 9.8
// us, 6.9 with fp32 alone, which puts 11 of 15.7 M keys on the wrong side of a rounding border; to
// fp16 and INT8 5.8 and 11.0. 8192 tokens of 32 + 8 to E5M2 51 us, to INT8 64.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pagedkv.h"
#include "pkv_codec.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryBatch = 2;          // items a thread loads before it stores any
constexpr int kRotaryMaxPairs = 64;      // head size 128
constexpr int kRotaryMaxTokens = 8;      // tokens of a CTA's tile

struct RotaryArgs {
  const uint16_t* q;           // rotated to q_out; token strides in elements
  const uint16_t* key;
  const uint16_t* value;
  uint16_t* q_out;
  long long q_stride, q_out_stride, key_stride, value_stride;
  const void* positions;
  const int32_t* slot_mapping; // null: no cache (queries only)
  const double* inv_freq;      // [rotary_dim / 2]
  void* k_cache;
  void* v_cache;
  float* scales;
  int32_t* status;
  long long num_slots;
  int32_t num_tokens, num_q_heads, num_kv_heads;
  int32_t items_row;           // D / 16, a power of two
  int32_t log_items_row;
  int32_t rot_items;           // rotary_dim / 16
  int32_t tile;                // tokens of a CTA's tile
  int32_t pos64, interleaved;
  float factor, sign;          // sign -1 turns the other way
  double factor64;
};

// f / 2 pi modulo one turn in units of 2^-64, to the nearest (|f| below 2^52): a long multiplication of
// f's 53 bits with 2^128 / 2 pi.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(f));
  const int field = static_cast<int>(bits >> 52) & 0x7FF;
  const unsigned long long m = (bits & ((1ull << 52) - 1)) | (1ull << 52);
  const int down = 1075 - field;   // f = m 2^-down, and p = m 2^64 / 2 pi
  if (down < 0 || down > 127) return 0;
  unsigned __int128 p = static_cast<unsigned __int128>(m) * 0x28BE60DB9391054Aull + __umul64hi(m, 0x7F09D5F47D4D3770ull);
  if (down > 0) p = (p + (static_cast<unsigned __int128>(1) << (down - 1))) >> down;
  const unsigned long long r = static_cast<unsigned long long>(p);
  return (bits >> 63) ? 0ull - r : r;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = BF16 ? pack_bf16x2(x[2 * i], x[2 * i + 1]) : pack_f16x2(x[2 * i], x[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// An item's E5M2 key bytes where fp32 leaves open on which side of a rounding border a value
// lies: `low` and `high` are the bytes of the values less and plus fp32's error; pairs in which they
// differ are turned again in fp64. Elements by their order in the item (first chunk, then second).
__device__ __noinline__ uint4 rotary_e5m2_exact(uint4 va, uint4 vb, uint4 low, uint4 high, unsigned long long pos,
                                                const unsigned long long* step, int interleaved, double factor,
                                                double sign) {
  const uint32_t src[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
  uint32_t w[4] = {low.x, low.y, low.z, low.w};
  const uint32_t u[4] = {high.x, high.y, high.z, high.w};
  auto value = [&](int e) {
    return static_cast<double>(__half2float(__ushort_as_half(static_cast<unsigned short>(src[e >> 1] >> (16 * (e & 1))))));
  };
  auto differs = [&](int e) { return (((w[e >> 2] ^ u[e >> 2]) >> (8 * (e & 3))) & 0xFFu) != 0; };
  auto put = [&](int e, double y) {
    // fp64 -> fp32 with the dropped bits kept in the last one, so that the next rounding is the only one
    float f = __double2float_rz(y);
    if (static_cast<double>(f) != y) f = __uint_as_float(__float_as_uint(f) | 1u);
    const uint32_t byte = e5m2x2_of_f32(f, 0.f) & 0xFFu;
    w[e >> 2] = (w[e >> 2] & ~(0xFFu << (8 * (e & 3)))) | (byte << (8 * (e & 3)));
  };
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    const int e0 = interleaved ? 2 * k : k, e1 = interleaved ? 2 * k + 1 : 8 + k;
    if (!differs(e0) && !differs(e1)) continue;
    // Quarter turns apart; of the rest z, at most pi / 4, the Taylor sums of sine to z^13 and cosine
    // to z^14 (2 10^-14 off).
    const unsigned long long phase = pos * step[k];
    const unsigned quarter = static_cast<unsigned>((phase + (1ull << 61)) >> 62);
    const double z = static_cast<double>(static_cast<long long>(phase - (static_cast<unsigned long long>(quarter) << 62))) *
                     3.4061215800865545e-19;   // 2^-63 pi
    const double zz = z * z;
    double sn = 1.0 / 6227020800.0, cn = -1.0 / 87178291200.0;
    sn = fma(sn, zz, -1.0 / 39916800.0);
    cn = fma(cn, zz, 1.0 / 479001600.0);
    sn = fma(sn, zz, 1.0 / 362880.0);
    cn = fma(cn, zz, -1.0 / 3628800.0);
    sn = fma(sn, zz, -1.0 / 5040.0);
    cn = fma(cn, zz, 1.0 / 40320.0);
    sn = fma(sn, zz, 1.0 / 120.0);
    cn = fma(cn, zz, -1.0 / 720.0);
    sn = fma(sn, zz, -1.0 / 6.0);
    cn = fma(cn, zz, 1.0 / 24.0);
    sn = fma(sn * zz, z, z);
    cn = fma(fma(cn, zz, -0.5), zz, 1.0);
    if (quarter & 1) {
      const double t = cn;
      cn = -sn;
      sn = t;
    }
    if (quarter & 2) {
      cn = -cn;
      sn = -sn;
    }
    sn *= sign;
    const double re = value(e0), im = value(e1);
    put(e0, factor * (re * cn - im * sn));
    put(e1, factor * (re * sn + im * cn));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// KV: the cache's element type (kKvBf16 means bf16 rows everywhere, the others fp16 rows).
template <int KV>
__global__ void __launch_bounds__(kRotaryThreads, KV == kKvE5m2 ? 4 : 0) rotary_kernel(const RotaryArgs a) {
  constexpr bool BF16 = KV == kKvBf16;
  __shared__ unsigned long long step[kRotaryMaxPairs];
  __shared__ float2 cs2[2][kRotaryMaxTokens * kRotaryMaxPairs];
  const int tid = threadIdx.x, lane = tid & 31;
  const int pairs = a.rot_items * 8;
  pdl_wait_prior_grid();
  const int heads = a.num_q_heads + 2 * a.num_kv_heads;
  const int per_token = heads << a.log_items_row;
  const int D = a.items_row * 16;
  const int second = a.interleaved ? 8 : a.rot_items * 8;   // distance of an item's second chunk
  const long long stride = static_cast<long long>(gridDim.x) * a.tile;
  auto tile_tokens = [&](long long t0) { return static_cast<int>(a.num_tokens - t0 < a.tile ? a.num_tokens - t0 : a.tile); };
  // Items i0, i0 + 256, ... of the tile at t0: both chunks of each.
  uint4 va[kRotaryBatch], vb[kRotaryBatch];
  auto load = [&](long long t0, int total, int i0) {
#pragma unroll
    for (int b = 0; b < kRotaryBatch; ++b) {
      const int i = i0 + b * kRotaryThreads;
      if (i >= total) break;
      const int row = i >> a.log_items_row, c = i & (a.items_row - 1);
      const int t = row / heads, h = row - t * heads;
      const uint16_t* src;
      if (h < a.num_q_heads) src = a.q + (t0 + t) * a.q_stride + h * D;
      else if (h < a.num_q_heads + a.num_kv_heads) src = a.key + (t0 + t) * a.key_stride + (h - a.num_q_heads) * D;
      else src = a.value + (t0 + t) * a.value_stride + (h - a.num_q_heads - a.num_kv_heads) * D;
      const bool turn = c < a.rot_items && h < a.num_q_heads + a.num_kv_heads;
      const int o1 = turn && !a.interleaved ? 8 * c : 16 * c;
      const int o2 = o1 + (turn ? second : 8);
      va[b] = *reinterpret_cast<const uint4*>(src + o1);
      vb[b] = *reinterpret_cast<const uint4*>(src + o2);
    }
  };
  // The cosines and sines of the tile at t0.
  auto angles = [&](long long t0, float2* cs) {
    const int nt = tile_tokens(t0);
    for (int i = tid; i < nt * pairs; i += kRotaryThreads) {
      const int t = i / pairs, j = i - t * pairs;
      const long long p = a.pos64 ? static_cast<const long long*>(a.positions)[t0 + t]
                                  : static_cast<const int32_t*>(a.positions)[t0 + t];
      const unsigned long long phase = static_cast<unsigned long long>(p) * step[j];
      // Quarter turns apart (exactly), the rest r within an eighth of a turn as hi + lo: rounded to
      // one fp32 number, an angle near half a turn would be off by more than the fp32 cosine (of 15.7 M
      // keys rounded to E5M2 27 fell on the wrong side of a border, 11 so; of fp64 cosines 12).
      const unsigned quarter = static_cast<unsigned>((phase + (1ull << 61)) >> 62);
      const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(quarter) << 62));
      const float hi = __ll2float_rn(rest), lo = __ll2float_rn(rest - __float2ll_rn(hi));
      float s0, c0;
      sincospif(hi * 1.0842021724855044e-19f, &s0, &c0);   // 2^-63: half turns in [-1/4, 1/4]
      const float e = lo * 3.4061215800865545e-19f;        // 2^-63 pi: sin(r + e) = sin r + e cos r, e^2 below 2^-48
      float s = fmaf(e, c0, s0), c = fmaf(-e, s0, c0);
      if (quarter & 1) {
        const float t = c;
        c = -s;
        s = t;
      }
      if (quarter & 2) {
        c = -c;
        s = -s;
      }
      cs[t * pairs + j] = make_float2(c * a.factor, s * a.factor * a.sign);
    }
  };
  long long t0 = static_cast<long long>(blockIdx.x) * a.tile;
  // A tile's first rows are under way while angles are worked out: the first tile's its own, a
  // later one's the tile's behind it.
  if (t0 < a.num_tokens) load(t0, tile_tokens(t0) * per_token, tid);
  if (tid < pairs) step[tid] = turn_fraction(a.inv_freq[tid]);
  __syncthreads();
  int buf = 0;
  if (t0 < a.num_tokens) angles(t0, cs2[0]);
  for (; t0 < a.num_tokens; t0 += stride, buf ^= 1) {
    __syncthreads();   // this tile's cosines are written, the last tile's read
    if (t0 + stride < a.num_tokens) angles(t0 + stride, cs2[buf ^ 1]);
    const float2* cs = cs2[buf];
    const int total = tile_tokens(t0) * per_token;
    for (int i0 = tid; i0 < total; i0 += kRotaryThreads * kRotaryBatch) {
      if (i0 != tid) load(t0, total, i0);
#pragma unroll
      for (int b = 0; b < kRotaryBatch; ++b) {
        const int i = i0 + b * kRotaryThreads;
        if (i >= total) break;
        const int row = i >> a.log_items_row, c = i & (a.items_row - 1);
        const int t = row / heads, h = row - t * heads;
        const bool is_v = h >= a.num_q_heads + a.num_kv_heads;
        const bool turn = c < a.rot_items && !is_v;
        const int o1 = turn && !a.interleaved ? 8 * c : 16 * c;
        const int o2 = o1 + (turn ? second : 8);
        float x[8], y[8];
        if (turn) {
          unpack8<BF16>(va[b], x);
          unpack8<BF16>(vb[b], y);
          const float2* w = cs + t * pairs + 8 * c;
          if (a.interleaved) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 w0 = w[k], w1 = w[4 + k];
              const float re0 = x[2 * k], im0 = x[2 * k + 1], re1 = y[2 * k], im1 = y[2 * k + 1];
              x[2 * k] = re0 * w0.x - im0 * w0.y;
              x[2 * k + 1] = re0 * w0.y + im0 * w0.x;
              y[2 * k] = re1 * w1.x - im1 * w1.y;
              y[2 * k + 1] = re1 * w1.y + im1 * w1.x;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 wk = w[k];
              const float re = x[k], im = y[k];
              x[k] = re * wk.x - im * wk.y;
              y[k] = re * wk.y + im * wk.x;
            }
          }
        }
        if (h < a.num_q_heads) {
          uint16_t* dst = a.q_out + (t0 + t) * a.q_out_stride + h * D;
          *reinterpret_cast<uint4*>(dst + o1) = turn ? pack8<BF16>(x) : va[b];
          *reinterpret_cast<uint4*>(dst + o2) = turn ? pack8<BF16>(y) : vb[b];
          continue;
        }
        const long long slot = a.slot_mapping[t0 + t];
        const bool bad = slot < -1 || slot >= a.num_slots;
        if (bad && a.status && c == 0) atomicOr(a.status, kDevBadSlot);
        if (bad || slot == -1) continue;   // the whole row's lanes together
        const int hk = h - a.num_q_heads - (is_v ? a.num_kv_heads : 0);
        // row of the cache: (block * Hkv + head) * 16 + offset
        const long long crow = ((slot >> 4) * a.num_kv_heads + hk) * kBlockSize + (slot & 15);
        void* cache = is_v ? a.v_cache : a.k_cache;
        if constexpr (KV == kKvF16 || KV == kKvBf16) {
          uint16_t* dst = static_cast<uint16_t*>(cache) + crow * D;
          *reinterpret_cast<uint4*>(dst + o1) = turn ? pack8<BF16>(x) : va[b];
          *reinterpret_cast<uint4*>(dst + o2) = turn ? pack8<BF16>(y) : vb[b];
        } else if constexpr (KV == kKvE5m2) {
          uint8_t* dst = static_cast<uint8_t*>(cache) + crow * D;
          uint2 w1, w2;
          if (turn) {
            // From fp32 in one rounding where its error d does not reach a border; two of 10^5 elements'
            // does. d is 8 u factor (|re| + |im|), u = 2^-24: the cosine and sine are within 2 u (two ulp of
            // sincospif below 1), their correction rounds by u / 2, the factor to fp32 by u, their product by
            // u, of the two products with re and im one by u, the sum by u, x - d and x + d by u.
            float ox[8], oy[8];
            unpack8<BF16>(va[b], ox);
            unpack8<BF16>(vb[b], oy);
            const float eps = fabsf(a.factor) * 4.76837158203125e-7f;
            uint32_t low[4], high[4];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              float dx[2], dy[2];
              if (a.interleaved) {
                dx[0] = dx[1] = (fabsf(ox[k]) + fabsf(ox[k + 1])) * eps;
                dy[0] = dy[1] = (fabsf(oy[k]) + fabsf(oy[k + 1])) * eps;
              } else {
                dx[0] = dy[0] = (fabsf(ox[k]) + fabsf(oy[k])) * eps;
                dx[1] = dy[1] = (fabsf(ox[k + 1]) + fabsf(oy[k + 1])) * eps;
              }
              const uint32_t lx = e5m2x2_of_f32(x[k] - dx[0], x[k + 1] - dx[1]);
              const uint32_t hx = e5m2x2_of_f32(x[k] + dx[0], x[k + 1] + dx[1]);
              const uint32_t ly = e5m2x2_of_f32(y[k] - dy[0], y[k + 1] - dy[1]);
              const uint32_t hy = e5m2x2_of_f32(y[k] + dy[0], y[k + 1] + dy[1]);
              const int at = k >> 2, sh = (k & 2) * 8;
              low[at] = sh ? low[at] | (lx << 16) : lx;
              high[at] = sh ? high[at] | (hx << 16) : hx;
              low[2 + at] = sh ? low[2 + at] | (ly << 16) : ly;
              high[2 + at] = sh ? high[2 + at] | (hy << 16) : hy;
            }
            uint4 w = make_uint4(low[0], low[1], low[2], low[3]);
            if ((low[0] ^ high[0]) | (low[1] ^ high[1]) | (low[2] ^ high[2]) | (low[3] ^ high[3])) {
              const long long p = a.pos64 ? static_cast<const long long*>(a.positions)[t0 + t]
                                          : static_cast<const int32_t*>(a.positions)[t0 + t];
              w = rotary_e5m2_exact(va[b], vb[b], w, make_uint4(high[0], high[1], high[2], high[3]),
                                    static_cast<unsigned long long>(p), step + 8 * c, a.interleaved, a.factor64, a.sign);
            }
            w1 = make_uint2(w.x, w.y);
            w2 = make_uint2(w.z, w.w);
          } else {
            w1 = make_uint2(e5m2x4(va[b].x, va[b].y), e5m2x4(va[b].z, va[b].w));
            w2 = make_uint2(e5m2x4(vb[b].x, vb[b].y), e5m2x4(vb[b].z, vb[b].w));
          }
          *reinterpret_cast<uint2*>(dst + o1) = w1;
          *reinterpret_cast<uint2*>(dst + o2) = w2;
        } else {
          if (!turn) {
            unpack8<BF16>(va[b], x);
            unpack8<BF16>(vb[b], y);
          }
          float amax = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(x[k]), fabsf(y[k])));
          // The row's items_row lanes are aligned and either all here or none.
          const unsigned group = ((1u << a.items_row) - 1u) << (lane & ~(a.items_row - 1));
          for (int o = a.items_row >> 1; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
          const float scale = int8_row_scale(amax);
          uint2 w1 = make_uint2(0u, 0u), w2 = make_uint2(0u, 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w1.x |= int8_byte(x[k], scale) << (8 * k);
            w1.y |= int8_byte(x[4 + k], scale) << (8 * k);
            w2.x |= int8_byte(y[k], scale) << (8 * k);
            w2.y |= int8_byte(y[4 + k], scale) << (8 * k);
          }
          uint8_t* dst = static_cast<uint8_t*>(cache) + crow * D;
          *reinterpret_cast<uint2*>(dst + o1) = w1;
          *reinterpret_cast<uint2*>(dst + o2) = w2;
          if (c == 0) a.scales[(crow >> 4) * 32 + (is_v ? 16 : 0) + (crow & 15)] = scale;
        }
      }
    }
    if (t0 + stride < a.num_tokens) load(t0 + stride, tile_tokens(t0 + stride) * per_token, tid);
  }
  pdl_launch_dependents();
}

}  // namespace pkv

namespace {

using namespace pkv;

// Arguments both entry points share: types, sizes, alignment. Token strides are in elements.
int rotary_common(RotaryArgs* a, pkv_dtype dtype, int32_t num_tokens, int32_t head_size, const void* positions,
                  int32_t position_bytes, const double* inv_freq, int32_t rotary_dim, double attn_factor) {
  if (dtype != PKV_FP16 && dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (num_tokens < 0) return PKV_ERR_INVALID_ARGUMENT;
  if (head_size != 64 && head_size != 128) return PKV_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > head_size || rotary_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (position_bytes != 4 && position_bytes != 8) return PKV_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(static_cast<float>(attn_factor))) return PKV_ERR_INVALID_ARGUMENT;
  if (num_tokens > 0 && (!positions || !inv_freq)) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(positions, static_cast<uintptr_t>(position_bytes)) || !aligned_to(inv_freq, 8))
    return PKV_ERR_INVALID_ARGUMENT;
  a->positions = positions;
  a->pos64 = position_bytes == 8;
  a->inv_freq = inv_freq;
  a->num_tokens = num_tokens;
  a->items_row = head_size / 16;
  a->log_items_row = head_size == 128 ? 3 : 2;
  a->rot_items = rotary_dim / 16;
  a->factor = static_cast<float>(attn_factor);
  a->factor64 = attn_factor;
  a->sign = 1.f;
  return PKV_OK;
}

// Rows of `heads` heads, 16-byte aligned, that do not overlap.
bool rows_ok(const void* p, long long stride, int32_t heads, int32_t head_size) {
  return p && aligned_to(p, 16) && stride % 8 == 0 && stride >= static_cast<long long>(heads) * head_size;
}

int rotary_launch(RotaryArgs& a, const void* fn, void* stream) {
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  const long long heads = a.num_q_heads + 2ll * a.num_kv_heads;
  if (heads * a.items_row * kRotaryMaxTokens >= (1ll << 31)) return PKV_ERR_UNSUPPORTED;
  // Tokens of a tile: about six items a thread, but no fewer tiles than the GPU holds CTAs.
  const long long per_token = heads * a.items_row;
  long long tile = (6ll * kRotaryThreads + per_token - 1) / per_token;
  const long long even = a.num_tokens / (sms * 4ll);
  if (tile > even) tile = even;
  if (tile > kRotaryMaxTokens) tile = kRotaryMaxTokens;
  if (tile < 1) tile = 1;
  a.tile = static_cast<int32_t>(tile);
  long long blocks = (a.num_tokens + tile - 1) / tile;
  if (blocks > sms * 4ll) blocks = sms * 4ll;
  void* args[1] = {&a};
  return launch_overlapped(fn, dim3(static_cast<unsigned>(blocks)), dim3(kRotaryThreads), 0, stream, args);
}

}  // namespace

extern "C" {

int pkv_rotary_embed(void* out, int64_t out_stride, const void* x, int64_t x_stride, pkv_dtype dtype,
                     int32_t num_tokens, int32_t num_heads, int32_t head_size, const void* positions,
                     int32_t position_bytes, const double* inv_freq, int32_t rotary_dim, int32_t interleaved,
                     double attn_factor, int32_t inverse, void* stream) {
  RotaryArgs a{};
  if (int rc = rotary_common(&a, dtype, num_tokens, head_size, positions, position_bytes, inv_freq, rotary_dim,
                             attn_factor))
    return rc;
  if (num_heads <= 0) return PKV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return PKV_OK;
  if (!rows_ok(out, out_stride, num_heads, head_size) || !rows_ok(x, x_stride, num_heads, head_size))
    return PKV_ERR_INVALID_ARGUMENT;
  a.q = static_cast<const uint16_t*>(x);
  a.q_out = static_cast<uint16_t*>(out);
  a.q_stride = x_stride;
  a.q_out_stride = out_stride;
  a.num_q_heads = num_heads;
  a.interleaved = interleaved != 0;
  if (inverse) a.sign = -1.f;
  return rotary_launch(a, dtype == PKV_BF16 ? reinterpret_cast<const void*>(&rotary_kernel<kKvBf16>)
                                            : reinterpret_cast<const void*>(&rotary_kernel<kKvF16>), stream);
}

int pkv_rotary_write(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* key,
                     int64_t key_stride, const void* value, int64_t value_stride, pkv_dtype src_dtype,
                     int32_t num_tokens, int32_t num_q_heads, const void* positions, int32_t position_bytes,
                     const int32_t* slot_mapping, const double* inv_freq, int32_t rotary_dim, int32_t interleaved,
                     double attn_factor, void* k_cache, void* v_cache, float* scales, pkv_dtype kv_dtype,
                     const pkv_cache_desc* cache, int32_t* device_status, void* stream) {
  if (!cache_desc_ok(cache)) return PKV_ERR_INVALID_ARGUMENT;
  const bool pair_ok = (src_dtype == PKV_FP16 && (kv_dtype == PKV_FP16 || kv_dtype == PKV_FP8_E5M2 ||
                                                  kv_dtype == PKV_INT8)) ||
                       (src_dtype == PKV_BF16 && kv_dtype == PKV_BF16);
  if (!pair_ok) return PKV_ERR_UNSUPPORTED;
  RotaryArgs a{};
  if (int rc = rotary_common(&a, src_dtype, num_tokens, cache->head_size, positions, position_bytes, inv_freq,
                             rotary_dim, attn_factor))
    return rc;
  if (num_q_heads <= 0 || (kv_dtype == PKV_INT8) != (scales != nullptr)) return PKV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return PKV_OK;
  const int D = cache->head_size, Hkv = cache->num_kv_heads;
  if (!rows_ok(q_out, q_out_stride, num_q_heads, D) || !rows_ok(q, q_stride, num_q_heads, D) ||
      !rows_ok(key, key_stride, Hkv, D) || !rows_ok(value, value_stride, Hkv, D))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!k_cache || !v_cache || !slot_mapping) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(scales, 16) ||
      !aligned_to(slot_mapping, 4) || !aligned_to(device_status, 4))
    return PKV_ERR_INVALID_ARGUMENT;
  a.q = static_cast<const uint16_t*>(q);
  a.key = static_cast<const uint16_t*>(key);
  a.value = static_cast<const uint16_t*>(value);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.slot_mapping = slot_mapping;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.scales = scales;
  a.status = device_status;
  a.num_slots = static_cast<long long>(cache->num_blocks) * kBlockSize;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = Hkv;
  a.interleaved = interleaved != 0;
  const void* fn = kv_dtype == PKV_FP16   ? reinterpret_cast<const void*>(&rotary_kernel<kKvF16>)
                   : kv_dtype == PKV_BF16 ? reinterpret_cast<const void*>(&rotary_kernel<kKvBf16>)
                   : kv_dtype == PKV_INT8 ? reinterpret_cast<const void*>(&rotary_kernel<kKvInt8>)
                                          : reinterpret_cast<const void*>(&rotary_kernel<kKvE5m2>);
  return rotary_launch(a, fn, stream);
}

}  // extern "C"
