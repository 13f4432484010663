// Quantising tokens into an INT4 cache, and reading rows of any cache back
// (declared in include/pagedkv.h; "KVCache Quant" of "AI大模型推理速度翻倍，Colossal-Inference开源发布"
// casts on the way in and out; the 4-bit codec is described in pkv_int4.cuh).
//
// Write: four threads a group of 64 dimensions, sixteen each; the group's least and largest value by two
// shuffles of a packed (least, -largest) pair, and both its numbers computed by each of the four.
// Bound by instructions: 365 a warp, issued on 65 % of the cycles (16.7 us for 8192 tokens of 8 heads of 128, where the bytes
// take 6.4); with eight dimensions of each group a thread and every code settled by itself it was 517 and 20.8 us.
// Read: D / 16 threads a row, sixteen dimensions each. Bound by memory: 65536 tokens of 8 heads of 128 from INT4 to fp16 in 59 us,
// 5.8 TB/s (86 % of a copy), to bf16 in 62; from INT8 in 68 (89 %), E5M2 in 64 (94 %), fp16 and bf16 in 94 to 103 (78 to 85 %).
// Products of INT8, and INT4 values on their way to bf16, are rounded to fp32 before the 16 bits. Rounded to the one of their
// two fp32 neighbours with an odd last bit they would round once; that took INT8 79 us in place of 68 and INT4 to bf16 94 in place of
// 62, for errors of 2^-24 beside a border.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pagedkv.h"
#include "pkv_int4.cuh"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

struct Int4WriteArgs {
  const uint4* src[2];         // key, value: [T][Hkv][D] 16-bit elements
  const int32_t* slot_mapping;
  uint32_t* codes[2];          // K, V caches
  uint32_t* scales;
  int32_t* status;
  long long num_slots;
  int32_t num_tokens, num_kv_heads;
};

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b, bool bf16) {
  uint32_t d;
  if (bf16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// th / heads: a 64-bit division costs more than all the rest of a row, so it is left to rows past 2^32.
__device__ __forceinline__ int token_of(long long th, int heads) {
  return static_cast<int>((th >> 32) == 0 ? static_cast<uint32_t>(th) / static_cast<uint32_t>(heads) : th / heads);
}

template <bool BF16>
__device__ __forceinline__ float2 floats_of(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <int G, bool BF16>
__global__ void __launch_bounds__(256) int4_write_kernel(const Int4WriteArgs a) {
  pdl_wait_prior_grid();
  constexpr int TPR = 4 * G;   // threads of a row: 16 dimensions each
  const long long rows = 2ll * a.num_tokens * a.num_kv_heads;
  const long long n = (rows * TPR + 31) / 32 * 32;   // whole warps: every lane takes part in the shuffles
  for (long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; idx < n;
       idx += static_cast<long long>(gridDim.x) * blockDim.x) {
    const bool real = idx < rows * TPR;
    const long long row = real ? idx / TPR : rows - 1;
    const int i = static_cast<int>(idx % TPR), g = i >> 2;
    const int which = row >= rows / 2;
    const long long th = which ? row - rows / 2 : row;
    const int t = token_of(th, a.num_kv_heads), h = static_cast<int>(th - static_cast<long long>(t) * a.num_kv_heads);
    const uint4* src = (which ? a.src[1] : a.src[0]) + th * (2 * TPR) + 2 * i;
    const uint4 v0 = src[0], v1 = src[1];
    const int slot = a.slot_mapping[t];
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    constexpr uint32_t kNeg = 0x80008000u;
    uint32_t lo2 = w[0], hi2 = w[0] ^ kNeg;
#pragma unroll
    for (int m = 1; m < 8; ++m) {
      lo2 = min2_nan(lo2, w[m], BF16);
      hi2 = min2_nan(hi2, w[m] ^ kNeg, BF16);
    }
    // (least, -largest) of the sixteen, then of the group
    uint32_t both = min2_nan(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632), BF16);
    both = min2_nan(both, __shfl_xor_sync(0xffffffffu, both, 1), BF16);
    both = min2_nan(both, __shfl_xor_sync(0xffffffffu, both, 2), BF16);
    if (!real || slot == -1) continue;
    if (slot < 0 || slot >= a.num_slots) {
      if (i == 0 && a.status) atomicOr(a.status, kDevBadSlot);
      continue;
    }
    const float2 lh = floats_of<BF16>(both);
    uint32_t words[2] = {0, 0}, meta = 0x00007FFFu;
    if (lh.x > -INFINITY && lh.y > -INFINITY && lh.x < INFINITY && lh.y < INFINITY) {
      const bool beyond = BF16 && (lh.x < -65504.f || -lh.y > 65504.f || -lh.y < -65504.f || lh.x > 65504.f);
      const Int4Group q = int4_group(fminf(fmaxf(lh.x, -65504.f), 65504.f), fminf(fmaxf(-lh.y, -65504.f), 65504.f));
      meta = pack_f16x2(q.s, q.z);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2 x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = floats_of<BF16>(w[4 * k + m]);
        if (beyond) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            x[m].x = fminf(fmaxf(x[m].x, -65504.f), 65504.f);
            x[m].y = fminf(fmaxf(x[m].y, -65504.f), 65504.f);
          }
        }
        words[k] = int4_word(x, q);
      }
    }
    const int blk = slot / kBlockSize, off = slot - blk * kBlockSize;
    const long long tile = static_cast<long long>(blk) * a.num_kv_heads + h;
    uint32_t* dst = (which ? a.codes[1] : a.codes[0]) + ((tile * kBlockSize + off) * 8 + 2 * (i & 3)) * G + g;
    dst[0] = words[0];
    dst[G] = words[1];
    if ((i & 3) == 0) a.scales[(tile * 2 * kBlockSize + which * kBlockSize + off) * G + g] = meta;
  }
  pdl_launch_dependents();
}

struct ReadArgs {
  uint16_t* dst[2];            // key, value: [T][Hkv][D]
  const int32_t* slot_mapping;
  const void* cache[2];
  const void* scales;
  int32_t* status;
  long long num_slots;
  int32_t num_tokens, num_kv_heads;
};

template <bool BF16>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
  return BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

// Sixteen dimensions of a row: dimensions 16 i .. 16 i + 15, of an INT4 row of 128 dimensions
// 8 i .. 8 i + 7 and 64 + 8 i .. + 7.
template <int KV, int D, bool BF16>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadArgs a) {
  pdl_wait_prior_grid();
  constexpr int TPR = D / 16;
  const long long rows = 2ll * a.num_tokens * a.num_kv_heads;
  for (long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; idx < rows * TPR;
       idx += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long row = idx / TPR;
    const int i = static_cast<int>(idx % TPR);
    const int which = row >= rows / 2;
    const long long th = which ? row - rows / 2 : row;
    const int t = token_of(th, a.num_kv_heads), h = static_cast<int>(th - static_cast<long long>(t) * a.num_kv_heads);
    const int slot = a.slot_mapping[t];
    if (slot == -1) continue;
    if (slot < 0 || slot >= a.num_slots) {
      if (i == 0 && a.status) atomicOr(a.status, kDevBadSlot);
      continue;
    }
    const int blk = slot / kBlockSize, off = slot - blk * kBlockSize;
    const long long tile = static_cast<long long>(blk) * a.num_kv_heads + h, at = tile * kBlockSize + off;
    const void* cache = which ? a.cache[1] : a.cache[0];
    uint32_t out[8];
    if constexpr (KV == kKvInt4) {
      constexpr int G = D / kInt4Group;
      const uint2 w = reinterpret_cast<const uint2*>(cache)[at * TPR + i];
      const uint32_t* sc = static_cast<const uint32_t*>(a.scales) + (tile * 2 * kBlockSize + which * kBlockSize + off) * G;
      const uint32_t word[2] = {w.x, w.y};
      uint32_t sz[2];
      if constexpr (G == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(sc);
        sz[0] = v.x;
        sz[1] = v.y;
      } else {
        sz[0] = sz[1] = *sc;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const __half2 p = *reinterpret_cast<const __half2*>(&sz[k]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if constexpr (!BF16) {
            const __half2 y = __hfma2(int4_pair(word[k], m), __low2half2(p), __high2half2(p));
            out[4 * k + m] = *reinterpret_cast<const uint32_t*>(&y);
          } else {
            const float2 c = __half22float2(int4_pair(word[k], m)), f = __half22float2(p);
            out[4 * k + m] = pack_bf16x2(fmaf(c.x, f.x, f.y), fmaf(c.y, f.x, f.y));
          }
        }
      }
    } else if constexpr (KV == kKvInt8 || KV == kKvE5m2) {
      const uint4 w = reinterpret_cast<const uint4*>(cache)[at * TPR + i];
      const uint32_t word[4] = {w.x, w.y, w.z, w.w};
      float s = 1.f;
      if constexpr (KV == kKvInt8) s = static_cast<const float*>(a.scales)[tile * 2 * kBlockSize + which * kBlockSize + off];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t two = word[k / 2] >> (16 * (k & 1));
        if constexpr (KV == kKvInt8) {
          out[k] = pack_out<BF16>(static_cast<float>(static_cast<int>(two & 0xFF) - 128) * s,
                                  static_cast<float>(static_cast<int>((two >> 8) & 0xFF) - 128) * s);
        } else {
          const uint32_t h2 = (two & 0xFF) << 8 | (two & 0xFF00) << 16;   // a byte is the top of its fp16 pattern
          if constexpr (BF16) {
            const float2 f = floats_of<false>(h2);
            out[k] = pack_bf16x2(f.x, f.y);
          } else {
            out[k] = h2;
          }
        }
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(cache) + (at * TPR + i) * 2;
      const uint4 x = p[0], y = p[1];
      const uint32_t word[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr ((KV == kKvBf16) == BF16) {
          out[k] = word[k];
        } else {
          const float2 f = floats_of<KV == kKvBf16>(word[k]);
          out[k] = pack_out<BF16>(f.x, f.y);
        }
      }
    }
    constexpr bool kApart = KV == kKvInt4 && D == 128;
    uint16_t* dst = (which ? a.dst[1] : a.dst[0]) + th * D + (kApart ? 8 : 16) * i;
    *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<uint4*>(dst + (kApart ? 64 : 8)) = make_uint4(out[4], out[5], out[6], out[7]);
  }
  pdl_launch_dependents();
}

template <int KV>
const void* read_kernel(int d, bool bf16) {
  if (d == 128)
    return bf16 ? reinterpret_cast<const void*>(&cache_read_kernel<KV, 128, true>)
                : reinterpret_cast<const void*>(&cache_read_kernel<KV, 128, false>);
  return bf16 ? reinterpret_cast<const void*>(&cache_read_kernel<KV, 64, true>)
              : reinterpret_cast<const void*>(&cache_read_kernel<KV, 64, false>);
}

// Blocks of 256 threads for n threads, at most eight a multiprocessor.
unsigned row_grid(long long n, int sms) {
  const long long blocks = (n + 255) / 256, most = 8ll * sms;
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

}  // namespace pkv

extern "C" {

int pkv_kv_cache_write_int4(const void* key, const void* value, pkv_dtype src_dtype, int32_t num_tokens,
                            const int32_t* slot_mapping, void* k_cache, void* v_cache, void* scales,
                            const pkv_cache_desc* cache, int32_t* device_status, void* stream) {
  using namespace pkv;
  if (num_tokens < 0 || !cache_desc_ok(cache)) return PKV_ERR_INVALID_ARGUMENT;
  if (src_dtype != PKV_FP16 && src_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!key || !value || !slot_mapping || !k_cache || !v_cache || !scales) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(key, 16) || !aligned_to(value, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(scales, 16) || !aligned_to(slot_mapping, 4) || !aligned_to(device_status, 4))
    return PKV_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  Int4WriteArgs a{};
  a.src[0] = static_cast<const uint4*>(key);
  a.src[1] = static_cast<const uint4*>(value);
  a.slot_mapping = slot_mapping;
  a.codes[0] = static_cast<uint32_t*>(k_cache);
  a.codes[1] = static_cast<uint32_t*>(v_cache);
  a.scales = static_cast<uint32_t*>(scales);
  a.status = device_status;
  a.num_slots = static_cast<long long>(cache->num_blocks) * kBlockSize;
  a.num_tokens = num_tokens;
  a.num_kv_heads = cache->num_kv_heads;
  const bool wide = cache->head_size == 128, bf16 = src_dtype == PKV_BF16;
  const void* fn = wide ? (bf16 ? reinterpret_cast<const void*>(&int4_write_kernel<2, true>)
                                : reinterpret_cast<const void*>(&int4_write_kernel<2, false>))
                        : (bf16 ? reinterpret_cast<const void*>(&int4_write_kernel<1, true>)
                                : reinterpret_cast<const void*>(&int4_write_kernel<1, false>));
  void* args[1] = {&a};
  return launch_overlapped(fn, dim3(row_grid(2ll * num_tokens * cache->num_kv_heads * (cache->head_size / 16), sms)), dim3(256), 0, stream, args);
}

int pkv_kv_cache_read(void* key, void* value, pkv_dtype dst_dtype, int32_t num_tokens, const int32_t* slot_mapping,
                      const void* k_cache, const void* v_cache, const void* scales, pkv_dtype kv_dtype,
                      const pkv_cache_desc* cache, int32_t* device_status, void* stream) {
  using namespace pkv;
  if (num_tokens < 0 || !cache_desc_ok(cache)) return PKV_ERR_INVALID_ARGUMENT;
  if (dst_dtype != PKV_FP16 && dst_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (kv_dtype != PKV_FP16 && kv_dtype != PKV_BF16 && kv_dtype != PKV_FP8_E5M2 && kv_dtype != PKV_INT8 &&
      kv_dtype != PKV_INT4)
    return PKV_ERR_UNSUPPORTED;
  if ((kv_dtype == PKV_INT8 || kv_dtype == PKV_INT4) != (scales != nullptr)) return PKV_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return PKV_OK;
  if (!key || !value || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(key, 16) || !aligned_to(value, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(scales, 16) || !aligned_to(slot_mapping, 4) || !aligned_to(device_status, 4))
    return PKV_ERR_INVALID_ARGUMENT;
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  ReadArgs a{};
  a.dst[0] = static_cast<uint16_t*>(key);
  a.dst[1] = static_cast<uint16_t*>(value);
  a.slot_mapping = slot_mapping;
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scales = scales;
  a.status = device_status;
  a.num_slots = static_cast<long long>(cache->num_blocks) * kBlockSize;
  a.num_tokens = num_tokens;
  a.num_kv_heads = cache->num_kv_heads;
  const int d = cache->head_size;
  const bool bf16 = dst_dtype == PKV_BF16;
  const void* fn = nullptr;
  switch (static_cast<int>(kv_dtype)) {
    case kKvF16: fn = read_kernel<kKvF16>(d, bf16); break;
    case kKvBf16: fn = read_kernel<kKvBf16>(d, bf16); break;
    case kKvE5m2: fn = read_kernel<kKvE5m2>(d, bf16); break;
    case kKvInt8: fn = read_kernel<kKvInt8>(d, bf16); break;
    default: fn = read_kernel<kKvInt4>(d, bf16); break;
  }
  void* args[1] = {&a};
  return launch_overlapped(fn, dim3(row_grid(2ll * num_tokens * cache->num_kv_heads * (d / 16), sms)), dim3(256), 0,
                           stream, args);
}

}  // extern "C"
