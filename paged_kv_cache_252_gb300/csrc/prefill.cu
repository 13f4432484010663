// Attention of a chunk of new tokens over the paged cache (declared in include/pagedkv.h).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pagedkv.h"
#include "pkv_internal.h"
#include "prefill_row.cuh"

namespace pkv {

constexpr int kPrefillSlices = 64;

// One warp per query row; a CTA takes one (sequence, query head) and every
// kPrefillSlices-th group of rows.
template <int KV, int D>
__global__ void __launch_bounds__(256) prefill_rows_kernel(const PrefillArgs a) {
  __shared__ float qs[8][D];
  const int s = blockIdx.x / a.num_q_heads, hq = blockIdx.x - s * a.num_q_heads;
  const int warp = threadIdx.x >> 5;
  pdl_wait_prior_grid();
  const PrefillSeq p = prefill_seq(a, s);
  if (p.bad && a.status && threadIdx.x == 0 && blockIdx.y == 0 && hq == 0) atomicOr(a.status, kDevBadCtx);
  for (int j = blockIdx.y * 8 + warp; j < p.n; j += kPrefillSlices * 8)
    prefill_row<KV, D>(a, s, p.qb + j, hq, max(p.past() + j + 1, 0), qs[warp]);
}

template <int KV>
const void* prefill_fn(int d) {
  return d == 128 ? reinterpret_cast<const void*>(&prefill_rows_kernel<KV, 128>)
                  : reinterpret_cast<const void*>(&prefill_rows_kernel<KV, 64>);
}

}  // namespace pkv

extern "C" {

size_t pkv_prefill_workspace_bytes(int32_t num_q_rows, int32_t num_seqs, int32_t num_q_heads,
                                   const pkv_cache_desc* cache) {
  if (num_q_rows < 0 || num_seqs < 0 || num_q_heads <= 0 || !pkv::cache_desc_ok(cache)) return 0;
  if (num_q_heads % cache->num_kv_heads != 0 || num_q_heads / cache->num_kv_heads > pkv::kMaxRows) return 0;
  return 256;
}

int pkv_paged_attention_prefill(void* out, const void* q, const int32_t* cu_q_lens, int32_t num_q_rows,
                                int32_t num_seqs, int32_t num_q_heads, const void* k_cache, const void* v_cache,
                                const float* scales, pkv_dtype kv_dtype, const pkv_cache_desc* cache,
                                const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                                float scale, void* workspace, size_t workspace_bytes, int32_t* device_status,
                                void* stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_q_rows < 0 || num_q_heads <= 0 || max_blocks_per_seq <= 0 || !cache_desc_ok(cache))
    return PKV_ERR_INVALID_ARGUMENT;
  if (kv_dtype != PKV_FP16 && kv_dtype != PKV_BF16 && kv_dtype != PKV_FP8_E5M2 && kv_dtype != PKV_INT8)
    return PKV_ERR_UNSUPPORTED;
  if (num_q_heads % cache->num_kv_heads != 0) return PKV_ERR_INVALID_ARGUMENT;
  if (num_q_heads / cache->num_kv_heads > kMaxRows) return PKV_ERR_UNSUPPORTED;
  // Scores keep their order under the scale: the running maxima are of the unscaled ones.
  if (!std::isfinite(scale) || scale <= 0.f) return PKV_ERR_INVALID_ARGUMENT;
  if ((kv_dtype == PKV_INT8) != (scales != nullptr)) return PKV_ERR_INVALID_ARGUMENT;
  if (static_cast<long long>(num_q_rows) * num_q_heads >= (1ll << 31) ||
      static_cast<long long>(num_seqs) * cache->num_kv_heads >= (1ll << 31) || max_blocks_per_seq > (1 << 26))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || num_q_rows == 0) return PKV_OK;
  if (!out || !q || !cu_q_lens || !k_cache || !v_cache || !block_tables || !context_lens || !workspace)
    return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(scales, 16) || !aligned_to(workspace, 16) || !aligned_to(cu_q_lens, 4) ||
      !aligned_to(block_tables, 4) || !aligned_to(context_lens, 4) || !aligned_to(device_status, 4))
    return PKV_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < pkv_prefill_workspace_bytes(num_q_rows, num_seqs, num_q_heads, cache))
    return PKV_ERR_WORKSPACE_TOO_SMALL;
  PrefillArgs a{};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.scales = scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_q_lens = cu_q_lens;
  a.status = device_status;
  a.q_rows = num_q_rows;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = num_q_heads / cache->num_kv_heads;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = cache->num_blocks;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int d = cache->head_size;
  const void* fn = kv_dtype == PKV_FP16   ? prefill_fn<kKvF16>(d)
                   : kv_dtype == PKV_BF16 ? prefill_fn<kKvBf16>(d)
                   : kv_dtype == PKV_INT8 ? prefill_fn<kKvInt8>(d)
                                          : prefill_fn<kKvE5m2>(d);
  void* args[1] = {&a};
  return launch_overlapped(fn, dim3(static_cast<unsigned>(num_seqs) * num_q_heads, kPrefillSlices), dim3(256), 0,
                           stream, args);
}

}  // extern "C"
