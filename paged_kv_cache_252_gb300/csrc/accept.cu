// Accepting verified draft tokens (declared in include/pagedkv.h): after a speculative
// verify ("投机采样", "AI大模型推理速度翻倍，Colossal-Inference开源发布"; token trees:
// FlexFlow Serve, survey of inference frameworks) the accepted drafts of a sequence, a
// path through its token tree, lie scattered over its last n_s positions. Row base + i
// of its cache becomes row base + accepted[i] (base = context_lens - n_s), and its new
// length is base + num_accepted.
//
// Source and destination rows overlap, so one CTA per (sequence, KV head) holds every row
// it moves in registers (at most 64 drafts x 256 bytes x K and V = 32 KB: sixteen
// 16-byte loads for each of 128 threads), passes a barrier, then stores. A draft already in
// its place is neither read nor written. Bound by its launch: a verify step moves a few
// rows a sequence.
#include <cuda_runtime.h>

#include <cstdint>

#include "pagedkv.h"
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kAcceptThreads = 128;
constexpr int kMaxDrafts = 64;

struct AcceptArgs {
  uint4* k_cache;
  uint4* v_cache;
  float* scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* cu_q_lens;
  const int32_t* accepted;      // [num_seqs][max_accepted]
  const int32_t* num_accepted;
  int32_t* new_context_lens;    // may be null
  int32_t* status;
  int32_t num_blocks, num_kv_heads, max_blocks_per_seq, max_q_per_seq, max_accepted;
  int32_t row_chunks;           // 16-byte chunks of one row (4, 8 or 16)
};

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptArgs a) {
  __shared__ long long src_row[kMaxDrafts], dst_row[kMaxDrafts];   // cache rows, -1: stays
  __shared__ int bad_s;
  const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x - s * a.num_kv_heads;
  const int tid = threadIdx.x;
  if (tid == 0) bad_s = 0;
  __syncthreads();
  pdl_wait_prior_grid();
  const int ctx = a.context_lens[s];
  const int cap = a.max_blocks_per_seq * kBlockSize;
  const int n = a.cu_q_lens ? a.cu_q_lens[s + 1] - a.cu_q_lens[s] : a.max_q_per_seq;
  const int m = a.num_accepted[s];
  const bool lens_ok = n >= 0 && n <= a.max_q_per_seq && ctx >= n && ctx <= cap && m >= 0 && m <= n && m <= a.max_accepted;
  const int base = ctx - n;
  int bad = lens_ok ? 0 : kDevBadCtx;
  if (lens_ok && tid < m) {
    const int j = a.accepted[static_cast<long long>(s) * a.max_accepted + tid];
    if (j < 0 || j >= n) {
      bad = kDevBadCtx;
    } else {
      const int32_t* bt = a.block_tables + static_cast<long long>(s) * a.max_blocks_per_seq;
      const int sp = base + j, dp = base + tid;
      const int sb = bt[sp >> 4], db = bt[dp >> 4];
      if (static_cast<unsigned>(sb) >= static_cast<unsigned>(a.num_blocks) ||
          static_cast<unsigned>(db) >= static_cast<unsigned>(a.num_blocks)) {
        bad = kDevBadBlock;
      } else {
        src_row[tid] = j == tid ? -1 : (static_cast<long long>(sb) * a.num_kv_heads + h) * kBlockSize + (sp & 15);
        dst_row[tid] = (static_cast<long long>(db) * a.num_kv_heads + h) * kBlockSize + (dp & 15);
      }
    }
  }
  if (bad) atomicOr(&bad_s, bad);
  __syncthreads();
  const int why = bad_s;
  if (h == 0 && tid == 0) {
    if (why && a.status) atomicOr(a.status, why);
    if (a.new_context_lens) a.new_context_lens[s] = why ? ctx : base + m;
  }
  if (why || m == 0) return;   // a sequence that breaks a rule is left as it is

  constexpr int kHeld = 2 * kMaxDrafts * 16 / kAcceptThreads;   // K and V rows of 256 bytes
  uint4 held[kHeld];
  const int per_cache = m * a.row_chunks, total = 2 * per_cache;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = tid + k * kAcceptThreads;
    if (i < total) {
      const int r = i < per_cache ? i : i - per_cache;
      const long long row = src_row[r / a.row_chunks];
      if (row >= 0) held[k] = (i < per_cache ? a.k_cache : a.v_cache)[row * a.row_chunks + r % a.row_chunks];
    }
  }
  float scale = 0.f;   // an INT8 cache's row scales: K of row tid, then V of row tid - m
  const bool has_scale = a.scales && tid < 2 * m;
  const int sr = tid < m ? tid : tid - m, sv = tid < m ? 0 : 16;
  if (has_scale && src_row[sr] >= 0) scale = a.scales[(src_row[sr] >> 4) * 32 + sv + (src_row[sr] & 15)];
  __syncthreads();   // every row is read before any is written
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = tid + k * kAcceptThreads;
    if (i < total) {
      const int r = i < per_cache ? i : i - per_cache;
      const int d = r / a.row_chunks;
      if (src_row[d] >= 0) (i < per_cache ? a.k_cache : a.v_cache)[dst_row[d] * a.row_chunks + r % a.row_chunks] = held[k];
    }
  }
  if (has_scale && src_row[sr] >= 0) a.scales[(dst_row[sr] >> 4) * 32 + sv + (dst_row[sr] & 15)] = scale;
}

}  // namespace pkv

extern "C" int pkv_kv_cache_accept(void* k_cache, void* v_cache, float* scales, pkv_dtype kv_dtype,
                                   const pkv_cache_desc* cache, const int32_t* block_tables,
                                   int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* cu_q_lens,
                                   int32_t num_seqs, int32_t max_q_per_seq, const int32_t* accepted,
                                   int32_t max_accepted, const int32_t* num_accepted, int32_t* new_context_lens,
                                   int32_t* device_status, void* stream) {
  using namespace pkv;
  if (!cache_desc_ok(cache) || num_seqs < 0 || max_q_per_seq <= 0 || max_accepted <= 0 || max_blocks_per_seq <= 0)
    return PKV_ERR_INVALID_ARGUMENT;
  if (kv_dtype != PKV_FP16 && kv_dtype != PKV_BF16 && kv_dtype != PKV_FP8_E5M2 && kv_dtype != PKV_INT8)
    return PKV_ERR_UNSUPPORTED;
  if (max_q_per_seq > kMaxDrafts || max_blocks_per_seq > (1 << 26)) return PKV_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_seqs) * cache->num_kv_heads >= (1ll << 31)) return PKV_ERR_UNSUPPORTED;
  if ((kv_dtype == PKV_INT8) != (scales != nullptr)) return PKV_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !accepted || !num_accepted)
    return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(scales, 16) || !aligned_to(block_tables, 4) ||
      !aligned_to(context_lens, 4) || !aligned_to(cu_q_lens, 4) || !aligned_to(accepted, 4) ||
      !aligned_to(num_accepted, 4) || !aligned_to(new_context_lens, 4) || !aligned_to(device_status, 4))
    return PKV_ERR_INVALID_ARGUMENT;
  // Every head's CTA reads what one of them would overwrite.
  auto written = [&](const int32_t* p, long long n) {
    return new_context_lens && p && new_context_lens < p + n && p < new_context_lens + num_seqs;
  };
  const long long seqs = num_seqs;
  if (written(context_lens, seqs) || written(num_accepted, seqs) || written(accepted, seqs * max_accepted) ||
      written(cu_q_lens, seqs + 1) || written(block_tables, seqs * max_blocks_per_seq))
    return PKV_ERR_INVALID_ARGUMENT;
  AcceptArgs a{};
  a.k_cache = static_cast<uint4*>(k_cache);
  a.v_cache = static_cast<uint4*>(v_cache);
  a.scales = scales;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_q_lens = cu_q_lens;
  a.accepted = accepted;
  a.num_accepted = num_accepted;
  a.new_context_lens = new_context_lens;
  a.status = device_status;
  a.num_blocks = cache->num_blocks;
  a.num_kv_heads = cache->num_kv_heads;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_q_per_seq = max_q_per_seq;
  a.max_accepted = max_accepted;
  a.row_chunks = tile_row_bytes(static_cast<int>(kv_dtype), cache->head_size) / 16;
  void* args[1] = {&a};
  const long long grid = static_cast<long long>(num_seqs) * cache->num_kv_heads;
  return launch_overlapped(reinterpret_cast<const void*>(&accept_kernel), dim3(static_cast<unsigned>(grid)),
                           dim3(kAcceptThreads), 0, stream, args);
}
