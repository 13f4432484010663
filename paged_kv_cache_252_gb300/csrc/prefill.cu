// Attention of a chunk of new tokens over the paged cache (declared in include/pagedkv.h).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "pagedkv.h"
#include "pkv_internal.h"
#include "prefill_kernel.cuh"

namespace {

using namespace pkv;

constexpr int kMaxDevices = 64;
constexpr size_t kCounterBytes = 4096;   // 2 per CTA: up to 256 multiprocessors
constexpr uintptr_t kSlotAlign = 32;     // slots are read and written 32 bytes a thread; a workspace has 16

struct Variant {
  const void* fn;
  int threads, launch_regs;
  size_t smem;
  bool widen;
};
template <int KV, int D>
Variant variant() {
  using Sh = PfShape<KV, D>;
  return {reinterpret_cast<const void*>(&prefill_kernel<KV, D>), Sh::kThreads, Sh::kLaunchRegs, Sh::kSmem, Sh::kWiden};
}
Variant variant_of(int kv, int d) {
  switch (kv) {
    case kKvF16: return d == 128 ? variant<kKvF16, 128>() : variant<kKvF16, 64>();
    case kKvBf16: return d == 128 ? variant<kKvBf16, 128>() : variant<kKvBf16, 64>();
    case kKvE5m2: return d == 128 ? variant<kKvE5m2, 128>() : variant<kKvE5m2, 64>();
    default: return d == 128 ? variant<kKvInt8, 128>() : variant<kKvInt8, 64>();
  }
}

std::mutex g_pf_mu;
bool g_pf_ready[kMaxDevices][4][2];

// Once per device and variant: the shared-memory limit, and that the launch holds the
// registers its warpgroups share out (a larger sum would wait forever).
int make_ready(const Variant& v, int kv, int d) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return PKV_ERR_NO_DEVICE;
  }
  std::lock_guard<std::mutex> lock(g_pf_mu);
  bool& ready = g_pf_ready[dev][kv][d == 128];
  if (ready) return PKV_OK;
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, v.fn) != cudaSuccess || fa.numRegs != v.launch_regs ||
      cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(v.smem)) !=
          cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  ready = true;
  return PKV_OK;
}

int prefill_slot_tiles(long long rows) { return rows > 128 ? 2 : 1; }

}  // namespace

extern "C" {

size_t pkv_prefill_workspace_bytes(int32_t num_q_rows, int32_t num_seqs, int32_t num_q_heads,
                                   const pkv_cache_desc* cache) {
  if (num_q_rows < 0 || num_seqs < 0 || num_q_heads <= 0 || !pkv::cache_desc_ok(cache)) return 0;
  if (num_q_heads % cache->num_kv_heads != 0 || num_q_heads / cache->num_kv_heads > kMaxRows) return 0;
  int sms = 0;
  if (device_sm_count(&sms)) return 0;
  const long long rows = static_cast<long long>(num_q_rows) * (num_q_heads / cache->num_kv_heads);
  return kCounterBytes + kSlotAlign + static_cast<size_t>(2) * sms * prefill_slot_tiles(rows) * pf_slot_floats(cache->head_size) *
                             sizeof(float);
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
  int sms = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  if (2ull * sms * sizeof(unsigned long long) > kCounterBytes) return PKV_ERR_UNSUPPORTED;
  if (workspace_bytes < pkv_prefill_workspace_bytes(num_q_rows, num_seqs, num_q_heads, cache))
    return PKV_ERR_WORKSPACE_TOO_SMALL;
  const int d = cache->head_size, kv = static_cast<int>(kv_dtype);
  const Variant v = variant_of(kv, d);
  if (int rc = make_ready(v, kv, d)) return rc;

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
  const PfBox box = pf_box(a.group);
  a.box_tokens = box.tokens;
  a.unit_tokens = box.unit;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.piece_counts = reinterpret_cast<unsigned long long*>(ws);
  a.partials = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(ws) + kCounterBytes + kSlotAlign - 1) &
                                        ~(kSlotAlign - 1));
  a.slot_tiles = prefill_slot_tiles(static_cast<long long>(num_q_rows) * a.group);
  a.epoch = next_call_epoch();

  // Query rows as [token][head][dimension]: boxes of 64 dimensions x the group's heads x tokens.
  CUtensorMap tq, tk0, tk1, tv;
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(num_q_heads),
                            static_cast<uint64_t>(num_q_rows)};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * 2, static_cast<uint64_t>(d) * 2 * num_q_heads};
  const uint32_t qbox[3] = {64, static_cast<uint32_t>(a.group), static_cast<uint32_t>(box.tokens)};
  if (int rc = encode_map_16bit(&tq, q, 3, dims, strides, qbox)) return rc;
  tk0 = tk1 = tv = tq;
  if (!v.widen) {
    const long long rows = static_cast<long long>(cache->num_blocks) * cache->num_kv_heads * kBlockSize;
    if (int rc = encode_tile_map(&tk0, k_cache, kv, d, rows, 0)) return rc;
    if (d == 128) {
      if (int rc = encode_tile_map(&tk1, k_cache, kv, d, rows, 1)) return rc;
    }
    // V: [half][token row][64 dimensions], a block's halves in one box.
    const uint32_t halves = static_cast<uint32_t>(d) / 64;
    const uint64_t vdims[3] = {64, static_cast<uint64_t>(rows), halves};
    const uint64_t vstrides[2] = {static_cast<uint64_t>(d) * 2, 128};
    const uint32_t vbox[3] = {64, kBlockSize, halves};
    if (int rc = encode_map_16bit(&tv, v_cache, 3, vdims, vstrides, vbox)) return rc;
  } else {
    const long long rows = static_cast<long long>(cache->num_blocks) * cache->num_kv_heads * kBlockSize;
    if (int rc = encode_tile_map(&tk0, k_cache, kv, d, rows, 0)) return rc;
    if (int rc = encode_tile_map(&tv, v_cache, kv, d, rows, 0)) return rc;
  }
  void* args[5] = {&tq, &tk0, &tk1, &tv, &a};
  return launch_overlapped(v.fn, dim3(static_cast<unsigned>(sms)), dim3(v.threads), v.smem, stream, args);
}

}  // extern "C"
