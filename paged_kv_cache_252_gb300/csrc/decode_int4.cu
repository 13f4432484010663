// Decode attention over an INT4 cache (declared in include/pagedkv.h): argument checks and launch.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "decode_int4.h"
#include "pagedkv.h"
#include "pkv_internal.h"

namespace {

using namespace pkv;

constexpr int kMaxDevices = 64;

std::mutex g_i4_mu;
struct Entry {
  int ctas;      // resident CTAs of the shape's largest row count; 0: not set up
};
Entry g_i4[kMaxDevices][2][5];   // [head size][rows]

// One a kernel: two entries that share one would set its shared-memory limit in turn.
int shape_index(int d, int rows) { return rows <= 4 && d == 128 ? 0 : rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 ? 3 : 4; }

// Fixed cost of a unit's piece on the work line, in blocks: 12 leaves 64 sequences at 34 us, 256 at 139 and 32 rows at 385, 20 at
// 30.6, 130 and 359, 32 at 30, 127 and 347, 56 at 30.6, 131 and 357.
constexpr int kPieceCostInt4 = 32;

// Once per device, head size and shape: shared-memory limits of both query types' kernels and the CTAs an
// SM holds (of the shape's largest row count, so that one workspace size serves the shape).
int resident_ctas(int d, int rows, int* ctas) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return PKV_ERR_NO_DEVICE;
  }
  const int x = shape_index(d, rows);
  std::lock_guard<std::mutex> lock(g_i4_mu);
  Entry& e = g_i4[dev][d == 128][x];
  if (e.ctas == 0) {
    const int most = 4 << x;
    int least = 0;
    for (int bf16 = 0; bf16 < 2; ++bf16) {
      const DecodeInt4Kernel k = decode_int4_kernel_of(d, most, bf16 != 0);
      int blocks = 0;
      if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem)) !=
              cudaSuccess ||
          cudaFuncSetAttribute(k.fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess ||
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, k.fn, k.threads, k.smem) != cudaSuccess || blocks <= 0) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
      }
      least = bf16 == 0 || blocks < least ? blocks : least;
    }
    e.ctas = least;   // (both kernels are set up)
  }
  *ctas = e.ctas;
  return PKV_OK;
}

// A call's workspace: units + CTAs slots, as a shared unit's pieces use slots unit + CTA, behind a counter for every slot.
struct Space {
  long long ctas;
  size_t counters, bytes;
};
int space_of(long long units, int d, int rows, Space* sp) {
  int sms = 0, per_sm = 0;
  if (int rc = device_sm_count(&sms)) return rc;
  if (int rc = resident_ctas(d, rows, &per_sm)) return rc;
  sp->ctas = static_cast<long long>(sms) * per_sm;
  if (sp->ctas > 4096) return PKV_ERR_UNSUPPORTED;   // four levels of eight
  sp->counters = decode_counter_bytes(units + sp->ctas);
  sp->bytes = sp->counters + static_cast<size_t>(units + sp->ctas) * partial_slot_floats(rows, d) * sizeof(float);
  return PKV_OK;
}

}  // namespace

namespace pkv {

size_t decode_int4_workspace_bytes(long long units, int d, int rows) {
  Space sp{};
  return space_of(units, d, rows, &sp) ? 0 : sp.bytes;
}

size_t decode_int4_counter_bytes(long long units, int d, int rows) {
  Space sp{};
  return space_of(units, d, rows, &sp) ? 0 : sp.counters;
}

}  // namespace pkv

extern "C" int pkv_paged_attention_decode_int4(void* out, const void* q, pkv_dtype q_dtype, const int32_t* cu_q_lens,
                                               const uint64_t* tree_masks, int32_t num_q_rows, int32_t num_seqs,
                                               int32_t num_q_heads, int32_t max_q_per_seq, const void* k_cache,
                                               const void* v_cache, const void* scales, const pkv_cache_desc* cache,
                                               const int32_t* block_tables, int32_t max_blocks_per_seq,
                                               const int32_t* context_lens, float scale, void* workspace,
                                               size_t workspace_bytes, int32_t* device_status, void* stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_q_heads <= 0 || max_q_per_seq <= 0 || max_blocks_per_seq <= 0 || !cache_desc_ok(cache))
    return PKV_ERR_INVALID_ARGUMENT;
  if (q_dtype != PKV_FP16 && q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (num_q_heads % cache->num_kv_heads != 0) return PKV_ERR_INVALID_ARGUMENT;
  const int group = num_q_heads / cache->num_kv_heads;
  const long long rows_ll = static_cast<long long>(group) * max_q_per_seq;
  if (rows_ll > kMaxRows || (tree_masks && max_q_per_seq > 64)) return PKV_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_seqs) * max_q_per_seq * num_q_heads >= (1ll << 31) ||
      static_cast<long long>(num_seqs) * max_blocks_per_seq >= (1ll << 31) || max_blocks_per_seq > (1 << 26))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !scales || !block_tables || !context_lens || !workspace)
    return PKV_ERR_INVALID_ARGUMENT;
  // Every row the kernel may touch lies below num_q_rows: with cu_q_lens that is checked on the device.
  if (num_q_rows < 1 || (!cu_q_lens && static_cast<long long>(num_seqs) * max_q_per_seq > num_q_rows))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) ||
      !aligned_to(scales, 16) || !aligned_to(workspace, 16) || !aligned_to(cu_q_lens, 4) || !aligned_to(tree_masks, 8) ||
      !aligned_to(block_tables, 4) || !aligned_to(context_lens, 4) || !aligned_to(device_status, 4))
    return PKV_ERR_INVALID_ARGUMENT;

  const int d = cache->head_size, rows = static_cast<int>(rows_ll);
  const long long units = static_cast<long long>(num_seqs) * cache->num_kv_heads;
  Space sp{};
  if (int rc = space_of(units, d, rows, &sp)) return rc;
  if (workspace_bytes < sp.bytes) return PKV_ERR_WORKSPACE_TOO_SMALL;
  // One wave: every CTA resident at once; never more CTAs than blocks could exist.
  const long long most = units * max_blocks_per_seq;
  const long long grid = sp.ctas < most ? sp.ctas : most;

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  DecodeInt4Args a{};
  a.out = out;
  a.q = q;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.cu_q_lens = cu_q_lens;
  a.q_rows = num_q_rows;
  a.tree_masks = reinterpret_cast<const unsigned long long*>(tree_masks);
  a.piece_counts = reinterpret_cast<unsigned long long*>(ws);
  a.partials = reinterpret_cast<float*>(ws + sp.counters);
  a.status = device_status;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.q_per_seq = max_q_per_seq;
  a.group = group;
  a.rows = rows;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_blocks = cache->num_blocks;
  a.slot_floats = partial_slot_floats(rows, d);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.epoch = next_call_epoch();
  a.piece_cost = kPieceCostInt4;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.meta = static_cast<const uint8_t*>(scales);
  const DecodeInt4Kernel k = decode_int4_kernel_of(d, rows, q_dtype == PKV_BF16);
  void* args[1] = {&a};
  return launch_overlapped(k.fn, dim3(static_cast<unsigned>(grid)), dim3(k.threads), k.smem, stream, args);
}
