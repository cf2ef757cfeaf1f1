// pkv_internal.h -- launchers shared between the C-ABI front end (pkv_api.cu)
// and the kernel translation units.  Arguments here are already validated.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>
#include <algorithm>
#include <atomic>
#include <utility>

#include "pkv.h"

namespace pkv {

constexpr int kBlockSize = 256;
constexpr int kHeadDim = 128;
constexpr int kMaxKvHeads = 8;
constexpr int kMaxGroup = 16;
constexpr int kMaxQHeads = 64;

// Raise `kernel`'s dynamic shared-memory limit on the current device to at
// least `bytes`, calling the runtime only when the request exceeds what was
// already set on that device (`marks` holds one high-water mark per device,
// zero-initialised static storage of the caller).
constexpr int kMaxDevices = 64;
template <typename... KArgs>
cudaError_t ensure_dyn_smem(void (*kernel)(KArgs...), size_t bytes, std::atomic<int>* marks) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int want = static_cast<int>(bytes);
  if (dev >= 0 && dev < kMaxDevices && want <= marks[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, want);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) {
    int cur = marks[dev].load(std::memory_order_relaxed);
    while (cur < want && !marks[dev].compare_exchange_weak(cur, want, std::memory_order_release)) {
    }
  }
  return e;
}

// Launch `kernel` on `stream` with programmatic stream serialization
// allowed, so it may start while the previous kernel drains (each kernel
// calls griddepcontrol.wait before touching global memory).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// ---- KV write
cudaError_t launch_kv_cache_write(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                  int64_t v_stride, const int32_t* slots, int32_t num_tokens,
                                  uint16_t* k_cache, uint16_t* v_cache, int64_t num_slots,
                                  int32_t row_elems, cudaStream_t stream);

// ---- decode
struct DecodeArgs {
  const uint16_t* q;
  const int32_t* context_lens;
  const int32_t* block_tables;
  uint16_t* out;
  int32_t max_blocks_per_seq;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t num_blocks;
  int32_t max_context_len;
  float scale;
  void* workspace;
  // Fused KV write (optional; all null for plain decode): each sequence's new
  // token row k_new[b] / v_new[b] (token strides in elements) is written to
  // k_cache / v_cache at slot_mapping[b] before it is read.
  const uint16_t* k_new = nullptr;
  const uint16_t* v_new = nullptr;
  int64_t k_stride = 0;
  int64_t v_stride = 0;
  const int32_t* slot_mapping = nullptr;
  uint16_t* k_cache = nullptr;
  uint16_t* v_cache = nullptr;
};
// Tensor maps over the caches, built by the front end (see pkv_api.cu).
// `per_head` selects the layout of the copy: one 5-D box per K (or V) tile,
// or 2 * num_kv_heads 3-D boxes with the same shared-memory image.
struct CacheMaps {
  CUtensorMap k;
  CUtensorMap v;
  int per_head;
};
size_t decode_workspace_bytes(int batch, int num_q_heads, int num_sms);
int decode_grid(int num_sms);
cudaError_t launch_paged_attn_decode(const DecodeArgs& a, const CacheMaps& maps, int num_sms,
                                     cudaStream_t stream);

// ---- prefill
struct PrefillArgs {
  const uint16_t* q;
  const int32_t* cu_seqlens_q;
  const int32_t* cu_seqlens_k;
  const int32_t* block_tables;
  uint16_t* out;
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t total_q;
  int32_t max_seqlen_q;
  int32_t max_seqlen_k;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t num_blocks;
  float scale;
  // Fused KV write (optional; all null for plain prefill): token i's new row
  // k_new[i] / v_new[i] (token strides in elements) goes to k_cache / v_cache
  // at slot_mapping[i] before any cache read; barrier_ws is the caller's
  // two-word grid-barrier workspace.
  const uint16_t* k_new = nullptr;
  const uint16_t* v_new = nullptr;
  int64_t k_stride = 0;
  int64_t v_stride = 0;
  const int32_t* slot_mapping = nullptr;
  uint16_t* k_cache = nullptr;
  uint16_t* v_cache = nullptr;
  unsigned int* barrier_ws = nullptr;
};
// Stated max_seqlen_q up to which the persistent kernel is used (prefill.cu
// dispatches; prefill_persistent.cu holds that kernel).
constexpr int kPersistentMaxSeqlenQ = 2048;
cudaError_t launch_paged_attn_prefill(const PrefillArgs& a, const CacheMaps& kv_maps,
                                      const CUtensorMap& q_map, const CUtensorMap& out_map, int num_sms,
                                      cudaStream_t stream);
cudaError_t launch_prefill_persistent(const PrefillArgs& a, const CacheMaps& kv_maps, const CUtensorMap& q_map,
                                      const CUtensorMap& out_map, int num_sms, cudaStream_t stream);

// ---- step metadata
struct MetaArgs {
  const int32_t* block_ids;
  const int32_t* table_offsets;
  const int32_t* num_cached;
  const int32_t* seq_lens;
  int32_t num_seqs, token_capacity, max_blocks_per_seq, block_size, num_blocks;
  int32_t* cu_seqlens_q;
  int32_t* cu_seqlens_k;
  int32_t* context_lens;
  int32_t* slot_mapping;
  int32_t* block_tables;
};
cudaError_t launch_prepare_metadata(const MetaArgs& a, int num_sms, cudaStream_t stream);

// ---- exponential-race sampler
struct SampleArgs {
  const float* logits;
  int64_t row_stride;
  const float* temperatures;
  int32_t batch, vocab;
  uint64_t seed, offset;
  int32_t* out;
  void* workspace;
};
size_t sample_workspace_bytes(int batch, int vocab);
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream);

// ---- the 4-bit cache (format in q4_device.cuh)
struct Q4Cache {
  uint8_t* k_data;    // [num_blocks, 256, Hkv, 64]
  uint8_t* k_scales;  // [num_blocks, 256, Hkv, 8]
  uint8_t* v_data;
  uint8_t* v_scales;
  float k_scale, v_scale;  // tensor scales
  float k_inv, v_inv;      // their reciprocals, rounded to fp32
  int32_t num_blocks, num_kv_heads;
};
cudaError_t launch_kv_write_q4(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                               const int32_t* slots, int32_t num_tokens, const Q4Cache& c, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_kv_read_q4(const int32_t* slots, int32_t num_tokens, const Q4Cache& c, uint16_t* k, uint16_t* v,
                              int num_sms, cudaStream_t stream);

// ---- attention over the 4-bit cache
struct AttnQ4Args {
  const uint16_t* q;
  uint16_t* out;
  const int32_t* context_lens;  // decode
  const int32_t* cu_seqlens_q;  // prefill
  const int32_t* cu_seqlens_k;  // prefill
  const int32_t* block_tables;
  int32_t max_blocks_per_seq;
  int32_t num_seqs, total_q, max_seqlen_q, max_seqlen_k;  // decode: batch rows, max_context_len
  int32_t num_q_heads;
  float scale;
  void* workspace;
  Q4Cache cache;
};
// Tensor maps over a layer's codes (num_blocks, 256, Hkv, 64 bytes) for boxes of
// `tokens` tokens of one block and `heads` kv heads, laid out in shared memory as
// [head][token][64 bytes] with the 64-byte swizzle (16-byte chunk c of token t at
// chunk c ^ ((t / 2) % 4)).
bool encode_q4_maps(const Q4Cache& c, int tokens, int heads, CUtensorMap* k, CUtensorMap* v);
size_t decode_q4_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int num_sms);
size_t prefill_q4_workspace_bytes(int total_q, int num_seqs, int max_seqlen_q, int max_seqlen_k, int num_q_heads,
                                  int num_kv_heads, int num_sms);
// Tensor map over q [total_q, Hq, 128] bf16 for boxes of 64 dims x 2^log2_heads
// heads x 128 / 2^log2_heads tokens with the 128-byte swizzle.
bool encode_q4_query_map(const uint16_t* q, int total_q, int num_q_heads, int log2_heads, CUtensorMap* m);
cudaError_t launch_paged_attn_decode_q4(const AttnQ4Args& a, int num_sms, cudaStream_t stream);
cudaError_t launch_paged_attn_prefill_q4(const AttnQ4Args& a, int num_sms, cudaStream_t stream);
// Prefill of at most 32 rows a kv head by the decode kernel (decode_q4.cu).
size_t rows_q4_workspace_bytes(int num_seqs, int max_seqlen_q, int num_q_heads, int num_sms);
cudaError_t launch_rows_q4(const AttnQ4Args& a, int num_sms, cudaStream_t stream);

// ---- norm + rotation of queries and keys
struct NormRopeArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  int32_t num_tokens, num_q_heads, num_kv_heads;
  const uint16_t* q_weight;  // null: rows are not normalised
  const uint16_t* k_weight;
  float eps;
  const int64_t* freqs;      // [rope_dim / 2] turns per position, Q0.64
  int32_t rope_dim, interleaved;
  const int32_t* positions;  // axis a of token t at a * position_axis_stride + t
  int64_t position_axis_stride;
  int32_t section_end0, section_end1;  // pairs below end0 follow axis 0, below end1 axis 1, else axis 2
  uint16_t* q_out;
  int64_t q_out_stride;
  uint16_t* k_out;  // dest 0
  int64_t k_out_stride;
  const int32_t* slots;  // dest 1, 2
  int32_t num_blocks;
  uint16_t* k_cache;  // dest 1
  uint16_t* v_cache;
  Q4Cache q4;  // dest 2
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, int dest, int num_sms, cudaStream_t stream);

// ---- blocks of a cache
struct ForkArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t num_seqs, max_blocks_per_seq;
  const int32_t* parents;
  int32_t num_forks;
  int32_t* ref_count;
  int32_t num_blocks;
  int32_t* child_tables;
  int32_t* child_lens;
  int32_t* copy_src;
  int32_t* copy_dst;
};
constexpr int kMaxForks = 8192;
cudaError_t launch_fork_blocks(const ForkArgs& a, cudaStream_t stream);
cudaError_t launch_free_blocks(const int32_t* block_tables, const int32_t* context_lens, int32_t num_seqs,
                               int32_t max_blocks_per_seq, int32_t* ref_count, int32_t num_blocks, int num_sms,
                               cudaStream_t stream);
struct CompactArgs {
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t num_seqs, max_blocks_per_seq;
  const int32_t* ref_count;
  int32_t num_blocks;
  int32_t* new_tables;
  int32_t* new_ref_count;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* num_moves;
};
cudaError_t launch_compact_blocks(const CompactArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_copy_blocks(void* cache, int32_t num_planes, int64_t plane_stride, int32_t num_blocks,
                               int64_t block_bytes, const int32_t* src, const int32_t* dst, int32_t num_copies,
                               cudaStream_t stream);

// Defines cudaError_t name(uint32_t* out, bool clear): read, and on request
// reset, the device error word `word` of a translation unit.
#define PKV_DEFINE_READ_ERROR(name, word)                                     \
  cudaError_t name(uint32_t* out, bool clear) {                               \
    unsigned int v = 0;                                                       \
    cudaError_t e = cudaMemcpyFromSymbol(&v, word, sizeof v);                 \
    if (e != cudaSuccess) return e;                                           \
    *out = v;                                                                 \
    if (clear) {                                                              \
      const unsigned int zero = 0;                                            \
      e = cudaMemcpyToSymbol(word, &zero, sizeof zero);                       \
    }                                                                         \
    return e;                                                                 \
  }

// ---- device error words (one per translation unit)
cudaError_t read_error_kv_q4(uint32_t* out, bool clear);
cudaError_t read_error_decode_q4(uint32_t* out, bool clear);
cudaError_t read_error_prefill_q4(uint32_t* out, bool clear);
cudaError_t read_error_norm_rope(uint32_t* out, bool clear);
cudaError_t read_error_blocks(uint32_t* out, bool clear);
cudaError_t read_error_kv_write(uint32_t* out, bool clear);
cudaError_t read_error_decode(uint32_t* out, bool clear);
cudaError_t read_error_prefill(uint32_t* out, bool clear);
cudaError_t read_error_prefill_persistent(uint32_t* out, bool clear);
cudaError_t read_error_metadata(uint32_t* out, bool clear);
cudaError_t read_error_sampler(uint32_t* out, bool clear);

}  // namespace pkv
