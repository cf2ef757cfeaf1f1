// pkv_api_q4.cu -- C ABI of the 4-bit cache, of norm + rotation and of the
// block operations: host-side argument validation and launches.  Nothing here
// allocates device memory or synchronises the host.
#include <cuda_runtime.h>

#include <cmath>

#include "pkv.h"
#include "pkv_internal.h"

namespace pkv {
namespace {

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pkv_status status_of(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

pkv_status check_cache_shape(int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim) {
  if (num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0) return PKV_ERR_SHAPE;
  if (block_size != kBlockSize || head_dim != kHeadDim || num_kv_heads > kMaxKvHeads) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * kBlockSize >= (int64_t{1} << 31)) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

// Sizes and tensor scales first (no pointer of the cache needs to be valid for them).
pkv_status check_q4_shape(const pkv_q4_cache* c) {
  if (!c) return PKV_ERR_NULL;
  const pkv_status st = check_cache_shape(c->num_blocks, c->block_size, c->num_kv_heads, c->head_dim);
  if (st != PKV_OK) return st;
  for (float s : {c->k_scale, c->v_scale})
    if (!(s > 0.f) || !std::isfinite(s) || !std::isfinite(1.f / s)) return PKV_ERR_SHAPE;
  return PKV_OK;
}

pkv_status check_q4_pointers(const pkv_q4_cache* c, Q4Cache* out) {
  for (const void* p : {c->k_data, c->k_scales, c->v_data, c->v_scales})
    if (!p) return PKV_ERR_NULL;
  for (const void* p : {c->k_data, c->k_scales, c->v_data, c->v_scales})
    if (!aligned16(p)) return PKV_ERR_ALIGN;
  out->k_data = c->k_data;
  out->k_scales = c->k_scales;
  out->v_data = c->v_data;
  out->v_scales = c->v_scales;
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  out->k_inv = 1.f / c->k_scale;
  out->v_inv = 1.f / c->v_scale;
  out->num_blocks = c->num_blocks;
  out->num_kv_heads = c->num_kv_heads;
  return PKV_OK;
}

pkv_status check_rows(const void* p, int64_t stride, int64_t row) {
  if (stride < row) return PKV_ERR_SHAPE;
  if (stride % 8 || !aligned16(p)) return PKV_ERR_ALIGN;
  return PKV_OK;
}

pkv_status check_attn_q4(const pkv_q4_cache* c, int32_t num_q_heads, int32_t max_blocks_per_seq, float scale) {
  const pkv_status st = check_q4_shape(c);
  if (st != PKV_OK) return st;
  if (num_q_heads <= 0 || max_blocks_per_seq <= 0 || num_q_heads % c->num_kv_heads) return PKV_ERR_SHAPE;
  if (!(scale > 0.f) || !std::isfinite(scale) || !std::isfinite(scale * c->k_scale)) return PKV_ERR_SHAPE;
  if (num_q_heads > kMaxQHeads || num_q_heads / c->num_kv_heads > kMaxGroup) return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

// Shared by the three norm + rotation calls: everything but the destination.
pkv_status norm_rope_common(const pkv_bf16* q, int64_t q_stride, const pkv_bf16* k, int64_t k_stride,
                            int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            const pkv_norm_rope* nr, pkv_bf16* q_out, int64_t q_out_stride, NormRopeArgs* a) {
  if (!nr) return PKV_ERR_NULL;
  if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads < 0 || head_dim <= 0 || !(nr->eps >= 0.f) ||
      !std::isfinite(nr->eps))
    return PKV_ERR_SHAPE;
  if (head_dim != kHeadDim || num_q_heads > kMaxQHeads || num_kv_heads > kMaxKvHeads) return PKV_ERR_UNSUPPORTED;
  if (nr->rope_dim < 0 || nr->rope_dim > head_dim || nr->rope_dim % 2) return PKV_ERR_SHAPE;
  if (nr->rope_dim % 32) return PKV_ERR_UNSUPPORTED;
  int end0 = 0, end1 = 0;
  if (nr->rope_dim > 0) {
    if (nr->num_axes < 1) return PKV_ERR_SHAPE;
    if (nr->num_axes > 3) return PKV_ERR_UNSUPPORTED;
    int total = 0;
    for (int i = 0; i < nr->num_axes; ++i) {
      if (nr->sections[i] < 0 || nr->sections[i] > nr->rope_dim) return PKV_ERR_SHAPE;
      total += nr->sections[i];
    }
    if (total != nr->rope_dim / 2) return PKV_ERR_SHAPE;
    if (nr->position_axis_stride < 0) return PKV_ERR_SHAPE;
    // axes that a call does not have follow nothing
    end0 = nr->sections[0];
    end1 = nr->num_axes > 1 ? end0 + nr->sections[1] : total;
    if (nr->num_axes == 1) end0 = total;
  }
  if (num_tokens == 0) return PKV_OK;
  if (!q || !q_out || (num_kv_heads && !k) || (nr->rope_dim && (!nr->freqs || !nr->positions))) return PKV_ERR_NULL;
  if (nr->rope_dim && (reinterpret_cast<uintptr_t>(nr->freqs) & 7u)) return PKV_ERR_ALIGN;
  if (!aligned16(nr->q_weight) || !aligned16(nr->k_weight)) return PKV_ERR_ALIGN;
  const int64_t q_row = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t k_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  pkv_status st = check_rows(q, q_stride, q_row);
  if (st == PKV_OK) st = check_rows(q_out, q_out_stride, q_row);
  if (st == PKV_OK && num_kv_heads) st = check_rows(k, k_stride, k_row);
  if (st != PKV_OK) return st;
  a->q = q;
  a->q_stride = q_stride;
  a->k = k;
  a->k_stride = k_stride;
  a->num_tokens = num_tokens;
  a->num_q_heads = num_q_heads;
  a->num_kv_heads = num_kv_heads;
  a->q_weight = nr->q_weight;
  a->k_weight = nr->k_weight;
  a->eps = nr->eps;
  a->freqs = nr->freqs;
  a->rope_dim = nr->rope_dim;
  a->interleaved = nr->interleaved;
  a->positions = nr->positions;
  a->position_axis_stride = nr->position_axis_stride;
  a->section_end0 = end0;
  a->section_end1 = end1;
  a->q_out = q_out;
  a->q_out_stride = q_out_stride;
  return PKV_OK;
}

pkv_status launch_norm(const NormRopeArgs& a, int dest, void* stream) {
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  return status_of(launch_norm_rope(a, dest, sms, static_cast<cudaStream_t>(stream)));
}

bool bad_pool(int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_blocks) {
  return num_seqs < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0;
}

bool pool_too_large(int32_t max_blocks_per_seq, int32_t num_blocks) {
  return static_cast<int64_t>(num_blocks) * kBlockSize >= (int64_t{1} << 31) ||
         static_cast<int64_t>(max_blocks_per_seq) * kBlockSize >= (int64_t{1} << 31);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_kv_cache_write_q4(const pkv_bf16* k, int64_t k_token_stride, const pkv_bf16* v,
                                 int64_t v_token_stride, const int32_t* slot_mapping, int32_t num_tokens,
                                 const pkv_q4_cache* cache, void* stream) {
  pkv_status st = check_q4_shape(cache);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  const int64_t row = static_cast<int64_t>(cache->num_kv_heads) * kHeadDim;
  if (k_token_stride < row || v_token_stride < row) return PKV_ERR_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping) return PKV_ERR_NULL;
  if (check_rows(k, k_token_stride, row) != PKV_OK || check_rows(v, v_token_stride, row) != PKV_OK)
    return PKV_ERR_ALIGN;
  Q4Cache c;
  st = check_q4_pointers(cache, &c);
  if (st != PKV_OK) return st;
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  return status_of(launch_kv_write_q4(k, k_token_stride, v, v_token_stride, slot_mapping, num_tokens, c, sms,
                                      static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_kv_cache_read_q4(const pkv_q4_cache* cache, const int32_t* slots, int32_t num_tokens, pkv_bf16* k_out,
                                pkv_bf16* v_out, void* stream) {
  pkv_status st = check_q4_shape(cache);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!slots || !k_out || !v_out) return PKV_ERR_NULL;
  if (!aligned16(k_out) || !aligned16(v_out)) return PKV_ERR_ALIGN;
  Q4Cache c;
  st = check_q4_pointers(cache, &c);
  if (st != PKV_OK) return st;
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  return status_of(launch_kv_read_q4(slots, num_tokens, c, k_out, v_out, sms, static_cast<cudaStream_t>(stream)));
}

size_t pkv_decode_q4_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads) {
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0) return 0;
  const int sms = sm_count();
  return sms > 0 ? decode_q4_workspace_bytes(batch, num_q_heads, num_kv_heads, sms) : 0;
}

pkv_status pkv_paged_attn_decode_q4(const pkv_bf16* q, const pkv_q4_cache* cache, const int32_t* context_lens,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t batch,
                                    int32_t num_q_heads, int32_t max_context_len, float scale, pkv_bf16* out,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  pkv_status st = check_attn_q4(cache, num_q_heads, max_blocks_per_seq, scale);
  if (st != PKV_OK) return st;
  if (batch < 0 || max_context_len < 0) return PKV_ERR_SHAPE;
  if (max_context_len >= (1 << 26)) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(batch) * num_q_heads >= (int64_t{1} << 31)) return PKV_ERR_UNSUPPORTED;
  if (batch == 0) return PKV_OK;
  if (!q || !context_lens || !block_tables || !out) return PKV_ERR_NULL;
  if (!aligned16(q) || !aligned16(out)) return PKV_ERR_ALIGN;
  AttnQ4Args a = {};
  st = check_q4_pointers(cache, &a.cache);
  if (st != PKV_OK) return st;
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  if (!workspace || workspace_bytes < decode_q4_workspace_bytes(batch, num_q_heads, cache->num_kv_heads, sms))
    return PKV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_ERR_ALIGN;
  a.q = q;
  a.out = out;
  a.context_lens = context_lens;
  a.block_tables = block_tables;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_seqs = batch;
  a.total_q = batch;
  a.max_seqlen_q = 1;
  a.max_seqlen_k = max_context_len;
  a.num_q_heads = num_q_heads;
  a.scale = scale;
  a.workspace = workspace;
  return status_of(launch_paged_attn_decode_q4(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t pkv_prefill_q4_workspace_bytes(int32_t total_q, int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                      int32_t num_q_heads, int32_t num_kv_heads) {
  if (total_q < 0 || num_seqs < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || num_q_heads <= 0 || num_kv_heads <= 0)
    return 0;
  const int sms = sm_count();
  if (sms <= 0) return 0;
  return prefill_q4_workspace_bytes(total_q, num_seqs, max_seqlen_q, max_seqlen_k, num_q_heads, num_kv_heads, sms);
}

pkv_status pkv_paged_attn_prefill_q4(const pkv_bf16* q, const pkv_q4_cache* cache, const int32_t* cu_seqlens_q,
                                     const int32_t* cu_seqlens_k, const int32_t* block_tables,
                                     int32_t max_blocks_per_seq, int32_t num_seqs, int32_t total_q,
                                     int32_t max_seqlen_q, int32_t max_seqlen_k, int32_t num_q_heads, float scale,
                                     pkv_bf16* out, void* workspace, size_t workspace_bytes, void* stream) {
  pkv_status st = check_attn_q4(cache, num_q_heads, max_blocks_per_seq, scale);
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || max_seqlen_q > max_seqlen_k)
    return PKV_ERR_SHAPE;
  if (num_seqs > 65535 || max_seqlen_q > (1 << 22) || max_seqlen_k >= (1 << 26)) return PKV_ERR_UNSUPPORTED;
  if (total_q == 0 || num_seqs == 0 || max_seqlen_q == 0) return PKV_OK;
  if (!q || !cu_seqlens_q || !cu_seqlens_k || !block_tables || !out) return PKV_ERR_NULL;
  if (!aligned16(q) || !aligned16(out)) return PKV_ERR_ALIGN;
  AttnQ4Args a = {};
  st = check_q4_pointers(cache, &a.cache);
  if (st != PKV_OK) return st;
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  const size_t need = prefill_q4_workspace_bytes(total_q, num_seqs, max_seqlen_q, max_seqlen_k, num_q_heads,
                                                 cache->num_kv_heads, sms);
  if (!workspace || workspace_bytes < need) return PKV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_ERR_ALIGN;
  a.q = q;
  a.out = out;
  a.cu_seqlens_q = cu_seqlens_q;
  a.cu_seqlens_k = cu_seqlens_k;
  a.block_tables = block_tables;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.max_seqlen_q = max_seqlen_q;
  a.max_seqlen_k = max_seqlen_k;
  a.num_q_heads = num_q_heads;
  a.scale = scale;
  a.workspace = workspace;
  return status_of(launch_paged_attn_prefill_q4(a, sms, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_qk_norm_rope(const pkv_bf16* q, int64_t q_token_stride, const pkv_bf16* k, int64_t k_token_stride,
                            int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            const pkv_norm_rope* nr, pkv_bf16* q_out, int64_t q_out_stride, pkv_bf16* k_out,
                            int64_t k_out_stride, void* stream) {
  NormRopeArgs a = {};
  pkv_status st = norm_rope_common(q, q_token_stride, k, k_token_stride, num_tokens, num_q_heads, num_kv_heads,
                                   head_dim, nr, q_out, q_out_stride, &a);
  if (st != PKV_OK || num_tokens == 0) return st;
  if (num_kv_heads) {
    if (!k_out) return PKV_ERR_NULL;
    st = check_rows(k_out, k_out_stride, static_cast<int64_t>(num_kv_heads) * head_dim);
    if (st != PKV_OK) return st;
  }
  a.k_out = k_out;
  a.k_out_stride = k_out_stride;
  return launch_norm(a, 0, stream);
}

pkv_status pkv_qk_norm_rope_write(const pkv_bf16* q, int64_t q_token_stride, const pkv_bf16* k,
                                  int64_t k_token_stride, const pkv_bf16* v, int64_t v_token_stride,
                                  int32_t num_tokens, int32_t num_q_heads, const pkv_norm_rope* nr,
                                  const int32_t* slot_mapping, pkv_bf16* k_cache, pkv_bf16* v_cache,
                                  int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                                  pkv_bf16* q_out, int64_t q_out_stride, void* stream) {
  pkv_status st = check_cache_shape(num_blocks, block_size, num_kv_heads, head_dim);
  if (st != PKV_OK) return st;
  NormRopeArgs a = {};
  st = norm_rope_common(q, q_token_stride, k, k_token_stride, num_tokens, num_q_heads, num_kv_heads, head_dim, nr,
                        q_out, q_out_stride, &a);
  if (st != PKV_OK || num_tokens == 0) return st;
  if (!v || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_NULL;
  st = check_rows(v, v_token_stride, static_cast<int64_t>(num_kv_heads) * head_dim);
  if (st != PKV_OK) return st;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
  a.v = v;
  a.v_stride = v_token_stride;
  a.slots = slot_mapping;
  a.num_blocks = num_blocks;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  return launch_norm(a, 1, stream);
}

pkv_status pkv_qk_norm_rope_write_q4(const pkv_bf16* q, int64_t q_token_stride, const pkv_bf16* k,
                                     int64_t k_token_stride, const pkv_bf16* v, int64_t v_token_stride,
                                     int32_t num_tokens, int32_t num_q_heads, const pkv_norm_rope* nr,
                                     const int32_t* slot_mapping, const pkv_q4_cache* cache, pkv_bf16* q_out,
                                     int64_t q_out_stride, void* stream) {
  pkv_status st = check_q4_shape(cache);
  if (st != PKV_OK) return st;
  NormRopeArgs a = {};
  st = norm_rope_common(q, q_token_stride, k, k_token_stride, num_tokens, num_q_heads, cache->num_kv_heads, kHeadDim,
                        nr, q_out, q_out_stride, &a);
  if (st != PKV_OK || num_tokens == 0) return st;
  if (!v || !slot_mapping) return PKV_ERR_NULL;
  st = check_rows(v, v_token_stride, static_cast<int64_t>(cache->num_kv_heads) * kHeadDim);
  if (st != PKV_OK) return st;
  st = check_q4_pointers(cache, &a.q4);
  if (st != PKV_OK) return st;
  a.v = v;
  a.v_stride = v_token_stride;
  a.slots = slot_mapping;
  a.num_blocks = cache->num_blocks;
  return launch_norm(a, 2, stream);
}

pkv_status pkv_fork_blocks(const int32_t* block_tables, const int32_t* context_lens, int32_t num_seqs,
                           int32_t max_blocks_per_seq, const int32_t* parents, int32_t num_forks, int32_t* ref_count,
                           int32_t num_blocks, int32_t* child_tables, int32_t* child_lens, int32_t* copy_src,
                           int32_t* copy_dst, void* stream) {
  if (bad_pool(num_seqs, max_blocks_per_seq, num_blocks) || num_forks < 0) return PKV_ERR_SHAPE;
  if (pool_too_large(max_blocks_per_seq, num_blocks) || num_forks > kMaxForks) return PKV_ERR_UNSUPPORTED;
  if (num_forks == 0) return PKV_OK;
  if ((num_seqs && (!block_tables || !context_lens)) || !parents || !ref_count || !child_tables || !child_lens ||
      !copy_src || !copy_dst)
    return PKV_ERR_NULL;
  const ForkArgs a = {block_tables, context_lens, num_seqs,   max_blocks_per_seq, parents,  num_forks,
                      ref_count,    num_blocks,   child_tables, child_lens,       copy_src, copy_dst};
  return status_of(launch_fork_blocks(a, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_free_blocks(const int32_t* block_tables, const int32_t* context_lens, int32_t num_seqs,
                           int32_t max_blocks_per_seq, int32_t* ref_count, int32_t num_blocks, void* stream) {
  if (bad_pool(num_seqs, max_blocks_per_seq, num_blocks)) return PKV_ERR_SHAPE;
  if (pool_too_large(max_blocks_per_seq, num_blocks)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!block_tables || !context_lens || !ref_count) return PKV_ERR_NULL;
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  return status_of(launch_free_blocks(block_tables, context_lens, num_seqs, max_blocks_per_seq, ref_count, num_blocks,
                                      sms, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_compact_blocks(const int32_t* block_tables, const int32_t* context_lens, int32_t num_seqs,
                              int32_t max_blocks_per_seq, const int32_t* ref_count, int32_t num_blocks,
                              int32_t* new_tables, int32_t* new_ref_count, int32_t* copy_src, int32_t* copy_dst,
                              int32_t* num_moves, void* stream) {
  if (bad_pool(num_seqs, max_blocks_per_seq, num_blocks)) return PKV_ERR_SHAPE;
  if (pool_too_large(max_blocks_per_seq, num_blocks)) return PKV_ERR_UNSUPPORTED;
  if ((num_seqs && (!block_tables || !context_lens || !new_tables)) || !ref_count || !new_ref_count || !num_moves ||
      (num_blocks > 1 && (!copy_src || !copy_dst)))
    return PKV_ERR_NULL;
  const int sms = sm_count();
  if (sms <= 0) return PKV_ERR_CUDA;
  const CompactArgs a = {block_tables, context_lens,  num_seqs, max_blocks_per_seq, ref_count, num_blocks,
                         new_tables,   new_ref_count, copy_src, copy_dst,           num_moves};
  return status_of(launch_compact_blocks(a, sms, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_copy_blocks(void* cache, int32_t num_planes, int64_t plane_stride_bytes, int32_t num_blocks,
                           int64_t block_bytes, const int32_t* src, const int32_t* dst, int32_t num_copies,
                           void* stream) {
  if (num_planes < 0 || num_blocks <= 0 || block_bytes <= 0 || num_copies < 0) return PKV_ERR_SHAPE;
  if (block_bytes > INT64_MAX / num_blocks) return PKV_ERR_SHAPE;
  if (num_planes > 1 && plane_stride_bytes < block_bytes * num_blocks) return PKV_ERR_SHAPE;
  if (block_bytes % 16 || plane_stride_bytes % 16) return PKV_ERR_ALIGN;
  if (num_planes == 0 || num_copies == 0) return PKV_OK;
  if (!cache || !src || !dst) return PKV_ERR_NULL;
  if (!aligned16(cache)) return PKV_ERR_ALIGN;
  return status_of(launch_copy_blocks(cache, num_planes, plane_stride_bytes, num_blocks, block_bytes, src, dst,
                                      num_copies, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
