// prefill_q4.cu -- packed prompts against the 4-bit cache (plain form: a warp per
// query row and head walks the visible keys one at a time).
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "q4_device.cuh"

namespace pkv {
namespace {

__device__ unsigned int g_err_prefill_q4;

struct Acc {
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
};

}  // namespace

// Lane i holds dims 4i .. 4i+3 of the query; keys 0 .. len-1 of the sequence.
__device__ void attend_row_q4(const Q4Cache& c, const uint16_t* q, uint16_t* out, const int32_t* table, int len,
                              int kvh, float sl2, unsigned int* err) {
  const int lane = threadIdx.x & 31;
  const uint2 w = *reinterpret_cast<const uint2*>(q + 4 * lane);
  const float x[4] = {q4::bf_lo(w.x), q4::bf_hi(w.x), q4::bf_lo(w.y), q4::bf_hi(w.y)};
  Acc a;
  for (int t = 0; t < len; ++t) {
    int b = __ldg(table + t / kBlockSize);
    if (b < 0 || b >= c.num_blocks) {
      if (lane == 0) atomicOr(err, PKV_DEVERR_BLOCK_RANGE);
      b = 0;
    }
    const int64_t row = (static_cast<int64_t>(b) * kBlockSize + t % kBlockSize) * c.num_kv_heads + kvh;
    uint32_t h[4];
    q4::dec8(*reinterpret_cast<const uint16_t*>(c.k_data + row * 64 + 2 * lane), h);
    const float ks = q4::dec_scale(c.k_scales[row * 8 + (lane >> 2)]);
    float s = ks * (x[0] * q4::half_lo(h[0]) + x[1] * q4::half_hi(h[0]) + x[2] * q4::half_lo(h[1]) +
                    x[3] * q4::half_hi(h[1]));
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= sl2;
    const float m = fmaxf(a.m, s);
    const float alpha = fast_exp2(a.m - m), p = fast_exp2(s - m);
    a.m = m;
    a.l = a.l * alpha + p;
    q4::dec8(*reinterpret_cast<const uint16_t*>(c.v_data + row * 64 + 2 * lane), h);
    const float vs = p * q4::dec_scale(c.v_scales[row * 8 + (lane >> 2)]);
    a.o[0] = a.o[0] * alpha + vs * q4::half_lo(h[0]);
    a.o[1] = a.o[1] * alpha + vs * q4::half_hi(h[0]);
    a.o[2] = a.o[2] * alpha + vs * q4::half_lo(h[1]);
    a.o[3] = a.o[3] * alpha + vs * q4::half_hi(h[1]);
  }
  const float inv = len > 0 ? c.v_scale / a.l : 0.f;
  *reinterpret_cast<uint2*>(out + 4 * lane) =
      make_uint2(pack_bf16x2(a.o[0] * inv, a.o[1] * inv), pack_bf16x2(a.o[2] * inv, a.o[3] * inv));
}

__global__ void __launch_bounds__(128) prefill_q4_kernel(const AttnQ4Args p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int row = static_cast<int>(pair / p.num_q_heads), h = static_cast<int>(pair % p.num_q_heads);
  const int i = blockIdx.y;
  const int q0 = p.cu_seqlens_q[i], q1 = p.cu_seqlens_q[i + 1];
  const int n = q1 - q0, len = p.cu_seqlens_k[i + 1] - p.cu_seqlens_k[i];
  if (n <= 0) return;
  if (len < n || len > static_cast<long long>(p.max_blocks_per_seq) * kBlockSize || q1 > p.total_q || q0 < 0 ||
      n > p.max_seqlen_q || len > p.max_seqlen_k) {
    if (pair == 0 && threadIdx.x == 0) atomicOr(&g_err_prefill_q4, PKV_DEVERR_LEN_RANGE);
    return;
  }
  if (row >= n) return;
  const int64_t at = (static_cast<int64_t>(q0 + row) * p.num_q_heads + h) * kHeadDim;
  attend_row_q4(p.cache, p.q + at, p.out + at, p.block_tables + static_cast<int64_t>(i) * p.max_blocks_per_seq,
                len - n + row + 1, h / (p.num_q_heads / p.cache.num_kv_heads),
                p.scale * p.cache.k_scale * 1.4426950408889634f, &g_err_prefill_q4);
}

size_t prefill_q4_workspace_bytes(int, int, int, int, int, int, int) { return 256; }

cudaError_t launch_paged_attn_prefill_q4(const AttnQ4Args& a, int, cudaStream_t stream) {
  const int64_t pairs = static_cast<int64_t>(a.max_seqlen_q) * a.num_q_heads;
  return launch_pdl(prefill_q4_kernel, dim3(static_cast<unsigned>((pairs + 3) / 4), a.num_seqs), dim3(128), 0, stream, a);
}

PKV_DEFINE_READ_ERROR(read_error_prefill_q4, g_err_prefill_q4)

}  // namespace pkv
