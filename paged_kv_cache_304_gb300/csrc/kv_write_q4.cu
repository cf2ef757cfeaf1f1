// kv_write_q4.cu -- scatter K/V rows into the 4-bit cache, and read rows back.
//
// Per token and kv head 256 bytes of bf16 become 64 bytes of codes and 8 of
// scales (the read does the reverse); both are bound by HBM.  A lane owns one
// group of 16 dims (32 bytes in, 8 + 1 bytes out), eight lanes a head's row, so
// a group's maximum needs no exchange between lanes and a warp moves four heads
// at a time.  The slot is read once per warp.
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "q4_device.cuh"

namespace pkv {
namespace {

__device__ unsigned int g_err_kv_q4;

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps)
    kv_write_q4_kernel(const uint16_t* __restrict__ k, int64_t k_stride, const uint16_t* __restrict__ v,
                       int64_t v_stride, const int32_t* __restrict__ slots, int32_t num_tokens, Q4Cache c) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t num_slots = static_cast<int64_t>(c.num_blocks) * kBlockSize;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < num_tokens; t += step) {
    const int64_t s = __ldg(slots + t);
    if (s == -1) continue;
    if (s < 0 || s >= num_slots) {
      if (lane == 0) atomicOr(&g_err_kv_q4, PKV_DEVERR_SLOT_RANGE);
      continue;
    }
    // units: group u of the K row, then of the V row (8 groups a head)
    const int per = c.num_kv_heads * q4::kRowScales;
    for (int u = lane; u < 2 * per; u += 32) {
      const bool is_v = u >= per;
      const int g = is_v ? u - per : u;
      const uint4* src = reinterpret_cast<const uint4*>((is_v ? v + t * v_stride : k + t * k_stride) + g * 16);
      const uint4 a = __ldg(src), b = __ldg(src + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const float inv = is_v ? c.v_inv : c.k_inv;
      float y[16], m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[2 * i] = q4::bf_lo(w[i]) * inv;
        y[2 * i + 1] = q4::bf_hi(w[i]) * inv;
        m = q4::max_nan(m, q4::max_nan(fabsf(y[2 * i]), fabsf(y[2 * i + 1])));
      }
      const uint32_t sb = q4::group_scale(m);
      const float sc = q4::dec_scale(sb);
      const int64_t at = s * per + g;
      *reinterpret_cast<uint2*>((is_v ? c.v_data : c.k_data) + at * 8) =
          make_uint2(q4::enc8(y, sc), q4::enc8(y + 8, sc));
      (is_v ? c.v_scales : c.k_scales)[at] = static_cast<uint8_t>(sb);
    }
  }
}

// Rows of slots[i] back as bf16; slot -1 (and, flagged, a slot outside the
// cache) gives zeros.  The product code * s * tensor_scale is rounded once.
__global__ void __launch_bounds__(32 * kWarps)
    kv_read_q4_kernel(const int32_t* __restrict__ slots, int32_t num_tokens, Q4Cache c, uint16_t* __restrict__ k,
                      uint16_t* __restrict__ v) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t num_slots = static_cast<int64_t>(c.num_blocks) * kBlockSize;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int per = c.num_kv_heads * q4::kRowScales;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); t < num_tokens; t += step) {
    const int64_t s = __ldg(slots + t);
    const bool ok = s >= 0 && s < num_slots;
    if (!ok && s != -1 && lane == 0) atomicOr(&g_err_kv_q4, PKV_DEVERR_SLOT_RANGE);
    for (int u = lane; u < 2 * per; u += 32) {
      const bool is_v = u >= per;
      const int g = is_v ? u - per : u;
      uint32_t o[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      if (ok) {
        const int64_t at = s * per + g;
        const uint2 d = *reinterpret_cast<const uint2*>((is_v ? c.v_data : c.k_data) + at * 8);
        const uint32_t sb = (is_v ? c.v_scales : c.k_scales)[at];
        const uint32_t sh = q4::dec_scale2(sb | sb << 8);
        const float ts = is_v ? c.v_scale : c.k_scale;
        uint32_t h[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          q4::dec8(half ? d.y : d.x, h);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t p = q4::hmul2(h[i], sh);
            o[4 * half + i] = pack_bf16x2(q4::half_lo(p) * ts, q4::half_hi(p) * ts);
          }
        }
      }
      uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (t * per + g) * 16);
      dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

unsigned token_grid(int num_tokens, int num_sms) {
  const int64_t blocks = (static_cast<int64_t>(num_tokens) + kWarps - 1) / kWarps;
  return static_cast<unsigned>(std::min<int64_t>(blocks, static_cast<int64_t>(num_sms) * 8));
}

}  // namespace

cudaError_t launch_kv_write_q4(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                               const int32_t* slots, int32_t num_tokens, const Q4Cache& c, int num_sms,
                               cudaStream_t stream) {
  return launch_pdl(kv_write_q4_kernel, dim3(token_grid(num_tokens, num_sms)), dim3(32 * kWarps), 0, stream, k,
                    k_stride, v, v_stride, slots, num_tokens, c);
}

cudaError_t launch_kv_read_q4(const int32_t* slots, int32_t num_tokens, const Q4Cache& c, uint16_t* k, uint16_t* v,
                              int num_sms, cudaStream_t stream) {
  return launch_pdl(kv_read_q4_kernel, dim3(token_grid(num_tokens, num_sms)), dim3(32 * kWarps), 0, stream, slots,
                    num_tokens, c, k, v);
}

PKV_DEFINE_READ_ERROR(read_error_kv_q4, g_err_kv_q4)

}  // namespace pkv
