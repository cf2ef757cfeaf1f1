// norm_rope.cu -- RMS norm of every query and key head and the rotation of its
// position in one pass, alone or together with the KV-cache write.
//
// Per head row x of 128 dims (fp32 throughout, one rounding to bf16):
//   y_d = x_d * rsqrt(mean(x^2) + eps) * w_d
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t) for the pairs of the first
//   rope_dim dims, (i, i + rope_dim/2) or, interleaved, (2i, 2i + 1);
//   t = position[axis(i)] * frequency_i.
// The angle is exact integer arithmetic: a frequency is a 64-bit fraction of a
// turn per position (Q0.64), so position * frequency mod 2^64 is the angle's
// fraction of a turn with no reduction error at any position, and its top 32
// bits give the argument of sincospi.  No table of cosines is read.
//
// Bound by HBM (every row read and written once).  Eight lanes own a head, 16
// dims each as two 8-dim chunks chosen so that both partners of a rotated pair
// sit in one lane; a warp takes four heads at a time and computes its lanes'
// eight sines and cosines once for all heads of the token it handles.  With few
// tokens a token's heads are spread over several warps.
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "q4_device.cuh"

namespace pkv {
namespace {

__device__ unsigned int g_err_norm_rope;

constexpr int kWarps = 4;

__device__ __forceinline__ void unpack(const uint4& a, float* x) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = q4::bf_lo(w[i]);
    x[2 * i + 1] = q4::bf_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// Quantise the lane's chunk (the other half of its group of 16 is in lane ^ 1)
// and store it; `a` is the bf16 chunk.
__device__ __forceinline__ void store_q4(uint8_t* data, uint8_t* scales, int64_t row, int chunk, const uint4& a,
                                         float inv, bool write) {
  float y[8], m = 0.f;
  unpack(a, y);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    y[i] *= inv;
    y[i + 1] *= inv;
    m = q4::max3_nan(m, fabsf(y[i]), fabsf(y[i + 1]));
  }
  m = q4::max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t sb = q4::group_scale(m);
  const uint32_t w = q4::enc8_group(y, sb, m);
  if (!write) return;
  *reinterpret_cast<uint32_t*>(data + row * q4::kRowBytes + chunk * 4) = w;
  if (!(chunk & 1)) scales[row * q4::kRowScales + (chunk >> 1)] = static_cast<uint8_t>(sb);
}

// kDest: 0 = k_out, 1 = bf16 cache (K and V), 2 = 4-bit cache (K and V).
template <int kDest>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormRopeArgs p, int splits) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int l = lane & 7, sub = lane >> 3;
  const int half_chunks = p.rope_dim >> 4;  // chunks in half of the rotated dims
  const bool inter = p.interleaved != 0;
  // The lane's chunks of 8 dims.  Rotated halves: chunk j and its partner
  // j + rope_dim/16 share a lane, the dims behind rope_dim fill the other
  // lanes.  Chunks 2j and 2j+1 (one group of 16) always sit in lanes 2i, 2i+1.
  int c0 = l, c1 = l + 8;
  if (!inter && half_chunks > 0) {
    if (l < half_chunks) {
      c1 = l + half_chunks;
    } else {
      c0 = l + half_chunks;
      c1 = c0 + 8 - half_chunks;
    }
  }
  const uint4 kOne = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint4* wqp = reinterpret_cast<const uint4*>(p.q_weight);
  const uint4* wkp = reinterpret_cast<const uint4*>(p.k_weight);
  const uint4 wq0 = wqp ? __ldg(wqp + c0) : kOne, wq1 = wqp ? __ldg(wqp + c1) : kOne;
  const uint4 wk0 = wkp ? __ldg(wkp + c0) : kOne, wk1 = wkp ? __ldg(wkp + c1) : kOne;

  const int rope_heads = p.num_q_heads + p.num_kv_heads;
  const int rope_groups = (rope_heads + 3) >> 2;
  const int groups = rope_groups + (kDest ? (p.num_kv_heads + 3) >> 2 : 0);
  const int per = (groups + splits - 1) / splits;
  const int64_t items = static_cast<int64_t>(p.num_tokens) * splits;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t t = it / splits;
    const int g0 = static_cast<int>(it - t * splits) * per;
    const int g1 = min(groups, g0 + per);
    if (g0 >= g1) continue;
    int64_t slot = -1;
    if (kDest) {
      slot = __ldg(p.slots + t);
      if (slot < -1 || slot >= static_cast<int64_t>(p.num_blocks) * kBlockSize) {
        if (lane == 0) atomicOr(&g_err_norm_rope, PKV_DEVERR_SLOT_RANGE);
        slot = -1;
      }
    }
    float cs[8], sn[8];
    if (g0 < rope_groups) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // pair of element e (halves) or of elements 2e, 2e+1 (interleaved)
        const int i = inter ? (e < 4 ? 4 * c0 + e : 4 * c1 + e - 4) : 8 * l + e;
        const bool rot = inter ? 2 * i < p.rope_dim : l < half_chunks;
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (rot) {
          const int axis = i < p.section_end0 ? 0 : (i < p.section_end1 ? 1 : 2);
          const int pos = __ldg(p.positions + axis * p.position_axis_stride + t);
          const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) *
                                static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(p.freqs) + i));
          const int turn = static_cast<int>(frac >> 32);  // angle / 2 pi in [-2^31, 2^31)
          sincospif(static_cast<float>(turn) * 4.656612873077393e-10f, &sn[e], &cs[e]);
        }
      }
    }
    // Group g's row of this lane, the next one's requested while this one is in work.
    auto load = [&](int g, uint4& a0, uint4& a1) {
      const bool is_v = g >= rope_groups;
      const int head = is_v ? 4 * (g - rope_groups) + sub : 4 * g + sub;
      a0 = a1 = make_uint4(0u, 0u, 0u, 0u);
      if (g < g1 && head < (is_v ? p.num_kv_heads : rope_heads)) {
        const uint16_t* row = is_v ? p.v + t * p.v_stride + head * kHeadDim
                                   : (head < p.num_q_heads ? p.q + t * p.q_stride + head * kHeadDim
                                                           : p.k + t * p.k_stride + (head - p.num_q_heads) * kHeadDim);
        // plain loads: the output may be the input
        a0 = reinterpret_cast<const uint4*>(row)[c0];
        a1 = reinterpret_cast<const uint4*>(row)[c1];
      }
    };
    uint4 n0, n1;
    load(g0, n0, n1);
    for (int g = g0; g < g1; ++g) {
      uint4 a0 = n0, a1 = n1;
      load(g + 1, n0, n1);
      const bool is_v = g >= rope_groups;
      const int head = is_v ? 4 * (g - rope_groups) + sub : 4 * g + sub;
      const bool is_q = !is_v && head < p.num_q_heads;
      const int kvh = is_v ? head : head - p.num_q_heads;  // kv head of a K or V row
      const bool real = is_v ? head < p.num_kv_heads : head < rope_heads;
      if (!is_v) {
        float x[16], w[16];
        unpack(a0, x);
        unpack(a1, x + 8);
        const bool norm = is_q ? wqp != nullptr : wkp != nullptr;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        ss += __shfl_xor_sync(0xffffffffu, ss, 4);
        const float r = norm ? rsqrtf(ss * (1.f / kHeadDim) + p.eps) : 1.f;
        unpack(is_q ? wq0 : wk0, w);
        unpack(is_q ? wq1 : wk1, w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
        if (inter) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = x[2 * e], z = x[2 * e + 1];
            x[2 * e] = u * cs[e] - z * sn[e];
            x[2 * e + 1] = z * cs[e] + u * sn[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = x[e], z = x[e + 8];
            x[e] = u * cs[e] - z * sn[e];
            x[e + 8] = z * cs[e] + u * sn[e];
          }
        }
        a0 = pack(x);
        a1 = pack(x + 8);
      }
      if (is_q) {
        if (real) {
          uint4* o = reinterpret_cast<uint4*>(p.q_out + t * p.q_out_stride + head * kHeadDim);
          o[c0] = a0;
          o[c1] = a1;
        }
      } else if (kDest == 0) {
        if (real) {
          uint4* o = reinterpret_cast<uint4*>(p.k_out + t * p.k_out_stride + kvh * kHeadDim);
          o[c0] = a0;
          o[c1] = a1;
        }
      } else if (kDest == 1) {
        if (real && slot >= 0) {
          uint4* o = reinterpret_cast<uint4*>((is_v ? p.v_cache : p.k_cache) + (slot * p.num_kv_heads + kvh) * kHeadDim);
          o[c0] = a0;
          o[c1] = a1;
        }
      }
      if (kDest == 2) {  // all lanes take part: a group of heads may hold both q and k
        const int64_t row = slot * p.num_kv_heads + kvh;
        const bool wr = real && !is_q && slot >= 0;
        if (__any_sync(0xffffffffu, wr)) {
          store_q4(is_v ? p.q4.v_data : p.q4.k_data, is_v ? p.q4.v_scales : p.q4.k_scales, row, c0, a0,
                   is_v ? p.q4.v_inv : p.q4.k_inv, wr);
          store_q4(is_v ? p.q4.v_data : p.q4.k_data, is_v ? p.q4.v_scales : p.q4.k_scales, row, c1, a1,
                   is_v ? p.q4.v_inv : p.q4.k_inv, wr);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int dest, int num_sms, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int groups = (a.num_q_heads + a.num_kv_heads + 3) / 4 + (dest ? (a.num_kv_heads + 3) / 4 : 0);
  // Few tokens: spread a token's heads over warps until the GPU has ~8 warps an SM.
  int splits = 1;
  while (splits < groups && static_cast<int64_t>(a.num_tokens) * splits < static_cast<int64_t>(num_sms) * 8) ++splits;
  const int64_t items = static_cast<int64_t>(a.num_tokens) * splits;
  const int64_t blocks = std::min<int64_t>((items + kWarps - 1) / kWarps, static_cast<int64_t>(num_sms) * 32);
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * kWarps);
  switch (dest) {
    case 0: return launch_pdl(norm_rope_kernel<0>, grid, block, 0, stream, a, splits);
    case 1: return launch_pdl(norm_rope_kernel<1>, grid, block, 0, stream, a, splits);
    default: return launch_pdl(norm_rope_kernel<2>, grid, block, 0, stream, a, splits);
  }
}

PKV_DEFINE_READ_ERROR(read_error_norm_rope, g_err_norm_rope)

}  // namespace pkv
