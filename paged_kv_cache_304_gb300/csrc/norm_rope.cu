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
// fraction of a turn with no reduction error at any position; its top 32 bits,
// in [-pi, pi], go to the SFU's sine and cosine (within 2^-21 there, a few
// thousandths of the output's rounding).  No table of cosines is read.
//
// Bound by HBM (every row read and written once).  Eight lanes own a head, 16
// dims each as two 8-dim chunks chosen so that both partners of a rotated pair
// sit in one lane; a warp takes four heads at a time, the next four requested
// while it works, and computes its lanes' eight sines and cosines once for all
// heads of the token it handles.  With few tokens a token's heads are spread
// over several warps.  fp32 arithmetic is done on pairs (one instruction for
// two), which is what keeps the issue slots below the memory time.
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "q4_device.cuh"

namespace pkv {
namespace {

__device__ unsigned int g_err_norm_rope;

constexpr int kWarps = 4;

// Eight bf16 of a chunk as four pairs of floats, and back.
__device__ __forceinline__ void unpack(const uint4& a, float2* x) {
  x[0] = make_float2(q4::bf_lo(a.x), q4::bf_hi(a.x));
  x[1] = make_float2(q4::bf_lo(a.y), q4::bf_hi(a.y));
  x[2] = make_float2(q4::bf_lo(a.z), q4::bf_hi(a.z));
  x[3] = make_float2(q4::bf_lo(a.w), q4::bf_hi(a.w));
}

__device__ __forceinline__ uint4 pack(const float2* x) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Quantise the lane's chunk (the other half of its group of 16 is in lane ^ 1)
// and store it; `a` is the bf16 chunk.
__device__ __forceinline__ void store_q4(uint8_t* data, uint8_t* scales, int64_t row, int chunk, const uint4& a,
                                         float inv, bool write) {
  float2 y2[4];
  float y[8], m = 0.f;
  unpack(a, y2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y2[i] = fmul2(y2[i], both(inv));
    y[2 * i] = y2[i].x;
    y[2 * i + 1] = y2[i].y;
    m = q4::max3_nan(m, fabsf(y2[i].x), fabsf(y2[i].y));
  }
  m = q4::max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t sb = q4::group_scale(m);
  const uint32_t w = q4::enc8_group(y, sb, m);
  if (!write) return;
  *reinterpret_cast<uint32_t*>(data + row * q4::kRowBytes + chunk * 4) = w;
  if (!(chunk & 1)) scales[row * q4::kRowScales + (chunk >> 1)] = static_cast<uint8_t>(sb);
}

// kDest: 0 = k_out, 1 = bf16 cache (K and V), 2 = 4-bit cache (K and V).
// kInter: rotated pairs are (2i, 2i + 1).
template <int kDest, bool kInter>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormRopeArgs p, int splits) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int l = lane & 7, sub = lane >> 3;
  const int half_chunks = p.rope_dim >> 4;  // chunks in half of the rotated dims
  // The lane's chunks of 8 dims.  Rotated halves: chunk j and its partner
  // j + rope_dim/16 share a lane, the dims behind rope_dim fill the other
  // lanes.  Chunks 2j and 2j+1 (one group of 16) always sit in lanes 2i, 2i+1.
  int c0 = l, c1 = l + 8;
  if (!kInter && half_chunks > 0) {
    if (l < half_chunks) {
      c1 = l + half_chunks;
    } else {
      c0 = l + half_chunks;
      c1 = c0 + 8 - half_chunks;
    }
  }
  // Groups of four heads: queries, then keys, then (with a cache) values.
  const int q_groups = (p.num_q_heads + 3) >> 2, kv_groups = (p.num_kv_heads + 3) >> 2;
  const int rope_groups = q_groups + kv_groups;
  const int groups = rope_groups + (kDest ? kv_groups : 0);
  const int per = (groups + splits - 1) / splits;
  const int64_t items = static_cast<int64_t>(p.num_tokens) * splits;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t t = it / splits;
    const int g0 = static_cast<int>(it - t * splits) * per;
    const int g1 = min(groups, g0 + per);
    if (g0 >= g1) continue;
    // Group g's row of this lane (plain loads: the output may be the input).
    const uint16_t* q_row = p.q + t * p.q_stride;
    const uint16_t* k_row = p.k + t * p.k_stride;
    const uint16_t* v_row = p.v + t * p.v_stride;
    auto load = [&](int g, uint4& a0, uint4& a1) {
      const int head = 4 * (g < q_groups ? g : g < rope_groups ? g - q_groups : g - rope_groups) + sub;
      const uint16_t* row = g < q_groups ? q_row : g < rope_groups ? k_row : v_row;
      a0 = a1 = make_uint4(0u, 0u, 0u, 0u);
      if (g < g1 && head < (g < q_groups ? p.num_q_heads : p.num_kv_heads)) {
        const uint4* src = reinterpret_cast<const uint4*>(row + head * kHeadDim);
        a0 = src[c0];
        a1 = src[c1];
      }
    };
    uint4 n0, n1;
    load(g0, n0, n1);
    int64_t slot = -1;
    if (kDest) {
      slot = __ldg(p.slots + t);
      if (slot < -1 || slot >= static_cast<int64_t>(p.num_blocks) * kBlockSize) {
        if (lane == 0) atomicOr(&g_err_norm_rope, PKV_DEVERR_SLOT_RANGE);
        slot = -1;
      }
    }
    // Cosines and sines of the lane's pairs: elements (2e, 2e + 1) of chunk c0
    // with those of c1 (halves), or pair e of the lane's chunks (interleaved).
    float cs[8], sn[8];
    if (g0 < rope_groups) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = kInter ? (e < 4 ? 4 * c0 + e : 4 * c1 + e - 4) : 8 * l + e;
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (kInter ? 2 * i < p.rope_dim : l < half_chunks) {
          const int axis = i < p.section_end0 ? 0 : (i < p.section_end1 ? 1 : 2);
          const int pos = __ldg(p.positions + axis * p.position_axis_stride + t);
          const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) *
                                static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(p.freqs) + i));
          // angle in [-pi, pi): the top 32 bits times 2 pi / 2^32
          const float angle = static_cast<float>(static_cast<int>(frac >> 32)) * 1.4629180792671596e-9f;
          cs[e] = __cosf(angle);
          sn[e] = __sinf(angle);
        }
      }
    }
    float2 w[8];       // weights of the lane's 16 dims, of the phase's kind of row
    bool norm = false;
    for (int g = g0; g < g1; ++g) {
      uint4 a0 = n0, a1 = n1;
      load(g + 1, n0, n1);
      const bool is_q = g < q_groups, is_v = g >= rope_groups;
      const int head = 4 * (is_q ? g : is_v ? g - rope_groups : g - q_groups) + sub;
      const bool real = head < (is_q ? p.num_q_heads : p.num_kv_heads);
      if (!is_v) {
        if (g == g0 || g == q_groups) {
          const uint4* src = reinterpret_cast<const uint4*>(is_q ? p.q_weight : p.k_weight);
          norm = src != nullptr;
          if (norm) {
            unpack(__ldg(src + c0), w);
            unpack(__ldg(src + c1), w + 4);
          }
        }
        float2 x[8];
        unpack(a0, x);
        unpack(a1, x + 4);
        if (norm) {
          float2 ss = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = ffma2(x[i], x[i], ss);
          float sum = ss.x + ss.y;
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          const float r = rsqrtf(sum * (1.f / kHeadDim) + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fmul2(fmul2(x[i], both(r)), w[i]);
        }
        if (kInter) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[e] = ffma2(make_float2(x[e].y, x[e].x), make_float2(-sn[e], sn[e]), fmul2(x[e], both(cs[e])));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]), s = make_float2(sn[2 * e], sn[2 * e + 1]);
            const float2 u = x[e], z = x[e + 4];
            x[e] = ffma2(z, make_float2(-s.x, -s.y), fmul2(u, c));
            x[e + 4] = ffma2(u, s, fmul2(z, c));
          }
        }
        a0 = pack(x);
        a1 = pack(x + 4);
      }
      if (is_q || kDest == 0) {
        if (real) {
          uint4* o = reinterpret_cast<uint4*>((is_q ? p.q_out + t * p.q_out_stride : p.k_out + t * p.k_out_stride) +
                                              head * kHeadDim);
          o[c0] = a0;
          o[c1] = a1;
        }
      } else if (kDest == 1) {
        if (real && slot >= 0) {
          uint4* o = reinterpret_cast<uint4*>((is_v ? p.v_cache : p.k_cache) + (slot * p.num_kv_heads + head) * kHeadDim);
          o[c0] = a0;
          o[c1] = a1;
        }
      } else if (slot >= 0) {  // the whole warp
        const int64_t row = slot * p.num_kv_heads + head;
        uint8_t* data = is_v ? p.q4.v_data : p.q4.k_data;
        uint8_t* scales = is_v ? p.q4.v_scales : p.q4.k_scales;
        const float inv = is_v ? p.q4.v_inv : p.q4.k_inv;
        store_q4(data, scales, row, c0, a0, inv, real);
        store_q4(data, scales, row, c1, a1, inv, real);
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int dest, int num_sms, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int kv_groups = (a.num_kv_heads + 3) / 4;
  const int groups = (a.num_q_heads + 3) / 4 + kv_groups * (dest ? 2 : 1);
  // Few tokens: spread a token's heads over warps until the GPU has ~8 warps an SM.
  int splits = 1;
  while (splits < groups && static_cast<int64_t>(a.num_tokens) * splits < static_cast<int64_t>(num_sms) * 8) ++splits;
  const int64_t items = static_cast<int64_t>(a.num_tokens) * splits;
  const int64_t blocks = std::min<int64_t>((items + kWarps - 1) / kWarps, static_cast<int64_t>(num_sms) * 32);
  const dim3 grid(static_cast<unsigned>(blocks)), block(32 * kWarps);
  void (*kernel)(NormRopeArgs, int) = nullptr;
  if (a.interleaved)
    kernel = dest == 0 ? norm_rope_kernel<0, true> : dest == 1 ? norm_rope_kernel<1, true> : norm_rope_kernel<2, true>;
  else
    kernel = dest == 0 ? norm_rope_kernel<0, false> : dest == 1 ? norm_rope_kernel<1, false> : norm_rope_kernel<2, false>;
  return launch_pdl(kernel, grid, block, 0, stream, a, splits);
}

PKV_DEFINE_READ_ERROR(read_error_norm_rope, g_err_norm_rope)

}  // namespace pkv
