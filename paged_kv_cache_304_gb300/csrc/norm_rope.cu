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
// Bound by HBM (every row read and written once).  A CTA takes a few tokens: it
// puts their cosines and sines into shared memory, then its warps take units of
// four heads of a token, eight lanes a head, 16 dims a lane as two 8-dim chunks
// chosen so that both partners of a rotated pair sit in one lane.  Nothing is
// carried from unit to unit, so the next unit's rows are requested while one is in
// work and few registers leave room for many warps (with the angles and weights
// kept in registers, 15 warps an SM reached 60 % of the copy bandwidth).  fp32
// arithmetic is done on pairs (one instruction for two).
#include <cuda_runtime.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "q4_device.cuh"

namespace pkv {
namespace {

__device__ unsigned int g_err_norm_rope;

constexpr int kWarps = 8;
constexpr int kMaxTokens = 8;          // of a CTA
constexpr int kPairs = kHeadDim / 2;

__device__ __forceinline__ uint4 pack8(const float2* x) {
  return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y), pack_bf16x2(x[2].x, x[2].y),
                    pack_bf16x2(x[3].x, x[3].y));
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Eight floats from shared memory as four pairs.
__device__ __forceinline__ void read8(const float* p, float2* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = make_float2(a.x, a.y);
  x[1] = make_float2(a.z, a.w);
  x[2] = make_float2(b.x, b.y);
  x[3] = make_float2(b.z, b.w);
}

// kDest: 0 = k_out, 1 = bf16 cache (K and V), 2 = 4-bit cache (K and V).
// kInter: rotated pairs are (2i, 2i + 1).
template <int kDest, bool kInter>
__global__ void __launch_bounds__(32 * kWarps, 4) norm_rope_kernel(const NormRopeArgs p, int tokens) {
  __shared__ __align__(16) float s_cos[kMaxTokens][kPairs], s_sin[kMaxTokens][kPairs];
  __shared__ __align__(16) float s_weight[2][kHeadDim];
  __shared__ int s_slot[kMaxTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int n = static_cast<int>(min(static_cast<int64_t>(tokens), p.num_tokens - t0));

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
  // Units: groups of four heads (queries, then keys, then, with a cache, values)
  // of the CTA's tokens.
  const int q_groups = (p.num_q_heads + 3) >> 2, kv_groups = (p.num_kv_heads + 3) >> 2;
  const int rope_groups = q_groups + kv_groups;
  const int groups = rope_groups + (kDest ? kv_groups : 0);
  // Rows of unit (t, g), this lane's head of the four (plain loads: the output may be the input).
  auto load = [&](int t, int g, uint4& a0, uint4& a1) {
    a0 = a1 = make_uint4(0u, 0u, 0u, 0u);
    if (t >= n) return;
    const bool is_q = g < q_groups;
    const int head = 4 * (is_q ? g : g < rope_groups ? g - q_groups : g - rope_groups) + sub;
    if (head >= (is_q ? p.num_q_heads : p.num_kv_heads)) return;
    const uint16_t* row = is_q ? p.q + (t0 + t) * p.q_stride
                               : g < rope_groups ? p.k + (t0 + t) * p.k_stride : p.v + (t0 + t) * p.v_stride;
    const uint4* src = reinterpret_cast<const uint4*>(row + head * kHeadDim);
    a0 = src[c0];
    a1 = src[c1];
  };
  int t = warp / groups, g = warp - t * groups;
  uint4 n0, n1;
  load(t, g, n0, n1);

  // Cosines and sines of every token (pairs behind rope_dim do not turn), weights, slots.
  for (int i = threadIdx.x; i < n * kPairs; i += 32 * kWarps) {
    const int pair = i % kPairs, tok = i / kPairs;
    float c = 1.f, s = 0.f;
    if (2 * pair < p.rope_dim) {
      const int axis = pair < p.section_end0 ? 0 : (pair < p.section_end1 ? 1 : 2);
      const int pos = __ldg(p.positions + axis * p.position_axis_stride + t0 + tok);
      const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) *
                            static_cast<uint64_t>(__ldg(reinterpret_cast<const long long*>(p.freqs) + pair));
      // angle in [-pi, pi): the top 32 bits times 2 pi / 2^32
      const float angle = static_cast<float>(static_cast<int>(frac >> 32)) * 1.4629180792671596e-9f;
      c = __cosf(angle);
      s = __sinf(angle);
    }
    s_cos[tok][pair] = c;
    s_sin[tok][pair] = s;
  }
  {
    const uint16_t* w = threadIdx.x < kHeadDim ? p.q_weight : p.k_weight;
    const int d = threadIdx.x % kHeadDim;
    s_weight[threadIdx.x / kHeadDim][d] = w ? __uint_as_float(static_cast<uint32_t>(__ldg(w + d)) << 16) : 1.f;
  }
  if (kDest && threadIdx.x < n) {
    int s = __ldg(p.slots + t0 + threadIdx.x);
    if (s < -1 || s >= p.num_blocks * kBlockSize) {
      atomicOr(&g_err_norm_rope, PKV_DEVERR_SLOT_RANGE);
      s = -1;
    }
    s_slot[threadIdx.x] = s;
  }
  __syncthreads();

  while (t < n) {
    uint4 a0 = n0, a1 = n1;
    int tn = t, gn = g + kWarps;
    while (gn >= groups) {
      gn -= groups;
      ++tn;
    }
    load(tn, gn, n0, n1);
    const bool is_q = g < q_groups, is_v = g >= rope_groups;
    const int head = 4 * (is_q ? g : is_v ? g - rope_groups : g - q_groups) + sub;
    const bool real = head < (is_q ? p.num_q_heads : p.num_kv_heads);
    if (!is_v) {
      float2 x[8], w[8];
      q4::unpack8(a0, x);
      q4::unpack8(a1, x + 4);
      if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = ffma2(x[i], x[i], ss);
        float sum = ss.x + ss.y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        const float r = rsqrtf(sum * (1.f / kHeadDim) + p.eps);
        read8(s_weight[is_q ? 0 : 1] + 8 * c0, w);
        read8(s_weight[is_q ? 0 : 1] + 8 * c1, w + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmul2(fmul2(x[i], both(r)), w[i]);
      }
      // The lane's pairs: elements of chunk c0 with those of c1 (halves), or
      // neighbours within each chunk (interleaved).
      float2 c[4], s[4];
      if (kInter) {
        const float4 ca = *reinterpret_cast<const float4*>(&s_cos[t][4 * c0]);
        const float4 cb = *reinterpret_cast<const float4*>(&s_cos[t][4 * c1]);
        const float4 sa = *reinterpret_cast<const float4*>(&s_sin[t][4 * c0]);
        const float4 sb = *reinterpret_cast<const float4*>(&s_sin[t][4 * c1]);
        const float ce[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
        const float se[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          x[e] = ffma2(make_float2(x[e].y, x[e].x), make_float2(-se[e], se[e]), fmul2(x[e], both(ce[e])));
      } else {
        read8(&s_cos[t][8 * l], c);
        read8(&s_sin[t][8 * l], s);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u = x[e], z = x[e + 4];
          x[e] = ffma2(z, make_float2(-s[e].x, -s[e].y), fmul2(u, c[e]));
          x[e + 4] = ffma2(u, s[e], fmul2(z, c[e]));
        }
      }
      a0 = pack8(x);
      a1 = pack8(x + 4);
    }
    const int64_t slot = kDest ? s_slot[t] : 0;
    if (is_q || kDest < 2) {
      uint16_t* o = nullptr;
      if (is_q)
        o = p.q_out + (t0 + t) * p.q_out_stride;
      else if (kDest == 0)
        o = p.k_out + (t0 + t) * p.k_out_stride;
      else if (slot >= 0)
        o = (is_v ? p.v_cache : p.k_cache) + slot * p.num_kv_heads * kHeadDim;
      if (real && o) {
        uint4* dst = reinterpret_cast<uint4*>(o + head * kHeadDim);
        dst[c0] = a0;
        dst[c1] = a1;
      }
    } else if (slot >= 0) {  // the whole warp
      const int64_t row = slot * p.num_kv_heads + head;
      const float inv = is_v ? p.q4.v_inv : p.q4.k_inv;
      uint32_t b0, b1;
      const uint32_t w0 = q4::quantise_chunk(a0, inv, &b0), w1 = q4::quantise_chunk(a1, inv, &b1);
      if (real) {
        uint32_t* data = reinterpret_cast<uint32_t*>((is_v ? p.q4.v_data : p.q4.k_data) + row * q4::kRowBytes);
        uint8_t* scales = (is_v ? p.q4.v_scales : p.q4.k_scales) + row * q4::kRowScales;
        data[c0] = w0;
        data[c1] = w1;
        if (!(lane & 1)) {  // even chunks: the scale of a group of two
          scales[c0 >> 1] = static_cast<uint8_t>(b0);
          scales[c1 >> 1] = static_cast<uint8_t>(b1);
        }
      }
    }
    t = tn;
    g = gn;
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int dest, int num_sms, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  // Up to eight tokens a CTA (their angles are computed once), fewer while that
  // would leave SMs without two CTAs.
  const int tokens =
      static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxTokens, a.num_tokens / (2 * static_cast<int64_t>(num_sms)))));
  const dim3 grid(static_cast<unsigned>((a.num_tokens + tokens - 1) / tokens)), block(32 * kWarps);
  void (*kernel)(NormRopeArgs, int) = nullptr;
  if (a.interleaved)
    kernel = dest == 0 ? norm_rope_kernel<0, true> : dest == 1 ? norm_rope_kernel<1, true> : norm_rope_kernel<2, true>;
  else
    kernel = dest == 0 ? norm_rope_kernel<0, false> : dest == 1 ? norm_rope_kernel<1, false> : norm_rope_kernel<2, false>;
  return launch_pdl(kernel, grid, block, 0, stream, a, tokens);
}

PKV_DEFINE_READ_ERROR(read_error_norm_rope, g_err_norm_rope)

}  // namespace pkv
