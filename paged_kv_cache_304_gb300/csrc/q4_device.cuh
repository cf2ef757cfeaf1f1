// q4_device.cuh -- the 4-bit row format on the device.
//
// A row of 128 dims of one head is eight groups of 16 consecutive dims.  Group
// j holds a scale s_j (e4m3, one byte) and 16 codes (e2m1, two to a byte, the
// even dim in the low nibble); dim d stands for code_d * s_j * tensor_scale.
//   quantising   y = x * (1 / tensor_scale) in fp32,
//                s = e4m3(min(max|y| / 6, 448)), round to nearest even,
//                code = e2m1(y / s), round to nearest even, saturating at 6;
//                s == 0 gives codes 0 (a group below 2^-10 * 6 reads as zero);
//                a NaN in the group makes its scale NaN, so all 16 read as NaN;
//                an infinity reads as +-6 * 448 * tensor_scale.
// code * s has at most six significant bits: it is exact in fp16 and in bf16,
// so attention over the cache multiplies the held values themselves, and
// tensor_scale is applied in fp32 outside the products.
#pragma once

#include <cuda_fp16.h>
#include <cfloat>
#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {
namespace q4 {

constexpr int kGroup = 16;       // dims that share a scale
constexpr int kRowBytes = 64;    // codes of one head's row
constexpr int kRowScales = 8;    // scales of one head's row

// Two codes from two floats: `lo` in bits 0-3.
__device__ __forceinline__ uint32_t enc2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// The four bytes of a word as four fp16 pairs: out[i] = codes 2i (low half), 2i+1.
__device__ __forceinline__ void dec8(uint32_t w, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}

// e4m3 byte of a float (round to nearest even, saturating; NaN stays NaN).
__device__ __forceinline__ uint32_t enc_scale(float s) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(s));
  return r & 0xffu;
}

// Two e4m3 bytes (low 16 bits) as an fp16 pair.
__device__ __forceinline__ uint32_t dec_scale2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

__device__ __forceinline__ float half_lo(uint32_t h2) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xffffu)));
}
__device__ __forceinline__ float half_hi(uint32_t h2) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 >> 16)));
}
__device__ __forceinline__ float dec_scale(uint32_t byte) { return half_lo(dec_scale2(byte)); }

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Maximum that a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Maximum of three that a NaN wins.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale byte of a group whose largest |y| is `amax`: e4m3(amax / 6), the quotient
// correctly rounded (product with the reciprocal, corrected with its residual;
// see enc8).  Everything from 2688 = 6 * 448 on saturates.
__device__ __forceinline__ uint32_t group_scale(float amax) {
  const float a = min_nan(amax, 4096.f), sixth = 1.f / 6.f;
  const float q = a * sixth;
  return enc_scale(fmaf(fmaf(-6.f, q, a), sixth, q));
}

// Eight codes of eight floats y over scale s (as the float its byte stands for);
// `r` is 1 / s rounded to nearest.  A code depends on which side of a tie y / s
// lies, so the quotient is needed correctly rounded (a tie is representable, and
// a quotient that is none does not round to one): the product y r is corrected
// with its residual, q + (y - q s) r (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  An infinite y is
// taken as its largest code before.
__device__ __forceinline__ uint32_t enc8(const float* y, float s, float r) {
  uint32_t w = 0;
  if (s == 0.f) return 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = y[2 * i] * r, b = y[2 * i + 1] * r;
    w |= enc2(fmaf(fmaf(-a, s, y[2 * i]), r, a), fmaf(fmaf(-b, s, y[2 * i + 1]), r, b)) << (8 * i);
  }
  return w;
}

// Codes of eight floats whose group's scale byte is `sb`.
__device__ __forceinline__ uint32_t enc8_group(float* y, uint32_t sb, float amax) {
  if (amax == INFINITY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(y[i], -FLT_MAX), FLT_MAX);
  }
  // One Newton step on the approximate reciprocal (of four-bit numbers only).
  const float s = dec_scale(sb), r = fast_rcp(s);
  return enc8(y, s, fmaf(fmaf(-s, r, 1.f), r, r));
}

// bf16 pair word to two floats (exact).
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace q4
}  // namespace pkv
