// Element format of the block-scaled 8-bit cache: e4m3 codes (sign, 4 exponent bits of bias 7,
// 3 mantissa bits; largest value 448, least 2^-9, NaN 0x7f / 0xff, no infinity) and one fp32
// scale per (sequence, kv head, block of `block` tokens), K and V apart. A row reads back as
// code * scale.
//
// The append's scales are powers of two, which costs an e4m3 code no precision (its own
// exponent absorbs the shift) and buys exactness twice: x * 2^-k is exact, so a stored element
// is rounded once, and bringing a block's older codes to a larger scale moves their exponents
// only (a code that falls below e4m3's normal range, 2^-6, is rounded to the 2^-9 grid).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "td_device.cuh"
#include "td_mma.cuh"

namespace td {

// Infinities become NaN, everything else stays: x * 0 is NaN for an infinity and +-0 otherwise.
// Applied before a maximum (which passes NaN over, so it is taken over finite elements) and before
// the conversion to e4m3 (which would saturate an infinity).
__device__ __forceinline__ float2 finite_or_nan(float2 x) { return ffma2(x, make_float2(0.f, 0.f), x); }

// The least power of two s >= 2^-126 with amax <= 448 s (amax as bits, finite). 448 = 1.75 * 2^8:
// the exponent of s is that of amax less 8, plus one if amax's significand is above 1.75.
__device__ __forceinline__ float pow2_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
  return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

// Two values to e4m3 codes (x in the low byte): rounded to nearest even, saturating, NaN kept.
__device__ __forceinline__ uint16_t to_e4m3x2(float2 v) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(v.y), "f"(v.x));
  return d;
}

// Two elements to codes of x * inv; infinities become NaN codes.
__device__ __forceinline__ uint16_t quant2_e4m3(float2 x, float inv) {
  return to_e4m3x2(fmul2(finite_or_nan(x), make_float2(inv, inv)));
}

// Two codes to the fp16 pair of their values (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint16_t codes) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(codes));
  return d;
}

__device__ __forceinline__ float2 e4m3x2_float2(uint16_t codes) {
  const uint32_t h = e4m3x2_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Four codes of a word brought to another scale: value * r rounded to nearest even.
__device__ __forceinline__ uint32_t rescale4_e4m3(uint32_t w, float r) {
  const float2 a = e4m3x2_float2((uint16_t)w), b = e4m3x2_float2((uint16_t)(w >> 16));
  const float2 rr = make_float2(r, r);
  return (uint32_t)to_e4m3x2(fmul2(a, rr)) | ((uint32_t)to_e4m3x2(fmul2(b, rr)) << 16);
}

}  // namespace td
