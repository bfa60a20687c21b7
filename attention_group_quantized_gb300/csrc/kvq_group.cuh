// kvq_group.cuh -- arithmetic of the group quantiser that more than one kernel
// uses: exact rounded division of bf16 values by fp16 scales, bf16 widening.
#pragma once

#include <cstdint>

#include "kvq_device.cuh"

namespace kvq {

// 1.5 * 2^23: adding it to a float of magnitude below 2^22 rounds that value
// to the nearest integer (ties to even) -- floats in [2^23, 2^24) are spaced
// 1 apart -- and leaves the integer in the low mantissa bits (its bit pattern
// 0x4B400000 has a zero low byte).
constexpr float kRoundAdd = 12582912.0f;

// max(a, b, c), NaN if any input is NaN (three-input form, sm_100 and later)
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float rcp_approx(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// rne(a / s), ties to even, for a bf16 value a and an fp16 scale s with
// |a / s| <= 256, given any r within 2^-21 (relative) of 1/s:
//   u = rne(a * r) is at most one step from rne(a / s);
//   d = a - u * s is exact in fp32 (u * s has at most 20 significant bits and
//     |d| <= 1.5 s while s >= |a| / 256, so d fits in 24 bits);
//   u moves one step towards a / s when |d| > s / 2, or when |d| = s / 2
//     (a / s is a half-integer) and u is odd.
// For such a and s this is also rne(fl(a / s)), the IEEE fp32 quotient
// rounded: fl(a / s) equals a half-integer h only when a / s does (a nonzero
// a - h * s is a multiple of 2^(e_a - 20), while fl(a / s) = h needs
// |a - h * s| < s * ulp(h) / 2, about 2^(e_a - 23)), and otherwise stays on
// the same side of every half-integer as a / s.  (Checked against the IEEE
// quotient for every finite bf16 a and fp16 scales from 2^-24 to 2^8.)
__device__ __forceinline__ float rne_div(float a, float s, float r) {
  float u = __fsub_rn(__fmaf_rn(a, r, kRoundAdd), kRoundAdd);
  const float d = __fmaf_rn(-u, s, a);
  const float ad = fabsf(d), hs = 0.5f * s;
  if (ad > hs || (ad == hs && (static_cast<int>(u) & 1) != 0)) u = __fadd_rn(u, copysignf(1.0f, d));
  return u;
}

__device__ __forceinline__ float2 bf16x2_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b16) { return __uint_as_float(b16 << 16); }

}  // namespace kvq
