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

// A group's parameters: the range widened to contain 0, the fp16 scale
// s = round-up(range / qmax) (one IEEE division), the zero point
// z = clamp(rne(-lo / s), 0, qmax) (rne_div), and the fast path's constants.
// Non-finite input: an infinity makes the range, hence the scale, infinite; a
// NaN is dropped by the min/max but shows in the fast path's largest remainder
// (or, in an otherwise all-zero group, in group_has_nan).
struct GroupParams {
  __half scale_h;   // 1 when the range is 0
  float mn, mx;     // the group's min and max (before widening)
  float sf, rcp, zf, C;   // scale, approximate 1/scale, zero point, zero + 1.5 * 2^23
  int qmax;
  bool flat;        // range 0 (all zeros, or NaN among zeros): every code 0
  bool bad;         // non-finite scale
};

// From the group's least and greatest values.
__device__ __forceinline__ GroupParams group_params_of(float mn, float mx, int bits) {
  GroupParams g;
  g.mn = mn;
  g.mx = mx;
  g.qmax = (1 << bits) - 1;
  const float qf = static_cast<float>(g.qmax);
  const float lo = fminf(0.0f, g.mn);
  const float hi = fmaxf(0.0f, g.mx);
  const float range = __fsub_rn(hi, lo);
  g.flat = range == 0.0f;
  g.scale_h = __ushort_as_half(0x3C00);  // 1.0
  g.sf = 1.0f; g.rcp = 1.0f; g.zf = 0.0f; g.C = kRoundAdd;
  g.bad = false;
  if (!g.flat) {
    g.scale_h = __float2half_ru(__fdiv_rn(range, qf));
    g.sf = __half2float(g.scale_h);
    g.bad = !isfinite(g.sf);
    g.rcp = rcp_approx(g.sf);
    g.zf = fminf(fmaxf(rne_div(-lo, g.sf, g.rcp), 0.0f), qf);
    g.C = g.zf + kRoundAdd;   // exact
  }
  return g;
}

// Whether some code of the group is clamped: rne(mx / s) + z > qmax or
// rne(mn / s) + z < 0, decided exactly from the remainders against the
// half-integers k + 1/2 (k = qmax - z) and -z - 1/2 (exact as in rne_div), a
// remainder of 0 being a tie that rounds to the even side.  Codes are
// monotone in x, so no other value is clamped when these two are not.
__device__ __forceinline__ bool group_clamps(const GroupParams& g) {
  const float k = static_cast<float>(g.qmax) - g.zf;
  const float rt = __fmaf_rn(-(k + 0.5f), g.sf, g.mx);
  const float rb = __fmaf_rn(g.zf + 0.5f, g.sf, g.mn);
  return rt > 0.0f || (rt == 0.0f && (static_cast<int>(k) & 1) != 0) ||
         rb < 0.0f || (rb == 0.0f && (static_cast<int>(g.zf) & 1) != 0);
}

// The specification's code of one value (a NaN gives code 0, as the
// specification's clamp of a NaN quotient does).
__device__ __forceinline__ int code_exact(float x, const GroupParams& g) {
  return static_cast<int>(fminf(fmaxf(__fadd_rn(rne_div(x, g.sf, g.rcp), g.zf), 0.0f), static_cast<float>(g.qmax)));
}

__device__ __forceinline__ GroupParams group_params(const uint32_t (&w)[16], int bits) {
  // min and max over the 32 values in bf16 pairs (exact), then the two lanes
  __nv_bfloat162 mn2 = *reinterpret_cast<const __nv_bfloat162*>(&w[0]), mx2 = mn2;
#pragma unroll
  for (int k = 1; k < 16; ++k) {
    const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[k]);
    mn2 = __hmin2(mn2, v);
    mx2 = __hmax2(mx2, v);
  }
  return group_params_of(fminf(__low2float(mn2), __high2float(mn2)), fmaxf(__low2float(mx2), __high2float(mx2)), bits);
}

__device__ __forceinline__ bool group_has_nan(const uint32_t (&w)[16]) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 x2 = bf16x2_to_float2(w[k]);
    bad |= (x2.x != x2.x) || (x2.y != x2.y);
  }
  return bad;
}

// The values of a quarter of a group (8v .. 8v+7) passed to f(j, x) with j =
// 0..7.  Used by the rare paths, which run a quarter at a time in a rolled loop
// so the group's registers are not all live at once.
template <class F>
__device__ __forceinline__ void quarter_values(const uint4& raw, F f) {
  const uint32_t q4[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) f(j, bf16_bits_to_float((j & 1) ? (q4[j >> 1] >> 16) : (q4[j >> 1] & 0xFFFFu)));
}

// Quantise one group of 32 channels (this thread alone): w holds the 32 bf16
// values, quarter(v) their v-th quarter again (for the rare path: re-read from
// where they were loaded, an L1 hit, or picked from w); the codes go to cdst (32 bytes for
// 8-bit, 16 for 4-bit) and the fp16 (scale, zero) word to *szw.
// Fast path, per pair of values: m = fl(x * r + C) holds rne(x * r) + z in its
// low mantissa bits (C's low byte is zero, so a code 0 .. qmax is m's low byte
// or nibble, gathered by byte permutes), u = m - C = rne(x * r), d = x - u * s
// exact; the code is the specification's wherever |d| < s / 2 (then u is the
// integer nearest x / s) and no code is clamped (group_clamps).  A quarter
// with some |d| at least s / 2 (a tie, or u one step off) or a NaN (the
// quarter's largest |d| is then NaN), or a clamped group, is redone with
// code_exact and stored 8 codes at a time.
template <class Quarter>
__device__ __forceinline__ void quantize_group_of(const uint32_t (&w)[16], Quarter quarter, int bits, uint8_t* cdst,
                                                  uint32_t* szw, int32_t* status) {
  const GroupParams gp = group_params(w, bits);
  bool bad = gp.bad;
  uint32_t packed[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) packed[k] = 0u;
  unsigned redo = 0;   // quarters to redo, one bit each
  if (gp.flat) {
    bad |= group_has_nan(w);
  } else {
    const float2 r2 = make_float2(gp.rcp, gp.rcp), c2 = make_float2(gp.C, gp.C);
    const float2 nc2 = make_float2(-gp.C, -gp.C), ns2 = make_float2(-gp.sf, -gp.sf);
    const float hs = 0.5f * gp.sf;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      // the largest |d| of the quarter; a NaN anywhere makes it NaN
      float dmax = 0.0f;
      uint32_t mb[8];   // bits of m: C = z + 1.5 * 2^23 has a zero low byte, so the code is in the low bits
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float2 x2 = bf16x2_to_float2(w[4 * v + kk]);
        const float2 m2 = __ffma2_rn(x2, r2, c2);
        const float2 d2 = __ffma2_rn(__fadd2_rn(m2, nc2), ns2, x2);
        dmax = fmax3_nan(dmax, fabsf(d2.x), fabsf(d2.y));
        mb[2 * kk] = __float_as_uint(m2.x);
        mb[2 * kk + 1] = __float_as_uint(m2.y);
      }
      if (bits == 8) {   // low bytes of four m's per word
        packed[2 * v] = prmt(prmt(mb[0], mb[1], 0x0040u), prmt(mb[2], mb[3], 0x0040u), 0x5410u);
        packed[2 * v + 1] = prmt(prmt(mb[4], mb[5], 0x0040u), prmt(mb[6], mb[7], 0x0040u), 0x5410u);
      } else {           // low nibbles of eight m's, the first in bits 0-3
        uint32_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = (mb[2 * j] & 0x0Fu) | ((mb[2 * j + 1] << 4) & 0xF0u);
        packed[v] = prmt(prmt(b[0], b[1], 0x0040u), prmt(b[2], b[3], 0x0040u), 0x5410u);
      }
      redo |= (dmax < hs ? 0u : 1u) << v;   // false for a NaN
    }
    if (group_clamps(gp)) redo = 0xFu;
  }
  if (redo == 0u) {
    uint4* dst = reinterpret_cast<uint4*>(cdst);
    dst[0] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    if (bits == 8) dst[1] = make_uint4(packed[4], packed[5], packed[6], packed[7]);
  } else {   // rare: whole group stored quarter by quarter, the flagged quarters recomputed
#pragma unroll 1
    for (int v = 0; v < 4; ++v) {
      uint32_t c8[2];
      if ((redo >> v) & 1u) {
        c8[0] = 0u;
        c8[1] = 0u;
        quarter_values(quarter(v), [&](int j, float x) {
          bad |= x != x;
          const uint32_t c = static_cast<uint32_t>(code_exact(x, gp));
          if (bits == 8) c8[j >> 2] |= c << (8 * (j & 3));
          else c8[0] |= c << (4 * j);
        });
      } else if (bits == 8) {
        c8[0] = v == 0 ? packed[0] : v == 1 ? packed[2] : v == 2 ? packed[4] : packed[6];
        c8[1] = v == 0 ? packed[1] : v == 1 ? packed[3] : v == 2 ? packed[5] : packed[7];
      } else {
        c8[0] = v == 0 ? packed[0] : v == 1 ? packed[1] : v == 2 ? packed[2] : packed[3];
        c8[1] = 0u;
      }
      if (bits == 8) reinterpret_cast<uint2*>(cdst)[v] = make_uint2(c8[0], c8[1]);
      else reinterpret_cast<uint32_t*>(cdst)[v] = c8[0];
    }
  }
  if (bad) report(status, KVQ_ERR_NONFINITE);
  *szw = __half_as_ushort(gp.scale_h) |
         (static_cast<uint32_t>(__half_as_ushort(__int2half_rn(static_cast<int>(gp.zf)))) << 16);
}

}  // namespace kvq
