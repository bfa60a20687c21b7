// kvq_tile.cuh -- the 128-key operand tiles of the tensor-core attention
// kernels (prefill, chunk): how a warpgroup of 128 threads turns the codes of
// a key tile into the fp16 operand tile that tcgen05.mma reads (128-byte
// swizzle), and the two-wide fp32 arithmetic of their softmax.
#pragma once

#include <cstdint>

#include "kvq_device.cuh"

namespace kvq {
namespace tile {

constexpr int kT = 128;           // tile edge (query rows, keys)
constexpr int kSub = 2048;        // code bytes one dequant iteration reads: 128 threads x 16 B

// How the dequant warpgroup walks one code tile (the K or V part of a key
// tile) of a (D, BITS) head.  Iteration `it` covers RPI token rows of R
// bytes (2 KB), 16 bytes per thread; a 16-byte chunk holds VPC channels (16
// or 32) and becomes two or four 16-byte fp16 chunks of the swizzled operand
// tile.
template <int D, int BITS>
struct DqFmt {
  static constexpr int R = D * BITS / 8;     // code bytes per token row
  static constexpr int RPI = kSub / R;       // rows per iteration
  static constexpr int NI = kT / RPI;        // iterations (ring sub-chunks) per part
  static constexpr int VPC = 128 / BITS;     // channels per chunk
  static_assert(RPI * NI == kT, "whole iterations per part");
};

// Row (within an iteration) and chunk of the 16 code bytes thread t loads.
// A warp's 32 lanes cover whole consecutive rows (512 contiguous bytes).
// With the 128-byte swizzle, fp16 chunk x of row r sits at bank group
// x ^ (r & 7), and the D/64 blocks of a tile are 16 KB apart (the same
// banks).  Per format, the eight lanes of each store phase take:
//   8-bit, D 128: one half (64 B) of row r and the other half of row r + 1,
//                 so the stores (two chunks per lane) go to even chunk
//                 indices in one row and odd ones in the other;
//   4-bit, D 128: rows r .. r+3 (r a multiple of 4), the first 32 bytes of
//                 rows r, r+3 and the last 32 of rows r+1, r+2 (or the other
//                 way round): each store phase writes the four swizzle rows
//                 of a quad, once in the low and once in the high half of the
//                 chunk index;
//   D 64:         two (8-bit) or four (4-bit) whole consecutive rows.
template <int D, int BITS>
__device__ __forceinline__ void dq_lane(int t, int& row, int& c) {
  const int w = t >> 5, l = t & 31;
  if constexpr (D == 128 && BITS == 8) {
    const int sub = (l & 7) >> 2, ph = (l >> 3) & 1;
    row = 4 * w + 2 * (l >> 4) + sub;
    c = (l & 3) + 4 * (sub ^ ph);
  } else if constexpr (D == 128 && BITS == 4) {
    const int rr = (l & 7) >> 1, ph = (l >> 3) & 1;
    const int hi = (rr ^ (rr >> 1)) & 1;     // rows 1, 2 of the quad take the other half
    row = 8 * w + 4 * (l >> 4) + rr;
    c = 2 * (hi ^ ph) + (l & 1);
  } else if constexpr (BITS == 8) {          // D 64
    row = t >> 2;
    c = t & 3;
  } else {
    row = t >> 1;
    c = t & 1;
  }
}

// two-wide fp32 arithmetic (one instruction for a pair of values)
__device__ __forceinline__ void ffma2(float& d0, float& d1, float a0, float a1, float b, float c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %4};\n\t"
      "mov.b64 rc, {%5, %5};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void fadd2(float& d0, float& d1, float a0, float a1) {
  asm("{\n\t.reg .b64 ra, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rd, {%0, %1};\n\t"
      "add.f32x2 rd, rd, ra;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 bytes to a shared-window address
__device__ __forceinline__ void sts128(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// One code chunk (16 bytes, channels ch0 ..) -> OC fp16 chunks of (c - z) * s
// (exact difference, one rounding) in the 128-byte-swizzled K-major tile
// [D/64 blocks][128 rows][128 B] at dst.
template <int BITS>
__device__ __forceinline__ void dequant_chunk(uint32_t dst, int row, int ch0, uint4 w, uint32_t word) {
  constexpr int OC = BITS == 8 ? 2 : 4;
  const uint32_t zb = zero_biased2(word);
  const uint32_t s2 = (word & 0xFFFFu) | (word << 16);
  // 4-bit high nibbles: c - z = (1024 + 16 c) / 16 - 64 - z in one exact FMA
  const uint32_t mz = hsub2_u32(0x63806380u /* (960, 960) */, zb);   // -(64 + z), exact
  const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4 * OC];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BITS == 8) {
      // channels 4i .. 4i + 3 in order
      o[2 * i] = hmul2_u32(hsub2_u32(bytes01_biased(wv[i]), zb), s2);
      o[2 * i + 1] = hmul2_u32(hsub2_u32(bytes23_biased(wv[i]), zb), s2);
    } else {
      // channels 8i .. 8i + 7 in the order 0,4,1,5,2,6,3,7
      const uint32_t w8 = wv[i] >> 8;
      o[4 * i + 0] = hmul2_u32(hsub2_u32(nib_biased(wv[i]), zb), s2);
      o[4 * i + 1] = hmul2_u32(hfma2_u32((wv[i] & 0x00F000F0u) | 0x64006400u, kHalf2Sixteenth, mz), s2);
      o[4 * i + 2] = hmul2_u32(hsub2_u32(nib_biased(w8), zb), s2);
      o[4 * i + 3] = hmul2_u32(hfma2_u32((w8 & 0x00F000F0u) | 0x64006400u, kHalf2Sixteenth, mz), s2);
    }
  }
  const int kb = ch0 >> 6, cb = (ch0 & 63) >> 3, sw = row & 7;
  const uint32_t rowp = dst + kb * (kT * 128) + row * 128;
#pragma unroll
  for (int i = 0; i < OC; ++i) sts128(rowp + (((cb + i) ^ sw) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
}

}  // namespace tile
}  // namespace kvq
