// kvq_dequantize.cu -- the group-quantised cache read back as values
// (《分块稀疏注意力与KV Cache量化：长文本推理显存优化实践》 §2.4: x_hat = (c - z) s).
//
// HBM-bound: each code and scale/zero word is read once, each value written
// once; the output (256 bytes a row in bf16 at D = 128) is the larger side.  A
// lane takes 8 channels: 8 bytes of codes (4 of a 4-bit head) in, one 16-byte
// bf16 store out, so that a warp's loads cover whole consecutive cache rows of
// one head and its stores whole output rows.  c - z is exact in fp32 and so is
// its product with the fp16 scale (9 + 11 significant bits), so the only
// rounding is the one to bf16.
#include <algorithm>
#include <type_traits>

#include "kvq_chunk.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;

struct DqParams {
  chunk::View c;
  const uint8_t* codes;
  const uint32_t* sz;
  void* out;
  int32_t* status;
  int32_t Hkv, tiles;       // tiles: runs of a warp's rows
  int32_t zero_rest;        // rows of no usable sequence become zeros
  int64_t codes_bytes;      // size of the code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

// The 8 values of a lane's codes: (c - z) s.  The fp32 with the bits
// 0x4B0000cc is 2^23 + c, put together by one byte permute a value.
template <int BITS>
__device__ __forceinline__ void values8(float (&x)[8], uint2 c, uint32_t word) {
  const float zb = 8388608.0f + half_hi(word), s = half_lo(word);
  const uint32_t lo = c.x & 0x0F0F0F0Fu, hi = (c.x >> 4) & 0x0F0F0F0Fu;   // (4-bit: even and odd channels)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = BITS == 8 ? (i < 4 ? c.x : c.y) : (i & 1) ? hi : lo;
    const int byte = BITS == 8 ? i & 3 : i >> 1;
    x[i] = (__uint_as_float(prmt(w, 0x4B000000u, 0x7440u + byte)) - zb) * s;
  }
}

// NP: passes of 32 lanes whose loads are in flight together (NP x 256 / D rows
// a warp).  For bf16, eight amortise the rows' look-up best when there are warps
// enough and two spread a short call over more of them; with fp32's twice as
// many stores two are faster at every length.  Measured (us; two, eight passes):
//   rows           1024        2048        3040        4096        8192       24576
//   8 heads, D 128, INT8, bf16
//             2.4   2.7   2.9   3.0   3.9   3.4   4.5   3.7   7.1   6.5  16.6  14.0
//   4 heads, D 64, INT8, bf16 (a quarter of the warps of eight passes)
//             2.1   2.7   2.2   2.7   2.2   2.7   2.4   2.7   2.9   3.0   5.9   5.8
//   8 heads, D 128, INT4, fp32
//             3.1   3.2   4.1   4.7   5.3   5.8   6.3   6.9   9.5  11.6  21.6  25.8
// so eight from about eight warps an SM on.  In all: 14.9 us for 79 MB of mixed
// heads, 5.3 TB/s, 18.0 us for 105 MB of 8-bit ones, 5.8 TB/s, 16.4 us for 88 MB
// of 4-bit ones, 5.4 TB/s, 2.6 us for 5 MB.
template <int D, bool F32, int NP>
__global__ void __launch_bounds__(kWarps * 32) dequantize_kernel(const __grid_constant__ DqParams p) {
  constexpr int G = D / 32;
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPP = 32 / LPR;       // rows per pass
  constexpr int R = RPP * NP;         // rows per warp
  // launched as a programmatic dependent: the rows may have been written by
  // the kernel before it
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, blockDim.x, p.status);
  const int64_t nw = static_cast<int64_t>(p.tiles) * p.Hkv;
  const int64_t storage = static_cast<int64_t>(p.c.pB) * p.c.pT;
  const int col = lane % LPR;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < nw;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int tile = static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(p.Hkv));
    const int h = static_cast<int>(static_cast<uint32_t>(u) - static_cast<uint32_t>(tile) * p.Hkv);
    const int r0 = tile * R;
    const int64_t mine = chunk::locate_rows(p.c, r0, lane, R, h == 0, p.status);
    auto rows = [&](auto bits_of) {
      constexpr int BITS = decltype(bits_of)::value;
      int64_t pos[NP];
      uint2 c[NP];
      uint32_t word[NP];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        pos[k] = __shfl_sync(0xffffffffu, mine, k * RPP + lane / LPR);
        c[k] = make_uint2(0u, 0u);
        word[k] = 0u;                   // a page outside the pool (or, zero_rest, a row of no sequence) reads as zeros
        if (pos[k] < 0) continue;
        const int64_t off = p.plane_off[h] + pos[k] * (D * BITS / 8) + col * BITS;
        const int64_t si = (static_cast<int64_t>(h) * storage + pos[k]) * G + col / 4;
        if (!KVQ_IN_RANGE(off >= 0 && off + BITS <= p.codes_bytes && si < static_cast<int64_t>(p.Hkv) * storage * G,
                          p.status))
          continue;
        if constexpr (BITS == 8) c[k] = *reinterpret_cast<const uint2*>(p.codes + off);
        else c[k].x = *reinterpret_cast<const uint32_t*>(p.codes + off);
        word[k] = p.sz[si];
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        if (pos[k] == chunk::kNoRow && !(p.zero_rest && r0 + k * RPP + lane / LPR < p.c.rows)) continue;
        float x[8];
        values8<BITS>(x, c[k], word[k]);
        const int64_t o = (static_cast<int64_t>(r0 + k * RPP + lane / LPR) * p.Hkv + h) * D + col * 8;
        if constexpr (F32) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + o);
          dst[0] = make_float4(x[0], x[1], x[2], x[3]);
          dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            v[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + o) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    };
    if (p.bits[h] == 8) rows(std::integral_constant<int, 8>{});
    else rows(std::integral_constant<int, 4>{});
  }
}

}  // namespace

cudaError_t launch_dequantize(const DequantizeArgs& a, cudaStream_t stream) {
  DqParams p;
  const kvq_cache& s = *a.src;
  p.c = chunk::view_of(a.chunk, s);
  p.codes = s.codes;
  p.sz = s.sz;
  p.out = a.out;
  p.status = a.status;
  p.Hkv = s.Hkv;
  p.zero_rest = a.zero_rest ? 1 : 0;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * s.B * s.Tcap * (s.D / 2);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  auto tiles_of = [&](int np) { return (a.chunk.rows + np * (256 / s.D) - 1) / (np * (256 / s.D)); };
  const bool f32 = a.out_dtype == KVQ_OUT_F32;
  const bool many = !f32 && static_cast<int64_t>(tiles_of(8)) * p.Hkv >= 8 * device_sm_count();
  p.tiles = tiles_of(many ? 8 : 2);
  const int64_t warps = static_cast<int64_t>(p.tiles) * p.Hkv;
  const int64_t blocks = std::min<int64_t>((warps + kWarps - 1) / kWarps, int64_t(1) << 30);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, p); };
  if (s.D == 128)
    return f32    ? launch(dequantize_kernel<128, true, 2>)
           : many ? launch(dequantize_kernel<128, false, 8>)
                  : launch(dequantize_kernel<128, false, 2>);
  return f32    ? launch(dequantize_kernel<64, true, 2>)
         : many ? launch(dequantize_kernel<64, false, 8>)
                : launch(dequantize_kernel<64, false, 2>);
}

}  // namespace kvq
