// kvq_rotate.cu -- a chunk's projected rows on their way to attention: queries
// and keys normed per head (root mean square, weights) and rotated by their
// cache position, queries written out, keys and values quantised into the
// caches (《分块稀疏注意力与KV Cache量化：长文本推理显存优化实践》 §2.4) -- one pass over
// the rows, where a program would otherwise write the keys once more and read
// them again for the append.
//
//   y = x r w,  r = 1 / sqrt(mean(x^2) + eps);  (a, b) -> (a c - b s, b c + a s)
//
// Every operation is rounded on its own (no contraction), and the mean of
// squares is exact before its one rounding, so that a stored code is a
// function of the inputs that a program in any language can follow: a bf16
// square has 16 significant bits, exact in fp32, and the sum carries its
// rounding errors along (two-sum, Knuth 1969), across lanes as well.
//
// HBM-bound: 2 bytes a channel in, 2 out for a query, 1 or 1/2 and 1/8 for a
// key or value.  A lane takes 8 channels (16 bytes), so a row of a head is 16 or
// 8 lanes and a warp 2 or 4 consecutive rows; it takes NH heads of them, whose
// loads are all in flight together and which share the look-up of the rows'
// positions and the table's cosines and sines.  A pair's partner is in the lane
// rot_dim / 16 away (or, interleaved, in the lane itself); a quantisation group
// is four lanes.
#include <algorithm>

#include "kvq_chunk.cuh"
#include "kvq_group.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;

struct RParams {
  chunk::View c;
  const uint16_t* q;
  const uint16_t* x[2];     // k_new, v_new
  int64_t sq_row, sq_head, s_row, s_head;
  const float* table;       // [positions][rot] or null
  const uint16_t* w[2];     // q_weight, k_weight or null
  uint16_t* q_out;
  uint8_t* codes[2];
  uint32_t* sz[2];
  int32_t* status;
  int32_t Hq, Hkv, positions, rot, interleaved;
  float eps;
  int32_t head_runs;        // runs of NH heads: queries, keys, values in that order
  int32_t zero_rest;        // query rows of no usable sequence become zeros
  int64_t tiles;            // runs of a warp's rows
  int64_t codes_bytes;      // size of each code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

// (s, e) += v, with s + e the exact sum (but for e's own rounding, 2^-24 of a
// term that is 2^-24 of the sum)
__device__ __forceinline__ void add_exact(float& s, float& e, float v) {
  const float t = __fadd_rn(s, v), b = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(v, b)));
  s = t;
}

// What a lane needs of its row: its position and where the cache keeps it.
struct Row {
  int64_t store;            // storage row, kNoRow or kBadPage
  int32_t pos;              // cache position, -1: the row is left out
};

__device__ __forceinline__ Row find_row(const RParams& p, int r0, int lane, int count, bool reporter) {
  Row w;
  w.store = chunk::kNoRow;
  w.pos = -1;
  int b = chunk::find_sequence(p.c.start, p.c.B, r0, lane);
  const int r = r0 + lane;
  if (lane >= count || r >= p.c.rows) return w;
  while (b + 1 < p.c.B && p.c.start[b + 1] <= r) ++b;
  const chunk::Seq s = chunk::sequence(p.c, b);
  if (s.bad) {
    if (reporter) report(p.status, KVQ_ERR_INVALID_ARG);
    return w;
  }
  if (r < s.row0 || r >= s.row0 + s.n) return w;
  const int pos = s.len - s.n + (r - s.row0);
  if (p.table != nullptr && pos >= p.positions) {
    if (reporter) report(p.status, KVQ_ERR_INVALID_ARG);
    return w;
  }
  w.pos = pos;
  w.store = chunk::storage_row(p.c, b, pos);
  if (w.store < 0) {
    if (reporter) report(p.status, KVQ_ERR_INVALID_ARG);
    w.store = chunk::kBadPage;
  }
  return w;
}

__device__ __forceinline__ void widen8(float (&f)[8], const uint4& raw) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = bf16x2_to_float2(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The row's norm over its LPR lanes: f * (1 / sqrt(mean + eps)) * w.
template <int D>
__device__ __forceinline__ void norm8(float (&f)[8], const uint4& weight, float eps) {
  constexpr int LPR = D / 8;
  float s = 0.0f, e = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) add_exact(s, e, __fmul_rn(f[i], f[i]));
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
    add_exact(s, e, s2);
    e = __fadd_rn(e, e2);
  }
  // (a sum past fp32 is infinite; its error term is then no number)
  const float sum = isinf(s) ? s : __fadd_rn(s, e);
  const float mean = __fmul_rn(sum, 1.0f / D);   // exact: a power of two
  const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, eps)));
  float w[8];
  widen8(w, weight);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], r), w[i]);
}

// Quantise a group held by four lanes, 8 values each, as kvq_quantize does.
__device__ __forceinline__ void store_group(const float (&x)[8], int bits, bool live, uint8_t* codes, uint32_t* word,
                                            bool first, int32_t* status) {
  float mn = x[0], mx = x[0];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mn = fminf(mn, x[i]);
    mx = fmaxf(mx, x[i]);
    finite &= fabsf(x[i]) < INFINITY;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (!live) return;
  const float qf = bits == 8 ? 255.0f : 15.0f;
  const float lo = fminf(0.0f, mn), hi = fmaxf(0.0f, mx);
  const float range = __fsub_rn(hi, lo);
  __half scale = __ushort_as_half(0x3C00);   // 1, with zero point and codes 0, where every value is 0
  float z = 0.0f;
  uint32_t c[8] = {};
  if (range != 0.0f) {
    scale = __float2half_ru(__fdiv_rn(range, qf));
    const float s = __half2float(scale);
    finite &= s < INFINITY;
    const float rcp = rcp_approx(s);
    z = fminf(fmaxf(rne_div(-lo, s, rcp), 0.0f), qf);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = static_cast<uint32_t>(fminf(fmaxf(__fadd_rn(rne_div(x[i], s, rcp), z), 0.0f), qf));
  }
  if (!finite) report(status, KVQ_ERR_NONFINITE);
  if (bits == 8) {
    *reinterpret_cast<uint2*>(codes) = make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                                                  c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
  } else {
    uint32_t v = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) v |= c[i] << (4 * i);
    *reinterpret_cast<uint32_t*>(codes) = v;
  }
  if (first)
    *word = __half_as_ushort(scale) |
            (static_cast<uint32_t>(__half_as_ushort(__int2half_rn(static_cast<int>(z)))) << 16);
}

template <int D, int NH>
__global__ void __launch_bounds__(kWarps * 32) rotate_append_kernel(const __grid_constant__ RParams p) {
  constexpr int G = D / 32;
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int R = 32 / LPR;         // rows per warp
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, col = lane % LPR;
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, blockDim.x, p.status);
  const int64_t storage = static_cast<int64_t>(p.c.pB) * p.c.pT;
  const int64_t units = p.tiles * p.head_runs;
  const int heads = p.Hq + 2 * p.Hkv;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int tile = static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(p.head_runs));
    const int run = static_cast<int>(static_cast<uint32_t>(u) - static_cast<uint32_t>(tile) * p.head_runs);
    const int r0 = tile * R;
    const int r = r0 + lane / LPR;
    // the rows' loads need no look-up: rows of no sequence are read, not used
    uint4 raw[NH];
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      const int h = run * NH + j;
      raw[j] = make_uint4(0u, 0u, 0u, 0u);
      if (h >= heads || r >= p.c.rows) continue;
      const uint16_t* src = h < p.Hq ? p.q + r * p.sq_row + h * p.sq_head
                                     : p.x[h < p.Hq + p.Hkv ? 0 : 1] + r * p.s_row +
                                           (h < p.Hq + p.Hkv ? h - p.Hq : h - p.Hq - p.Hkv) * p.s_head;
      raw[j] = *reinterpret_cast<const uint4*>(src + col * 8);
    }
    const Row mine = find_row(p, r0, lane, R, run == 0);
    const int64_t store = __shfl_sync(0xffffffffu, mine.store, lane / LPR);
    const int pos = __shfl_sync(0xffffffffu, mine.pos, lane / LPR);
    const bool turns = p.table != nullptr && col * 8 < p.rot && run * NH < p.Hq + p.Hkv;
    const int half = p.rot / 2;
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.0f;
      sn[i] = 0.0f;
    }
    if (turns && pos >= 0) {
      const float* t = p.table + static_cast<int64_t>(pos) * p.rot;
      if (p.interleaved) {
        const float4 a = *reinterpret_cast<const float4*>(t + col * 4);
        const float4 b = *reinterpret_cast<const float4*>(t + half + col * 4);
        cs[0] = cs[1] = a.x; cs[2] = cs[3] = a.y; cs[4] = cs[5] = a.z; cs[6] = cs[7] = a.w;
        sn[0] = sn[1] = b.x; sn[2] = sn[3] = b.y; sn[4] = sn[5] = b.z; sn[6] = sn[7] = b.w;
      } else {
        const float* tc = t + (col * 8) % half;
        const float4 a = *reinterpret_cast<const float4*>(tc), b = *reinterpret_cast<const float4*>(tc + 4);
        const float4 c = *reinterpret_cast<const float4*>(tc + half), d = *reinterpret_cast<const float4*>(tc + half + 4);
        cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w; cs[4] = b.x; cs[5] = b.y; cs[6] = b.z; cs[7] = b.w;
        sn[0] = c.x; sn[1] = c.y; sn[2] = c.z; sn[3] = c.w; sn[4] = d.x; sn[5] = d.y; sn[6] = d.z; sn[7] = d.w;
      }
    }
    const bool second = col * 8 >= half;   // (half-split pairs) the lane holds the pairs' second channels
    const int partner = second ? lane - p.rot / 16 : lane + p.rot / 16;
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      const int h = run * NH + j;
      if (h >= heads) break;
      float f[8];
      widen8(f, raw[j]);
      const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
      if (kind < 2) {
        if (p.w[kind] != nullptr) norm8<D>(f, *reinterpret_cast<const uint4*>(p.w[kind] + col * 8), p.eps);
        if (p.table != nullptr) {
          float o[8];
          if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = f[i ^ 1];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, f[i], partner & 31);
          }
          if (turns) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const bool sub = p.interleaved ? (i & 1) == 0 : !second;
              const float a = __fmul_rn(f[i], cs[i]), b = __fmul_rn(o[i], sn[i]);
              f[i] = sub ? __fsub_rn(a, b) : __fadd_rn(a, b);
            }
          }
        }
        const uint4 y = round8(f);
        if (kind == 0) {
          if (r < p.c.rows && (pos >= 0 || p.zero_rest)) {
            const uint4 v = pos >= 0 ? y : make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(p.q_out + (static_cast<int64_t>(r) * p.Hq + h) * D + col * 8) = v;
          }
          continue;
        }
        widen8(f, y);
      }
      const int kh = h - p.Hq - (kind - 1) * p.Hkv, bits = p.bits[kh];
      const int64_t off = p.plane_off[kh] + store * (D * bits / 8) + col * bits;
      const int64_t si = (static_cast<int64_t>(kh) * storage + store) * G + col / 4;
      const bool live = store >= 0 && KVQ_IN_RANGE(off >= 0 && off + bits <= p.codes_bytes && si >= 0 &&
                                                       si < static_cast<int64_t>(p.Hkv) * storage * G, p.status);
      store_group(f, bits, live, p.codes[kind - 1] + off, p.sz[kind - 1] + si, col % 4 == 0, p.status);
    }
  }
}

}  // namespace

cudaError_t launch_rotate_append(const RotateArgs& a, cudaStream_t stream) {
  RParams p;
  const kvq_cache& k = *a.k;
  p.c = chunk::view_of(a.chunk, k);
  p.q = a.q;
  p.x[0] = a.k_new; p.x[1] = a.v_new;
  p.sq_row = a.sq_row; p.sq_head = a.sq_head; p.s_row = a.s_row; p.s_head = a.s_head;
  p.table = a.rot.table;
  p.w[0] = static_cast<const uint16_t*>(a.rot.q_weight);
  p.w[1] = static_cast<const uint16_t*>(a.rot.k_weight);
  p.q_out = a.q_out;
  p.codes[0] = k.codes; p.codes[1] = a.v->codes;
  p.sz[0] = k.sz; p.sz[1] = a.v->sz;
  p.status = a.status;
  p.Hq = a.Hq; p.Hkv = k.Hkv;
  p.positions = a.rot.positions;
  p.rot = a.rot.table != nullptr ? a.rot.rot_dim : 16;
  p.interleaved = a.rot.interleaved;
  p.eps = a.rot.eps;
  p.zero_rest = a.zero_rest ? 1 : 0;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * k.B * k.Tcap * (k.D / 2);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  const int R = 256 / k.D, heads = a.Hq + 2 * k.Hkv;
  p.tiles = (a.chunk.rows + R - 1) / R;
  // several heads a warp once that leaves a few warps an SM
  const bool many = p.tiles * ((heads + 3) / 4) >= 8 * device_sm_count();
  p.head_runs = many ? (heads + 3) / 4 : heads;
  const int64_t warps = p.tiles * p.head_runs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((warps + kWarps - 1) / kWarps, int64_t(1) << 30)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, p); };
  if (k.D == 128) return many ? launch(rotate_append_kernel<128, 4>) : launch(rotate_append_kernel<128, 1>);
  return many ? launch(rotate_append_kernel<64, 4>) : launch(rotate_append_kernel<64, 1>);
}

}  // namespace kvq
