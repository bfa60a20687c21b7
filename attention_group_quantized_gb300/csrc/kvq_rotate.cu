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
// is four lanes, which exchange quarters so that each has a head's whole group
// and works out its scale once.
//
// Measured: 32K rows of 32 + 8 + 8 heads, half of the channels turned, INT4, 722
// MB, 205 us, 3.5 TB/s (its floor is 107 us at 6.78 TB/s).  Neither HBM nor issue
// is full: 212 instructions a warp and head (the norm about 90, the rotation 45,
// a key's or value's quantisation 90) in chains, and 14 warps an SM (of the 16
// that 128 registers allow) that fill 60 % of its issue slots.
#include <algorithm>
#include <type_traits>

#include "kvq_chunk.cuh"
#include "kvq_group.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kBlocksPerSM = 4;   // (five or six, on fewer registers: the same)
// Warps an SM that are left where a warp takes four heads (one against four of
// them: 100 rows of 32 + 8 + 8 heads 4.6 and 4.9 us, 128 6.2 and 5.1, 400 11.6
// and 6.1; 512 rows of 4 + 1 + 1 heads 4.3 and 4.7, 1024 6.1 and 5.5) ...
constexpr int kWarpsPerSM = 4;
// ... and where it takes twice as many runs of rows: one, two, four and eight of
// them take, 48 heads, 560 rows: 9.1, 9.6, 13.3 and 20.9 us, 2048: 20.8, 19.8,
// 21.6 and 28.0, 4096: 38.3, 34.7, 35.0 and 40.3, 8192: 76.7, 66.6, 64.1 and
// 67.0, 32K: 270, 228, 210 and 205.
constexpr int kPassWarpsPerSM = 32;
constexpr int kMaxPasses = 8;

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
  int32_t Hq, Hkv, positions, rot;
  float eps;
  int32_t zero_rest;        // query rows of no usable sequence become zeros
  int32_t passes;           // runs of 32 / LPR rows that a warp takes one after the other
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

// The sum of a lane's eight squares over 2 D as s + e, exact likewise: half of
// what the lane adds to the mean, so that no sum across lanes passes fp32
// unless the mean does.  Added to a power of two M above the sum, a square is
// cut at M's last place: what the sum grew by is exact, what was cut off as
// well (both fused, so the square itself is never rounded), and the sums of
// the former stay exact.  Four two-wide instructions a pair of values.
__device__ __forceinline__ int top_exponent(const uint4& raw) {   // |x| < 2^(top - 126) for the lane's values
  const __nv_bfloat162 a = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x)), b = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
  const __nv_bfloat162 c = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw.z)), d = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&raw.w));
  const __nv_bfloat162 m2 = __hmax2(__hmax2(a, b), __hmax2(c, d));   // (drops NaN: the sum then is NaN anyway)
  const uint32_t m = *reinterpret_cast<const uint32_t*>(&m2);
  return static_cast<int>(max(m >> 16, m & 0xFFFFu) >> 7);
}
template <int D>
__device__ __forceinline__ void square_sum(float& s, float& e, int top, float2 (&f)[4]) {
  const bool large = top > 180;       // squares that near fp32's end or pass it: summed 2^-200 times as large
  if (large) {
    const float2 down = make_float2(0x1p-100f, 0x1p-100f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], down);
    top -= 100;
  }
  // four squares of at most 2^(2 top - 252) on each side of the pair: M = 2^(2 top - 249)
  const float M = __int_as_float(max(2 * top - 122, 1) << 23);
  const float2 minus = make_float2(-1.0f, -1.0f);
  float2 S = make_float2(M, M), E = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 next = __ffma2_rn(f[i], f[i], S);
    const float2 less = __ffma2_rn(next, minus, S);                    // minus what the sum grew by
    E = __fadd2_rn(E, __ffma2_rn(f[i], f[i], less));
    S = next;
  }
  s = __fadd_rn(__fsub_rn(S.x, M), __fsub_rn(S.y, M));
  e = __fadd_rn(E.x, E.y);
  float up = 0.5f / D;
  if (large) {                        // (the first 2^100 passes fp32 only where the lane's part of the mean does)
    s = __fmul_rn(s, 0x1p100f);
    e = __fmul_rn(e, 0x1p100f);
    up *= 0x1p100f;
  }
  const float2 se = __fmul2_rn(make_float2(s, e), make_float2(up, up));
  s = se.x;
  e = se.y;
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

__device__ __forceinline__ void widen8(float2 (&f)[4], const uint4& raw) {
  f[0] = bf16x2_to_float2(raw.x);
  f[1] = bf16x2_to_float2(raw.y);
  f[2] = bf16x2_to_float2(raw.z);
  f[3] = bf16x2_to_float2(raw.w);
}

__device__ __forceinline__ uint4 round8(const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / sqrt(mean + eps) of half a mean s + e.
__device__ __forceinline__ float inverse_root(float s, float e, float eps) {
  // (a half past fp32 is infinite; its error term is then no number)
  const float half = isinf(s) ? s : __fadd_rn(s, e);
  const float mean = __fmul_rn(half, 2.0f);   // exact, and infinite where the mean rounds to that
  return __frcp_rn(__fsqrt_rn(__fadd_rn(mean, eps)));
}

__device__ __forceinline__ void add_across(float& s, float& e, int o) {
  const float s2 = __shfl_xor_sync(0xffffffffu, s, o), e2 = __shfl_xor_sync(0xffffffffu, e, o);
  add_exact(s, e, s2);
  e = __fadd_rn(e, e2);
}

// The norms' factors of NH heads' rows, f[head] the lane's 8 channels.  Of four
// heads, the first two exchanges leave each quarter of a row's lanes with one
// head (half of the heads go each way), so that the rest, and the root, are
// worked out once for all of them.
template <int D, int NH>
__device__ __forceinline__ void norm_factors(float (&r)[NH], const uint4 (&raw)[NH], float eps, int lane) {
  constexpr int LPR = D / 8;
  float s[NH], e[NH];
#pragma unroll
  for (int j = 0; j < NH; ++j) {
    float2 f[4];
    widen8(f, raw[j]);
    square_sum<D>(s[j], e[j], top_exponent(raw[j]), f);
  }
  if constexpr (NH == 4) {
    const bool up = lane & (LPR / 2), right = lane & (LPR / 4);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float s2 = __shfl_xor_sync(0xffffffffu, up ? s[j] : s[j + 2], LPR / 2);
      const float e2 = __shfl_xor_sync(0xffffffffu, up ? e[j] : e[j + 2], LPR / 2);
      s[j] = up ? s[j + 2] : s[j];
      e[j] = up ? e[j + 2] : e[j];
      add_exact(s[j], e[j], s2);
      e[j] = __fadd_rn(e[j], e2);
    }
    const float s2 = __shfl_xor_sync(0xffffffffu, right ? s[0] : s[1], LPR / 4);
    const float e2 = __shfl_xor_sync(0xffffffffu, right ? e[0] : e[1], LPR / 4);
    float st = right ? s[1] : s[0], et = right ? e[1] : e[0];
    add_exact(st, et, s2);
    et = __fadd_rn(et, e2);
#pragma unroll
    for (int o = LPR / 8; o > 0; o >>= 1) add_across(st, et, o);
    const float mine = inverse_root(st, et, eps);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = __shfl_sync(0xffffffffu, mine, (lane & ~(LPR - 1)) + (j >> 1) * (LPR / 2) + (j & 1) * (LPR / 4));
  } else {
#pragma unroll
    for (int j = 0; j < NH; ++j) {
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) add_across(s[j], e[j], o);
      r[j] = inverse_root(s[j], e[j], eps);
    }
  }
}

// The 32 values of a lane's own group, from four lanes that hold a quarter of
// a group each of four heads: lane j of the four gets head j's.  (A 4 x 4
// transposition: pairs of lanes, then of pairs, exchange what is the other's.)
__device__ __forceinline__ void own_group(uint32_t (&w)[16], const uint4 (&y)[4], int lane) {
  uint32_t m[4][4];                   // [quarter][word], of the heads as they come
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j][0] = y[j].x; m[j][1] = y[j].y; m[j][2] = y[j].z; m[j][3] = y[j].w;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & o) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, up ? m[j][i] : m[j | o][i], o);
        if (up) m[j][i] = other;
        else m[j | o][i] = other;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * j + i] = m[j][i];
}

// The same for one head: every lane gets its group's values.
__device__ __forceinline__ void own_group(uint32_t (&w)[16], const uint4 (&y)[1], int lane) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int from = (lane & ~3) + j;
    w[4 * j] = __shfl_sync(0xffffffffu, y[0].x, from);
    w[4 * j + 1] = __shfl_sync(0xffffffffu, y[0].y, from);
    w[4 * j + 2] = __shfl_sync(0xffffffffu, y[0].z, from);
    w[4 * j + 3] = __shfl_sync(0xffffffffu, y[0].w, from);
  }
}

// A warp's unit: `passes` runs of 32 / LPR rows for NH heads of one kind (0
// queries, 1 keys, 2 values), h0 the first.  (One piece of code for all three:
// with a copy for each the kernel outgrew the instruction cache and took half as
// long again.  INTERLEAVED is its own instantiation for the same reason.)  The unit's rows (32 at most) are
// looked up at once, a lane each, and the next rows' loads are in flight while
// the present ones are worked on.
template <int D, int NH, bool INTERLEAVED>
__device__ __forceinline__ void unit_of(const RParams& p, int kind, int r0, int h0, bool reporter, int lane) {
  constexpr int G = D / 32;
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int R = 32 / LPR;         // rows per pass
  const int col = lane % LPR, half = p.rot / 2;
  const int count = min(NH, (kind == 0 ? p.Hq : p.Hkv) - h0);   // heads
  const int64_t s_row = kind == 0 ? p.sq_row : p.s_row, s_head = kind == 0 ? p.sq_head : p.s_head;
  const uint16_t* src = (kind == 0 ? p.q : p.x[kind - 1]) + (r0 + lane / LPR) * s_row + h0 * s_head + col * 8;
  // (the rows' loads need no look-up: rows of no sequence are read, not used)
  uint4 raw[NH];
  auto load = [&](int r) {
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      raw[j] = make_uint4(0u, 0u, 0u, 0u);
      if (r < p.c.rows && j < count) raw[j] = *reinterpret_cast<const uint4*>(src + j * s_head);
    }
    src += R * s_row;
  };
  load(r0 + lane / LPR);
  const Row mine = find_row(p, r0, lane, p.passes * R, reporter);
  const bool norm = kind < 2 && p.w[kind & 1] != nullptr;
  const bool rotate = kind < 2 && p.table != nullptr, turns = rotate && col * 8 < p.rot;
  const bool second = col * 8 >= half;   // (half-split pairs) the lane holds the pairs' second channels
  const int partner = (second ? lane - p.rot / 16 : lane + p.rot / 16) & 31;
  uint4 weight = make_uint4(0u, 0u, 0u, 0u);
  if (norm) weight = *reinterpret_cast<const uint4*>(p.w[kind & 1] + col * 8);
  const int64_t storage = static_cast<int64_t>(p.c.pB) * p.c.pT;
#pragma unroll 1
  for (int pass = 0; pass < p.passes && r0 + pass * R < p.c.rows; ++pass) {
    const int r = r0 + pass * R + lane / LPR;
    const int64_t store = __shfl_sync(0xffffffffu, mine.store, pass * R + lane / LPR);
    const int pos = __shfl_sync(0xffffffffu, mine.pos, pass * R + lane / LPR);
    uint4 y[NH];
#pragma unroll
    for (int j = 0; j < NH; ++j) y[j] = raw[j];
    if (pass + 1 < p.passes) load(r + R);
    if (norm || rotate) {
      float rn[NH];
      if (norm) norm_factors<D, NH>(rn, y, p.eps, lane);
      // cosines of the lane's channels, and what its partners are multiplied by:
      // minus the sine for a pair's first channel, the sine for its second
      float2 cs[4], sn[4];
      if (turns && pos >= 0) {
        const float* t = p.table + static_cast<int64_t>(pos) * p.rot;
        if constexpr (INTERLEAVED) {
          const float4 a = *reinterpret_cast<const float4*>(t + col * 4);
          const float4 b = *reinterpret_cast<const float4*>(t + half + col * 4);
          cs[0] = make_float2(a.x, a.x); cs[1] = make_float2(a.y, a.y); cs[2] = make_float2(a.z, a.z); cs[3] = make_float2(a.w, a.w);
          sn[0] = make_float2(-b.x, b.x); sn[1] = make_float2(-b.y, b.y); sn[2] = make_float2(-b.z, b.z); sn[3] = make_float2(-b.w, b.w);
        } else {
          const float* tc = t + (second ? col * 8 - half : col * 8);
          const float4 a = *reinterpret_cast<const float4*>(tc), b = *reinterpret_cast<const float4*>(tc + 4);
          const float4 c = *reinterpret_cast<const float4*>(tc + half), d = *reinterpret_cast<const float4*>(tc + half + 4);
          const float sg = second ? 1.0f : -1.0f;
          cs[0] = make_float2(a.x, a.y); cs[1] = make_float2(a.z, a.w); cs[2] = make_float2(b.x, b.y); cs[3] = make_float2(b.z, b.w);
          sn[0] = make_float2(sg * c.x, sg * c.y); sn[1] = make_float2(sg * c.z, sg * c.w);
          sn[2] = make_float2(sg * d.x, sg * d.y); sn[3] = make_float2(sg * d.z, sg * d.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cs[i] = make_float2(1.0f, 1.0f);
          sn[i] = make_float2(0.0f, 0.0f);
        }
      }
      float2 w[4];
      widen8(w, weight);
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        float2 f[4];
        widen8(f, y[j]);
        if (norm) {
          const float2 r2 = make_float2(rn[j], rn[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(__fmul2_rn(f[i], r2), w[i]);
        }
        if (rotate) {
          float2 o[4];
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_float2(f[i].y, f[i].x);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[i].x = __shfl_sync(0xffffffffu, f[i].x, partner);
              o[i].y = __shfl_sync(0xffffffffu, f[i].y, partner);
            }
          }
          if (turns) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (one-wide sums: two-wide ones were fused with the products, `.rn` or not)
              const float2 a = __fmul2_rn(f[i], cs[i]), b = __fmul2_rn(o[i], sn[i]);
              f[i] = make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
            }
          }
        }
        y[j] = round8(f);
      }
    }
    if (kind == 0) {
      if (r < p.c.rows && (pos >= 0 || p.zero_rest)) {
        uint16_t* dst = p.q_out + (static_cast<int64_t>(r) * p.Hq + h0) * D + col * 8;
#pragma unroll
        for (int j = 0; j < NH; ++j)
          if (j < count) *reinterpret_cast<uint4*>(dst + j * D) = pos >= 0 ? y[j] : make_uint4(0u, 0u, 0u, 0u);
      }
    } else {
      uint32_t v[16];
      own_group(v, y, lane);
      const int j = NH == 1 ? 0 : lane & 3, h = h0 + j;
      if (j < count && store >= 0 && (NH > 1 || (lane & 3) == 0)) {
        const int bits = p.bits[h];
        const int64_t off = p.plane_off[h] + store * (D * bits / 8) + col / 4 * (4 * bits);
        const int64_t si = (static_cast<int64_t>(h) * storage + store) * G + col / 4;
        if (KVQ_IN_RANGE(off >= 0 && off + 4 * bits <= p.codes_bytes && si >= 0 &&
                             si < static_cast<int64_t>(p.Hkv) * storage * G, p.status))
          quantize_group_of(v, [&](int i) {
            return i == 0 ? make_uint4(v[0], v[1], v[2], v[3]) : i == 1 ? make_uint4(v[4], v[5], v[6], v[7])
                 : i == 2 ? make_uint4(v[8], v[9], v[10], v[11]) : make_uint4(v[12], v[13], v[14], v[15]);
          }, bits, p.codes[kind - 1] + off, p.sz[kind - 1] + si, p.status);
      }
    }
  }
}

template <int D, int NH, bool INTERLEAVED>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSM) rotate_append_kernel(const __grid_constant__ RParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, blockDim.x, p.status);
  const int q_runs = (p.Hq + NH - 1) / NH, kv_runs = (p.Hkv + NH - 1) / NH;   // runs of heads: of one kind each
  const int runs = q_runs + 2 * kv_runs;
  const int64_t units = p.tiles * runs;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int tile = static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(runs));
    const int run = static_cast<int>(static_cast<uint32_t>(u) - static_cast<uint32_t>(tile) * runs);
    const int r0 = tile * p.passes * (256 / D);
    const int kind = run < q_runs ? 0 : run < q_runs + kv_runs ? 1 : 2;
    const int first = kind == 0 ? run : run - q_runs - (kind - 1) * kv_runs;
    unit_of<D, NH, INTERLEAVED>(p, kind, r0, first * NH, run == 0, lane);
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
  p.eps = a.rot.eps;
  p.zero_rest = a.zero_rest ? 1 : 0;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * k.B * k.Tcap * (k.D / 2);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  // several heads, and then several runs of rows, a warp where that leaves
  // warps enough to fill the GPU
  const int R = 256 / k.D;
  const int64_t want = int64_t(kWarpsPerSM) * device_sm_count(), runs = (a.chunk.rows + R - 1) / R;
  const int fours = (a.Hq + 3) / 4 + 2 * ((k.Hkv + 3) / 4);
  const bool many = runs * fours >= want;
  const int64_t heads = many ? fours : a.Hq + 2 * k.Hkv;
  p.passes = 1;
  while (p.passes < kMaxPasses && runs * heads >= int64_t(2 * kPassWarpsPerSM) * device_sm_count() * p.passes) p.passes *= 2;
  p.tiles = (runs + p.passes - 1) / p.passes;
  const int64_t warps = p.tiles * heads;
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
  auto choose = [&](auto d, auto nh) {
    constexpr int D = decltype(d)::value, NH = decltype(nh)::value;
    return a.rot.interleaved ? launch(rotate_append_kernel<D, NH, true>) : launch(rotate_append_kernel<D, NH, false>);
  };
  using std::integral_constant;
  if (k.D == 128)
    return many ? choose(integral_constant<int, 128>{}, integral_constant<int, 4>{})
                : choose(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  return many ? choose(integral_constant<int, 64>{}, integral_constant<int, 4>{})
              : choose(integral_constant<int, 64>{}, integral_constant<int, 1>{});
}

}  // namespace kvq
