// kvq_quantize.cu -- quantise-on-write of bf16 K/V rows into the group-quantised
// cache (《分块稀疏注意力与KV Cache量化：长文本推理显存优化实践》 §2.4, group of 32
// channels per the hook of §3.2), and per-head quantisation-error statistics
// for the per-head bit allocation of the same section.
//
// HBM-bound: every input byte is read once and every code/scale byte written
// once.  One thread quantises one group of 32 channels on its own: four
// 16-byte loads, the group's range, one IEEE division for the scale, then
// each code from x times an approximate reciprocal of the scale, rounded by a
// 1.5 * 2^23 addend inside the same FMA, two values per instruction (paired
// fp32).  The exact remainder x - u * s tells whether that rounding is the
// specification's (see rne_div); the rare quarter-groups where it might not
// be are redone value by value.  One 32-byte (INT8) or 16-byte (INT4) store
// of codes per group; a warp's stores cover whole contiguous rows.  The result
// is bit-identical to the specification's IEEE fp32 arithmetic.
#include <algorithm>

#include "kvq_chunk.cuh"
#include "kvq_device.cuh"
#include "kvq_group.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// Division of 32-bit unsigned numerators by a divisor fixed for the launch
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994, the round-up multiplier of their Figure 4.1):
// with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
//   q = (t + ((n - t) >> 1)) >> (l - 1),  t = mulhi(m, n),   for d >= 2.
struct FastDiv {
  uint32_t d, m, l;
  static FastDiv make(uint32_t d) {
    FastDiv f;
    f.d = d;
    f.l = 0;
    while ((uint64_t(1) << f.l) < d) ++f.l;
    f.m = d <= 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << f.l) - d)) / d + 1);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    if (d <= 1) return n;
    const uint32_t t = __umulhi(m, n);
    return (t + ((n - t) >> 1)) >> (l - 1);
  }
};

struct QParams {
  FastDiv div_nt, div_hkv;   // row -> (b, h, t): row = (b * Hkv + h) * nt + t
  // optional block table: the cache is a pool of B pages of Tcap = 64 tokens
  // and sequence b's token t sits in page bt[b * bt_stride + t / 64]
  const int32_t* bt;
  int32_t bt_stride;
  const int32_t* lens;      // optional per-sequence lengths (contiguous caches only)
  const uint16_t* x;
  int64_t sx_b, sx_h, sx_t;
  uint8_t* codes;
  uint32_t* sz;
  int32_t* status;
  int32_t B, Hkv, Tcap, t0, nt;
  int64_t rows;
  int64_t codes_bytes;      // size of the code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

// Debug build: a group's codes (nbytes from byte offset off) and its
// scale/zero word (index si) inside their buffers.
__device__ __forceinline__ bool group_dst_ok(int64_t off, int nbytes, int64_t si, int64_t codes_bytes,
                                             int64_t sz_words, int32_t* status) {
  return KVQ_IN_RANGE(off >= 0 && off + nbytes <= codes_bytes && si >= 0 && si < sz_words, status);
}

// Load one group of 32 bf16 values (64 bytes, 16-byte aligned source) as 16
// words of raw bf16 pairs; they stay packed and are widened where used.
__device__ __forceinline__ void load_group(uint32_t (&w)[16], const uint16_t* src) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const uint4 raw = reinterpret_cast<const uint4*>(src)[v];
    w[4 * v] = raw.x; w[4 * v + 1] = raw.y; w[4 * v + 2] = raw.z; w[4 * v + 3] = raw.w;
  }
}

// quantize_group_of values loaded by load_group from src.
__device__ __forceinline__ void quantize_group(const uint32_t (&w)[16], const uint16_t* src, int bits, uint8_t* cdst,
                                               uint32_t* szw, int32_t* status) {
  quantize_group_of(w, [&](int v) { return reinterpret_cast<const uint4*>(src)[v]; }, bits, cdst, szw, status);
}

// Squared quantisation error of one group, sum_i (x_i - x_hat_i)^2 with
// x_hat = (code - z) * s the value the cache would hold at `bits` bits, and
// its squared norm sum_i x_i^2, two values per instruction.  With u and d as
// in quantize_group, x - x_hat = d wherever |d| <= s / 2 and no code is
// clamped (at a tie, |d| = s / 2, either neighbour gives the same error).  A
// quarter with some |d| > s / 2, or a NaN, or a clamped group, is redone with
// code_exact.  Each square-and-add rounds once.
__device__ __forceinline__ float2 group_sq_error(const uint32_t (&w)[16], const uint16_t* src, int bits, bool& bad) {
  const GroupParams gp = group_params(w, bits);
  bad |= gp.bad;
  if (gp.flat) {   // every value 0 (x_hat = 0): no error; a NaN among zeros is reported
    bad |= group_has_nan(w);
    return make_float2(0.0f, 0.0f);
  }
  const float2 r2 = make_float2(gp.rcp, gp.rcp), c2 = make_float2(gp.C, gp.C);
  const float2 nc2 = make_float2(-gp.C, -gp.C), ns2 = make_float2(-gp.sf, -gp.sf);
  const float hs = 0.5f * gp.sf;
  float2 nrm2 = make_float2(0.0f, 0.0f);
  float errq[4];
  unsigned redo = 0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float2 err2 = make_float2(0.0f, 0.0f);
    float dmax = 0.0f;
#pragma unroll
    for (int k = 4 * v; k < 4 * v + 4; ++k) {
      const float2 x2 = bf16x2_to_float2(w[k]);
      nrm2 = __ffma2_rn(x2, x2, nrm2);
      const float2 d2 = __ffma2_rn(__fadd2_rn(__ffma2_rn(x2, r2, c2), nc2), ns2, x2);
      dmax = fmaxf(dmax, fmaxf(fabsf(d2.x), fabsf(d2.y)));
      err2 = __ffma2_rn(d2, d2, err2);
    }
    errq[v] = __fadd_rn(err2.x, err2.y);
    redo |= (dmax <= hs && errq[v] == errq[v] ? 0u : 1u) << v;   // a NaN makes the sum NaN
  }
  if (group_clamps(gp)) redo = 0xFu;
  if (redo != 0u) {
    const int zero = static_cast<int>(gp.zf);
#pragma unroll 1
    for (int v = 0; v < 4; ++v) {
      if (!((redo >> v) & 1u)) continue;
      float e = 0.0f;
      quarter_values(reinterpret_cast<const uint4*>(src)[v], [&](int, float x) {
        bad |= x != x;
        const float d = __fmaf_rn(-static_cast<float>(code_exact(x, gp) - zero), gp.sf, x);
        e = __fmaf_rn(d, d, e);
      });
      errq[v] = e;
    }
  }
  return make_float2(__fadd_rn(__fadd_rn(errq[0], errq[1]), __fadd_rn(errq[2], errq[3])),
                     __fadd_rn(nrm2.x, nrm2.y));
}

// resident blocks of 256 threads per SM the register budget is sized for (tunable at build time)
#ifndef KVQ_QUANT_MIN_BLOCKS
#define KVQ_QUANT_MIN_BLOCKS 5
#endif

// One thread per (row, group): row = (b * Hkv + h) * nt + t.  (A persistent
// loop that issued the next group's loads before this group's arithmetic
// measured slower: the extra registers cost more occupancy than it gained.)
// PAGED: the cache is a page pool addressed through p.bt; LENS: rows at
// positions t0 + t >= p.lens[b] are not quantised, and those before the end
// of that length's 128-token tile are cleared (codes and scale/zero word 0,
// which dequantise to exact zeros for the prefill's last tile); separate
// instantiations, so the plain kernel carries none of it.
template <int D, bool PAGED, bool LENS>
__global__ void __launch_bounds__(256, KVQ_QUANT_MIN_BLOCKS) quantize_kernel(const __grid_constant__ QParams p) {
  constexpr int G = D / 32;
  const int64_t n = p.rows * G;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const uint32_t r = static_cast<uint32_t>(i / G);
    const int g = static_cast<int>(i % G);
    const uint32_t bh = p.div_nt.div(r);
    const int t = static_cast<int>(r - bh * p.div_nt.d);
    const uint32_t bq = p.div_hkv.div(bh);
    const int h = static_cast<int>(bh - bq * p.div_hkv.d);
    const int b = static_cast<int>(bq);
    const int bits = p.bits[h];
    int64_t pos = static_cast<int64_t>(b) * p.Tcap + p.t0 + t;
    if constexpr (LENS) {
      const int len = min(max(p.lens[b], 0), p.Tcap);
      if (p.t0 + t >= len) {
        const int64_t off = p.plane_off[h] + pos * (D * bits / 8) + g * (32 * bits / 8);
        const int64_t si = (static_cast<int64_t>(h) * p.B * p.Tcap + pos) * G + g;
        if (p.t0 + t < ((len + 127) & ~127) &&
            group_dst_ok(off, 4 * bits, si, p.codes_bytes, static_cast<int64_t>(p.Hkv) * p.B * p.Tcap * G, p.status)) {
          uint4* dst = reinterpret_cast<uint4*>(p.codes + off);
          dst[0] = make_uint4(0u, 0u, 0u, 0u);
          if (bits == 8) dst[1] = make_uint4(0u, 0u, 0u, 0u);
          p.sz[si] = 0u;
        }
        continue;
      }
    }
    if constexpr (PAGED) {
      const int tl = p.t0 + t;
      if (!KVQ_IN_RANGE(tl / 64 < p.bt_stride, p.status)) continue;
      const int page = p.bt[static_cast<int64_t>(b) * p.bt_stride + tl / 64];
      if (page < 0 || page >= p.B) {   // a page outside the pool: report, write nothing
        if (g == 0) report(p.status, KVQ_ERR_INVALID_ARG);
        continue;
      }
      pos = static_cast<int64_t>(page) * 64 + tl % 64;
    }
    const int64_t off = p.plane_off[h] + pos * (D * bits / 8) + g * (32 * bits / 8);
    const int64_t si = (static_cast<int64_t>(h) * p.B * p.Tcap + pos) * G + g;
    if (!group_dst_ok(off, 4 * bits, si, p.codes_bytes, static_cast<int64_t>(p.Hkv) * p.B * p.Tcap * G, p.status))
      continue;
    uint32_t w[16];
    const uint16_t* src = p.x + b * p.sx_b + h * p.sx_h + t * p.sx_t + g * 32;
    load_group(w, src);
    quantize_group(w, src, bits, p.codes + off, p.sz + si, p.status);
  }
}

// Append: the new token of every (sequence b, KV head h) of K and of V, rows
// [k rows | v rows] of [b][h], written at cache position seq_lens[b] - 1.
struct AParams {
  const int32_t* bt;        // optional block table (the caches are page pools), as in QParams
  int32_t bt_stride;
  const uint4* q_src;       // optional: q vectors to stage for the decode (host memory read in place)
  uint4* q_dst;
  int64_t q_vec;            // 16-byte vectors to copy
  const uint16_t* x[2];     // k_new, v_new: bf16 [B][Hkv][D]
  uint8_t* codes[2];
  uint32_t* sz[2];
  const int32_t* seq_lens;
  int32_t* status;
  int32_t B, Hkv, Tcap;     // storage: B sequences (or pages) of Tcap tokens
  int32_t nseq, cap;        // sequences and their capacity in tokens
  int64_t codes_bytes;      // size of each code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

template <int D, bool PAGED>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AParams p) {
  constexpr int G = D / 32;
  // the decode launched after this kernel may begin its prologue now; it
  // waits for this grid's completion before reading memory
  grid_launch_dependents();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < p.q_vec;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    p.q_dst[i] = p.q_src[i];
  const int64_t bhn = static_cast<int64_t>(p.nseq) * p.Hkv;
  const int64_t n = 2 * bhn * G;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / G;                 // [k rows | v rows] of [b][h]
    const int g = static_cast<int>(i % G);
    const int job = static_cast<int>(r / bhn);
    const int64_t bh = r % bhn;
    const int h = static_cast<int>(bh % p.Hkv);
    const int b = static_cast<int>(bh / p.Hkv);
    const int len = p.seq_lens[b];
    if (len < 1 || len > p.cap) {
      if (job == 0 && h == 0 && g == 0) report(p.status, KVQ_ERR_INVALID_ARG);
      continue;
    }
    const int bits = p.bits[h];
    int64_t pos = static_cast<int64_t>(b) * p.Tcap + len - 1;
    if constexpr (PAGED) {
      if (!KVQ_IN_RANGE((len - 1) / 64 < p.bt_stride, p.status)) continue;
      const int page = p.bt[static_cast<int64_t>(b) * p.bt_stride + (len - 1) / 64];
      if (page < 0 || page >= p.B) {
        if (job == 0 && h == 0 && g == 0) report(p.status, KVQ_ERR_INVALID_ARG);
        continue;
      }
      pos = static_cast<int64_t>(page) * 64 + (len - 1) % 64;
    }
    const int64_t off = p.plane_off[h] + pos * (D * bits / 8) + g * (32 * bits / 8);
    const int64_t si = (static_cast<int64_t>(h) * p.B * p.Tcap + pos) * G + g;
    if (!group_dst_ok(off, 4 * bits, si, p.codes_bytes, static_cast<int64_t>(p.Hkv) * p.B * p.Tcap * G, p.status))
      continue;
    uint32_t w[16];
    const uint16_t* src = p.x[job] + bh * D + g * 32;
    load_group(w, src);
    quantize_group(w, src, bits, p.codes[job] + off, p.sz[job] + si, p.status);
  }
}

// Append of a chunk: packed rows of K and V ([row][head], strided) written at
// their sequences' positions.  One thread per group of 32 channels, as in
// quantize_kernel; a warp takes one KV head and 32 / G consecutive rows, so
// that its code stores cover whole consecutive cache rows and its scale/zero
// stores one contiguous run, while its loads are whole 128- or 256-byte rows.
// The rows' positions are looked up once per warp, a lane per row.
struct ACParams {
  chunk::View c;
  const uint16_t* x[2];     // k_new, v_new
  int64_t s_row, s_head;
  uint8_t* codes[2];
  uint32_t* sz[2];
  int32_t* status;
  int32_t Hkv;
  int32_t tiles;            // runs of 32 / G rows
  int64_t codes_bytes;      // size of each code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

constexpr int kAppendWarps = 4;   // per block (eight: 53.4 us for 176 MB against 51.6)

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32, 2 * KVQ_QUANT_MIN_BLOCKS) append_chunk_kernel(const __grid_constant__ ACParams p) {
  constexpr int G = D / 32;
  constexpr int R = 32 / G;                   // rows per warp
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, blockDim.x, p.status);
  const int64_t nw = static_cast<int64_t>(p.tiles) * p.Hkv * 2;
  const int64_t storage = static_cast<int64_t>(p.c.pB) * p.c.pT;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5); u < nw;
       u += static_cast<int64_t>(gridDim.x) * kAppendWarps) {
    const int job = static_cast<int>(u & 1);  // K and V of the same rows side by side: they share the look-up's lines
    const uint32_t th = static_cast<uint32_t>(u >> 1);
    const int tile = static_cast<int>(th / static_cast<uint32_t>(p.Hkv));
    const int h = static_cast<int>(th - static_cast<uint32_t>(tile) * p.Hkv);
    const int r0 = tile * R;
    const int64_t mine = chunk::locate_rows(p.c, r0, lane, R, h == 0 && job == 0, p.status);
    const int64_t pos = __shfl_sync(0xffffffffu, mine, lane / G);
    if (pos < 0) continue;
    const int g = lane % G, bits = p.bits[h];
    const int64_t off = p.plane_off[h] + pos * (D * bits / 8) + g * (32 * bits / 8);
    const int64_t si = (static_cast<int64_t>(h) * storage + pos) * G + g;
    if (!group_dst_ok(off, 4 * bits, si, p.codes_bytes, static_cast<int64_t>(p.Hkv) * storage * G, p.status)) continue;
    uint32_t w[16];
    const uint16_t* src = p.x[job] + (r0 + lane / G) * p.s_row + h * p.s_head + g * 32;
    load_group(w, src);
    quantize_group(w, src, bits, p.codes[job] + off, p.sz[job] + si, p.status);
  }
}

// Per-head error statistics: grid (chunks, H); block (c, h) takes groups
// c * 256 + tid, then every chunks * 256, of head h's B * T * G groups
// (row r = b * T + t, group g), and writes its (error, norm) sums in fp64 to
// part[h][c]; head_stats_reduce adds the chunks in a fixed order, so the
// result does not depend on scheduling.
struct SParams {
  FastDiv div_t;            // r -> (b, t)
  const uint16_t* x;        // bf16 [B][H][T][D]
  const float* w;           // [B][H][T] or null (1)
  const int32_t* lens;      // [B] or null (T)
  double* part;             // [H][chunks][2]
  int32_t* status;
  int32_t B, H, T, bits, chunks;
};

constexpr int kStatThreads = 256;
// Resident blocks the register budget is sized for.  Measured alternatives
// (3, 5 or 6 blocks; two groups per iteration; a register prefetch of the
// next group) were no faster.
constexpr int kStatBlocksPerSM = 4;

template <int D>
__global__ void __launch_bounds__(kStatThreads, kStatBlocksPerSM) head_stats_kernel(const __grid_constant__ SParams p) {
  constexpr int G = D / 32;
  const int h = blockIdx.y;
  // the reduction launched after this kernel may be scheduled now; it waits
  // for this grid's completion before reading the partial sums
  grid_launch_dependents();
  const int64_t n = static_cast<int64_t>(p.B) * p.T * G;
  // (error, norm) summed in fp32 with Kahan's compensation (sum - comp is the
  // running total), widened to fp64 once for the block's reduction
  float2 sum = make_float2(0.0f, 0.0f), comp = make_float2(0.0f, 0.0f);
  const float2 m1 = make_float2(-1.0f, -1.0f);
  bool bad = false;
  auto accumulate = [&](float2 e, float wt) {
    e = __fmul2_rn(e, make_float2(wt, wt));
    const float2 y = __ffma2_rn(comp, m1, e);              // e - comp
    const float2 nsum = __fadd2_rn(sum, y);
    comp = __ffma2_rn(y, m1, __ffma2_rn(sum, m1, nsum));   // (nsum - sum) - y
    sum = nsum;
  };
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kStatThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(p.chunks) * kStatThreads) {
    const uint32_t r = static_cast<uint32_t>(i / G);
    const int g = static_cast<int>(i % G);
    const uint32_t b = p.div_t.div(r);
    const int t = static_cast<int>(r - b * p.div_t.d);
    if (p.lens != nullptr && t >= p.lens[b]) continue;
    const int64_t row = (static_cast<int64_t>(b) * p.H + h) * p.T + t;
    uint32_t v[16];
    const uint16_t* src = p.x + row * D + g * 32;
    load_group(v, src);
    accumulate(group_sq_error(v, src, p.bits, bad), p.w != nullptr ? p.w[row] : 1.0f);
  }
  if (bad) report(p.status, KVQ_ERR_NONFINITE);
  // the block's sum in fp32 (a tree of depth 8 over compensated per-thread
  // totals: a few units of 2^-24 relative), then fp64 across blocks (the fp64
  // pipe is narrow, so it is kept out of the per-thread tail)
  float2 tot = __ffma2_rn(comp, m1, sum);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tot.x = __fadd_rn(tot.x, __shfl_down_sync(0xffffffffu, tot.x, o));
    tot.y = __fadd_rn(tot.y, __shfl_down_sync(0xffffffffu, tot.y, o));
  }
  __shared__ float2 red[kStatThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[warp] = tot;
  __syncthreads();
  if (threadIdx.x == 0) {
    double e = 0.0, m = 0.0;
    for (int k = 0; k < kStatThreads / 32; ++k) { e += static_cast<double>(red[k].x); m += static_cast<double>(red[k].y); }
    double* out = p.part + (static_cast<int64_t>(h) * p.chunks + blockIdx.x) * 2;
    out[0] = e;
    out[1] = m;
  }
}

// One warp per head: stats[h] = the sum of part[h][0 .. chunks) in a fixed order.
__global__ void __launch_bounds__(32) head_stats_reduce(const double* part, int chunks, double* stats) {
  const int h = blockIdx.x, lane = threadIdx.x;
  grid_dependency_wait();   // launched as a dependent of head_stats_kernel
  double e = 0.0, m = 0.0;
  for (int c = lane; c < chunks; c += 32) {
    e += part[(static_cast<int64_t>(h) * chunks + c) * 2];
    m += part[(static_cast<int64_t>(h) * chunks + c) * 2 + 1];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    e += __shfl_xor_sync(0xffffffffu, e, o);
    m += __shfl_xor_sync(0xffffffffu, m, o);
  }
  if (lane == 0) {
    stats[2 * h] = e;
    stats[2 * h + 1] = m;
  }
}

}  // namespace

int head_stats_chunks(int B, int H, int T, int D) {
  const int64_t groups = static_cast<int64_t>(B) * T * (D / 32);
  // one resident wave over all heads
  int64_t c = (static_cast<int64_t>(device_sm_count()) * kStatBlocksPerSM + H - 1) / H;
  const int64_t need = (groups + kStatThreads - 1) / kStatThreads;
  if (c > need) c = need;
  if (c > kHeadStatsMaxChunks) c = kHeadStatsMaxChunks;
  return c < 1 ? 1 : static_cast<int>(c);
}

cudaError_t launch_head_stats(const HeadStatsArgs& a, cudaStream_t stream) {
  SParams p;
  p.div_t = FastDiv::make(static_cast<uint32_t>(a.T));
  p.x = a.x; p.w = a.w; p.lens = a.lens;
  p.part = a.part; p.status = a.status;
  p.B = a.B; p.H = a.H; p.T = a.T; p.bits = a.bits;
  p.chunks = head_stats_chunks(a.B, a.H, a.T, a.D);
  const dim3 grid(static_cast<unsigned>(p.chunks), static_cast<unsigned>(a.H));
  if (a.D == 128) head_stats_kernel<128><<<grid, kStatThreads, 0, stream>>>(p);
  else head_stats_kernel<64><<<grid, kStatThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the fixed-order sum, launched while the statistics kernel still runs
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.H));
  cfg.blockDim = dim3(32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, head_stats_reduce, static_cast<const double*>(a.part), p.chunks, a.stats);
}

cudaError_t launch_quantize(const QuantizeArgs& a, cudaStream_t stream) {
  QParams p;
  p.x = a.x;
  p.sx_b = a.sx_b; p.sx_h = a.sx_h; p.sx_t = a.sx_t;
  p.codes = a.codes; p.sz = a.sz; p.status = a.status;
  p.B = a.B; p.Hkv = a.Hkv; p.Tcap = a.Tcap; p.t0 = a.t0; p.nt = a.nt;
  p.bt = a.bt;
  p.bt_stride = a.bt_max_pages;
  p.lens = a.lens;
  if (p.lens != nullptr && p.bt != nullptr) return cudaErrorInvalidValue;
  p.rows = static_cast<int64_t>(a.bt != nullptr ? a.bt_B : a.B) * a.Hkv * a.nt;
  if (p.rows >= (int64_t(1) << 31)) return cudaErrorInvalidValue;   // rows are indexed in 32 bits
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * a.B * a.Tcap * (a.D / 2);
  p.div_nt = FastDiv::make(static_cast<uint32_t>(a.nt));
  p.div_hkv = FastDiv::make(static_cast<uint32_t>(a.Hkv));
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  if (p.rows == 0) return cudaSuccess;
  int64_t blocks = (p.rows * (a.D / 32) + 255) / 256;   // one thread per (row, group)
  const int64_t cap = int64_t(1) << 30;                   // grid-stride beyond that
  if (blocks > cap) blocks = cap;
  const unsigned g = static_cast<unsigned>(blocks);
  if (a.D == 128) {
    if (p.bt != nullptr) quantize_kernel<128, true, false><<<g, 256, 0, stream>>>(p);
    else if (p.lens != nullptr) quantize_kernel<128, false, true><<<g, 256, 0, stream>>>(p);
    else quantize_kernel<128, false, false><<<g, 256, 0, stream>>>(p);
  } else {
    if (p.bt != nullptr) quantize_kernel<64, true, false><<<g, 256, 0, stream>>>(p);
    else if (p.lens != nullptr) quantize_kernel<64, false, true><<<g, 256, 0, stream>>>(p);
    else quantize_kernel<64, false, false><<<g, 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  AParams p;
  p.q_src = static_cast<const uint4*>(a.q_src);
  p.q_dst = static_cast<uint4*>(a.q_dst);
  p.q_vec = a.q_src != nullptr ? static_cast<int64_t>(a.q_bytes / 16) : 0;
  p.x[0] = a.k_new; p.x[1] = a.v_new;
  p.codes[0] = a.k_codes; p.codes[1] = a.v_codes;
  p.sz[0] = a.k_sz; p.sz[1] = a.v_sz;
  p.seq_lens = a.seq_lens;
  p.status = a.status;
  p.B = a.B; p.Hkv = a.Hkv; p.Tcap = a.Tcap;
  p.bt = a.bt;
  p.bt_stride = a.bt_max_pages;
  p.nseq = a.bt != nullptr ? a.bt_B : a.B;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * a.B * a.Tcap * (a.D / 2);
  p.cap = a.bt != nullptr ? a.bt_max_pages * 64 : a.Tcap;
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  const int64_t rows = 2 * static_cast<int64_t>(p.nseq) * a.Hkv;
  int64_t blocks = (rows * (a.D / 32) + 255) / 256;   // one thread per (row, group)
  const int64_t qblocks = (p.q_vec + 255) / 256;   // one 16-byte vector per thread
  if (qblocks > blocks) blocks = qblocks;
  const int64_t cap = static_cast<int64_t>(device_sm_count()) * 16;
  if (blocks > cap) blocks = cap;
  const unsigned g = static_cast<unsigned>(blocks);
  if (a.D == 128) {
    if (p.bt != nullptr) append_kernel<128, true><<<g, 256, 0, stream>>>(p);
    else append_kernel<128, false><<<g, 256, 0, stream>>>(p);
  } else {
    if (p.bt != nullptr) append_kernel<64, true><<<g, 256, 0, stream>>>(p);
    else append_kernel<64, false><<<g, 256, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_append_chunk(const AppendChunkArgs& a, cudaStream_t stream) {
  ACParams p;
  p.c = chunk::view_of(a.chunk, *a.k);
  p.x[0] = a.k_new; p.x[1] = a.v_new;
  p.s_row = a.s_row; p.s_head = a.s_head;
  p.codes[0] = a.k->codes; p.codes[1] = a.v->codes;
  p.sz[0] = a.k->sz; p.sz[1] = a.v->sz;
  p.status = a.status;
  p.Hkv = a.k->Hkv;
  const int R = 32 / (a.k->D / 32);
  p.tiles = (a.chunk.rows + R - 1) / R;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * a.k->B * a.k->Tcap * (a.k->D / 2);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  // one warp per (run of rows, head, K or V); grid-stride beyond 2^30 blocks
  const int64_t warps = static_cast<int64_t>(p.tiles) * p.Hkv * 2;
  const int64_t blocks = std::min<int64_t>((warps + kAppendWarps - 1) / kAppendWarps, int64_t(1) << 30);
  const unsigned g = static_cast<unsigned>(blocks);
  if (a.k->D == 128) append_chunk_kernel<128><<<g, kAppendWarps * 32, 0, stream>>>(p);
  else append_chunk_kernel<64><<<g, kAppendWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kvq
