// kvq_blocks.cu -- which 64-token blocks of a cached sequence a query needs:
// every block's channel bounds kept in 8 bits beside the K cache, a score per
// block from them, and the n best blocks of each query row and KV head.  (The
// pages' block-sparse attention skips whole key tiles judged unnecessary,
// 《分块稀疏注意力与KV Cache量化：长文本推理显存优化实践》 §1.3, §2.3; this is a
// judgement made at decode time, per query.)
//
// The score bounds the best product that any token of the block can give, but
// for the rounding of the query to 8 bits:
//   sum_h q_h . k <= sum_d qp_d max_d + qn_d min_d,
//   qp = sum_h max(q_h, 0), qn = sum_h min(q_h, 0)
// over the query heads h of a KV head, so a group of heads costs no more than
// one.  Bounds and query are held in 8 bits with a scale per 32 channels; the
// products of whole numbers are exact, and the few fp32 operations that join
// the groups have a fixed order: a selection is a function of the inputs.
#include <algorithm>

#include "kvq_chunk.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// bounds of blocks
// ---------------------------------------------------------------------------

constexpr int kBoundsWarps = 4;
constexpr int kBoundsBlocks = 8;    // an SM (four prompts of 32K: 8 38.5 us, 6 40.0, 5 44.0)

struct BParams {
  chunk::View c;
  const uint8_t* codes;
  const uint32_t* sz;
  int8_t* b_codes;
  float* b_scales;
  int32_t* status;
  int32_t Hkv;
  int64_t tiles;            // runs of R rows
  int64_t codes_bytes;      // size of the code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max2(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min2(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The 8 values (c - z) s of a lane's codes, exact in fp32 (9 + 11 significant
// bits): the fp32 with the bits 0x4B0000cc is 2^23 + c.
template <int BITS>
__device__ __forceinline__ void values8(float2 (&x)[4], uint2 c, uint32_t word) {
  const float zb = -(8388608.0f + half_hi(word)), s = half_lo(word);
  const float2 zb2 = make_float2(zb, zb), s2 = make_float2(s, s);
  const uint32_t lo = c.x & 0x0F0F0F0Fu, hi = (c.x >> 4) & 0x0F0F0F0Fu;   // (4-bit: even and odd channels)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v;
    if constexpr (BITS == 8) {
      const uint32_t w = i < 2 ? c.x : c.y;
      v.x = __uint_as_float(prmt(w, 0x4B000000u, 0x7440u + 2 * (i & 1)));
      v.y = __uint_as_float(prmt(w, 0x4B000000u, 0x7441u + 2 * (i & 1)));
    } else {
      v.x = __uint_as_float(prmt(lo, 0x4B000000u, 0x7440u + i));
      v.y = __uint_as_float(prmt(hi, 0x4B000000u, 0x7440u + i));
    }
    x[i] = __fmul2_rn(__fadd2_rn(v, zb2), s2);
  }
}

// Bounds of one block of n tokens, by a warp: a lane has 8 channels of every
// RPP-th token, so that a load of the warp covers whole consecutive rows.
template <int D, int BITS>
__device__ __forceinline__ void block_of(const BParams& p, int h, int sb, int n, int lane) {
  constexpr int G = D / 32;
  constexpr int LPR = D / 8;          // lanes per row
  constexpr int RPP = 32 / LPR;       // rows per pass
  constexpr int U = 8;                // passes whose loads are in flight together
  const int col = lane % LPR, part = lane / LPR;
  const int64_t blocks = static_cast<int64_t>(p.c.pB) * (p.c.pT / KVQ_TILE_TOKENS);
  const int64_t row0 = static_cast<int64_t>(sb) * KVQ_TILE_TOKENS;
  const int64_t off0 = p.plane_off[h] + row0 * (D * BITS / 8) + col * BITS;
  const int64_t si0 = (static_cast<int64_t>(h) * blocks * KVQ_TILE_TOKENS + row0) * G + col / 4;
  if (!KVQ_IN_RANGE(sb >= 0 && sb < blocks && off0 + (KVQ_TILE_TOKENS - 1) * (D * BITS / 8) + BITS <= p.codes_bytes,
                    p.status))
    return;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  // the lane's rows at fixed distances from two pointers; of a block that is
  // cut, whole rows are read (they are the storage's) and those past its end
  // replaced by the lane's first
  const uint8_t* src = p.codes + off0 + part * (D * BITS / 8);
  const uint32_t* sw = p.sz + si0 + part * G;
  uint2 c0 = make_uint2(0u, 0u);
  uint32_t word0 = 0u;
  if (n < KVQ_TILE_TOKENS) {          // (token 0 for lanes whose first one is past the end)
    const int back = part < n ? 0 : part;
    if constexpr (BITS == 8) c0 = *reinterpret_cast<const uint2*>(src - back * (D * BITS / 8));
    else c0.x = *reinterpret_cast<const uint32_t*>(src - back * (D * BITS / 8));
    word0 = *(sw - back * G);
  }
#pragma unroll 1
  for (int t0 = 0; t0 < n; t0 += RPP * U) {
    uint2 c[U];
    uint32_t word[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      c[j] = make_uint2(0u, 0u);
      if constexpr (BITS == 8) c[j] = *reinterpret_cast<const uint2*>(src + j * RPP * (D * BITS / 8));
      else c[j].x = *reinterpret_cast<const uint32_t*>(src + j * RPP * (D * BITS / 8));
      word[j] = sw[j * RPP * G];
    }
    src += RPP * U * (D * BITS / 8);
    sw += RPP * U * G;
    if (n < KVQ_TILE_TOKENS) {
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (t0 + j * RPP + part >= n) {
          c[j] = c0;
          word[j] = word0;
        }
    }
#pragma unroll
    for (int j = 0; j < U; j += 2) {
      float2 x[4], y[4];
      values8<BITS>(x, c[j], word[j]);
      values8<BITS>(y, c[j + 1], word[j + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[2 * i] = min3(lo[2 * i], x[i].x, y[i].x);
        hi[2 * i] = max3(hi[2 * i], x[i].x, y[i].x);
        lo[2 * i + 1] = min3(lo[2 * i + 1], x[i].y, y[i].y);
        hi[2 * i + 1] = max3(hi[2 * i + 1], x[i].y, y[i].y);
      }
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = min2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = max2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  }
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max3(a, fabsf(lo[i]), fabsf(hi[i]));
  a = max2(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max2(a, __shfl_xor_sync(0xffffffffu, a, 2));
  if (part > 1) return;               // lanes of part 0 write the greatest values, of part 1 the least
  const float s = __fdiv_rn(a, 127.0f);
  uint32_t v[2] = {0u, 0u};
  if (!(a < INFINITY)) {
    report(p.status, KVQ_ERR_NONFINITE);
  } else if (s > 0.0f) {              // (s rounds to 0 only where every value is 0: the least stored one is 2^-24)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = part == 0 ? ceilf(__fdiv_rn(hi[i], s)) : floorf(__fdiv_rn(lo[i], s));
      const int code = static_cast<int>(fminf(fmaxf(f, -127.0f), 127.0f));
      v[i / 4] |= (static_cast<uint32_t>(code) & 0xFFu) << (8 * (i % 4));
    }
  }
  const int64_t g = (static_cast<int64_t>(h) * blocks + sb) * G + col / 4;
  *reinterpret_cast<uint2*>(p.b_codes + g * 64 + part * 32 + (col % 4) * 8) = make_uint2(v[0], v[1]);
  if (part == 0 && col % 4 == 0) p.b_scales[g] = a < INFINITY ? s : 0.0f;
}

// HBM reads each code and word of a touched block once; what bounds it is the
// ALU pipe (a permute a code, a three-input minimum and maximum a pair) and issue
// slots: four prompts of 30K-32K, 8 heads, INT8, 151 MB, 38.5 us, 3.9 TB/s;
// one new token in each of 16 sequences 6.1 us, of which a launch, two
// look-ups and a block's loads.
//
// A block is the work of the row that holds its first new token: a sequence's
// first new row, or one at the start of a block.  A warp looks at R rows for
// one head: one while the rows are few or mostly sequences' first (each may own
// a block), 64 once they are many (mostly prompts, one owner in 64).
template <int D, int R>
__global__ void __launch_bounds__(kBoundsWarps * 32, kBoundsBlocks) block_bounds_kernel(const __grid_constant__ BParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, blockDim.x, p.status);
  const int64_t units = p.tiles * p.Hkv;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kBoundsWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kBoundsWarps) {
    const int tile = static_cast<int>(static_cast<uint32_t>(u) / static_cast<uint32_t>(p.Hkv));
    const int h = static_cast<int>(static_cast<uint32_t>(u) - static_cast<uint32_t>(tile) * p.Hkv);
#pragma unroll 1
    for (int r0 = tile * R; r0 < min((tile + 1) * R, p.c.rows); r0 += 32) {
      int b = chunk::find_sequence(p.c.start, p.c.B, r0, lane);
      const int r = r0 + lane;
      int sb = -1, n = 0;
      if (lane < R && r < p.c.rows) {
        while (b + 1 < p.c.B && p.c.start[b + 1] <= r) ++b;
        const chunk::Seq s = chunk::sequence(p.c, b);
        const int pos = s.len - s.n + (r - s.row0);
        if (!s.bad && r >= s.row0 && r < s.row0 + s.n && (r == s.row0 || pos % KVQ_TILE_TOKENS == 0)) {
          const int i = pos / KVQ_TILE_TOKENS;
          const int64_t row = chunk::storage_row(p.c, b, i * KVQ_TILE_TOKENS);
          if (row >= 0) sb = static_cast<int>(row / KVQ_TILE_TOKENS);
          else if (h == 0) report(p.status, KVQ_ERR_INVALID_ARG);
          n = min(KVQ_TILE_TOKENS, s.len - i * KVQ_TILE_TOKENS);
        }
      }
      for (unsigned m = __ballot_sync(0xffffffffu, sb >= 0); m != 0; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int block = __shfl_sync(0xffffffffu, sb, src), count = __shfl_sync(0xffffffffu, n, src);
        if (p.bits[h] == 8) block_of<D, 8>(p, h, block, count, lane);
        else block_of<D, 4>(p, h, block, count, lane);
        __syncwarp();
      }
    }
  }
}

// Listed blocks' bounds as values: a warp per (KV head, block), 4 channels a lane
// at a time (16 bytes out, 4 of codes in).
__global__ void __launch_bounds__(kBoundsWarps * 32) bounds_values_kernel(const int8_t* codes, const float* scales,
                                                                          const int32_t* ids, int n, int Hkv, int64_t NB,
                                                                          int D, float* out, int32_t* status) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t total = static_cast<int64_t>(Hkv) * n;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kBoundsWarps + (threadIdx.x >> 5); u < total;
       u += static_cast<int64_t>(gridDim.x) * kBoundsWarps) {
    const int64_t h = u / n;
    const int id = ids[u - h * n];
    const bool ok = id >= 0 && id < NB;
    if (!ok && h == 0 && lane == 0) report(status, KVQ_ERR_INVALID_ARG);
    const int64_t g0 = ok ? (h * NB + id) * (D / 32) : 0;
    for (int e = lane * 4; e < 2 * D; e += 128) {          // row e / D (greatest, least), channel e % D
      const int d = e % D;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (ok) {
        const char4 c = *reinterpret_cast<const char4*>(codes + (g0 + d / 32) * 64 + (e / D) * 32 + d % 32);
        const float s = scales[g0 + d / 32];
        v = make_float4(static_cast<signed char>(c.x) * s, static_cast<signed char>(c.y) * s,
                        static_cast<signed char>(c.z) * s, static_cast<signed char>(c.w) * s);
      }
      *reinterpret_cast<float4*>(out + u * 2 * D + e) = v;
    }
  }
}

// ---------------------------------------------------------------------------
// selection
// ---------------------------------------------------------------------------

constexpr int kSelThreads = 256;
constexpr int kSelectPer = 128;     // blocks of a CTA at least
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSmemKeys = 8192;     // keys selected from in shared memory (sequences up to 524,288 tokens)
constexpr int kMaxChunks = 64;      // CTAs of one (row, KV head)

struct SParams {
  const uint16_t* q;
  const int8_t* b_codes;
  const float* b_scales;
  const int32_t* bt;
  const int32_t* row_seq;
  const int32_t* row_lens;
  int32_t* blocks;
  int32_t* cnt;             // [rows * Hkv] chunks scored; zero between calls
  uint32_t* keys;           // [rows * Hkv][key_stride]
  int32_t* status;
  int64_t NB, key_stride;
  int32_t seqs, bt_stride, cap, pB;
  int32_t rows, Hq, Hkv, rep, n_select, first, last;
  int32_t per_chunk, chunks;
};

// Larger scores have larger keys; -0 and 0 the same.
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(__fadd_rn(score, 0.0f));
  return u ^ ((u >> 31) != 0u ? 0xFFFFFFFFu : 0x80000000u);
}

// Shared memory of a selection's last part.
struct SelectSmem {
  int hist[2][256];
  uint32_t lo[kSelWarps], hi[kSelWarps];   // each warp's least and greatest key
  int2 sums[kSelWarps];
  int digit, above, count;
};

// The indices (plus `base`) of the `want` largest of n keys (0 < want < n),
// ascending, ties to the lower index.  The key of rank `want` is found digit by
// digit, 8 bits at a time from the highest bit in which any two keys differ
// (scores of one row share sign and most of their exponents), with a histogram
// of the keys that agree so far; it ends early where all keys of the rank's
// digit are wanted.  Then one ordered pass.  mn, mx: this thread's least and
// greatest key.
template <class Load>
__device__ __forceinline__ void select_largest(Load key, int n, int want, int base, int32_t* out, uint32_t mn, uint32_t mx,
                                               SelectSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) {
    sm.lo[w] = mn;
    sm.hi[w] = mx;
  }
  if (tid < 256) sm.hist[0][tid] = 0;
  __syncthreads();
  mn = __reduce_min_sync(0xffffffffu, sm.lo[lane % kSelWarps]);
  mx = __reduce_max_sync(0xffffffffu, sm.hi[lane % kSelWarps]);
  int shift = mn == mx ? 0 : max(24 - __clz(mn ^ mx), 0);      // the first digit's lowest bit
  uint32_t mask = shift >= 24 ? 0u : 0xFFFFFFFFu << (shift + 8);   // bits that all keys looked at agree in
  uint32_t prefix = mx & mask;
  int left = want;                    // rank among the keys that agree with the prefix
  bool whole = mn == mx;              // every key from the prefix on is wanted (mn == mx: ties, by index below)
  if (whole) {
    mask = 0xFFFFFFFFu;
    prefix = mx;
  }
  for (int pass = 0; !whole; ++pass) {
    int* hist = sm.hist[pass & 1];
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    if (tid < 256) sm.hist[(pass & 1) ^ 1][tid] = 0;
    __syncthreads();
    if (w == 0) {                     // lane l: digits 255 - 8 l .. 248 - 8 l
      int c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * lane - j];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (before < left && before + c[j] >= left) {
          sm.digit = 255 - 8 * lane - j;
          sm.above = before;
          sm.count = c[j];
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(sm.digit) << shift;
    mask |= 255u << shift;
    left -= sm.above;
    whole = left == sm.count || shift == 0;
    shift = max(shift - 8, 0);
    // (a last digit of fewer than 8 new bits overlaps the one before: those bits agree)
  }
  // keys whose known digits are above the prefix, and the first `left` of those equal to it
  const int per = (n + kSelThreads - 1) / kSelThreads;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int2 mine = make_int2(0, 0);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i) & mask;
    mine.x += k > prefix;
    mine.y += k == prefix;
  }
  int2 x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y0 = __shfl_up_sync(0xffffffffu, x.x, o), y1 = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) {
      x.x += y0;
      x.y += y1;
    }
  }
  if (lane == 31) sm.sums[w] = x;
  __syncthreads();
  int above = x.x - mine.x, equal = x.y - mine.y;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i)
    if (i < w) {
      above += sm.sums[i].x;
      equal += sm.sums[i].y;
    }
  int at = above + min(equal, left);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i) & mask;
    if (k > prefix || (k == prefix && equal++ < left)) out[at++] = base + i;
  }
}

// A chain of short steps, bound by latency: 8 blocks of one sequence 3.7 us, 512
// blocks of 8 sequences and 8 heads (9 MB of bounds, 1.3 us at the copy rate)
// 8.3 us, 1800 blocks of four 9.4 us.
//
// One CTA scores per_chunk blocks of a (row, KV head), its threads G lanes a
// block (one per group, 64 bytes of bounds each); where there are several
// CTAs, the last to arrive selects from all the keys.  The blocks that are
// always taken are left out of all this: the others are `first` .. nblk -
// `last` - 1, candidate i being block first + i.
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const __grid_constant__ SParams p) {
  constexpr int G = D / 32;
  constexpr int U = 2;                // blocks of a lane whose loads are in flight together
  constexpr int kRound = U * kSelThreads / G;
  __shared__ __align__(16) uint32_t s_q[G][16];   // the group's 32 greatest-side codes, then the least-side ones
  __shared__ float s_u[G];
  __shared__ uint32_t s_keys[kSmemKeys];
  __shared__ SelectSmem sm;
  __shared__ int s_last;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const int seg = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.chunks));
  const int chunk = static_cast<int>(blockIdx.x) - seg * p.chunks;
  const int row = seg / p.Hkv, kvh = seg - row * p.Hkv;
  int len = p.row_lens[row];
  const int seq = p.row_seq != nullptr ? p.row_seq[row] : row;
  uint32_t qv[8];                     // the lane's channel of the group's queries
  if (tid < D) {
    const uint16_t* src = p.q + (static_cast<int64_t>(row) * p.Hq + kvh * p.rep) * D + tid;
#pragma unroll
    for (int r = 0; r < 8; ++r) qv[r] = r < p.rep ? src[r * D] : 0u;
  }
  if (len < 0 || len > p.cap || seq < 0 || seq >= p.seqs) {
    if (tid == 0) report(p.status, KVQ_ERR_INVALID_ARG);
    len = 0;
  }
  const int nblk = (len + KVQ_TILE_TOKENS - 1) / KVQ_TILE_TOKENS;
  int32_t* out = p.blocks + static_cast<int64_t>(seg) * p.n_select;
  if (nblk <= p.n_select) {           // all of them
    if (chunk == 0)
      for (int i = tid; i < p.n_select; i += kSelThreads) out[i] = i < nblk ? i : -1;
    return;
  }
  const int n = nblk - p.first - p.last, want = p.n_select - p.first - p.last;   // (n > want >= 0)
  if (chunk == 0) {
    for (int i = tid; i < p.first; i += kSelThreads) out[i] = i;
    for (int i = tid; i < p.last; i += kSelThreads) out[p.n_select - p.last + i] = nblk - p.last + i;
  }
  const int c0 = chunk * p.per_chunk, c1 = min(c0 + p.per_chunk, n);
  if (want == 0 || c0 >= n) return;
  const int used = (n + p.per_chunk - 1) / p.per_chunk;   // CTAs with blocks to score

  const int g = lane % G;
  uint4 w[U][4];
  float sc[U];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = p.first + min(i0 + (j * kSelThreads + tid) / G, c1 - 1);   // (past the end: the last block again)
      int64_t sb = static_cast<int64_t>(seq) * (p.cap / KVQ_TILE_TOKENS) + i;
      if (p.bt != nullptr) {
        int page = KVQ_IN_RANGE(i < p.bt_stride, p.status) ? p.bt[static_cast<int64_t>(seq) * p.bt_stride + i] : 0;
        if (page < 0 || page >= p.pB) {
          report(p.status, KVQ_ERR_INVALID_ARG);
          page = 0;
        }
        sb = page;
      }
      if (!KVQ_IN_RANGE(sb >= 0 && sb < p.NB, p.status)) sb = 0;
      const int64_t at = (kvh * p.NB + sb) * G + g;
      const uint4* src = reinterpret_cast<const uint4*>(p.b_codes + at * 64);
#pragma unroll
      for (int v = 0; v < 4; ++v) w[j][v] = src[v];
      sc[j] = p.b_scales[at];
    }
  };
  fetch(c0);
  // the query in 8 bits: warp g has group g, lane l its channel l
  if (tid < D) {
    float up = 0.0f, down = 0.0f;
    bool finite = true;
#pragma unroll
    for (int r = 0; r < 8; ++r) {     // (heads past the group's add nothing)
      const float v = __uint_as_float(qv[r] << 16);
      finite &= fabsf(v) < INFINITY;
      up = __fadd_rn(up, fmaxf(v, 0.0f));
      down = __fadd_rn(down, fminf(v, 0.0f));
    }
    if (!finite) report(p.status, KVQ_ERR_NONFINITE);
    float a = fmaxf(up, -down);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float u = __fdiv_rn(a, 127.0f);
    const float cp = u > 0.0f ? rintf(__fdiv_rn(up, u)) : 0.0f, cn = u > 0.0f ? rintf(__fdiv_rn(down, u)) : 0.0f;
    int8_t* dst = reinterpret_cast<int8_t*>(s_q[tid / 32]);
    dst[lane] = static_cast<int8_t>(static_cast<int>(fminf(fmaxf(cp, -127.0f), 127.0f)));
    dst[32 + lane] = static_cast<int8_t>(static_cast<int>(fminf(fmaxf(cn, -127.0f), 127.0f)));
    if (lane == 0) s_u[tid / 32] = u;
  }
  __syncthreads();
  uint32_t qc[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(&s_q[g][4 * i]);
    qc[4 * i] = v.x; qc[4 * i + 1] = v.y; qc[4 * i + 2] = v.z; qc[4 * i + 3] = v.w;
  }
  const float u = s_u[g];
  const bool in_smem = n <= kSmemKeys;
  const bool alone = used == 1;
  uint32_t* gkeys = p.keys + static_cast<int64_t>(seg) * p.key_stride;
  uint32_t mn = 0xFFFFFFFFu, mx = 0u;
  for (int i0 = c0; i0 < c1; i0 += kRound) {
    if (i0 != c0) fetch(i0);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      int dots = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        dots = __dp4a(static_cast<int>(w[j][v].x), static_cast<int>(qc[4 * v]), dots);
        dots = __dp4a(static_cast<int>(w[j][v].y), static_cast<int>(qc[4 * v + 1]), dots);
        dots = __dp4a(static_cast<int>(w[j][v].z), static_cast<int>(qc[4 * v + 2]), dots);
        dots = __dp4a(static_cast<int>(w[j][v].w), static_cast<int>(qc[4 * v + 3]), dots);
      }
      const float t = __fmul_rn(__fmul_rn(u, sc[j]), static_cast<float>(dots));
      float score = __shfl_sync(0xffffffffu, t, lane - g);
#pragma unroll
      for (int k = 1; k < G; ++k) score = __fadd_rn(score, __shfl_sync(0xffffffffu, t, lane - g + k));
      const int i = i0 + (j * kSelThreads + tid) / G;
      if (g == 0 && i < c1) {
        const uint32_t key = key_of(score);
        mn = min(mn, key);
        mx = max(mx, key);
        if (alone && in_smem) s_keys[i] = key;
        else if (KVQ_IN_RANGE(i < p.key_stride, p.status)) gkeys[i] = key;
      }
    }
  }
  __syncthreads();
  if (!alone) {
    // publish the chunk's keys and count the arrivals: after the barrier the
    // release orders every thread's keys before the count, and for the last
    // to arrive its acquire orders the others' keys before the reads below
    if (tid == 0) s_last = atom_add_acq_rel_gpu(p.cnt + seg, 1) + 1 == used;
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) p.cnt[seg] = 0;     // ready for the next call
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t key = __ldcg(gkeys + i);
      mn = min(mn, key);
      mx = max(mx, key);
      if (in_smem) s_keys[i] = key;
    }
    // (select_largest's first barrier orders these before its reads)
  }
  out += p.first;
  if (in_smem) select_largest([&](int i) { return s_keys[i]; }, n, want, p.first, out, mn, mx, sm);
  else select_largest([&](int i) { return __ldcg(gkeys + i); }, n, want, p.first, out, mn, mx, sm);
}

cudaLaunchConfig_t config(int64_t blocks, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(blocks, int64_t(1) << 30)));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsArgs& a, cudaStream_t stream) {
  BParams p;
  const kvq_cache& k = *a.k;
  p.c = chunk::view_of(a.chunk, k);
  p.codes = k.codes;
  p.sz = k.sz;
  p.b_codes = a.bounds.codes;
  p.b_scales = a.bounds.scales;
  p.status = a.status;
  p.Hkv = k.Hkv;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * k.B * k.Tcap * (k.D / 2);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  // A row a warp costs by rows, 64 by the first new rows that lie in one run of
  // 64.  Up to 4096 rows (8 heads, INT8, one against 64): a prompt of 512 5.0
  // and 4.8 us, of 2048 8.3 and 5.1, of 4096 12.3 and 5.1, at worst 7 us lost;
  // but 256 sequences of one row 7.6 and 170, of four 10.4 and 46.  Above: a
  // prompt of 8192 20.5 and 5.8, 1000 sequences of sixteen 57 and 28, unless
  // most rows are a sequence's first: 3000 sequences of two 58 and 148, of
  // four 73 and 86, of sixteen 166 and 66.
  const bool few = a.chunk.rows <= std::max<int64_t>(4096, int64_t(4) * a.chunk.B);
  p.tiles = few ? a.chunk.rows : (static_cast<int64_t>(a.chunk.rows) + 63) / 64;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config((p.tiles * p.Hkv + kBoundsWarps - 1) / kBoundsWarps, kBoundsWarps * 32, stream, &attr);
  auto launch = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, p); };
  if (k.D == 128) return few ? launch(block_bounds_kernel<128, 1>) : launch(block_bounds_kernel<128, 64>);
  return few ? launch(block_bounds_kernel<64, 1>) : launch(block_bounds_kernel<64, 64>);
}

cudaError_t launch_bounds_values(const kvq_cache& k, const kvq_bounds& bounds, const int32_t* blocks, int32_t n,
                                 float* out, int32_t* status, cudaStream_t stream) {
  const int64_t warps = static_cast<int64_t>(k.Hkv) * n;
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config((warps + kBoundsWarps - 1) / kBoundsWarps, kBoundsWarps * 32, stream, &attr);
  return cudaLaunchKernelEx(&cfg, bounds_values_kernel, static_cast<const int8_t*>(bounds.codes),
                            static_cast<const float*>(bounds.scales), blocks, static_cast<int>(n),
                            static_cast<int>(k.Hkv), static_cast<int64_t>(k.B) * (k.Tcap / KVQ_TILE_TOKENS),
                            static_cast<int>(k.D), out, status);
}

// workspace: [cnt: a counter for every possible (row, KV head), so that their
// place does not depend on a call's shape][keys]
constexpr size_t kCountBytes = static_cast<size_t>(kMaxRows) * KVQ_MAX_HKV * 4;

size_t select_workspace_bytes(int rows, int Hkv, int64_t cap) {
  const size_t stride = static_cast<size_t>((cap / KVQ_TILE_TOKENS + 3) / 4 * 4);
  return kCountBytes + static_cast<size_t>(rows) * Hkv * stride * 4;
}

cudaError_t launch_select_blocks(const SelectArgs& a, cudaStream_t stream) {
  SParams p;
  const kvq_cache& k = *a.k;
  p.q = a.q;
  p.b_codes = a.bounds.codes;
  p.b_scales = a.bounds.scales;
  p.bt = a.bt;
  p.row_seq = a.row_seq;
  p.row_lens = a.row_lens;
  p.blocks = a.blocks;
  p.cnt = static_cast<int32_t*>(a.ws);
  p.keys = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.ws) + kCountBytes);
  p.status = a.status;
  const int nb = a.cap / KVQ_TILE_TOKENS;
  p.key_stride = (nb + 3) / 4 * 4;
  p.NB = static_cast<int64_t>(k.B) * (k.Tcap / KVQ_TILE_TOKENS);
  p.seqs = a.seqs;
  p.bt_stride = a.bt_max_pages;
  p.cap = a.cap;
  p.pB = k.B;
  p.rows = a.rows;
  p.Hq = a.Hq;
  p.Hkv = k.Hkv;
  p.rep = a.Hq / k.Hkv;
  p.n_select = a.n_select;
  p.first = a.first;
  p.last = a.last;
  // about four CTAs an SM: blocks are cut finer while the rows are few
  const int64_t segs = static_cast<int64_t>(a.rows) * k.Hkv;
  int64_t per = (segs * nb + 4 * device_sm_count() - 1) / (4 * device_sm_count());
  per = std::max<int64_t>(per, (nb + kMaxChunks - 1) / kMaxChunks);
  per = std::max<int64_t>((per + 127) / 128 * 128, kSelectPer);
  p.per_chunk = static_cast<int32_t>(per);
  p.chunks = static_cast<int32_t>(std::max<int64_t>((nb + per - 1) / per, 1));
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = config(segs * p.chunks, kSelThreads, stream, &attr);
  return k.D == 128 ? cudaLaunchKernelEx(&cfg, select_blocks_kernel<128>, p)
                    : cudaLaunchKernelEx(&cfg, select_blocks_kernel<64>, p);
}

}  // namespace kvq
