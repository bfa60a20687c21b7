// kvq_chunk_narrow.cu -- chunk attention of few rows per KV head (drafted
// tokens, short chunks, single tokens next to them): the same work as
// kvq_chunk_attn.cu, with the keys on the tensor cores' row side.
//
// With at most 32 packed rows (token * rep + head) a 128-row query tile is
// mostly empty, and what bounds the call is the cache read.  So a key tile is
// the M side of both products,
//   S^T [128 keys x NR rows]      = K [keys x D]      Q^T [D x rows]
//   O^T [D channels x NR rows]   += V^T [channels x keys] P^T [keys x rows]
// and the softmax works on NR = 16 or 32 columns: a thread has one key's
// scores, a row's running max lives in shared memory and moves only when a
// score exceeds it by more than 2^8 (a vote of the four warps a tile), and the
// sums are per thread until the piece ends.
//
// One CTA (896 threads, one per SM) walks its range of the work list
// (kvq_chunk_walk.cuh):
//   warps 0, 1   issue V^T P^T and K Q^T (a warp each: neither waits for what
//                only the other needs); warp 0 also allocates and frees TMEM;
//   warps 2, 3   keep rings of raw slots (64 tokens: codes and words) of K and
//                V full by bulk copies, about 50 KB in flight an SM;
//   warps 4-11   K codes (and the piece's queries) to fp16 operand tiles, warps
//   12-19        V codes likewise (two warps a scheduler for each part: one
//                alone took 1.2 us a tile, most of it latency);
//   warps 20-27  softmax in two states, of even and of odd tiles, each with its
//                own maxima, sums and O^T, so that one's waits run under the
//                other's; rescaling, the piece's output or partial, the merge.
// TMEM: S^T and O^T of each state, NR columns each.
//
// Measured: long contexts are bound by HBM's reads (eight sequences of 32K, 16
// rows, INT8: 590 MB in 118 us, 5.0 TB/s over the call, 0.95 us per 36 KB tile an
// SM); a call of one tile takes 10 us, and a segment's cut about 9 us (eight
// sequences of 8K: 42 us).  Fetching the codes into L2 further ahead was slower (54 us against 49 for
// eight sequences of 8K), and so were slots of 32 tokens (more copies).
#include <cmath>
#include <mutex>

#include "kvq_chunk_walk.cuh"
#include "kvq_internal.h"
#include "kvq_tc.cuh"
#include "kvq_tile.cuh"

namespace kvq {
namespace {

using namespace tile;
using namespace chunk_walk;

constexpr int kThreads = 896;
constexpr int kRing = 3;               // raw slots of K, and as many of V

enum {
  B_QREADY = 0, B_QEMPTY, B_FULL0, B_EMPTY0 = B_FULL0 + 4, B_SFULL0 = B_EMPTY0 + 4, B_PFULL0 = B_SFULL0 + 2,
  B_PDONE0 = B_PFULL0 + 2, B_OFREE = B_PDONE0 + 2, B_STATE, B_MMADONE0, B_EXIT = B_MMADONE0 + 2, B_RAW0,
  B_RFREE0 = B_RAW0 + 2 * kRing, B_COUNT = B_RFREE0 + 2 * kRing
};   // FULL and EMPTY: K stages 0, 1, V stages 0, 1; SFULL, PFULL, PDONE: states; RAW and RFREE: K slots, V slots
// Every warp but warp 0 arrives once on B_EXIT when it is done with shared
// memory, TMEM and its asynchronous operations; warp 0 frees TMEM after that.
constexpr int kExitArrivals = kThreads / 32 - 1;

template <int D, int NR>
struct NLayout {
  static constexpr int kTile = kT * D * 2;              // one K or V operand tile
  static constexpr int kOffK = 0;                       // 2 stages
  static constexpr int kOffV = kOffK + 2 * kTile;       // 2 stages; with D = 64 the products read 16 KB past each
  // P^T of both states: [128 keys][64 rows] fp16, the second state's rows 32 on
  static constexpr int kOffP = kOffV + 2 * kTile;
  static constexpr int kPStep = 64;                     // bytes
  static constexpr int kOffQ = kOffP + kT * 128;        // [D / 64][NR][128 B]
  // raw slots: kST tokens' codes (8-bit heads fill the room), then their words
  static constexpr int kST = 64;
  static constexpr int kRawWords = kST * D;
  static constexpr int kRawBytes = kRawWords + kST * (D / 32) * 4;
  static constexpr int kOffRaw = kOffQ + NR * D * 2;
  static constexpr int kOffBar = kOffRaw + 2 * kRing * kRawBytes;
  static constexpr int kOffMisc = kOffBar + B_COUNT * 8;     // TMEM address
  static constexpr int kOffRow = (kOffMisc + 16 + 15) / 16 * 16;   // per state and row: position, max, factor, four warps' values
  static constexpr int kOffSplit = kOffRow + NR * 2 * 7 * 4;   // Split
  static constexpr int kOffWalk = kOffSplit + 16;
  static constexpr int kOffPre = kOffWalk + kThreads / 32 * 128;
  static constexpr size_t bytes(int B) { return 1024 + kOffPre + static_cast<size_t>(B + 1) * 4; }
};
constexpr int kMaxB = 2048;            // sequences (their unit counts lie in shared memory)
static_assert(NLayout<128, 32>::bytes(kMaxB) <= 232448, "shared memory");
static_assert(32 * 128 * 4 <= kT * 128, "a piece's output rows fit the P tile");

// Whether any of a softmax warpgroup's 128 threads says so (all take part);
// id: the warpgroup's barrier.
__device__ __forceinline__ bool group_or(bool x, int id) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// Floats as integers of the same order (for the integer warp maximum).
__device__ __forceinline__ int to_ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_ordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// The warp's sums of NR rows' values to dst[NR]: at each step a lane keeps half
// of the rows that it has and gives away the others (31 shuffles for 32 rows;
// 80 for 16 rows one by one).
template <int NR>
__device__ __forceinline__ void sum_rows(float (&l)[NR], int lane, int32_t* dst) {
  static_assert(NR == 16 || NR == 32, "at most a row a lane");
  int row = 0;
#pragma unroll
  for (int o = 16, n = NR / 2; o > 0; o >>= 1, n >>= 1) {
    if (n > 0) {
      const bool up = lane & o;           // keeps rows n .. 2n - 1 of those it has
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float give = up ? l[i] : l[n + i];
        const float keep = up ? l[n + i] : l[i];
        l[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
      row += up ? n : 0;
    } else {
      l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);   // (16 rows: both lanes of a pair have the row)
    }
  }
  dst[row] = __float_as_int(l[0]);
}

// One part (0: K, 1: V) of a piece's tiles by its two warpgroups: raw slots (64
// tokens) to rows of the operand tile, warpgroup `sub` taking every second
// iteration.
template <int D, int NR, int BITS>
__device__ __forceinline__ bool dequant_piece(const CParams& p, uint8_t* smem, uint64_t* bar, const Walk& w, int which,
                                              int sub, uint32_t& jj, uint32_t& slot, uint32_t& round, uint32_t& marks, int t,
                                              int lane) {
  using L = NLayout<D, NR>;
  using F = DqFmt<D, BITS>;
  constexpr int H = F::NI / 2;              // iterations per slot, both warpgroups'
  static_assert(H * F::RPI == 64, "whole iterations per slot");
  constexpr int N = H > 1 ? H / 2 : 1;      // this warpgroup's (of a slot with one: every second slot)
  int row, c;
  dq_lane<D, BITS>(t, row, c);
  for (int j = 0; j < w.n; ++j, ++jj) {
    const uint32_t st = jj & 1;
    if (jj >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bar[B_EMPTY0 + 2 * which + st], ((jj >> 1) - 1) & 1, p.status,
                                                      p.wait_ns)))
      return false;
    const uint32_t dst = smem_u32(smem + (which ? L::kOffV : L::kOffK) + st * L::kTile);
    uint32_t most = 0;                      // the largest scale in the low half
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = which * kRing + static_cast<int>(slot);
      if (!__all_sync(0xffffffffu, mbar_wait(&bar[B_RAW0 + k], round & 1, p.status, p.wait_ns))) return false;
      const bool mine = H > 1 || s == sub;
      const uint8_t* raw = smem + L::kOffRaw + k * L::kRawBytes;
      const uint4* codes = reinterpret_cast<const uint4*>(raw + row * F::R + c * 16);
      const uint32_t* words = reinterpret_cast<const uint32_t*>(raw + L::kRawWords) + row * (D / 32) + c * F::VPC / 32;
      uint4 v[N];
      uint32_t word[N];
      if (mine) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int it = H > 1 ? 2 * i + sub : 0;
          v[i] = codes[it * F::RPI * F::R / 16];
          word[i] = words[it * F::RPI * (D / 32)];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_RFREE0 + k]);
      if (mine) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int it = s * H + (H > 1 ? 2 * i + sub : 0);
          dequant_chunk<BITS>(dst, F::RPI * it + row, c * F::VPC, v[i], word[i]);
          most = __vmaxu2(most, word[i]);
        }
      }
      if (++slot == kRing) {
        slot = 0;
        ++round;
      }
    }
    mark_big<BITS>(marks, most, j);
    if (which) clear_unseen<D, BITS>(dst, p, w, w.t.tile(w.i + j) * kT, row, c, sub, F::NI, 2);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_FULL0 + 2 * which + st]);
  }
  return true;
}

// Four channels of an output row to global memory.
template <int D>
__device__ __forceinline__ void store_out4(const CParams& p, int64_t off, float4 o) {
  if (!KVQ_IN_RANGE(off >= 0 && off + 4 <= static_cast<int64_t>(p.c.rows) * p.Hq * D, p.status)) return;
  if (p.out_dtype == KVQ_OUT_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + off) = o;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o.x, o.y), b = __floats2bfloat162_rn(o.z, o.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + off) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// The rows of a cut segment merged by log-sum-exp over its pieces, in CTA
// order: a thread takes four channels of a row, two such at a time and four
// pieces' loads of each in flight (row by row, a warp each, it took 4.7 us).
template <int D>
__device__ __forceinline__ void merge_rows(const CParams& p, const Walk& w, const Cut& cut, int rows_per_block, int rows,
                                           int t) {
  constexpr int Q = D / 4, U = 2, P = 4;
  const int np = cut.c1 - cut.c0 + 1;
#pragma unroll 1
  for (int i0 = t; i0 < rows * Q; i0 += U * 128) {
    float M[U], L[U];
    float4 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      M[u] = -INFINITY;
      L[u] = 0.0f;
      acc[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll 1
    for (int k0 = 0; k0 < np; k0 += P) {
      float lse[U][P];
      float4 v[U][P];
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const int64_t part = static_cast<int64_t>(cut.partial(cut.c0 + min(k0 + k, np - 1))) * p.slot_rows;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * 128, rows * Q - 1), r = i / Q;
          lse[u][k] = k0 + k < np ? __ldcg(p.ws_lse + part + r) : -INFINITY;
          v[u][k] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (part + r) * D) + i % Q);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float m = M[u];
#pragma unroll
        for (int k = 0; k < P; ++k) m = fmaxf(m, lse[u][k]);
        if (m == -INFINITY) continue;   // no piece with weight yet
        const float a = fast_exp2(M[u] - m);
        acc[u].x *= a; acc[u].y *= a; acc[u].z *= a; acc[u].w *= a;
        L[u] *= a;
#pragma unroll
        for (int k = 0; k < P; ++k) {
          const float b = fast_exp2(lse[u][k] - m);
          acc[u].x = fmaf(b, v[u][k].x, acc[u].x);
          acc[u].y = fmaf(b, v[u][k].y, acc[u].y);
          acc[u].z = fmaf(b, v[u][k].z, acc[u].z);
          acc[u].w = fmaf(b, v[u][k].w, acc[u].w);
          L[u] += b;
        }
        M[u] = m;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 128;
      if (i >= rows * Q) break;
      const float inv = L[u] > 0.0f ? 1.0f / L[u] : 0.0f;
      store_out4<D>(p, out_offset(p, w, w.rt * rows_per_block + i / Q, D) + i % Q * 4,
                    make_float4(acc[u].x * inv, acc[u].y * inv, acc[u].z * inv, acc[u].w * inv));
    }
  }
}

template <int D, int NR>
__global__ void __launch_bounds__(kThreads, 1) chunk_narrow_kernel(const __grid_constant__ CParams p) {
  using L = NLayout<D, NR>;
  constexpr uint32_t kCols = 4 * NR;                                 // TMEM: S^T and O^T of both states
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  int32_t* pre = reinterpret_cast<int32_t*>(smem + L::kOffPre);
  Walk* walks = reinterpret_cast<Walk*>(smem + L::kOffWalk);
  Split& split = *reinterpret_cast<Split*>(smem + L::kOffSplit);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bar[B_QREADY], 4);
    mbar_init(&bar[B_QEMPTY], 1);
    for (int k = 0; k < 4; ++k) {
      mbar_init(&bar[B_FULL0 + k], 8);
      mbar_init(&bar[B_EMPTY0 + k], 1);
    }
    mbar_init(&bar[B_SFULL0], 1);
    mbar_init(&bar[B_SFULL0 + 1], 1);
    mbar_init(&bar[B_PFULL0], 4);
    mbar_init(&bar[B_PFULL0 + 1], 4);
    mbar_init(&bar[B_PDONE0], 1);
    mbar_init(&bar[B_PDONE0 + 1], 1);
    mbar_init(&bar[B_OFREE], 4);
    mbar_init(&bar[B_STATE], 4);
    mbar_init(&bar[B_MMADONE0], 1);
    mbar_init(&bar[B_MMADONE0 + 1], 1);
    mbar_init(&bar[B_EXIT], kExitArrivals);
    for (int k = 0; k < 2 * kRing; ++k) {
      mbar_init(&bar[B_RAW0 + k], 1);
      mbar_init(&bar[B_RFREE0 + k], 8);
    }
    fence_barrier_init();
  }
  // (before the dependency wait: the registers of two CTAs with TMEM do not fit
  // an SM, so this never waits for a CTA that could wait for this kernel)
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, kCols);
    tc::tmem_relinquish();
  }
  // the caches, queries and lengths may come from the kernel before this one
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, kThreads, p.status);
  // (starts that descend: the units may be anything)
  const bool disorder = __syncthreads_or(count_units<NR>(p, pre, warp, lane, kThreads / 32));
  if (disorder) {
    // nothing to do
  } else if (warp == 1) {
    sum_units(p, pre, lane);
    start_walk<NR>(p, pre, walks[1], split.N, lane);
  } else if (warp == 2) {
    const int most = start_parts<NR>(p, walks[2], lane);
    if (lane == 0) split.most = most;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  Walk& w = walks[warp];
  const int from = !disorder && split.parts<NR>(p) ? 2 : 1;   // the warp whose split it is
  const int64_t total = disorder ? 0 : walks[from].left;
  if (total <= 0) {   // the whole CTA: nothing was started
    if (warp == 0) tc::tmem_dealloc(tmem, kCols);
    if (warp == 1 && p.zero_rest) zero_rest_rows<D>(p, disorder, lane);
    return;
  }
  if (warp != from) copy_walk(w, walks[from], lane);
  __syncthreads();   // (that warp's own walk goes on from here)
  auto wait_all = [&](int which, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(&bar[which], parity & 1, p.status, p.wait_ns));
  };
  auto drain = [&](int which, uint32_t parity) { mbar_wait(&bar[which], parity & 1, p.status, kDrainNs); };

  // Registers: launched with 72 per thread (checked on the host); per
  // warpgroup 56 + 4 x 56 + 2 x 112 = 7 x 72.
  if (warp < 4) tc::reg_dealloc<56>();
  if (warp == 0) {
    // ---------------- issuer of O^T (+)= V^T P^T, then the end of the CTA ----------------
    constexpr uint32_t id_pv = tc::idesc_f16_f32(kT, NR, true, true);
    const uint32_t pt = smem_u32(smem + L::kOffP), vb = smem_u32(smem + L::kOffV);
    uint32_t k = 0, piece = 0, cnt[2] = {0, 0};   // tiles, and each state's
    bool ok = true;
    do {
      const int n = w.n;
      for (int j = 0; j < n && ok; ++j, ++k) {
        const int x = j & 1;                        // the tile's state
        ok = wait_all(B_FULL0 + 2 + (k & 1), k >> 1) && wait_all(B_PFULL0 + x, cnt[x]);
        if (ok && j == 0 && piece > 0) ok = wait_all(B_OFREE, piece - 1);   // the previous piece's O has been read
        if (!ok) break;
        ++cnt[x];
        tc::fence_after_sync();
        if (tc::elect_one()) {
          // (D = 64: channels 64-127 of the A operand are whatever follows the
          // tile; their rows of O^T are never read)
          const uint32_t vs = vb + (k & 1) * L::kTile, d_o = tmem + 2 * NR + x * NR;
          const uint64_t da = tc::smem_desc_sw128(vs, kT * 128, 1024);
          const uint64_t db = tc::smem_desc_sw128(pt + x * L::kPStep, kT * 128, 1024);
          if (j < 2) tc::mma_ss<false>(d_o, da, db, id_pv);
          else tc::mma_ss<true>(d_o, da, db, id_pv);
#pragma unroll
          for (int s = 1; s < kT / 16; ++s)   // 16 keys on: 2 KB, 128 in the descriptors' address field
            tc::mma_ss<true>(d_o, da + s * 128, db + s * 128, id_pv);
          tc::commit(&bar[B_EMPTY0 + 2 + (k & 1)]);
          tc::commit(&bar[B_PDONE0 + x]);
        }
        __syncwarp();
      }
      ++piece;
    } while (ok && next_piece<NR>(p, w, lane));
    if (tc::elect_one()) tc::commit(&bar[B_MMADONE0 + 1]);
    __syncwarp();
    drain(B_MMADONE0 + 1, 0);
    // The other roles finish in bounded time: each stops at its first wait
    // that runs out, and a role waits at most a few times per tile.
    const uint64_t deadline = p.wait_ns * static_cast<uint64_t>(16 * min(total, int64_t(1) << 20) + 16) + 4 * kDrainNs;
    const uint64_t t0 = global_ns();
    uint32_t n = 0;
    while (!mbar_try_wait(&bar[B_EXIT], 0)) {
      if ((++n & 255u) == 0 && global_ns() - t0 > deadline) {
        report(p.status, KVQ_ERR_TIMEOUT);
        break;
      }
    }
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kCols);
    return;
  }

  if (warp == 1) {
    // ---------------- issuer of S^T = K Q^T ----------------
    constexpr uint32_t id_qk = tc::idesc_f16_f32(kT, NR, false);
    const uint32_t q = smem_u32(smem + L::kOffQ), kb = smem_u32(smem + L::kOffK);
    uint32_t jj = 0, piece = 0, cnt[2] = {0, 0};
    bool ok = true;
    do {
      const int n = w.n;
      ok = wait_all(B_QREADY, piece);
      for (int j = 0; j < n && ok; ++j, ++jj) {
        const int x = j & 1;
        ok = wait_all(B_FULL0 + (jj & 1), jj >> 1);
        if (ok && cnt[x] > 0) ok = wait_all(B_PFULL0 + x, cnt[x] - 1);   // the state's S has been read
        if (!ok) break;
        ++cnt[x];
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint32_t d_s = tmem + x * NR;
          const uint64_t da = tc::smem_desc_sw128(kb + (jj & 1) * L::kTile, 16, 1024);
          const uint64_t db = tc::smem_desc_sw128(q, 16, 1024);
          tc::mma_ss<false>(d_s, da, db, id_qk);
#pragma unroll
          for (int s = 1; s < D / 16; ++s)    // 16 channels on: 32 B, or the next 64-channel block
            tc::mma_ss<true>(d_s, da + (s >> 2) * (kT * 8) + (s & 3) * 2, db + (s >> 2) * (NR * 8) + (s & 3) * 2, id_qk);
          tc::commit(&bar[B_SFULL0 + x]);
          tc::commit(&bar[B_EMPTY0 + (jj & 1)]);
          if (j + 1 == n) tc::commit(&bar[B_QEMPTY]);
        }
        __syncwarp();
      }
      ++piece;
    } while (ok && next_piece<NR>(p, w, lane));
    // every product this warp issued has completed (a commit with none
    // pending arrives at once) before the warp reports that it is done
    if (tc::elect_one()) tc::commit(&bar[B_MMADONE0]);
    __syncwarp();
    drain(B_MMADONE0, 0);
    tc::fence_before_sync();
    if (lane == 0) mbar_arrive(&bar[B_EXIT]);
    return;
  }

  if (warp < 4) {
    // ---------------- copies: raw slots of K (warp 2) and of V (warp 3) ----------------
    // (a warp each: one warp for both held K's copies back while V's ring was full)
    const int x = warp - 2;
    const int64_t blocks = static_cast<int64_t>(p.c.pB) * (p.c.pT / 64);
    const uint64_t pol = l2_evict_first_policy();
    uint32_t slot = 0, round = 0;
    bool ok = true;
    do {
      const Seen seen(p, w);
      const int rb = D * p.bits[w.kvh] / 8;                        // code bytes of a token
      const uint32_t cb = L::kST * rb, wb = L::kST * (D / 32) * 4;
      const uint8_t* codes = p.codes[x] + p.plane_off[w.kvh];
      const uint32_t* words = p.sz[x] + w.kvh * blocks * (64 * (D / 32));
      int half[2] = {0, 0};
      for (int j = 0; j < w.n && ok; ++j) {
        if ((j & 31) == 0 && j + lane < w.n) {                     // 32 tiles' pages at a time, a lane each
          const int t0 = w.t.tile(w.i + j + lane) * kT;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int a = t0 + 64 * h;
            const bool is_seen = a < seen.end && (a + 64 > seen.lo || a < p.sinks);
            // (a half that nothing sees stands for the other: its rows are masked)
            const int b = is_seen ? a : (h == 0 ? a + 64 : a - 64);
            half[h] = chunk::storage_block(p.c, w.b, b / 64, p.status);
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          int64_t blk = __shfl_sync(0xffffffffu, half[s], j & 31);
          const int k = x * kRing + static_cast<int>(slot);
          if (round > 0) ok = wait_all(B_RFREE0 + k, round - 1);
          if (!ok) break;
          if (lane == 0) {
            uint8_t* raw = smem + L::kOffRaw + k * L::kRawBytes;
            if (!KVQ_IN_RANGE(blk >= 0 && blk < blocks && p.plane_off[w.kvh] + (blk + 1) * 64 * rb <= p.codes_bytes,
                              p.status))
              blk = 0;
            const int64_t at = blk * 64;
            mbar_arrive_expect_tx(&bar[B_RAW0 + k], cb + wb);
            bulk_g2s_hint(raw, codes + at * rb, cb, &bar[B_RAW0 + k], pol);
            bulk_g2s_hint(raw + L::kRawWords, words + at * (D / 32), wb, &bar[B_RAW0 + k], pol);
          }
          if (++slot == kRing) {
            slot = 0;
            ++round;
          }
          __syncwarp();
        }
      }
    } while (ok && next_piece<NR>(p, w, lane));
    // every copy has landed before the CTA can exit, whether or not the
    // dequant warps got to read it: the last one into each slot
    if (lane == 0) {
#pragma unroll 1
      for (uint32_t k = 0; k < kRing; ++k) {
        const uint32_t fills = round + (k < slot ? 1 : 0);
        if (fills > 0) drain(B_RAW0 + x * kRing + static_cast<int>(k), fills - 1);
      }
      mbar_arrive(&bar[B_EXIT]);
    }
    __syncwarp();
    return;
  }

  if (warp < 20) {
    tc::reg_dealloc<56>();
    // ---------------- dequant warpgroups: two for K (the first also the queries), two for V ----------------
    const int wg = (warp - 4) >> 2, which = wg >> 1, sub = wg & 1;
    const int t = threadIdx.x & 127;
    uint32_t jj = 0, slot = 0, round = 0, piece = 0;
    bool ok = true, big = false;
    do {
      if (wg == 0) {
        ok = load_queries<D, NR>(p, smem_u32(smem + L::kOffQ), &bar[B_QEMPTY], w, t, (piece - 1) & 1, piece > 0);
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && piece < p.issue_limit) mbar_arrive(&bar[B_QREADY]);
      }
      uint32_t marks = 0;
      ok = p.bits[w.kvh] == 4 ? dequant_piece<D, NR, 4>(p, smem, bar, w, which, sub, jj, slot, round, marks, t, lane)
                              : dequant_piece<D, NR, 8>(p, smem, bar, w, which, sub, jj, slot, round, marks, t, lane);
      big |= marked_overflow<D>(p, w, marks, which, which + 1, lane);
      ++piece;
    } while (ok && next_piece<NR>(p, w, lane));
    if (big) report(p.status, KVQ_ERR_NONFINITE);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_EXIT]);
    return;
  }

  tc::reg_alloc<112>();
  // (a warp whose first tile is the piece's second)
  if (warp == kThreads / 32 - 1 && p.zero_rest) zero_rest_rows<D>(p, false, lane);
  // ---------------- softmax warpgroups: thread = key of the tile, then channel of O^T ----------------
  // Two states of the online softmax, each with its own maxima, sums and O^T:
  // warpgroup x takes the piece's tiles j with j % 2 == x, so that a tile's
  // chain of waits (scores, vote, weights, products) runs under the other's;
  // at the piece's end warpgroup 0 joins the two.  (A warpgroup's four warps
  // take every decision together, so that its barriers are always met by all:
  // a wait that ran out is a vote.)
  const int x = (warp - 20) >> 2, id = 1 + x;
  const int q4 = warp & 3, key = q4 * 32 + lane;
  // positions of the rows (each warpgroup has its own copy), the running
  // maxima (log2 domain), the factors of their last move, four warps' values
  constexpr int kState = 7 * NR;
  int32_t* row_pos = reinterpret_cast<int32_t*>(smem + L::kOffRow) + x * kState;
  float* row_m = reinterpret_cast<float*>(row_pos + NR);
  float* row_a = row_m + NR;
  int32_t* row_w = reinterpret_cast<int32_t*>(row_a + NR);
  const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
  const uint32_t s_addr = tmem + lanes + x * NR;
  const uint32_t o_addr = tmem + lanes + 2 * NR + x * NR;
  const uint32_t p_row = smem_u32(smem + L::kOffP) + key * 128;
  const float sl2 = p.scale_log2;
  uint32_t cnt = 0, piece = 0;                             // this state's tiles; pieces
  bool ok = true, stop = false;
  do {
    // the piece's rows: positions (a row past the segment's end as the last
    // one), no maximum yet -- once warpgroup 0 has read the previous piece's
    if (x == 1 && piece > 0) ok = wait_all(B_OFREE, piece - 1) && ok;
    if (key < NR) {
      const int R = w.rt * NR + key;
      row_pos[key] = key < w.t.rows ? w.s.len - w.s.n + R / p.rep : w.t.pos_hi;
      row_m[key] = -INFINITY;
    }
    if (group_or(!ok, id)) break;
    float l[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) l[i] = 0.0f;
    const int n = w.n;
    for (int j = x; j < n; j += 2, ++cnt) {
      const int t0 = w.t.tile(w.i + j) * kT, tok = t0 + key;
      // some row of the block does not see some key of the tile
      const bool masked = t0 + kT - 1 > w.t.pos_lo ||
                          (p.window > 0 && t0 < w.t.pos_hi - p.window + 1 && t0 + kT > p.sinks);
      const bool always = tok < p.sinks || p.window == 0;  // no window for this key
      ok = wait_all(B_SFULL0 + x, cnt) && ok;
      tc::fence_after_sync();
      float s[NR];
      {
        uint32_t v[NR];
        if constexpr (NR == 16) tc::ld_32x32b_x16(s_addr, v);
        else tc::ld_32x32b_x32(s_addr, v);
        tc::wait_ld(v);
#pragma unroll
        for (int i = 0; i < NR; ++i) s[i] = __uint_as_float(v[i]) * sl2;
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
          const int4 pos = *reinterpret_cast<const int4*>(row_pos + i);
          const int ps[4] = {pos.x, pos.y, pos.z, pos.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(ps[e] >= tok && (always || ps[e] - p.window < tok))) s[i + e] = -INFINITY;
        }
      }
      bool move = !ok;
#pragma unroll
      for (int i = 0; i < NR; i += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(row_m + i);
        move |= s[i] > m4.x + kRescaleThreshold || s[i + 1] > m4.y + kRescaleThreshold ||
                s[i + 2] > m4.z + kRescaleThreshold || s[i + 3] > m4.w + kRescaleThreshold;
      }
      if (group_or(move, id)) {
        if (group_or(!ok, id)) {
          stop = true;
          break;
        }
        // new maxima of the rows that need one, the sums and O^T rescaled
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const int mx = __reduce_max_sync(0xffffffffu, to_ordered(s[i]));
          if (lane == i) row_w[q4 * NR + i] = mx;
        }
        group_sync(id);
        if (key < NR) {
          const float M = fmaxf(fmaxf(from_ordered(row_w[key]), from_ordered(row_w[NR + key])),
                                fmaxf(from_ordered(row_w[2 * NR + key]), from_ordered(row_w[3 * NR + key])));
          const float mo = row_m[key];
          const float mn = M > mo + kRescaleThreshold ? M : mo;   // (mo -infinity: any M)
          row_a[key] = mo == -INFINITY ? 1.0f : fast_exp2(mo - mn);
          row_m[key] = mn;
        }
        group_sync(id);
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
          const float4 a4 = *reinterpret_cast<const float4*>(row_a + i);
          l[i] *= a4.x; l[i + 1] *= a4.y; l[i + 2] *= a4.z; l[i + 3] *= a4.w;
        }
        if (j > x) {
          ok = wait_all(B_PDONE0 + x, cnt - 1) && ok;
          tc::fence_after_sync();
#pragma unroll
          for (int c0 = 0; c0 < NR; c0 += 16) {
            uint32_t v[16];
            tc::ld_32x32b_x16(o_addr + c0, v);
            tc::wait_ld(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * row_a[c0 + i]);
            tc::st_32x32b_x16(o_addr + c0, v);
          }
          tc::wait_st();
        }
      }
      // P^T = 2^(S - m): this key's row of the operand tile, once the state's previous product has read it
      uint32_t pk[NR / 2];
#pragma unroll
      for (int i = 0; i < NR; i += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(row_m + i);
        const float mm[4] = {m4.x, m4.y, m4.z, m4.w};
        float e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // (a row that sees nothing yet has no maximum: its weights are 2^-infinity = 0)
          e[u] = fast_exp2(s[i + u] - (mm[u] == -INFINITY ? 0.0f : mm[u]));
          l[i + u] += e[u];
        }
        pk[i / 2] = pack_half2(e[0], e[1]);
        pk[i / 2 + 1] = pack_half2(e[2], e[3]);
      }
      if (cnt > 0) ok = wait_all(B_PDONE0 + x, cnt - 1) && ok;
#pragma unroll
      for (int i = 0; i < NR / 8; ++i)
        sts128(p_row + (((i + x * (L::kPStep / 16)) ^ (key & 7)) << 4), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_PFULL0 + x]);
    }
    if (stop) break;
    // ---- end of the piece: sums over the keys; the two states joined; O^T / sum ----
    if (n > x) ok = wait_all(B_PDONE0 + x, cnt - 1) && ok;
    if (group_or(!ok, id)) break;
    tc::fence_after_sync();
    sum_rows<NR>(l, lane, row_w + q4 * NR);
    if (x == 1) {   // maxima and sums are in shared memory, O^T in TMEM: warpgroup 0's from here
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_STATE]);
      ++piece;
      continue;
    }
    ok = wait_all(B_STATE, piece) && ok;
    if (group_or(!ok, id)) break;
    tc::fence_after_sync();
    const int rows = w.t.rows;
    const bool whole = n == w.t.n, four = p.bits[w.kvh] == 4;
    const Cut cut(w, kLead<NR>);
    const int part = cut.partial(blockIdx.x);
    // a row's factors of the two O^T, each in its state's row_a
    if (key < NR) {
      float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        sum0 += __int_as_float(row_w[q * NR + key]);
        sum1 += __int_as_float(row_w[kState + q * NR + key]);
      }
      const float m0 = row_m[key], m1 = row_m[kState + key], M = fmaxf(m0, m1);
      const float f0 = m0 == -INFINITY ? 0.0f : fast_exp2(m0 - M);
      const float f1 = m1 == -INFINITY ? 0.0f : fast_exp2(m1 - M);
      const float sum = f0 * sum0 + f1 * sum1, inv = sum > 0.0f ? 1.0f / sum : 0.0f;
      row_a[key] = f0 * inv;
      row_a[kState + key] = f1 * inv;
      if (!whole && key < rows)
        p.ws_lse[static_cast<int64_t>(part) * p.slot_rows + key] = sum > 0.0f ? M + __log2f(sum) : -INFINITY;
    }
    group_sync(id);
    // The rows' outputs to shared memory ([row][channel] over the P buffers,
    // which no product reads any more), then to global memory in a rolled loop:
    // a piece's end runs once, and straight-line code for every row took 2.6 us
    // of it to fetch.
    float* stage = reinterpret_cast<float*>(smem + L::kOffP);
    {
      // operand column `key` holds this channel (4-bit heads: order 0,4,1,5,2,6,3,7 within eight)
      const int ch = four ? (key & ~7) | ((key & 1) << 2) | ((key & 7) >> 1) : key;
#pragma unroll 1
      for (int c0 = 0; c0 < rows; c0 += 16) {
        uint32_t v0[16], v1[16];
        tc::ld_32x32b_x16(o_addr + c0, v0);
        if (n > 1) tc::ld_32x32b_x16(o_addr + NR + c0, v1);   // (a piece of one tile has no second state)
        tc::wait_ld(v0);
        if (n > 1) tc::wait_ld(v1);
        if (key < D) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float o = __uint_as_float(v0[i]) * row_a[c0 + i];
            if (n > 1) o = fmaf(__uint_as_float(v1[i]), row_a[kState + c0 + i], o);
            stage[(c0 + i) * D + ch] = o;
          }
        }
      }
    }
    group_sync(id);
#pragma unroll 1
    for (int i = key; i < rows * (D / 4); i += 128) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      const float4 o = reinterpret_cast<const float4*>(stage)[i];
      if (!whole) {
        *reinterpret_cast<float4*>(p.ws_o + (static_cast<int64_t>(part) * p.slot_rows + r) * D + c) = o;
        continue;
      }
      store_out4<D>(p, out_offset(p, w, w.rt * NR + r, D) + c, o);
    }
    tc::fence_before_sync();
    group_sync(id);   // the rows' values have been read; every partial is stored
    if (lane == 0) mbar_arrive(&bar[B_OFREE]);
    if (!whole) {
      // one acquire-release atomic after the group's barrier, and a vote that
      // hands its outcome (and what it acquired) to the group
      bool last = false;
      if (key == 0) last = atom_add_acq_rel_gpu(p.cnt + 2 * cut.c0, 1) + 1 == cut.c1 - cut.c0 + 1;
      if (group_or(last, id)) {
        merge_rows<D>(p, w, cut, NR, rows, key);
        if (key == 0) p.cnt[2 * cut.c0] = 0;   // ready for the next call
      }
    }
    ++piece;
  } while (next_piece<NR>(p, w, lane));
  tc::wait_st();
  tc::fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar[B_EXIT]);
}

// Per device and instantiation, set once under a lock: the kernel's dynamic
// shared-memory limit, and its registers checked.
std::mutex g_prep_mu;
bool g_prep[64][4] = {};

template <int D, int NR>
kvq_status launch_n(const CParams& p, cudaStream_t stream) {
  using L = NLayout<D, NR>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(g_prep_mu);
    bool& ready = g_prep[dev][(D == 128 ? 2 : 0) + (NR == 16 ? 0 : 1)];
    if (!ready) {
      // the register split inside the kernel assumes 72 per thread at launch
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, chunk_narrow_kernel<D, NR>) != cudaSuccess) return KVQ_ERR_CUDA;
      if (fa.numRegs != 72) return KVQ_ERR_UNSUPPORTED;
      if (cudaFuncSetAttribute(chunk_narrow_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(L::bytes(kMaxB))) != cudaSuccess)
        return KVQ_ERR_CUDA;
      ready = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::bytes(p.c.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_narrow_kernel<D, NR>, p) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

// At most 32 rows: with 64 columns a softmax thread's scores and sums do not fit
// its registers (even 32 spill some), and 64 rows on 8000 tokens took 108 us to
// the 256-row kernel's 66.  Measured (us; this kernel, the 256-row one; eight
// sequences, 8 KV heads, D = 128):
//   tokens        200       1000       2000       4000       8000       32000
//   INT8 16   11.0 12.5  16.6 21.8  20.1 27.1  27.7 40.6  41.8 65.5  118  189
//        24   14.3 12.7  21.4 22.0  25.7 27.5  34.3 40.7  54.7 65.6  135  189
//        32   14.7 12.6  21.8 22.0  26.8 27.2  35.3 40.9  55.9 65.0  137  188
//   INT4 16   11.4 12.7  18.2 22.0  21.3 27.7  30.5 40.9  46.6 66.7  136  199
//        32   14.7 12.5  22.6 22.1  27.6 27.8  36.7 40.9  59.3 66.5  150  198
// (of 17 to 32 rows on a few hundred tokens the other would be 2 us faster)
bool chunk_narrow_takes(int B, int64_t max_rows) { return B <= kMaxB && max_rows <= 32; }

kvq_status launch_chunk_narrow(const CParams& p, int D, int64_t max_rows, cudaStream_t stream) {
  if (D == 128) return max_rows <= 16 ? launch_n<128, 16>(p, stream) : launch_n<128, 32>(p, stream);
  return max_rows <= 16 ? launch_n<64, 16>(p, stream) : launch_n<64, 32>(p, stream);
}

}  // namespace kvq
