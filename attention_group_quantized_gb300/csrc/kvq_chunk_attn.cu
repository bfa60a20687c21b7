// kvq_chunk_attn.cu -- attention of a chunk of new tokens over the
// group-quantised cache, on the 5th-generation tensor cores.
//
// Method: the query of packed row r, at cache position p, attends tokens
// j <= p of its sequence, with a window only j > p - window or j < sinks; the
// cache holds integer codes with a scale and a zero point per 32 channels
// (《分块稀疏注意力与KV Cache量化：长文本推理显存优化实践》 §2.4), dequantised inside
// the attention read (§1.3); the keys are visited in 128-token tiles with an
// online softmax (§2.2).
//
// Work: the query heads that share a KV head are packed with the chunk's
// tokens into one list of rows (row = token * rep + head), so every
// dequantised K/V tile serves them all; 256 rows (two slots of 128, one
// tcgen05 tile each) are a segment's rows, and the key tiles that any of them
// sees its tiles.  The list of all (sequence, KV head, row block, key tile) is
// cut into equal ranges, one per persistent CTA ("stream-K"): ragged lengths
// and few rows over a long cache load every SM alike.  A segment that is cut
// leaves one partial (o, lse) per piece in the workspace, and the CTA that
// completes it merges them in a fixed order.
//
// One CTA (640 threads, one per SM):
//   warp 0      zeroes rows of no sequence, if asked to; allocates TMEM and
//               frees it once every other role is done;
//   warps 1, 2  issue slot h = warp - 1's tcgen05.mma (S_h = Q_h K^T from
//               shared memory, O_h += P_h V with P from TMEM), taking turns so
//               that one slot's softmax runs under the other's products;
//   warp 3      fetches the next piece's queries into L2;
//   warps 4-11  per piece, its query rows to fp16 (a warpgroup per slot); per
//               key tile, K and V codes to fp16 operand tiles (two stages, a
//               warpgroup per 64-token half), the next part's codes in flight
//               in registers meanwhile;
//   warps 12-19 softmax of slot 0 and slot 1, one thread per row; at a piece's
//               end O / sum to the output or the workspace.
// TMEM (512 columns): S_0 [0,128) O_0 [128,128+D) S_1 [256,384) O_1 [384,384+D).
// The running max only moves (and O is rescaled) when it grows by more than
// 2^8; P is rounded to fp16, sums and O stay in fp32.
//
// Measured (32 query heads on 8, D = 128): 2048 tokens on 32K cached, INT8,
// 865 to 890 us (from GPU to GPU) = 1270 to 1310 TFLOP/s, 68 to 70 % of a bf16
// GEMM's burst rate -- 1.87 us a tile of
// 256 rows, of which the products take 1.37 at that rate and the softmax's 2^x
// 1.1, next to them; what is left is the chain between them.  Shorter pieces
// add about 10 us each (first queries and codes, partials, merge): 16 sequences
// of 1 to 286 new tokens on 1K to 8K, from pages, 172 us; 3500 tokens with a
// window of 4096 on 55K to 84K, INT4, 237 us.  One dequant warpgroup for whole
// tiles took 246 and 257 us where the two took 187 and 236 (the loads of one
// thread's K and V wait for each other); an L2 prefetch of the codes was slower.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "kvq_chunk_walk.cuh"
#include "kvq_internal.h"
#include "kvq_tc.cuh"
#include "kvq_tile.cuh"

namespace kvq {
namespace {

using namespace tile;
using namespace chunk_walk;

constexpr int kThreads = 640;
constexpr int kRows = 2 * kT;          // packed rows per segment
constexpr uint32_t kTmemCols = 512;

enum {
  B_QREADY = 0, B_QEMPTY, B_KFULL0, B_KFULL1, B_VFULL0, B_VFULL1, B_KVEMPTY0, B_KVEMPTY1, B_SFULL0, B_SFULL1,
  B_PFIRST0, B_PFIRST1, B_PFULL0, B_PFULL1, B_ORDY0, B_ORDY1, B_OFREE0, B_OFREE1, B_TURN0, B_TURN1, B_GROUP0, B_GROUP1,
  B_MMADONE, B_EXIT, B_COUNT
};
// Every warp but warp 0 arrives once on B_EXIT when it is done with shared
// memory, TMEM and its asynchronous operations, on the normal path and after
// a timed-out wait alike; warp 0 frees TMEM only after that.
constexpr int kExitArrivals = kThreads / 32 - 1;

template <int D>
struct CLayout {
  static constexpr int kQBytes = kT * D * 2;            // one slot's fp16 rows / one K or V tile
  static constexpr int kOffQ = 0;                       // 2 slots
  static constexpr int kOffK = kOffQ + 2 * kQBytes;     // 2 stages
  static constexpr int kOffV = kOffK + 2 * kQBytes;     // 2 stages
  static constexpr int kOffBar = kOffV + 2 * kQBytes;
  static constexpr int kOffMisc = kOffBar + (B_COUNT + 1) / 2 * 16;  // TMEM address, merge flags
  static constexpr int kOffSplit = kOffMisc + 16;         // Split
  static constexpr int kOffWalk = kOffSplit + 16;          // Walk of each warp
  static constexpr int kOffPre = kOffWalk + kThreads / 32 * 128;   // int32 [B + 1]
  static size_t bytes(int B) { return 1024 + kOffPre + static_cast<size_t>(B + 1) * 4; }
};

// Half a key tile (64 tokens: a page, or that much of a sequence) as its dequant
// warpgroup reads it; a half that nothing sees stands in for the other, its
// rows are masked.  Looked up one tile ahead of the loads that use it and free
// of branches: a branch between a load and its use waits for every load in
// flight.
template <bool PAGED>
struct HalfTile {
  int t0;                // the tile's first token
  int block;             // a page id as it stands in the table, or a block
  __device__ __forceinline__ void look_up(const CParams& p, const Walk& w, int j, int x) {
    const Seen s(p, w);
    t0 = w.t.tile(w.i + j) * kT;
    const int i0 = t0 / 64, i1 = i0 + 1;
    const bool seen0 = t0 + 64 > s.lo || t0 < p.sinks;
    const bool seen1 = t0 + 64 < s.end && (t0 + kT > s.lo || t0 + 64 < p.sinks);
    const int i = (x == 0 ? seen0 : !seen1) ? i0 : i1;
    if constexpr (PAGED) {
      const bool ok = KVQ_IN_RANGE(i >= 0 && i < p.c.bt_stride, p.status);
      block = ok ? p.c.bt[static_cast<int64_t>(w.b) * p.c.bt_stride + i] : 0;
    } else {
      block = w.b * (p.c.pT / 64) + i;
    }
  }
  // A page outside the pool reads as page 0 (and is reported at the piece's end).
  __device__ __forceinline__ void check(const CParams& p, bool& bad) {
    if constexpr (PAGED) {
      const bool out = static_cast<uint32_t>(block) >= static_cast<uint32_t>(p.c.pB);
      bad |= out;
      block = out ? 0 : block;
    }
  }
};

// Half of a part (64 tokens' codes and words of K or V) in registers.
template <int D, int BITS>
struct HalfRegs {
  static constexpr int N = DqFmt<D, BITS>::NI / 2;
  static_assert(2 * N == DqFmt<D, BITS>::NI, "whole iterations per half tile");
  uint4 c[N];
  uint32_t w[N];
};

// codes, sz: the thread's place in block 0 of the head's codes and words (each
// byte is used once per CTA: no L1 line).
template <int D, int BITS>
__device__ __forceinline__ void load_half(const CParams& p, HalfRegs<D, BITS>& r, const uint8_t* codes,
                                          const uint32_t* sz, int block) {
  using F = DqFmt<D, BITS>;
  const int blk = KVQ_IN_RANGE(block >= 0 && block < static_cast<int64_t>(p.c.pB) * (p.c.pT / 64), p.status) ? block : 0;
  codes += blk * int64_t(64 * F::R);
  sz += blk * int64_t(64 * (D / 32));
#pragma unroll
  for (int it = 0; it < r.N; ++it) {
    r.c[it] = __ldcg(reinterpret_cast<const uint4*>(codes + it * F::RPI * F::R));
    r.w[it] = __ldcg(sz + it * F::RPI * (D / 32));
  }
}

template <int D, int BITS>
__device__ __forceinline__ void store_half(uint32_t dst, const HalfRegs<D, BITS>& r, int x, int row, int c) {
  using F = DqFmt<D, BITS>;
#pragma unroll
  for (int it = 0; it < r.N; ++it)
    dequant_chunk<BITS>(dst, F::RPI * (x * r.N + it) + row, c * F::VPC, r.c[it], r.w[it]);
}

template <int D, int BITS>
__device__ __forceinline__ uint32_t max_word(const HalfRegs<D, BITS>& r) {
  uint32_t m = r.w[0];
#pragma unroll
  for (int it = 1; it < r.N; ++it) m = __vmaxu2(m, r.w[it]);
  return m;
}

// 16 bytes from global to shared memory without a register, zeros for n = 0.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr) : "memory");
  return v;
}

// The piece's query rows of slot x (rows past the segment's end zero) into its swizzled
// tile and there, each thread its own 16-byte chunks, to fp16.  All of a
// piece's loads are in flight together: through registers, in batches of
// eight, the next piece's first product waited 2 us longer.
template <int D>
__device__ __forceinline__ bool fetch_queries(const CParams& p, uint32_t dst, uint64_t* empty, const Walk& w, int x,
                                              int t, uint32_t piece) {
  constexpr int CPR = D / 8;              // 16-byte chunks per row
  constexpr int RPP = 128 / CPR;          // rows per pass
  const int ch = t % CPR, row = t / CPR;
  const int rows = w.t.rows - x * kT, end = rows > 0 ? kT : 0;   // the slot's
  if (piece > 0 && !__all_sync(0xffffffffu, mbar_wait(empty, (piece - 1) & 1, p.status, p.wait_ns))) return false;
  const uint16_t* base = p.q + static_cast<int64_t>(w.s.row0) * p.sq_row + w.kvh * p.rep * p.sq_head + ch * 8;
  const int R0 = w.rt * kRows + x * kT + row;   // token and head of this thread's row, stepped from pass to pass
  int tok = R0 / p.rep, hh = R0 - tok * p.rep;
  const int dtok = RPP / p.rep, dhh = RPP - dtok * p.rep;
  auto at = [&](int r) { return dst + x * (kT * D * 2) + (ch >> 3) * (kT * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4); };
#pragma unroll 4
  for (int r = row; r < end; r += RPP) {
    const bool live = r < rows;
    cp_async16(at(r), live ? base + tok * p.sq_row + hh * p.sq_head : base, live ? 16u : 0u);
    tok += dtok;
    hh += dhh;
    if (hh >= p.rep) {
      hh -= p.rep;
      ++tok;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  const bool four = p.bits[w.kvh] == 4;
  uint32_t big = 0;
#pragma unroll 4
  for (int r = row; r < end; r += RPP) {
    const uint4 x = query_chunk(lds128(at(r)), four, big);
    sts128(at(r), x.x, x.y, x.z, x.w);
  }
  check_queries(p, big);
  return true;
}

// Half x of the key tiles of one piece: codes to fp16 operand tiles.  jj counts
// the CTA's tiles (stage jj & 1).  False after a wait that ran out.
template <int D, int BITS, bool PAGED>
__device__ __forceinline__ bool dequant_piece(const CParams& p, uint8_t* smem, uint64_t* bar, const Walk& w, int x,
                                              uint32_t& jj, uint32_t piece, bool& bad, uint32_t& marks, int t,
                                              int lane) {
  using L = CLayout<D>;
  using F = DqFmt<D, BITS>;
  constexpr int G = D / 32, N = HalfRegs<D, BITS>::N;
  int row, c;
  dq_lane<D, BITS>(t, row, c);
  const uint32_t kdst = smem_u32(smem + L::kOffK);
  constexpr uint32_t kToV = L::kOffV - L::kOffK;
  const int64_t blocks = static_cast<int64_t>(p.c.pB) * (p.c.pT / 64);
  const int64_t coff = p.plane_off[w.kvh] + row * F::R + c * 16;
  const int64_t soff = w.kvh * blocks * (64 * G) + row * G + c * F::VPC / 32;
  HalfTile<PAGED> cur, next;
  HalfRegs<D, BITS> k, v;
  auto done = [&](int which, bool tell = true) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && tell) mbar_arrive(&bar[which]);
  };
  cur.look_up(p, w, 0, x);
  next.look_up(p, w, min(1, w.n - 1), x);
  cur.check(p, bad);
  auto load_k = [&]() { load_half<D, BITS>(p, k, p.codes[0] + coff, p.sz[0] + soff, cur.block); };
  auto load_v = [&]() { load_half<D, BITS>(p, v, p.codes[1] + coff, p.sz[1] + soff, cur.block); };
  load_k();
  if (!fetch_queries<D>(p, smem_u32(smem + L::kOffQ), &bar[B_QEMPTY], w, x, t, piece)) return false;
  done(B_QREADY, piece < p.issue_limit);
  for (int j = 0; j < w.n; ++j, ++jj) {
    const uint32_t st = jj & 1, dst = kdst + st * L::kQBytes;
    load_v();
    const int t0 = cur.t0;
    next.check(p, bad);
    cur = next;
    next.look_up(p, w, min(j + 2, w.n - 1), x);
    if (jj >= 2 && !__all_sync(0xffffffffu, mbar_wait(&bar[B_KVEMPTY0 + st], ((jj >> 1) - 1) & 1, p.status, p.wait_ns)))
      return false;
    store_half<D, BITS>(dst, k, x, row, c);
    uint32_t most = max_word<D, BITS>(k);   // (branch-free: a branch on a loaded word would wait for every load in flight)
    done(B_KFULL0 + st);
    if (j + 1 < w.n) load_k();
    store_half<D, BITS>(dst + kToV, v, x, row, c);
    most = __vmaxu2(most, max_word<D, BITS>(v));
    mark_big<BITS>(marks, most, j);
    clear_unseen<D, BITS>(dst + kToV, p, w, t0, row, c, x * N, (x + 1) * N);
    done(B_VFULL0 + st);
  }
  return true;
}

// 32 output values of one row, from channel offset `off` of the output.
__device__ __forceinline__ void store_row32(const CParams& p, int D, int64_t off, const float (&o)[32]) {
  if (!KVQ_IN_RANGE(off >= 0 && off + 32 <= static_cast<int64_t>(p.c.rows) * p.Hq * D, p.status)) return;
  if (p.out_dtype == KVQ_OUT_F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * i + 2 * e], o[8 * i + 2 * e + 1]);
        v[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// Partial sums in the workspace, [2 * CTAs][D / 4][slot_rows][4]: partial k's value 4 i + e of row r at
// ws_o[((k * D / 4 + i) * slot_rows + r) * 4 + e], so that the threads of a
// slot, one row each, write and read whole lines.
template <int D>
__device__ __forceinline__ float4* partial_o(const CParams& p, int k, int r) {
  return reinterpret_cast<float4*>(p.ws_o) + static_cast<int64_t>(k) * (D / 4) * p.slot_rows + r;
}

// This row's pieces merged by log-sum-exp in CTA order; the normalised row
// goes to offset orow of the output.  Two pieces' loads are in flight together
// (one at a time took 9.9 us a merge).
template <int D>
__device__ __forceinline__ void merge_row(const CParams& p, const Cut& cut, int r, int64_t orow) {
  auto lse_of = [&](int c) {
    return c <= cut.c1 ? __ldcg(p.ws_lse + static_cast<int64_t>(cut.partial(c)) * p.slot_rows + r) : -INFINITY;
  };
  float M = -INFINITY, L = 0.0f;
#pragma unroll 1
  for (int c = cut.c0; c <= cut.c1; c += 4) {
    float lse[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) lse[k] = lse_of(c + k);
    const float mn = fmaxf(M, fmaxf(fmaxf(lse[0], lse[1]), fmaxf(lse[2], lse[3])));
    if (mn == -INFINITY) continue;   // no piece with weight yet
    L *= fast_exp2(M - mn);
#pragma unroll
    for (int k = 0; k < 4; ++k) L += fast_exp2(lse[k] - mn);
    M = mn;
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
#pragma unroll 1
  for (int i0 = 0; i0 < D / 4; i0 += 8) {
    float o[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
#pragma unroll 1
    for (int c = cut.c0; c <= cut.c1; c += 2) {
      const float la = lse_of(c), lb = lse_of(c + 1);
      const int64_t at = static_cast<int64_t>(i0) * p.slot_rows;
      const float4* sa = partial_o<D>(p, cut.partial(c), r) + at;
      const float4* sb = partial_o<D>(p, cut.partial(min(c + 1, cut.c1)), r) + at;
      float4 va[8], vb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) va[i] = __ldcg(sa + i * p.slot_rows);
#pragma unroll
      for (int i = 0; i < 8; ++i) vb[i] = __ldcg(sb + i * p.slot_rows);
      const float wa = la == -INFINITY ? 0.0f : fast_exp2(la - M) * inv;
      const float wb = lb == -INFINITY ? 0.0f : fast_exp2(lb - M) * inv;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[4 * i] = fmaf(wb, vb[i].x, fmaf(wa, va[i].x, o[4 * i]));
        o[4 * i + 1] = fmaf(wb, vb[i].y, fmaf(wa, va[i].y, o[4 * i + 1]));
        o[4 * i + 2] = fmaf(wb, vb[i].z, fmaf(wa, va[i].z, o[4 * i + 2]));
        o[4 * i + 3] = fmaf(wb, vb[i].w, fmaf(wa, va[i].w, o[4 * i + 3]));
      }
    }
    store_row32(p, D, orow + 4 * i0, o);
  }
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) chunk_attention_kernel(const __grid_constant__ CParams p) {
  using L = CLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  // (by an offset: a pointer rounded up as an integer would lose its address
  // space, and every access would carry a 64-bit generic address)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  int32_t* flag = reinterpret_cast<int32_t*>(smem + L::kOffMisc) + 1;   // merge flags of the two slots
  int32_t* pre = reinterpret_cast<int32_t*>(smem + L::kOffPre);         // units of sequences 0 .. b-1, per KV head
  Walk* walks = reinterpret_cast<Walk*>(smem + L::kOffWalk);
  Split& split = *reinterpret_cast<Split*>(smem + L::kOffSplit);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bar[B_QREADY], 8);
    mbar_init(&bar[B_QEMPTY], 3);   // both issuers, and warp 3
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[B_KFULL0 + s], 8);
      mbar_init(&bar[B_VFULL0 + s], 8);
      mbar_init(&bar[B_KVEMPTY0 + s], 2);
      mbar_init(&bar[B_SFULL0 + s], 1);
      mbar_init(&bar[B_PFIRST0 + s], 4);
      mbar_init(&bar[B_PFULL0 + s], 4);
      mbar_init(&bar[B_ORDY0 + s], 1);
      mbar_init(&bar[B_OFREE0 + s], 4);
      mbar_init(&bar[B_TURN0 + s], 1);
      mbar_init(&bar[B_GROUP0 + s], 4);
    }
    mbar_init(&bar[B_MMADONE], 2);
    mbar_init(&bar[B_EXIT], kExitArrivals);
    fence_barrier_init();
  }
  // (before the dependency wait: the registers of two CTAs with TMEM do not fit
  // an SM, so this never waits for a CTA that could wait for this kernel)
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  // the caches, queries and lengths may come from the kernel before this one
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, kThreads, p.status);
  // (starts that descend: the units may be anything)
  const bool disorder = __syncthreads_or(count_units<kRows>(p, pre, warp, lane, kThreads / 32));
  if (disorder) {
    // nothing to do
  } else if (warp == 1) {
    sum_units(p, pre, lane);
    start_walk<kRows>(p, pre, walks[1], split.N, lane);
  } else if (warp == 2) {
    const int most = start_parts<kRows>(p, walks[2], lane);
    if (lane == 0) split.most = most;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Walk& w = walks[warp];
  const int from = !disorder && split.parts<kRows>(p) ? 2 : 1;   // the warp whose split it is
  const int64_t total = disorder ? 0 : walks[from].left;
  if (total <= 0) {   // the whole CTA: nothing was started
    if (warp == 0) tc::tmem_dealloc(tmem, kTmemCols);
    if (warp == 1 && p.zero_rest) zero_rest_rows<D>(p, disorder, lane);
    return;
  }
  if (warp != from) copy_walk(w, walks[from], lane);
  __syncthreads();   // (that warp's own walk goes on from here)

  // Registers: launched with 96 per thread (checked on the host); per
  // warpgroup 64 + 2 x 88 + 2 x 120 = 5 x 96 (of six such splits the fastest:
  // 48 + 2 x 96 + 2 x 120 takes 1015 us for 2048 tokens on 32K, 72 + 2 x 80 +
  // 2 x 120 911 us).
  if (warp < 4) {
    tc::reg_dealloc<64>();
    if (warp == 0) {
      if (p.zero_rest) zero_rest_rows<D>(p, false, lane);
      // The other roles finish in bounded time: each stops at its first wait
      // that runs out, and a role waits at most a few times per tile.
      const uint64_t deadline = p.wait_ns * static_cast<uint64_t>(8 * min(total, int64_t(1) << 20) + 16) + 4 * kDrainNs;
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
      tc::tmem_dealloc(tmem, kTmemCols);
      return;
    }
    if (warp == 3) {
      // ---------------- the next piece's queries into L2 ----------------
      // One piece ahead of the dequant warps: this warp waits for each piece's
      // queries to be in shared memory and counts among those that free them,
      // so it meets every phase of that barrier in order (a waiter that the
      // others do not wait for can miss two phases and take a later one for its own).
      bool ok = true, more;
      uint32_t piece = 0;
      do {
        more = next_piece<kRows>(p, w, lane);
        for (int r = lane; more && r < w.t.rows; r += 32) {
          const int R = w.rt * kRows + r, tok = R / p.rep, hh = R - tok * p.rep;
          prefetch_l2_bulk(p.q + (w.s.row0 + tok) * p.sq_row + (w.kvh * p.rep + hh) * p.sq_head, D * 2);
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_QREADY], piece & 1, p.status, p.wait_ns));
        if (ok && lane == 0) mbar_arrive(&bar[B_QEMPTY]);
        ++piece;
      } while (ok && more);
      if (lane == 0) mbar_arrive(&bar[B_EXIT]);
      return;
    }
    // ---------------- MMA issuers, one warp per slot ----------------
    const int h = warp - 1;
    const uint32_t id_qk = tc::idesc_f16_f32(kT, kT, false);
    const uint32_t id_pv = tc::idesc_f16_f32(kT, D, true);
    const uint32_t qh = smem_u32(smem + L::kOffQ) + h * L::kQBytes;
    const uint32_t k_base = smem_u32(smem + L::kOffK);
    const uint32_t v_base = smem_u32(smem + L::kOffV);
    const uint32_t d_s = tmem + h * 256, d_o = d_s + 128;
    auto wait_all = [&](int which, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(&bar[which], parity & 1, p.status, p.wait_ns));
    };
    auto issue_qk = [&](int st) {
      const uint32_t kh = k_base + st * L::kQBytes;
      tc::mma_ss<false>(d_s, tc::smem_desc_sw128(qh, 16, 1024), tc::smem_desc_sw128(kh, 16, 1024), id_qk);
#pragma unroll
      for (int s = 1; s < D / 16; ++s) {
        const uint32_t off = (s >> 2) * (kT * 128) + (s & 3) * 32;
        tc::mma_ss<true>(d_s, tc::smem_desc_sw128(qh + off, 16, 1024), tc::smem_desc_sw128(kh + off, 16, 1024), id_qk);
      }
      tc::commit(&bar[B_SFULL0 + h]);
    };
    auto issue_pv = [&](int st, bool first, int hf) {
      const uint32_t vs = v_base + st * L::kQBytes;
      if (hf == 0) {
        const uint64_t v0 = tc::smem_desc_sw128(vs, kT * 128, 1024);
        if (first) tc::mma_ts<false>(d_o, d_s, v0, id_pv);
        else tc::mma_ts<true>(d_o, d_s, v0, id_pv);
      }
#pragma unroll
      for (int s = hf == 0 ? 1 : 2; s < (hf == 0 ? 2 : kT / 16); ++s)
        tc::mma_ts<true>(d_o, d_s + s * 8, tc::smem_desc_sw128(vs + s * 2048, kT * 128, 1024), id_pv);
    };
    // Turns (pieces with both slots): in block g a slot issues P.V of one tile
    // and Q.K^T of the next.  Slot 0 goes after slot 1's block g - 1, slot 1
    // after slot 0's block g; g runs on from piece to piece.
    uint32_t g = 0, jj = 0, sj = 0, mine = 0, piece = 0;
    bool ok = true;
    do {
      const int nh = w.t.rows > kT ? 2 : 1, n = w.n;
      if (h >= nh) {
        // a piece without slot 1: its issuer only frees what the piece's
        // barriers expect of it (and so meets every phase of them in order)
        ok = wait_all(B_QREADY, piece);
        if (ok && lane == 0) mbar_arrive(&bar[B_QEMPTY]);
        for (int j = 0; j < n && ok; ++j, ++jj) {
          ok = wait_all(B_KFULL0 + (jj & 1), jj >> 1) && wait_all(B_VFULL0 + (jj & 1), jj >> 1);
          if (ok && lane == 0) mbar_arrive(&bar[B_KVEMPTY0 + (jj & 1)]);
        }
        if (!ok) break;
        ++piece;
        continue;
      }
      const bool turns = nh == 2;
      auto take_turn = [&]() -> bool {
        if (!turns || (h == 0 && g == 0)) return true;
        return h == 0 ? wait_all(B_TURN0, g - 1) : wait_all(B_TURN1, g);
      };
      auto pass_turn = [&]() {
        if (turns) mbar_arrive(&bar[h == 0 ? B_TURN1 : B_TURN0]);
      };
      // the query rows are free once the piece's last Q.K^T is done
      auto free_queries = [&]() { tc::commit(&bar[B_QEMPTY]); };
      ok = wait_all(B_QREADY, piece) && wait_all(B_KFULL0 + (jj & 1), jj >> 1) && take_turn();
      if (!ok) break;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        issue_qk(jj & 1);
        if (n == 1) free_queries();
        pass_turn();
      }
      __syncwarp();
      if (turns) ++g;
      for (int j = 0; j < n && ok; ++j, ++jj, ++sj) {
        const int st = jj & 1;
        ok = wait_all(B_VFULL0 + st, jj >> 1) && wait_all(B_PFIRST0 + h, sj) && take_turn();
        // the first P.V overwrites O: the previous piece's has been read
        if (ok && j == 0 && mine > 0) ok = wait_all(B_OFREE0 + h, mine - 1);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) issue_pv(st, j == 0, 0);
        __syncwarp();
        ok = wait_all(B_PFULL0 + h, sj);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          issue_pv(st, false, 1);
          tc::commit(&bar[B_ORDY0 + h]);
          tc::commit(&bar[B_KVEMPTY0 + st]);
        }
        __syncwarp();
        if (j + 1 < n) {
          ok = wait_all(B_KFULL0 + ((jj + 1) & 1), (jj + 1) >> 1);
          if (!ok) break;
          tc::fence_after_sync();
        }
        if (tc::elect_one()) {
          if (j + 1 < n) {
            issue_qk((jj + 1) & 1);
            if (j + 2 == n) free_queries();
          }
          pass_turn();
        }
        __syncwarp();
        if (turns) ++g;
      }
      if (!ok) break;
      ++piece;
      ++mine;
    } while (next_piece<kRows>(p, w, lane));
    // every product this warp issued has completed (a commit with none
    // pending arrives at once) before the warp reports that it is done
    if (tc::elect_one()) tc::commit(&bar[B_MMADONE]);
    __syncwarp();
    mbar_wait(&bar[B_MMADONE], 0, p.status, kDrainNs);
    __syncwarp();
    tc::fence_before_sync();
    if (lane == 0) mbar_arrive(&bar[B_EXIT]);
    return;
  }

  if (warp < 12) {
    tc::reg_dealloc<88>();
    // ---------------- dequant warpgroups: half x of the tiles, slot x's queries ----------------
    const int x = (warp - 4) >> 2, t = threadIdx.x & 127;
    uint32_t jj = 0, piece = 0;
    bool ok, bad = false, big = false;
    do {
      uint32_t marks = 0;
      ok = p.bits[w.kvh] == 4 ? dequant_piece<D, 4, PAGED>(p, smem, bar, w, x, jj, piece, bad, marks, t, lane)
                              : dequant_piece<D, 8, PAGED>(p, smem, bar, w, x, jj, piece, bad, marks, t, lane);
      big |= marked_overflow<D>(p, w, marks, 0, 2, lane);
      ++piece;
    } while (ok && next_piece<kRows>(p, w, lane));
    if (bad) report(p.status, KVQ_ERR_INVALID_ARG);
    if (big) report(p.status, KVQ_ERR_NONFINITE);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_EXIT]);
    return;
  }

  // ---------------- softmax warpgroups ----------------
  tc::reg_alloc<120>();
  const int h = (warp - 12) >> 2;           // slot 0 or 1
  const int q4 = warp & 3;                  // TMEM lane quarter
  const int r = q4 * 32 + lane;             // row within the slot
  const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
  const uint32_t s_addr = tmem + lane_off + h * 256;
  const uint32_t o_addr = s_addr + 128;
  const float sl2 = p.scale_log2;
  uint32_t sj = 0, group = 0;
  bool ok = true;
  // the slot's four warps, without a wait that could last for ever
  auto group_sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_GROUP0 + h]);
    ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_GROUP0 + h], group & 1, p.status, p.wait_ns)) && ok;
    ++group;
  };
  do {
    if (h * kT >= w.t.rows) continue;       // a piece without this slot
    const bool four = p.bits[w.kvh] == 4;
    const int R = w.rt * kRows + h * kT + r;
    const bool live = h * kT + r < w.t.rows;
    const int pos0 = w.s.len - w.s.n;
    const int pos = live ? pos0 + R / p.rep : w.t.pos_hi;
    // tiles with columns that some row of the slot does not see: those that
    // begin after mask_from or before mask_below
    const int mask_from = pos0 + (w.rt * kRows + h * kT) / p.rep - (kT - 1);
    const int mask_below =
        p.window > 0 ? pos0 + (w.rt * kRows + min(h * kT + kT, w.t.rows) - 1) / p.rep - p.window + 1 : 0;
    float m_run = -INFINITY, l_run = 0.0f;
    for (int j = 0; j < w.n; ++j, ++sj) {
      const int t0 = w.t.tile(w.i + j) * kT;
      const bool masked = t0 > mask_from || (t0 < mask_below && t0 + kT > p.sinks);
      ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_SFULL0 + h], sj & 1, p.status, p.wait_ns));
      if (!ok) break;
      tc::fence_after_sync();
      // the columns of 32-column chunk c that this row sees, one bit each:
      // up to `lim`, but for those from `sk` to `lo` - 1
      auto seen_bits = [&](int c) -> uint32_t {
        const int lim = pos - t0, lo = p.window > 0 ? pos - p.window + 1 - t0 : 0, sk = p.sinks - t0;
        auto below = [](int x) -> uint32_t { return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u; };
        return below(lim + 1 - 32 * c) & (~below(lo - 32 * c) | below(sk - 32 * c));
      };
      float mxa = -INFINITY, mxb = -INFINITY;
      if (!masked) {
        uint32_t va[32], vb[32];
        auto mx_chunk = [&](const uint32_t (&v)[32]) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            mxa = fmax3(mxa, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            mxb = fmax3(mxb, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
          }
        };
        tc::ld_32x32b_x32(s_addr, va);
        tc::wait_ld(va);
        tc::ld_32x32b_x32(s_addr + 32, vb);
        mx_chunk(va);
        tc::wait_ld(vb);
        tc::ld_32x32b_x32(s_addr + 64, va);
        mx_chunk(vb);
        tc::wait_ld(va);
        tc::ld_32x32b_x32(s_addr + 96, vb);
        mx_chunk(va);
        tc::wait_ld(vb);
        mx_chunk(vb);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // a score that is not seen becomes -infinity, here and in TMEM: the
          // second pass is the same for every tile (2^-infinity = 0)
          uint32_t v[32];
          tc::ld_32x32b_x32(s_addr + c * 32, v);
          const uint32_t m = seen_bits(c);
          tc::wait_ld(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!(m & (1u << i))) v[i] = 0xFF800000u;
            if (i & 1) mxa = fmax3(mxa, __uint_as_float(v[i - 1]), __uint_as_float(v[i]));
          }
          tc::st_32x32b_x32(s_addr + c * 32, v);
        }
        tc::wait_st();
      }
      const float m_tile = fmaxf(mxa, mxb) * sl2;
      float m_use = m_run, alpha = 1.0f;
      if (m_run == -INFINITY || m_tile > m_run + kRescaleThreshold) {
        m_use = fmaxf(m_run, m_tile);
        alpha = (m_run == -INFINITY) ? 0.0f : fast_exp2(m_run - m_use);
        m_run = m_use;
      }
      // rescale O (rare) before any P.V of this tile is issued
      if (__any_sync(0xffffffffu, alpha != 1.0f) && j > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_ORDY0 + h], (sj - 1) & 1, p.status, p.wait_ns));
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tc::ld_32x32b_x32(o_addr + c * 32, v);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tc::st_32x32b_x32(o_addr + c * 32, v);
        }
      }
      auto p_first = [&]() {
        tc::wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B_PFIRST0 + h]);
      };
      float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
      const float neg_m = m_use == -INFINITY ? 0.0f : -m_use;   // (a row that sees nothing yet: every weight is 0)
      uint32_t va[32], vb[32];
      auto p_chunk = [&](const uint32_t (&v)[32], int c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float x0, x1, x2, x3;
          ffma2(x0, x1, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), sl2, neg_m);
          ffma2(x2, x3, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]), sl2, neg_m);
          const float p0 = fast_exp2(x0), p1 = fast_exp2(x1), p2 = fast_exp2(x2), p3 = fast_exp2(x3);
          fadd2(s0, s1, p0, p1);
          fadd2(s2, s3, p2, p3);
          pk[i / 2] = pack_half2(p0, p1);
          pk[i / 2 + 1] = pack_half2(p2, p3);
        }
        tc::st_32x32b_x16(s_addr + c * 16, pk);
      };
      tc::ld_32x32b_x32(s_addr, va);
      tc::wait_ld(va);
      tc::ld_32x32b_x32(s_addr + 32, vb);
      p_chunk(va, 0);
      p_first();
      tc::wait_ld(vb);
      tc::ld_32x32b_x32(s_addr + 64, va);
      p_chunk(vb, 1);
      tc::wait_ld(va);
      tc::ld_32x32b_x32(s_addr + 96, vb);
      p_chunk(va, 2);
      tc::wait_ld(vb);
      p_chunk(vb, 3);
      l_run = l_run * alpha + ((s0 + s1) + (s2 + s3));
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[B_PFULL0 + h]);
    }
    if (!ok) break;
    // ---- end of the piece ----
    ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_ORDY0 + h], (sj - 1) & 1, p.status, p.wait_ns));
    if (!ok) break;
    tc::fence_after_sync();
    const float inv = l_run > 0.0f ? 1.0f / l_run : 0.0f;
    const bool whole = w.n == w.t.n;
    const Cut cut(w, kLead<kRows>);
    const int part = cut.partial(blockIdx.x);
    const int64_t orow = out_offset(p, w, R, D);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t v[32];
      tc::ld_32x32b_x32(o_addr + c * 32, v);
      tc::wait_ld();
      float o[32];
      if (four) {   // column 8m + 2k holds channel 8m + k, column 8m + 2k + 1 channel 8m + 4 + k
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[(i & ~7) | ((i & 3) << 1) | ((i >> 2) & 1)]) * inv;
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[i]) * inv;
      }
      if (!live) continue;
      if (whole) {
        store_row32(p, D, orow + c * 32, o);
      } else {
        float4* dst = partial_o<D>(p, part, h * kT + r) + static_cast<int64_t>(8 * c) * p.slot_rows;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[static_cast<int64_t>(i) * p.slot_rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        if (c == 0)
          p.ws_lse[static_cast<int64_t>(part) * p.slot_rows + h * kT + r] =
              l_run > 0.0f ? m_run + __log2f(l_run) : -INFINITY;
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[B_OFREE0 + h]);
    if (!whole) {
      group_sync();   // every thread's partial is stored
      if (!ok) break;
      // one acquire-release atomic after the group's barrier: its release
      // covers the group's stores, its acquire the other pieces' (released by
      // their own arrivals) for the last arriver
      if (threadIdx.x == 384 + h * kT)
        flag[h] = atom_add_acq_rel_gpu(p.cnt + 2 * cut.c0 + h, 1) + 1 == cut.c1 - cut.c0 + 1 ? 1 : 0;
      group_sync();
      if (!ok) break;
      if (flag[h] == 1) {
        if (live) merge_row<D>(p, cut, h * kT + r, orow);
        if (threadIdx.x == 384 + h * kT) p.cnt[2 * cut.c0 + h] = 0;   // ready for the next call
      }
      group_sync();   // the flag has been read
      if (!ok) break;
    }
  } while (next_piece<kRows>(p, w, lane));
  tc::wait_st();   // P and rescaled O stores of a loop left early have landed
  tc::fence_before_sync();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar[B_EXIT]);
}

// Per device and instantiation, set once under a lock: the kernel's dynamic
// shared-memory limit, and whether it was built with the 96 registers per
// thread that the register split above assumes.  1 = ready, -2 = not usable.
std::mutex g_prep_mu;
int g_prep[64][4] = {};

template <int D, bool PAGED>
int prepare_on_current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -1;
  std::lock_guard<std::mutex> lock(g_prep_mu);
  int& st = g_prep[dev][(D == 128 ? 1 : 0) + (PAGED ? 2 : 0)];
  if (st == 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, chunk_attention_kernel<D, PAGED>) != cudaSuccess || fa.numRegs != 96) {
      st = -2;
    } else if (cudaFuncSetAttribute(chunk_attention_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(CLayout<D>::bytes(4096))) != cudaSuccess) {
      return -1;   // a CUDA error; try again on the next call
    } else {
      st = 1;
    }
  }
  return st;
}
static_assert(CLayout<128>::kOffPre + 1024 + 4097 * 4 <= 232448, "shared memory of the D = 128 kernel");

size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

// Workspace: [cnt: 2 per CTA][lse: 2 partials per CTA][o: the same, D values a row]
int slot_rows(int rows, int rep) {
  const int64_t all = static_cast<int64_t>(rows) * rep;
  return all < kRows ? static_cast<int>(all < 1 ? 1 : all) : kRows;
}
size_t counter_bytes(int ctas) { return align16(static_cast<size_t>(ctas) * 2 * 4); }
size_t lse_bytes(int ctas, int sr) { return align16(static_cast<size_t>(ctas) * 2 * sr * 4); }

template <int D, bool PAGED>
kvq_status launch_d(const CParams& p, cudaStream_t stream) {
  const int prep = prepare_on_current_device<D, PAGED>();
  if (prep == -2) return KVQ_ERR_UNSUPPORTED;
  if (prep != 1) return KVQ_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = CLayout<D>::bytes(p.c.B);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_attention_kernel<D, PAGED>, p) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

size_t chunk_workspace_bytes(int rows, int B, int Hq, int Hkv, int D) {
  (void)B;
  const int ctas = device_sm_count(), sr = slot_rows(rows, Hq / Hkv);
  return counter_bytes(ctas) + lse_bytes(ctas, sr) + static_cast<size_t>(ctas) * 2 * sr * D * 4;
}

kvq_status launch_chunk_attention(const ChunkAttnArgs& a, cudaStream_t stream) {
  CParams p;
  memset(&p, 0, sizeof(p));
  const int D = a.k->D;
  p.c = chunk::view_of(a.chunk, *a.k);
  p.q = a.q;
  p.sq_row = a.sq_row; p.sq_head = a.sq_head;
  p.codes[0] = a.k->codes; p.codes[1] = a.v->codes;
  p.sz[0] = a.k->sz; p.sz[1] = a.v->sz;
  p.out = a.out;
  p.status = a.status;
  p.out_dtype = a.out_dtype; p.Hq = a.Hq; p.Hkv = a.k->Hkv; p.rep = a.Hq / a.k->Hkv;
  p.zero_rest = a.zero_rest ? 1 : 0;
  p.window = a.window; p.sinks = a.sinks;
  p.wait_ns = a.pol.wait_ns;
  p.issue_limit = static_cast<uint32_t>(a.pol.issue_limit);   // (negative: more pieces than any call has)
  p.num_ctas = device_sm_count();
  p.slot_rows = slot_rows(a.chunk.rows, p.rep);
  // units of all sequences (one KV head) are counted in 32 bits
  const int64_t blocks = static_cast<int64_t>(a.chunk.rows) * p.rep / kRows + a.chunk.B;
  if (blocks * (a.chunk.cap / kT + 1 + std::max(kLead<kRows>, kLead<16>)) >= (int64_t(1) << 31)) return KVQ_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.cnt = reinterpret_cast<int32_t*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + counter_bytes(p.num_ctas));
  p.ws_o = reinterpret_cast<float*>(ws + counter_bytes(p.num_ctas) + lse_bytes(p.num_ctas, p.slot_rows));
  const float scale = a.softmax_scale > 0.0f ? a.softmax_scale : 1.0f / sqrtf(static_cast<float>(D));
  p.scale_log2 = scale * 1.4426950408889634f;
  p.codes_bytes = kvq_cache_codes_bytes(a.k);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  // Few rows of a (sequence, KV head): the kernel that puts the keys on the
  // rows' side (a 128-row query tile would be mostly empty).
  const int64_t max_rows = static_cast<int64_t>(p.c.max_chunk) * p.rep;
  if (chunk_narrow_takes(p.c.B, max_rows)) return launch_chunk_narrow(p, D, max_rows, stream);
  if (p.c.bt != nullptr) return D == 128 ? launch_d<128, true>(p, stream) : launch_d<64, true>(p, stream);
  return D == 128 ? launch_d<128, false>(p, stream) : launch_d<64, false>(p, stream);
}

}  // namespace kvq
