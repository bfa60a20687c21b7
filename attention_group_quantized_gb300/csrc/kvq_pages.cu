// kvq_pages.cu -- who has the pages of a pool: room for new tokens, forks that
// share full pages, pages let go, live pages moved together, pages copied.
//
// The decisions are prefix sums over the pool's counts and the slots, small
// (a few KB to a few hundred) and bound by latency: one CTA makes them, each
// thread with a run of its own (two passes over the run around one scan of the
// CTA), so that pages are handed out in a fixed order, lowest first.  The data
// movement they lead to is HBM-bound and goes to a second launch over the
// whole GPU, a programmatic dependent of the first, which finds the list of
// page pairs in the workspace.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyWarps = 4;

// workspace (int32): [pairs, padded][list, src, dst: n_pages + slots each][mark, size: slots each]
struct Scratch {
  int32_t* pairs;           // entries of src and dst
  int32_t* list;            // free pages in order (reserve, fork); where a page goes (compact)
  int32_t* src;
  int32_t* dst;
  int32_t* mark;            // fork: the first pair that names a slot as its to
  int32_t* size;            // fork: the length of a pair's from
};

inline size_t list_words(int n_pages, int slots) {
  return (static_cast<size_t>(n_pages) + slots + 3) / 4 * 4;
}

Scratch scratch_of(int32_t* ws, int n_pages, int slots) {
  const size_t w = list_words(n_pages, slots), m = list_words(0, slots);
  return Scratch{ws, ws + 4, ws + 4 + w, ws + 4 + 2 * w, ws + 4 + 3 * w, ws + 4 + 3 * w + m};
}
constexpr size_t scratch_words(size_t list, size_t marks) { return 4 + 3 * list + 2 * marks; }

struct PParams {
  kvq_page_table t;
  Scratch s;
  const int32_t* from;      // fork: from; free: which; reserve: add
  const int32_t* to;
  int32_t* n_live;
  int32_t* status;
  int32_t n;
};

// Exclusive prefix sum over the CTA's threads; *total gets the sum.
__device__ __forceinline__ int scan_cta(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  if (w == 0) {
    int y = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    warp_sums[lane] = y;
  }
  __syncthreads();
  const int before = (w > 0 ? warp_sums[w - 1] : 0) + x - v;
  *total = warp_sums[kPlanWarps - 1];
  __syncthreads();
  return before;
}

// The run of n items that a thread has.
__device__ __forceinline__ void run_of(int n, int& i0, int& i1) {
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  i0 = min(static_cast<int>(threadIdx.x) * per, n);
  i1 = min(i0 + per, n);
}

__device__ __forceinline__ int pages_of(int len) { return (len + KVQ_TILE_TOKENS - 1) / KVQ_TILE_TOKENS; }

// The lowest `want` free pages (all of them where there are fewer), in order,
// to list; returns the number of free pages.
__device__ __forceinline__ int list_free(const PParams& p, int want, int* warp_sums) {
  int i0, i1, total, n = 0;
  run_of(p.t.n_pages, i0, i1);
#pragma unroll 4
  for (int i = i0; i < i1; ++i) n += p.t.refs[i] == 0;
  int at = scan_cta(n, warp_sums, &total);
  if (n > 0)
    for (int i = i0; i < i1 && at < want; ++i)
      if (p.t.refs[i] == 0) p.s.list[at++] = i;
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const __grid_constant__ PParams p) {
  __shared__ int sums[32];
  grid_dependency_wait();
  grid_launch_dependents();
  int i0, i1, need_all;
  run_of(p.t.slots, i0, i1);
  // pages that a slot needs; -1: nothing to do for it
  auto need_of = [&](int s, int& len, int& add, bool reporter) -> int {
    add = p.from[s];
    len = p.t.seq_lens[s];
    const int64_t cap = static_cast<int64_t>(p.t.max_pages) * KVQ_TILE_TOKENS;
    if (add == 0 && len >= 0 && len <= cap) return -1;
    if (add < 0 || len < 0 || static_cast<int64_t>(len) + add > cap) {
      if (reporter) report(p.status, KVQ_ERR_INVALID_ARG);
      return -1;
    }
    return pages_of(len + add) - pages_of(len);
  };
  int n = 0, len, add;
  for (int s = i0; s < i1; ++s) n += max(need_of(s, len, add, true), 0);
  int at = scan_cta(n, sums, &need_all);
  const int have = list_free(p, need_all, sums);
  for (int s = i0; s < i1; ++s) {
    const int need = need_of(s, len, add, false);
    if (need < 0) continue;
    if (need > 0 && at + need > have) {
      report(p.status, KVQ_ERR_NO_PAGES);
    } else {
      int32_t* row = p.t.table + static_cast<int64_t>(s) * p.t.max_pages + pages_of(len);
      for (int j = 0; j < need; ++j) {
        const int page = p.s.list[at + j];
        row[j] = page;
        p.t.refs[page] = 1;
      }
      p.t.seq_lens[s] = len + add;
    }
    at += need;
  }
}

__global__ void __launch_bounds__(kPlanThreads) fork_kernel(const __grid_constant__ PParams p) {
  __shared__ int sums[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, slots = p.t.slots;
  const int64_t cap = static_cast<int64_t>(p.t.max_pages) * KVQ_TILE_TOKENS;
  for (int s = tid; s < slots; s += kPlanThreads) p.s.mark[s] = INT32_MAX;
  __syncthreads();
  // pairs that hold: size[i] = the length to copy, else -1, and src[i] the
  // partly filled last page, -1 where there is none in the pool (lengths are
  // read before any is written)
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int f = p.from[i], t = p.to[i];
    int size = -1, last = -1;
    if (f >= 0 && f < slots && t >= 0 && t < slots && p.t.seq_lens[t] == 0) {
      const int len = p.t.seq_lens[f];
      if (len >= 0 && len <= cap) {
        size = len;
        atomicMin(&p.s.mark[t], i);
        if (len % KVQ_TILE_TOKENS != 0) {
          last = p.t.table[static_cast<int64_t>(f) * p.t.max_pages + len / KVQ_TILE_TOKENS];
          if (last < 0 || last >= p.t.n_pages) last = -1;
        }
      }
    }
    if (size < 0) report(p.status, KVQ_ERR_INVALID_ARG);
    p.s.size[i] = size;
    p.s.src[i] = last;
    p.s.dst[i] = -1;
  }
  if (tid == 0) *p.s.pairs = p.n;
  __syncthreads();
  int i0, i1, need_all, n = 0;
  run_of(p.n, i0, i1);
  for (int i = i0; i < i1; ++i) {
    if (p.s.size[i] >= 0 && p.s.mark[p.to[i]] != i) {   // another pair's to
      report(p.status, KVQ_ERR_INVALID_ARG);
      p.s.size[i] = p.s.src[i] = -1;
    }
    n += p.s.src[i] >= 0;
  }
  int at = scan_cta(n, sums, &need_all);
  const int have = list_free(p, need_all, sums);
  for (int i = i0; i < i1; ++i) {
    const int size = p.s.size[i];
    if (size < 0) continue;
    const int f = p.from[i], t = p.to[i], last = size / KVQ_TILE_TOKENS;
    if (p.s.src[i] >= 0) {
      if (at >= have) {
        report(p.status, KVQ_ERR_NO_PAGES);
        p.s.size[i] = p.s.src[i] = -1;
        ++at;
        continue;
      }
      const int page = p.s.list[at++];
      p.s.dst[i] = page;
      p.t.table[static_cast<int64_t>(t) * p.t.max_pages + last] = page;
      p.t.refs[page] = 1;
    } else if (size % KVQ_TILE_TOKENS != 0) {            // outside the pool: copied as it stands
      report(p.status, KVQ_ERR_INVALID_ARG);
      p.t.table[static_cast<int64_t>(t) * p.t.max_pages + last] =
          p.t.table[static_cast<int64_t>(f) * p.t.max_pages + last];
    }
    p.t.seq_lens[t] = size;
  }
}

// A warp per listed slot.
__global__ void __launch_bounds__(128) free_kernel(const __grid_constant__ PParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (i >= p.n) return;
  const int s = p.from[i];
  if (s < 0 || s >= p.t.slots) {
    if (lane == 0) report(p.status, KVQ_ERR_INVALID_ARG);
    return;
  }
  // (the exchange: of two that list the same slot, one gets its length)
  int len = lane == 0 ? atomicExch(&p.t.seq_lens[s], 0) : 0;
  len = __shfl_sync(0xffffffffu, len, 0);
  if (len < 0 || len > static_cast<int64_t>(p.t.max_pages) * KVQ_TILE_TOKENS) {
    if (lane == 0) report(p.status, KVQ_ERR_INVALID_ARG);
    return;
  }
  const int32_t* row = p.t.table + static_cast<int64_t>(s) * p.t.max_pages;
  for (int j = lane; j < pages_of(len); j += 32) {
    const int page = row[j];
    if (page < 0 || page >= p.t.n_pages) {
      report(p.status, KVQ_ERR_INVALID_ARG);
    } else if (atomicSub(&p.t.refs[page], 1) <= 0) {   // free already
      atomicAdd(&p.t.refs[page], 1);
      report(p.status, KVQ_ERR_INVALID_ARG);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_kernel(const __grid_constant__ PParams p) {
  __shared__ int sums[32];
  grid_dependency_wait();
  grid_launch_dependents();
  int i0, i1, live_all, moves;
  run_of(p.t.n_pages, i0, i1);
  int n = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) n += p.t.refs[i] > 0;
  scan_cta(n, sums, &live_all);
  if (threadIdx.x == 0 && p.n_live != nullptr) *p.n_live = live_all;
  // sources: live pages from live_all on; destinations: the other pages before
  // it -- as many
  int ns = 0, nd = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const bool live = p.t.refs[i] > 0;
    ns += live && i >= live_all;
    nd += !live && i < live_all;
  }
  int as = scan_cta(ns, sums, &moves), ad = scan_cta(nd, sums, &moves);
  for (int i = i0; i < i1; ++i) {
    const bool live = p.t.refs[i] > 0;
    p.s.list[i] = i;
    if (live && i >= live_all) p.s.src[as++] = i;
    if (!live && i < live_all) p.s.dst[ad++] = i;
  }
  if (threadIdx.x == 0) *p.s.pairs = moves;
  __syncthreads();
  for (int m = threadIdx.x; m < moves; m += kPlanThreads) {
    const int src = p.s.src[m], dst = p.s.dst[m];
    p.s.list[src] = dst;
    p.t.refs[dst] = p.t.refs[src];
    p.t.refs[src] = 0;
  }
}

// Page pairs copied: a warp per (pair, KV head, K or V), whole rows of 16-byte
// words.  After a plan the pairs are in the workspace, and the same launch does
// what else takes more than one CTA: the entries of the full pages that a fork
// shares, a warp per pair (in the planning CTA they took most of its time: 128
// forks of up to 125 pages with what goes with them 24.3 us, 18.5 us here), or the page table's
// entries renamed after a compaction, a warp per slot.
struct CParams {
  const int32_t* pairs;     // number of pairs, null: n
  const int32_t* src;
  const int32_t* dst;
  uint8_t* codes[2];
  uint32_t* sz[2];
  int8_t* b_codes;
  float* b_scales;
  const int32_t* remap;     // compact: where a page goes, null: nothing to rename
  const int32_t* from;      // fork: the pairs' slots and lengths (-1: not forked), null: none
  const int32_t* to;
  const int32_t* size;
  kvq_page_table t;
  int32_t* status;
  int32_t n, n_pages, Hkv, D;
  int64_t codes_bytes;      // size of each code buffer (the debug build's index checks)
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

// `words` 16-byte words by a warp, 8 in flight a lane.
__device__ __forceinline__ void copy_words(uint4* dst, const uint4* src, int words, int lane) {
  for (int i0 = 0; i0 < words; i0 += 256) {
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j * 32 + lane < words) v[j] = src[i0 + j * 32 + lane];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j * 32 + lane < words) dst[i0 + j * 32 + lane] = v[j];
  }
}

__global__ void __launch_bounds__(kCopyWarps * 32) copy_pages_kernel(const __grid_constant__ CParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w0 = static_cast<int64_t>(blockIdx.x) * kCopyWarps + (threadIdx.x >> 5);
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kCopyWarps;
  const int n = p.pairs != nullptr ? *p.pairs : p.n;
  const int G = p.D / KVQ_GROUP;
  const int64_t units = static_cast<int64_t>(n) * p.Hkv * 2;
  for (int64_t u = w0; u < units; u += nw) {
    const int64_t ph = u >> 1;
    const int job = static_cast<int>(u & 1);
    const int i = static_cast<int>(ph / p.Hkv), h = static_cast<int>(ph - static_cast<int64_t>(i) * p.Hkv);
    const int s = p.src[i], d = p.dst[i];
    if (s < 0 || d < 0) continue;
    if (s >= p.n_pages || d >= p.n_pages) {
      if (lane == 0) report(p.status, KVQ_ERR_INVALID_ARG);
      continue;
    }
    if (s == d) continue;
    const int bytes = KVQ_TILE_TOKENS * p.D * p.bits[h] / 8;
    const int64_t so = p.plane_off[h] + static_cast<int64_t>(s) * bytes, dO = p.plane_off[h] + static_cast<int64_t>(d) * bytes;
    if (!KVQ_IN_RANGE(so + bytes <= p.codes_bytes && dO + bytes <= p.codes_bytes, p.status)) continue;
    copy_words(reinterpret_cast<uint4*>(p.codes[job] + dO), reinterpret_cast<const uint4*>(p.codes[job] + so), bytes / 16,
               lane);
    const int64_t hs = static_cast<int64_t>(h) * p.n_pages + s, hd = static_cast<int64_t>(h) * p.n_pages + d;
    uint4* sz = reinterpret_cast<uint4*>(p.sz[job]);
    copy_words(sz + hd * (KVQ_TILE_TOKENS * G / 4), sz + hs * (KVQ_TILE_TOKENS * G / 4), KVQ_TILE_TOKENS * G / 4, lane);
    if (job == 0 && p.b_codes != nullptr) {
      uint4* bc = reinterpret_cast<uint4*>(p.b_codes);
      if (lane < 4 * G) bc[hd * 4 * G + lane] = bc[hs * 4 * G + lane];
      if (lane < G) p.b_scales[hd * G + lane] = p.b_scales[hs * G + lane];
    }
  }
  if (p.size != nullptr) {
    // (from the last warp down: the first ones copy)
    for (int64_t i = nw - 1 - w0; i < n; i += nw) {
      const int full = p.size[i] / KVQ_TILE_TOKENS;   // (-1: 0)
      const int32_t* row = p.t.table + static_cast<int64_t>(p.from[i]) * p.t.max_pages;
      int32_t* out = p.t.table + static_cast<int64_t>(p.to[i]) * p.t.max_pages;
#pragma unroll 4
      for (int j = lane; j < full; j += 32) {
        const int page = row[j];
        out[j] = page;
        if (page >= 0 && page < p.n_pages) atomicAdd(&p.t.refs[page], 1);
        else report(p.status, KVQ_ERR_INVALID_ARG);
      }
    }
  }
  if (p.remap == nullptr) return;
  for (int64_t s = w0; s < p.t.slots; s += nw) {
    const int len = p.t.seq_lens[s];
    if (len < 0 || len > static_cast<int64_t>(p.t.max_pages) * KVQ_TILE_TOKENS) {
      if (lane == 0) report(p.status, KVQ_ERR_INVALID_ARG);
      continue;
    }
    int32_t* row = p.t.table + s * p.t.max_pages;
    for (int j = lane; j < pages_of(len); j += 32) {
      const int page = row[j];
      if (page >= 0 && page < p.n_pages) row[j] = p.remap[page];
      else report(p.status, KVQ_ERR_INVALID_ARG);
    }
  }
}

template <class Kernel, class Params>
cudaError_t launch(Kernel kernel, const Params& p, int64_t blocks, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

PParams plan_params(const PagesArgs& a) {
  PParams p;
  p.t = a.t;
  p.s = scratch_of(a.ws, a.t.n_pages, a.t.slots);
  p.from = a.from;
  p.to = a.to;
  p.n_live = a.n_live;
  p.status = a.status;
  p.n = a.n;
  return p;
}

// most: pairs that the list can have
cudaError_t launch_copy(const PagesArgs& a, const int32_t* pairs, const int32_t* src, const int32_t* dst, int64_t most,
                        const int32_t* remap, const int32_t* size, cudaStream_t stream) {
  CParams p;
  const kvq_cache& k = *a.k;
  p.pairs = pairs;
  p.src = src;
  p.dst = dst;
  p.codes[0] = k.codes; p.codes[1] = a.v->codes;
  p.sz[0] = k.sz; p.sz[1] = a.v->sz;
  p.b_codes = a.bounds.codes;
  p.b_scales = a.bounds.scales;
  p.remap = remap;
  p.from = a.from;
  p.to = a.to;
  p.size = size;
  p.t = a.t;
  p.status = a.status;
  p.n = a.n;
  p.n_pages = k.B;
  p.Hkv = k.Hkv;
  p.D = k.D;
  p.codes_bytes = a.layout.off4 + static_cast<int64_t>(a.layout.n4) * k.B * k.Tcap * (k.D / 2);
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  int64_t warps = most * k.Hkv * 2;
  if (remap != nullptr) warps = std::max<int64_t>(warps, a.t.slots);
  if (size != nullptr) warps += a.n;
  const int64_t blocks = std::min<int64_t>((warps + kCopyWarps - 1) / kCopyWarps, int64_t(32) * device_sm_count());
  return launch(copy_pages_kernel, p, std::max<int64_t>(blocks, 1), kCopyWarps * 32, stream);
}

}  // namespace

size_t pages_workspace_bytes(int n_pages, int slots) {
  return scratch_words(list_words(n_pages, slots), list_words(0, slots)) * 4;
}

cudaError_t launch_pages_reserve(const PagesArgs& a, cudaStream_t stream) {
  return launch(reserve_kernel, plan_params(a), 1, kPlanThreads, stream);
}

cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t stream) {
  const PParams p = plan_params(a);
  const cudaError_t e = launch(fork_kernel, p, 1, kPlanThreads, stream);
  if (e != cudaSuccess) return e;
  return launch_copy(a, p.s.pairs, p.s.src, p.s.dst, a.n, nullptr, p.s.size, stream);
}

cudaError_t launch_pages_free(const PagesArgs& a, cudaStream_t stream) {
  PParams p = {};
  p.t = a.t;
  p.from = a.from;
  p.status = a.status;
  p.n = a.n;
  return launch(free_kernel, p, (static_cast<int64_t>(a.n) + 3) / 4, 128, stream);
}

cudaError_t launch_pages_compact(const PagesArgs& a, cudaStream_t stream) {
  const PParams p = plan_params(a);
  const cudaError_t e = launch(compact_kernel, p, 1, kPlanThreads, stream);
  if (e != cudaSuccess) return e;
  return launch_copy(a, p.s.pairs, p.s.src, p.s.dst, a.t.n_pages / 2, p.s.list, nullptr, stream);
}

cudaError_t launch_copy_pages(const PagesArgs& a, cudaStream_t stream) {
  return launch_copy(a, nullptr, a.from, a.to, a.n, nullptr, nullptr, stream);
}

}  // namespace kvq
