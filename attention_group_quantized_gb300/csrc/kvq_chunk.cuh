// kvq_chunk.cuh -- where the packed rows of a ragged chunk live: row r of
// sequence b (start[b] <= r < start[b + 1]) is cache position
// seq_lens[b] - (start[b + 1] - r).  Shared by the chunk append, the read-back
// and the chunk attention.
#pragma once

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace chunk {

// A chunk and the cache storage its positions index (a page pool when bt is set).
struct View {
  const int32_t* start;      // [B + 1]
  const int32_t* seq_lens;   // [B]
  const int32_t* bt;         // [B][bt_stride] page ids or null
  int32_t B, rows, max_chunk;
  int32_t bt_stride;
  int32_t cap;               // tokens a sequence may have
  int32_t pB, pT;            // storage: pB sequences (or pages) of pT tokens
};

inline View view_of(const ChunkDesc& c, const kvq_cache& storage) {
  View v;
  v.start = c.start; v.seq_lens = c.seq_lens; v.bt = c.bt;
  v.B = c.B; v.rows = c.rows; v.max_chunk = c.max_chunk;
  v.bt_stride = c.bt_max_pages;
  v.cap = c.cap;
  v.pB = storage.B; v.pT = storage.Tcap;
  return v;
}

// Sequence b's new tokens: its first row and their number (0 when the
// description is unusable, which `bad` tells), and its length.
struct Seq {
  int32_t row0, n, len;
  bool bad, down;   // down: it ends before it starts
};
__device__ __forceinline__ Seq sequence(const View& c, int b) {
  Seq s;
  s.row0 = c.start[b];
  const int32_t end = c.start[b + 1];
  s.len = c.seq_lens[b];
  s.down = end < s.row0;
  s.bad = s.row0 < 0 || end < s.row0 || end > c.rows || s.len < 0 || s.len > c.cap;
  s.n = s.bad ? 0 : end - s.row0;
  if (s.n > s.len || s.n > c.max_chunk) {
    s.bad = true;
    s.n = 0;
  }
  return s;
}

// The last b in [0, B) with start[b] <= r: the sequence of row r when the
// starts ascend.  32 candidates per step (one load each), by a whole warp for
// one r; start[0] is taken as <= r.
__device__ __forceinline__ int find_sequence(const int32_t* start, int B, int r, int lane) {
  int lo = 0, n = B;   // answer in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane == 0 || (lane * step < n && start[i] <= r);
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = 31 - __clz(m);     // (ascending starts: a run of ones)
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// Where a token of the cache is stored: its row among a head's rows
// (storage * pT + slot), -1 for a page id outside the pool.
__device__ __forceinline__ int64_t storage_row(const View& c, int b, int pos) {
  if (c.bt == nullptr) return static_cast<int64_t>(b) * c.pT + pos;
  const int page = c.bt[static_cast<int64_t>(b) * c.bt_stride + pos / KVQ_TILE_TOKENS];
  if (page < 0 || page >= c.pB) return -1;
  return static_cast<int64_t>(page) * KVQ_TILE_TOKENS + pos % KVQ_TILE_TOKENS;
}

// The 64-token storage block (a page, or that much of a sequence) of tokens
// 64 i .. 64 i + 63 of sequence b; a page id outside the pool is reported and
// block 0 returned.  (int: the host refuses storage of 2^31 blocks.)
__device__ __forceinline__ int storage_block(const View& c, int b, int i, int32_t* status) {
  if (c.bt == nullptr) return b * (c.pT / KVQ_TILE_TOKENS) + i;
  if (!KVQ_IN_RANGE(i < c.bt_stride, status)) return 0;
  const int page = c.bt[static_cast<int64_t>(b) * c.bt_stride + i];
  if (page >= 0 && page < c.pB) return page;
  report(status, KVQ_ERR_INVALID_ARG);
  return 0;
}

// Whether packed row r0 + lane (of those below c.rows) is one that no usable
// sequence has (the whole warp).
__device__ __forceinline__ bool row_is_free(const View& c, int r0, int lane) {
  int b = find_sequence(c.start, c.B, r0, lane);
  const int r = r0 + lane;
  if (r >= c.rows) return false;
  while (b + 1 < c.B && c.start[b + 1] <= r) ++b;
  const Seq s = sequence(c, b);
  return r < s.row0 || r >= s.row0 + s.n;   // (n = 0 for one that is left out)
}

constexpr int64_t kNoRow = -1;     // belongs to no usable sequence
constexpr int64_t kBadPage = -2;   // its page lies outside the pool

// Storage rows of the packed rows r0 + lane (lanes whose row is >= c.rows get
// kNoRow).  The whole warp takes part; `report` says whether this warp is
// the one that reports what is wrong.
__device__ __forceinline__ int64_t locate_rows(const View& c, int r0, int lane, int count, bool reporter,
                                               int32_t* status) {
  int b = find_sequence(c.start, c.B, r0, lane);
  const int r = r0 + lane;
  if (lane >= count || r >= c.rows) return kNoRow;
  while (b + 1 < c.B && c.start[b + 1] <= r) ++b;
  const Seq s = sequence(c, b);
  if (s.bad) {
    if (reporter) report(status, KVQ_ERR_INVALID_ARG);
    return kNoRow;
  }
  if (r < s.row0 || r >= s.row0 + s.n) return kNoRow;
  const int64_t row = storage_row(c, b, s.len - s.n + (r - s.row0));
  if (row < 0) {
    if (reporter) report(status, KVQ_ERR_INVALID_ARG);
    return kBadPage;
  }
  return row;
}

// A bad sequence without rows of its own would go unseen by the rows' own
// checks: one block of a launch looks at every sequence.
__device__ __forceinline__ void check_sequences(const View& c, int tid, int nthr, int32_t* status) {
  for (int b = tid; b < c.B; b += nthr)
    if (sequence(c, b).bad) report(status, KVQ_ERR_INVALID_ARG);
  if (tid == 0 && c.start[0] != 0) report(status, KVQ_ERR_INVALID_ARG);
}

}  // namespace chunk
}  // namespace kvq
