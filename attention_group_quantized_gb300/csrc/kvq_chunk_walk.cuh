// kvq_chunk_walk.cuh -- the work list of the chunk attention kernels: every
// (sequence, KV head, row block, 128-token key tile) in order, cut into equal
// contiguous ranges, one per CTA ("stream-K"), so that ragged lengths and few
// rows over a long cache load every SM alike.  A segment is a row block (ROWS
// packed rows, token * rep + head) of one (sequence, KV head); the run of a
// segment's tiles inside one CTA's range is a piece.  The ranges are equal in
// units: a unit per tile, and kLead<ROWS> before each segment's first for what
// a segment costs whatever its length (queries, first codes, output) -- with
// equal tiles alone, CTAs of many short segments finished last.
#pragma once

#include <cstdint>

#include "kvq_chunk.cuh"
#include "kvq_tile.cuh"

namespace kvq {
namespace chunk_walk {

using tile::kT;

constexpr float kRescaleThreshold = 8.0f;  // log2 units: the running max moves (and O is rescaled) beyond it
// What a kernel waits for before it may end (its own products and copies in
// flight) takes microseconds, and is given this long whatever the call's limit.
constexpr uint64_t kDrainNs = kDefaultWaitLimitNs;

struct CParams {
  chunk::View c;
  const uint16_t* q;
  int64_t sq_row, sq_head;
  const uint8_t* codes[2];          // K, V code buffers
  const uint32_t* sz[2];
  int32_t* cnt;                     // [CTAs][2] arrivals at a cut segment, by its first CTA and slot
  float* ws_lse;                    // [2 * CTAs][slot_rows], log2 domain
  float* ws_o;                      // [2 * CTAs][slot_rows * D], in the kernel's own order
  void* out;
  int32_t* status;
  int32_t out_dtype, zero_rest, Hq, Hkv, rep, window, sinks, num_ctas, slot_rows;
  float scale_log2;
  int64_t codes_bytes;              // size of each code buffer (the debug build's index checks)
  uint64_t wait_ns;                 // bounded-wait limit
  uint32_t issue_limit;             // test only: pieces whose queries a CTA makes ready
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

// (0, 2, 3, 4, 6 measured in the 256-row kernel for 16 sequences of 1 to 286 new
// tokens: 189, 172, 170, 170, 171 us; 0, 2, 4, 6, 8 in the narrow one for 32
// sequences of 1 to 4 new tokens on 100 to 6000: 84, 64, 59, 59, 59 us)
template <int ROWS>
constexpr int kLead = ROWS == 256 ? 4 : 6;

// A segment's key tiles: those that some row of the block sees, in order.
// Index i of the list is tile (i < ns ? i : i + skip).
struct Tiles {
  int n, ns, skip;
  int pos_lo, pos_hi;    // positions of the block's first and last row
  int rows;              // its rows
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : i + skip; }
};
template <int ROWS>
__device__ __forceinline__ Tiles segment_tiles(const CParams& p, const chunk::Seq& s, int rt) {
  Tiles t;
  t.rows = min(ROWS, s.n * p.rep - rt * ROWS);
  t.pos_lo = s.len - s.n + rt * ROWS / p.rep;
  t.pos_hi = s.len - s.n + (rt * ROWS + t.rows - 1) / p.rep;
  t.n = t.pos_hi / kT + 1;
  t.ns = t.skip = 0;
  if (p.window > 0) {
    const int fw = max(t.pos_lo - p.window + 1, 0) / kT;
    t.ns = min((min(p.sinks, t.pos_hi + 1) + kT - 1) / kT, fw);
    t.skip = fw - t.ns;
    t.n -= t.skip;
  }
  return t;
}
template <int ROWS>
__device__ __forceinline__ int row_blocks(const CParams& p, const chunk::Seq& s) {
  return (s.n * p.rep + ROWS - 1) / ROWS;
}

// A warp's walk through its CTA's range of the work list, piece by piece.  It
// lives in shared memory: the roles' loops need their registers.
struct Walk {
  int64_t left;          // units of the range from the piece's first on
  int64_t seg;           // the first unit of the piece's segment
  int b, kvh, rt, i;     // the piece starts at tile index i of this segment
  chunk::Seq s;
  Tiles t;
  int n, units;          // tiles and units of the piece
  int C;                 // CTAs that share the N units of the work list (N = 0: parts of the segment, start_parts)
  int64_t N;
};
static_assert(sizeof(Walk) <= 128, "room for a Walk per warp");

// u: the piece's first unit within its segment.  A range that ends in a
// segment's lead has no piece there.
template <int ROWS>
__device__ __forceinline__ void open_piece(const CParams& p, Walk& w, int u) {
  w.t = segment_tiles<ROWS>(p, w.s, w.rt);
  w.units = static_cast<int>(min(static_cast<int64_t>(w.t.n + kLead<ROWS> - u), w.left));
  w.i = max(u - kLead<ROWS>, 0);
  w.n = u + w.units - kLead<ROWS> - w.i;
  if (w.n <= 0) w.left = 0;
}
// To the next piece (the whole warp; lane 0 does it); false at the range's end.
template <int ROWS>
__device__ __forceinline__ bool next_piece(const CParams& p, Walk& w, int lane) {
  __syncwarp();
  if (lane == 0) {
    w.left -= w.units;
    w.seg += w.t.n + kLead<ROWS>;   // (a piece with another after it ends its segment)
    if (w.left > 0) {
      if (++w.rt >= row_blocks<ROWS>(p, w.s)) {
        w.rt = 0;
        if (++w.kvh >= p.Hkv) {
          w.kvh = 0;
          do {
            ++w.b;
            w.s = chunk::sequence(p.c, w.b);
          } while (w.s.n == 0);
        }
      }
      open_piece<ROWS>(p, w, 0);
    }
  }
  __syncwarp();
  return w.left > 0;
}

// Tokens that a segment's queries see: below `end`, from `lo` on or below the sinks.
struct Seen {
  int end, lo;
  __device__ __forceinline__ Seen(const CParams& p, const Walk& w)
      : end(w.t.pos_hi + 1), lo(p.window > 0 ? w.t.pos_lo - p.window + 1 : 0) {}
};

// The operands are fp16: a group whose scale and zero point can stand for a
// value that rounds to infinity there (65520 and more) is reported if a query
// sees it.  Smaller scales than kBigScale (as fp16 bits) never do.
template <int BITS>
constexpr uint32_t kBigScale = BITS == 8 ? 0x5C04u /* 257 */ : 0x6C44u /* 4368 */;
__device__ __forceinline__ bool overflows(uint32_t word, int bits) {
  const float qmax = static_cast<float>((1 << bits) - 1);
  const float s = fabsf(half_lo(word)), z = half_hi(word);
  return !(s * fmaxf(z, qmax - z) < 65520.0f);
}

// Output offset of packed row R of a sequence and KV head.
__device__ __forceinline__ int64_t out_offset(const CParams& p, const Walk& w, int R, int D) {
  const int tok = R / p.rep, hh = R - tok * p.rep;
  return ((static_cast<int64_t>(w.s.row0) + tok) * p.Hq + w.kvh * p.rep + hh) * D;
}

// The rows that no usable sequence has become zeros (zero_rest), by one warp of
// each CTA, 32 rows in turn; all rows where the starts descend.
template <int D>
__device__ __forceinline__ void zero_rest_rows(const CParams& p, bool disorder, int lane) {
  const int n = p.Hq * D / (p.out_dtype == KVQ_OUT_F32 ? 4 : 8);   // 16-byte stores of a row
#pragma unroll 1
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * 32; r0 < p.c.rows; r0 += static_cast<int64_t>(p.num_ctas) * 32) {
    const int first = static_cast<int>(r0);
    const bool mine = disorder ? first + lane < p.c.rows : chunk::row_is_free(p.c, first, lane);
    for (unsigned left = __ballot_sync(0xffffffffu, mine); left != 0u; left &= left - 1) {
      uint4* row = static_cast<uint4*>(p.out) + (r0 + __ffs(left) - 1) * n;
      for (int i = lane; i < n; i += 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// Units of a sequence for one KV head (the whole warp, a lane per row block).
template <int ROWS>
__device__ __forceinline__ int32_t sequence_units(const CParams& p, const chunk::Seq& s, int lane) {
  const int nrt = row_blocks<ROWS>(p, s);
  int32_t n = 0;
  for (int rt = lane; rt < nrt; rt += 32) n += segment_tiles<ROWS>(p, s, rt).n + kLead<ROWS>;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// pre[b + 1] = units of sequence b for one KV head: a warp per sequence.
// Returns whether the starts of this warp's sequences descend somewhere:
// sequences that ascend share no row, so their rows are at most the call's; of
// others two could write one row, and the units could pass 32 bits.
template <int ROWS>
__device__ __forceinline__ bool count_units(const CParams& p, int32_t* pre, int warp, int lane, int warps) {
  bool down = false;
  for (int b = warp; b < p.c.B; b += warps) {
    const chunk::Seq s = chunk::sequence(p.c, b);
    down |= s.down;
    const int32_t n = sequence_units<ROWS>(p, s, lane);
    if (lane == 0) pre[b + 1] = n;
  }
  return down;
}

// The counts' prefix sums in place: pre[b] = units of sequences 0 .. b - 1 (one warp).
__device__ __forceinline__ void sum_units(const CParams& p, int32_t* pre, int lane) {
  int32_t carry = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    int32_t n = b0 + lane < p.c.B ? pre[b0 + lane + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += v;
    }
    if (b0 + lane < p.c.B) pre[b0 + lane + 1] = carry + n;
    carry += __shfl_sync(0xffffffffu, n, 31);
  }
  if (lane == 0) pre[0] = 0;
}

// a b / c for a, b, c >= 0: in 32 bits when the product fits (a 64-bit division
// is a long software sequence, and a CTA's start and every piece's end wait
// for a few of them).
__device__ __forceinline__ int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  const int64_t ab = a * b;
  if (((ab | c) >> 32) == 0) return static_cast<uint32_t>(ab) / static_cast<uint32_t>(c);
  return ab / c;
}

// Costs in units (about one tile's time).  kCutCost: what ranges that ignore the
// segments' ends cost a CTA over one piece each (second pieces, partials,
// merges); kJoinCost: what parts of a segment cost over all of it, kPartsSlack
// more than that before they are preferred to such ranges; kMaxParts: with more
// parts the ranges were as fast or faster.  Measured (us; ranges, whole
// segments, parts), 64 segments of 16 rows on 500, 1000, 2000, 3000, 4000, 8000
// tokens: 15.3 18.8 23.0 25.7 28.4 41.4, 12.5 16.3 23.7 31.3 38.8 69.7, - - 20.2
// 23.9 27.7 43.0; of 120 rows on 100, 1000, 2000, 3000: 17.3 29.3 34.1 39.8, 12.7
// 23.8 34.8 47.2, - 25.3 29.9 35.9; 8 segments of 256 rows on 2000 in 17 parts:
// 50 against 53.
constexpr int kCutCost = 14, kJoinCost = 4, kPartsSlack = 3, kMaxParts = 3;

// How the work was split (one per CTA, in shared memory).
struct Split {
  int64_t N;       // units of the work list
  int most;        // start_parts' tiles of a CTA, or -1
  template <int ROWS>
  __device__ __forceinline__ bool parts(const CParams& p) const {
    return most >= 0 && static_cast<int64_t>(most + kLead<ROWS> - kCutCost) * p.num_ctas <= N;
  }
};

// No more segments than CTAs: an equal number m of CTAs for each, which take
// equal parts of its tiles (m = 1 cuts none), so that every CTA has one piece at
// most.  Opens this CTA's, if it has one; the tiles that a CTA has at most (with
// m > 1 and what the parts cost), or -1 for more segments than CTAs (one warp,
// while another one runs start_walk).
template <int ROWS>
__device__ __forceinline__ int start_parts(const CParams& p, Walk& w, int lane) {
  if (p.c.B > p.num_ctas) return -1;
  int segs = 0, longest = 0, nrt = 0;
  chunk::Seq s;
  auto look = [&](int b0) {
    s.n = 0;
    if (b0 + lane < p.c.B) s = chunk::sequence(p.c, b0 + lane);
    nrt = row_blocks<ROWS>(p, s);
  };
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    look(b0);
    segs += __reduce_add_sync(0xffffffffu, nrt);
    if (static_cast<int64_t>(segs) * p.Hkv > p.num_ctas) return -1;
    for (int rt = 0; rt < nrt; ++rt) longest = max(longest, segment_tiles<ROWS>(p, s, rt).n);
  }
  if (lane == 0) w.left = 0;
  __syncwarp();
  if (segs == 0) return 0;
  longest = __reduce_max_sync(0xffffffffu, longest);
  int m = p.num_ctas / (segs * p.Hkv), most = (longest + m - 1) / m + kJoinCost;
  if (m == 1 || m > kMaxParts || longest <= most) {
    m = 1;
    most = longest;
  } else {
    most += kPartsSlack;
  }
  // this CTA's segment, counted by sequence, KV head, row block
  const int mine = blockIdx.x / m, part = blockIdx.x - mine * m;
  for (int b0 = 0, before = 0; b0 < p.c.B; b0 += 32) {
    if (p.c.B > 32) look(b0);
    int incl = nrt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int off = mine - p.Hkv * (before + incl - nrt);
    if (off >= 0 && off < p.Hkv * nrt) {
      w.b = b0 + lane;
      w.s = s;
      w.kvh = off / nrt;
      w.rt = off - w.kvh * nrt;
      w.t = segment_tiles<ROWS>(p, s, w.rt);
      const int parts = min(m, w.t.n);
      w.N = 0;                        // (see Cut)
      w.C = parts;
      w.seg = mine * m;
      if (part < parts) {
        w.i = static_cast<int>(mul_div(w.t.n, part, parts));
        w.n = static_cast<int>(mul_div(w.t.n, part + 1, parts)) - w.i;
        w.left = w.units = w.n;
      }
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
  return most;
}

// Opens the first piece of this CTA's range [N c / C, N (c + 1) / C) of the N
// units (one warp; never more CTAs than units in the split).  w.left is the
// range's length, 0 for a CTA without a piece.  The other warps copy w
// (copy_walk): computed by all of them it took 1.8 us of a CTA's start.
template <int ROWS>
__device__ __forceinline__ void start_walk(const CParams& p, const int32_t* pre, Walk& w, int64_t& units, int lane) {
  const int64_t N = static_cast<int64_t>(p.Hkv) * pre[p.c.B];
  if (lane == 0) units = N;
  const int C = N < p.num_ctas ? static_cast<int>(N) : p.num_ctas;
  if (static_cast<int>(blockIdx.x) >= C) {
    if (lane == 0) w.left = 0;
    __syncwarp();
    return;
  }
  const int64_t f0 = mul_div(N, blockIdx.x, C), total = mul_div(N, blockIdx.x + 1, C) - f0;
  int lo = 0, hi = p.c.B - 1;   // the last b with Hkv * pre[b] <= f0: a sequence with units
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(p.Hkv) * pre[mid] <= f0) lo = mid; else hi = mid - 1;
  }
  const chunk::Seq s = chunk::sequence(p.c, lo);
  const int per = pre[lo + 1] - pre[lo];
  const int64_t off = f0 - static_cast<int64_t>(p.Hkv) * pre[lo];
  const int kvh = static_cast<int>(mul_div(off, 1, per));
  int rem = static_cast<int>(off - static_cast<int64_t>(kvh) * per);
  // the row block: prefix sums over 32 blocks at a time
  const int nrt = row_blocks<ROWS>(p, s);
  int rt = 0;
  for (int r0 = 0; nrt > 1 && r0 < nrt; r0 += 32) {
    const int mine = r0 + lane < nrt ? segment_tiles<ROWS>(p, s, r0 + lane).n + kLead<ROWS> : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, r0 + lane < nrt && incl > rem);
    if (past != 0u) {
      const int k = __ffs(past) - 1;
      rt = r0 + k;
      rem -= __shfl_sync(0xffffffffu, incl, k) - __shfl_sync(0xffffffffu, mine, k);
      break;
    }
    rem -= __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    w.C = C;
    w.N = N;
    w.seg = f0 - rem;
    w.left = total;
    w.b = lo;
    w.kvh = kvh;
    w.rt = rt;
    w.s = s;
    open_piece<ROWS>(p, w, rem);
  }
  __syncwarp();
}

__device__ __forceinline__ void copy_walk(Walk& to, const Walk& from, int lane) {
  static_assert(sizeof(Walk) % 4 == 0 && sizeof(Walk) <= 128, "a word per lane");
  if (lane < static_cast<int>(sizeof(Walk) / 4))
    reinterpret_cast<uint32_t*>(&to)[lane] = reinterpret_cast<const uint32_t*>(&from)[lane];
  __syncwarp();
}

// A cut segment: CTAs c0 .. c1 hold its tiles.  A CTA's piece of it is partial
// 0 of the CTA's two when it is the first of the CTA's range (which then began
// in the segment, its lead at the earliest), else 1.
struct Cut {
  int c0, c1, slot0;
  __device__ __forceinline__ static int owner(const Walk& w, int64_t f) {
    const int64_t x = f * w.C + w.C - 1;   // the CTA of unit f: floor(((f + 1) C - 1) / N)
    return static_cast<int>(mul_div(x, 1, w.N));
  }
  __device__ __forceinline__ Cut(const Walk& w, int lead) {
    if (w.N == 0) {   // start_parts: the CTAs from w.seg on have a part each
      c0 = static_cast<int>(w.seg);
      c1 = c0 + w.C - 1;
      slot0 = 0;
      return;
    }
    c0 = owner(w, w.seg + lead);
    c1 = owner(w, w.seg + lead + w.t.n - 1);
    slot0 = w.seg <= mul_div(w.N, c0, w.C) ? 0 : 1;
  }
  __device__ __forceinline__ int partial(int c) const { return 2 * c + (c == c0 ? slot0 : 0); }
};

// Rows of the V tile at token t0 that no query of the segment sees become zeros
// in the operand tile, whatever is stored there: a masked weight of 0 must not
// meet an infinity or a NaN (K needs none of it, its scores are replaced).  Run
// by the threads that wrote the rows, after they did: a test on the registers
// themselves cost 15 % of the 256-row kernel, because a branch there waits for
// every load in flight.
// (iterations it0, it0 + step, .. below it1 of the part)
template <int D, int BITS>
__device__ __forceinline__ void clear_unseen(uint32_t dst, const CParams& p, const Walk& w, int t0, int row, int c,
                                             int it0 = 0, int it1 = tile::DqFmt<D, BITS>::NI, int step = 1) {
  using F = tile::DqFmt<D, BITS>;
  const Seen s(p, w);
  if (t0 + kT <= s.end && (t0 >= s.lo || t0 + kT <= p.sinks)) return;   // the whole tile is seen by someone
#pragma unroll 1
  for (int it = it0; it < it1; it += step) {
    const int r = F::RPI * it + row, j = t0 + r;
    if (j < s.end && (j >= s.lo || j < p.sinks)) continue;
    const int ch0 = c * F::VPC;
    const uint32_t rowp = dst + (ch0 >> 6) * (kT * 128) + r * 128;
    for (int i = 0; i < F::VPC / 8; ++i) tile::sts128(rowp + (((((ch0 & 63) >> 3) + i) ^ (r & 7)) << 4), 0u, 0u, 0u, 0u);
  }
}

// A dequant warp marks the tiles of its piece (bit j % 32 for tile j) in which
// it met a scale of kBigScale or more, perhaps in rows that nothing sees; after
// the piece it looks at the words of those tiles once more: whether one that is
// seen overflows.  (By the whole warp; parts x0 .. x1 - 1 of K, V.)
template <int BITS>
__device__ __forceinline__ void mark_big(uint32_t& marks, uint32_t most, int j) {
  if ((most & 0xFFFFu) >= kBigScale<BITS>) marks |= 1u << (j & 31);
}
template <int D>
__device__ __forceinline__ bool marked_overflow(const CParams& p, const Walk& w, uint32_t marks, int x0, int x1, int lane) {
  marks = __reduce_or_sync(0xffffffffu, marks);
  if (marks == 0u || p.status == nullptr) return false;
  const Seen s(p, w);
  const int64_t storage = static_cast<int64_t>(p.c.pB) * p.c.pT;
  bool big = false;
#pragma unroll 1
  for (int j = 0; j < w.n; ++j) {
    if (!(marks >> (j & 31) & 1u)) continue;
#pragma unroll 1
    for (int tok = w.t.tile(w.i + j) * kT + lane, k = 0; k < kT / 32; tok += 32, ++k) {
      if (tok >= s.end || (tok < s.lo && tok >= p.sinks)) continue;
      const int64_t at = chunk::storage_row(p.c, w.b, tok);
      if (at < 0) continue;   // (reported; page 0 stands in for it)
#pragma unroll 1
      for (int x = x0; x < x1; ++x)
        for (int g = 0; g < D / 32; ++g)
          big |= overflows(p.sz[x][(w.kvh * storage + at) * (D / 32) + g], p.bits[w.kvh]);
    }
  }
  return big;
}

// Eight query channels, bf16 to fp16 (for a 4-bit head in the channel order of
// its K tiles, 0,4,1,5,2,6,3,7); big: the largest magnitude seen, as two bf16
// bit patterns.
__device__ __forceinline__ uint4 query_chunk(uint4 v, bool four, uint32_t& big) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    big = __vmaxu2(big, x[e] & 0x7FFF7FFFu);
    x[e] = pack_half2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xFFFF0000u));
  }
  if (!four) return make_uint4(x[0], x[1], x[2], x[3]);
  return make_uint4(prmt(x[0], x[2], 0x5410u), prmt(x[0], x[2], 0x7632u), prmt(x[1], x[3], 0x5410u),
                    prmt(x[1], x[3], 0x7632u));
}
__device__ __forceinline__ void check_queries(const CParams& p, uint32_t big) {
  // 0x4780 is 65536, the first bf16 beyond fp16's range (infinities and NaN lie above it)
  if ((big & 0xFFFFu) >= 0x4780u || (big >> 16) >= 0x4780u) report(p.status, KVQ_ERR_NONFINITE);
}

// The piece's query rows to fp16 in the swizzled layout (rows past the
// segment's end zero); for a 4-bit head in the channel order of its K tiles.
// dst: [D / 64 blocks][ROWS rows][128 B]; empty: the barrier that says that the
// buffer is free.
template <int D, int ROWS>
__device__ __forceinline__ bool load_queries(const CParams& p, uint32_t dst, uint64_t* empty, const Walk& w, int t,
                                             uint32_t parity, bool wait) {
  constexpr int CPR = D / 8;              // 16-byte chunks per row
  constexpr int RPP = 128 / CPR;          // rows per pass
  constexpr int NB = ROWS / RPP < 8 ? ROWS / RPP : 8;   // passes in flight
  const int ch = t % CPR;
  const bool four = p.bits[w.kvh] == 4;
  const uint16_t* base = p.q + static_cast<int64_t>(w.s.row0) * p.sq_row + w.kvh * p.rep * p.sq_head + ch * 8;
  const int rows = w.t.rows;
  // token and head of this thread's row, stepped from pass to pass
  const int R0 = w.rt * ROWS + t / CPR;
  int tok = R0 / p.rep, hh = R0 - tok * p.rep;
  const int dtok = RPP / p.rep, dhh = RPP - dtok * p.rep;
  uint32_t big = 0;
  for (int r0 = 0; r0 < ROWS; r0 += RPP * NB) {
    uint4 v[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int r = r0 + k * RPP + t / CPR;
      v[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) v[k] = *reinterpret_cast<const uint4*>(base + tok * p.sq_row + hh * p.sq_head);
      tok += dtok;
      hh += dhh;
      if (hh >= p.rep) {
        hh -= p.rep;
        ++tok;
      }
    }
    if (r0 == 0 && wait && !__all_sync(0xffffffffu, mbar_wait(empty, parity, p.status, p.wait_ns))) return false;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int r = r0 + k * RPP + t / CPR;
      const uint4 x = query_chunk(v[k], four, big);
      const uint32_t rowp = dst + (ch >> 3) * (ROWS * 128) + r * 128;
      tile::sts128(rowp + (((ch & 7) ^ (r & 7)) << 4), x.x, x.y, x.z, x.w);
    }
  }
  check_queries(p, big);
  return true;
}

}  // namespace chunk_walk

// The kernel for few rows per (sequence, KV head), where it applies.
bool chunk_narrow_takes(int B, int64_t max_rows);
kvq_status launch_chunk_narrow(const chunk_walk::CParams& p, int D, int64_t max_rows, cudaStream_t stream);

}  // namespace kvq
