// kvq_chunk_attn.cu -- attention of a chunk of new tokens over the
// group-quantised cache: the query of packed row r, at cache position p,
// attends tokens j <= p of its sequence, with a window only j > p - window or
// j < sinks.
//
// One warp per (packed row, query head): the lanes hold the query's channels
// and walk the visible keys with an online softmax.
#include <cmath>

#include "kvq_chunk.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct CParams {
  chunk::View c;
  const uint16_t* q;
  int64_t sq_row, sq_head;
  const uint8_t* codes[2];
  const uint32_t* sz[2];
  void* out;
  int32_t* status;
  int32_t out_dtype, Hq, Hkv, window, sinks;
  float scale_log2;
  int64_t plane_off[KVQ_MAX_HKV];
  int8_t bits[KVQ_MAX_HKV];
};

// CPL consecutive channels (a lane's share) of one stored row
template <int D>
__device__ __forceinline__ void lane_values(float (&x)[D / 32], const CParams& p, int which, int h, int64_t row,
                                            int lane) {
  constexpr int N = D / 32;
  const int bits = p.bits[h];
  const int64_t storage = static_cast<int64_t>(p.c.pB) * p.c.pT;
  const uint32_t word = p.sz[which][(h * storage + row) * N + lane * N / 32];
  const uint8_t* c = p.codes[which] + p.plane_off[h] + row * (D * bits / 8) + lane * N * bits / 8;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int code = bits == 8 ? c[i] : (c[i / 2] >> (4 * (i & 1))) & 15;
    x[i] = (static_cast<float>(code) - half_hi(word)) * half_lo(word);
  }
}

template <int D>
__global__ void __launch_bounds__(256) chunk_attention_kernel(const __grid_constant__ CParams p) {
  constexpr int N = D / 32;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) chunk::check_sequences(p.c, threadIdx.x, blockDim.x, p.status);
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int r = static_cast<int>(u / p.Hq), h = static_cast<int>(u % p.Hq);
  if (r >= p.c.rows) return;
  int b = chunk::find_sequence(p.c.start, p.c.B, r, lane);
  const chunk::Seq s = chunk::sequence(p.c, b);
  if (r < s.row0 || r >= s.row0 + s.n) return;
  const int pos = s.len - s.n + (r - s.row0);
  const int kvh = h / (p.Hq / p.Hkv);
  float q[N], o[N], m = -INFINITY, l = 0.0f;
  bool ok = true;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __uint_as_float(static_cast<uint32_t>(p.q[r * p.sq_row + h * p.sq_head + lane * N + i]) << 16);
    ok &= fabsf(q[i]) < 65504.0f;
    o[i] = 0.0f;
  }
  if (!ok) report(p.status, KVQ_ERR_NONFINITE);
  const int first = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
  for (int j = first > 0 && p.sinks > 0 ? 0 : first; j <= pos; ++j) {
    if (j < first && j >= p.sinks) j = first;
    int64_t row = chunk::storage_row(p.c, b, j);
    if (row < 0) {
      report(p.status, KVQ_ERR_INVALID_ARG);
      row = j % KVQ_TILE_TOKENS;
    }
    float x[N], dot = 0.0f;
    lane_values<D>(x, p, 0, kvh, row, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) dot = fmaf(q[i], x[i], dot);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
    dot *= p.scale_log2;
    const float mn = fmaxf(m, dot), a = fast_exp2(m - mn), w = fast_exp2(dot - mn);
    lane_values<D>(x, p, 1, kvh, row, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(w, x[i], o[i] * a);
    l = l * a + w;
    m = mn;
  }
  const int64_t at = (static_cast<int64_t>(r) * p.Hq + h) * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (p.out_dtype == KVQ_OUT_F32) static_cast<float*>(p.out)[at + i] = o[i] / l;
    else static_cast<__nv_bfloat16*>(p.out)[at + i] = __float2bfloat16_rn(o[i] / l);
  }
}

}  // namespace

size_t chunk_workspace_bytes(int, int, int, int, int) { return 16; }

kvq_status launch_chunk_attention(const ChunkAttnArgs& a, cudaStream_t stream) {
  CParams p;
  p.c.start = a.chunk.start; p.c.seq_lens = a.chunk.seq_lens; p.c.bt = a.chunk.bt;
  p.c.B = a.chunk.B; p.c.rows = a.chunk.rows; p.c.max_chunk = a.chunk.max_chunk;
  p.c.bt_stride = a.chunk.bt_max_pages;
  p.c.cap = a.chunk.cap;
  p.c.pB = a.k->B; p.c.pT = a.k->Tcap;
  p.q = a.q;
  p.sq_row = a.sq_row; p.sq_head = a.sq_head;
  p.codes[0] = a.k->codes; p.codes[1] = a.v->codes;
  p.sz[0] = a.k->sz; p.sz[1] = a.v->sz;
  p.out = a.out;
  p.status = a.status;
  p.out_dtype = a.out_dtype; p.Hq = a.Hq; p.Hkv = a.k->Hkv; p.window = a.window; p.sinks = a.sinks;
  const float scale = a.softmax_scale > 0.0f ? a.softmax_scale : 1.0f / sqrtf(static_cast<float>(a.k->D));
  p.scale_log2 = scale * 1.4426950408889634f;
  for (int h = 0; h < KVQ_MAX_HKV; ++h) {
    p.plane_off[h] = a.layout.plane_off[h];
    p.bits[h] = a.layout.bits[h];
  }
  const int64_t blocks = (static_cast<int64_t>(a.chunk.rows) * a.Hq + 7) / 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.k->D == 128 ? cudaLaunchKernelEx(&cfg, chunk_attention_kernel<128>, p)
                                      : cudaLaunchKernelEx(&cfg, chunk_attention_kernel<64>, p);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
