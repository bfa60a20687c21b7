/*
 * kvq.h -- C ABI of libkvq: group-quantised KV-cache attention on GB300 (sm_103a).
 *
 * The method (source pages: 《分块稀疏注意力与KV Cache量化：长文本推理显存优化实践》,
 * xdnf.cn, here "P4"; and 《一只"兔子"如何搅动大模型推理赛道的底层逻辑》, m.xxqk.cn, "P1"):
 *   - the KV cache is stored as integer codes, quantised in groups of 32
 *     adjacent head_dim channels, each group with its own scale and zero point
 *     (P4 §2.4 "KV Cache分组量化"; group size 32 from the hook in P4 §3.2);
 *   - attention softmax(Q K^T / sqrt(d)) V (P1 §3.1) is computed tile by tile
 *     with an online softmax whose running max and normaliser are merged
 *     across tiles (P4 §2.2);
 *   - dequantisation happens inside the attention read, not as a separate pass
 *     (P4 §1.3);
 *   - prefill may skip whole key tiles with a block-sparse mask (P4 §1.3, §2.3).
 *
 * Conventions for every call:
 *   - Ownership: the caller owns every buffer.  The library never allocates or
 *     frees the caller's memory, never synchronises, and launches only on
 *     `stream` (a cudaStream_t; NULL = the legacy default stream).  All calls
 *     are asynchronous with respect to the host.  The one exception to "no
 *     allocation" is kvq_decode_step_host, which keeps up to 16 CUDA graphs
 *     (driver resources) to replay repeated steps; see that call.
 *   - Errors: argument problems are detected on the host; the call returns a
 *     status and launches nothing.  A failed launch returns KVQ_ERR_CUDA.
 *   - Device status: conditions only the device can see (non-finite input,
 *     fp16 scale overflow, a sequence length beyond capacity, a bounded wait
 *     that timed out) are written to the optional device word `dev_status`
 *     (first error wins; the caller zeroes it and reads it after its own
 *     synchronisation).  NULL disables the report.
 *   - bf16 tensors are raw 16-bit bfloat16 values; fp16 values are IEEE binary16.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KVQ_API __attribute__((visibility("default")))
#else
#define KVQ_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kvq_status {
  KVQ_OK = 0,
  KVQ_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned buffer, ... */
  KVQ_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. D not 64/128) */
  KVQ_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
  KVQ_ERR_WORKSPACE = 4,     /* workspace missing or too small */
  KVQ_ERR_TIMEOUT = 5,       /* (device) a bounded wait gave up */
  KVQ_ERR_NONFINITE = 6,     /* (device) non-finite input or fp16 overflow */
  KVQ_ERR_BOUNDS = 7,        /* (device, libkvq_debug.so only) an index check failed; the access was skipped */
  KVQ_ERR_NO_PAGES = 8       /* (device) a page pool has too few free pages */
} kvq_status;

#define KVQ_GROUP 32          /* channels per quantisation group (P4 §3.2) */
#define KVQ_MAX_HKV 64        /* most KV heads a cache may have */
#define KVQ_TILE_TOKENS 64    /* cache capacity granularity */
#define KVQ_OUT_F32 0
#define KVQ_OUT_BF16 1
#define KVQ_OUT_ZERO_REST 0x100   /* or-ed to either by calls that say so (see kvq_chunk) */

/*
 * A quantised KV cache (one for K, one for V).  Group quantisation of P4 §2.4:
 * per (sequence b, KV head h, token t, group g of 32 channels) one fp16 scale
 * s and one fp16 integer zero point z; each channel value x is stored as the
 * code c with x_hat = (c - z) * s.  Per-head bit-width (P4 §2.4: sensitive
 * heads keep more bits) is 8 (one code per byte) or 4 (two codes per byte,
 * even channel in the low nibble).
 *
 * Layout (fixed by the library; all device memory, 16-byte aligned):
 *   codes: one plane per KV head.  Planes of 8-bit heads come first, in head
 *          order, then planes of 4-bit heads, in head order.  A plane is
 *          [B][Tcap][D*bits/8] bytes, row-major.  kvq_cache_head_offset()
 *          gives a plane's byte offset; kvq_cache_codes_bytes() the total.
 *   sz:    [Hkv][B][Tcap][D/32] 32-bit words; low 16 bits = fp16 scale,
 *          high 16 bits = fp16 zero point.  kvq_cache_sz_bytes() is the size.
 * head_bits is a HOST array of Hkv entries, each 4 or 8; it must stay valid
 * for the duration of each call that takes the cache.  Tcap must be a
 * multiple of KVQ_TILE_TOKENS; D is 64 or 128.
 */
typedef struct kvq_cache {
  uint8_t* codes;
  uint32_t* sz;
  const int8_t* head_bits;
  int32_t B, Hkv, Tcap, D;
} kvq_cache;

/* Total bytes of the code planes / the scale-zero words; -1 on invalid shape. */
KVQ_API int64_t kvq_cache_codes_bytes(const kvq_cache* cache);
KVQ_API int64_t kvq_cache_sz_bytes(const kvq_cache* cache);
/* Byte offset of KV head h's code plane within `codes`; -1 on invalid input. */
KVQ_API int64_t kvq_cache_head_offset(const kvq_cache* cache, int32_t h);

/*
 * kvq_quantize -- quantise-on-write (P4 §2.4, group 32 per P4 §3.2).
 *
 * x: device bf16, element (b, h, t, d) at x[b*sx_b + h*sx_h + t*sx_t + d]
 *    (element strides; channels contiguous; every row 16-byte aligned), for
 *    b < dst->B, h < dst->Hkv, t < nt.
 * Writes cache positions t0 .. t0+nt-1 of every (b, h) of `dst`.
 * Per group of 32 channels, qmax = 2^bits - 1, all arithmetic IEEE fp32:
 *   lo = min(0, min x), hi = max(0, max x), r = hi - lo;
 *   r == 0: s = 1, z = 0, codes 0;
 *   else s = fp16 rounded up from r / qmax, z = clamp(rne(-lo / s), 0, qmax),
 *        c = clamp(rne(x / s) + z, 0, qmax)   (rne = round half to even).
 * A non-finite input or a scale beyond fp16 range reports KVQ_ERR_NONFINITE
 * in dev_status; that group's stored values are then unspecified.
 */
KVQ_API kvq_status kvq_quantize(const void* x, int64_t sx_b, int64_t sx_h, int64_t sx_t,
                        int32_t t0, int32_t nt, const kvq_cache* dst,
                        int32_t* dev_status, void* stream);

/*
 * Workspace bytes kvq_decode_attention needs for this shape on the CURRENT
 * device (the split count depends on its SM count).  0 on invalid shape.
 */
KVQ_API size_t kvq_decode_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D);

/*
 * kvq_decode_attention -- one query token per (sequence, query head) over the
 * quantised cache, dequantised inside the attention read (P4 §1.3), tiled
 * online softmax (P4 §2.2) split across CTAs, then a log-sum-exp merge.
 *
 * q:        device bf16 [B][Hq][D], contiguous, 16-byte aligned.
 * k, v:     caches with identical B, Hkv, Tcap, D and head_bits.
 * seq_lens: device int32 [B]; sequence b attends cache tokens 0 .. len_b-1.
 *           len_b == 0 gives a zero output row; len_b outside [0, Tcap]
 *           reports KVQ_ERR_INVALID_ARG in dev_status and is clamped.
 * Hq:       query heads; Hq % Hkv == 0 and Hq / Hkv <= 8.  Query head h
 *           reads KV head h / (Hq / Hkv).
 * softmax_scale: multiplies Q.K; <= 0 selects 1/sqrt(D).
 * out:      device [B][Hq][D], fp32 (out_dtype KVQ_OUT_F32) or bf16 (KVQ_OUT_BF16).
 * workspace: device scratch of >= kvq_decode_workspace_bytes(B, Hq, Hkv, D)
 *           bytes, 16-byte aligned.  Zero-fill it once before its first use
 *           (e.g. cudaMemsetAsync): it holds per-segment arrival counters that
 *           every successful call leaves at zero again.  After a call that
 *           reported a device error, zero-fill it again.  Calls that share a
 *           workspace must be ordered on the GPU.
 * q values must lie within fp16 range (|q| < 65504): the kernel's tensor-core
 * products take Q in fp16 (exact for bf16 values in that range).
 */
KVQ_API kvq_status kvq_decode_attention(const void* q, const kvq_cache* k, const kvq_cache* v,
                                const int32_t* seq_lens, int32_t Hq, float softmax_scale,
                                void* out, int32_t out_dtype,
                                void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, void* stream);

/*
 * kvq_prefill_attention -- prefill (causal or not) over a group-quantised KV cache.
 *
 * Quantises K and V into k_cache / v_cache (positions 0 .. S-1, exactly as
 * kvq_quantize), then computes, per query head h and query position i,
 *   O[i] = softmax_j(scale * Q[i] . K_hat[j]) V_hat[j]
 * over keys j <= i when causal == 1 (P1 §3.1 with the causal rule), over all
 * keys j < S when causal == 0, where K_hat, V_hat are the dequantised cache
 * rows, tile by tile with an online softmax (P4 §2.2).
 * With a tile mask (P4 §1.3, §2.3: skipped blocks are not computed), an
 * off-diagonal key tile kt of query tile qt takes part only if
 * tile_mask[qt * nT + kt] != 0, where nT = S / tile; the keys of a skipped
 * tile are left out of the softmax.  Causal prefill reads only kt < qt of the
 * mask; non-causal reads every off-diagonal entry.  Diagonal tiles are always
 * computed (element-wise causal rule when causal == 1, whole when 0).
 *
 * q:    device bf16 [B][Hq][S][D]; k, v: device bf16 [B][Hkv][S][D];
 *       contiguous, 16-byte aligned.
 * causal 0 or 1; tile must be 128; S a multiple of 128; D 64 or 128;
 * Hq % Hkv == 0; caches with any per-head bits (8 or 4, e.g. from
 * kvq_allocate_head_bits), Tcap >= S.
 * tile_mask: device uint8 [nT][nT] or NULL (every tile kept); with a mask,
 *       nT * nT must stay below 2^31 (S up to 5,931,520), else
 *       KVQ_ERR_UNSUPPORTED.
 * out:  device [B][Hq][S][D], fp32 or bf16.
 * The tensor-core operands are fp16: |q| < 65504, else KVQ_ERR_NONFINITE; K_hat,
 * V_hat and the weights are rounded to it, and stored values of 65520 and more
 * become infinities there, which is not reported.
 */
KVQ_API kvq_status kvq_prefill_attention(const void* q, const void* k, const void* v,
                                 int32_t B, int32_t Hq, int32_t Hkv, int32_t S, int32_t D,
                                 int32_t causal, float softmax_scale,
                                 const uint8_t* tile_mask, int32_t tile,
                                 const kvq_cache* k_cache, const kvq_cache* v_cache,
                                 void* out, int32_t out_dtype,
                                 int32_t* dev_status, void* stream);

/*
 * kvq_head_error_stats -- per-head quantisation-error statistics, the input
 * of a sensitivity-driven per-head bit allocation (P4 §2.4: every attention
 * head gets a sensitivity score; sensitive heads are stored at the higher
 * bit-width, the rest at the lower one).
 *
 * For each head h, with x_hat the dequantised value that kvq_quantize would
 * store at `bits` bits (the same codes, bit for bit):
 *   stats[h][0] = sum_{b, t < len_b} w[b][h][t] * sum_d (x - x_hat)^2
 *   stats[h][1] = sum_{b, t < len_b} w[b][h][t] * sum_d x^2
 * x:        device bf16 [B][H][T][D], contiguous, 16-byte aligned; D 64 or 128.
 * seq_lens: device int32 [B] or NULL (every sequence T tokens); tokens
 *           t >= len_b are left out.
 * weights:  device float [B][H][T] or NULL (1): a per-token attention mass,
 *           expected >= 0.
 * bits:     4 or 8.
 * stats:    device double [H][2], written whole.
 * workspace: device, at least kvq_head_error_stats_workspace_bytes(H) bytes,
 *           16-byte aligned, else KVQ_ERR_WORKSPACE.
 * The sums are fp32 within a 32-channel group and fp64 beyond it, in an order
 * fixed by the sizes and the device (the same result on every call).
 * Non-finite input reports KVQ_ERR_NONFINITE in dev_status.  Two launches.
 */
KVQ_API size_t kvq_head_error_stats_workspace_bytes(int32_t H);
KVQ_API kvq_status kvq_head_error_stats(const void* x, int32_t B, int32_t H, int32_t T, int32_t D,
                                const int32_t* seq_lens, const float* weights, int32_t bits,
                                double* stats, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, void* stream);

/*
 * kvq_allocate_head_bits -- per-head bit-widths from K and V error statistics
 * (host function; P4 §2.4, and P4 §3.4: keeping more heads at high precision
 * trades compression, about 4x down to 2.5x, for accuracy).
 *
 * score[h] = k_stats[h][0] / k_stats[h][1] + v_stats[h][0] / v_stats[h][1]
 * (a term with a zero norm counts 0): the relative error of the head's K and
 * V at the low bit-width.  The n_high heads with the largest scores get 8
 * bits, ties going to the smaller head index; the others get low_bits.
 * k_stats, v_stats: host double [H][2] (kvq_head_error_stats, copied back);
 * head_bits: host int8 [H], written; score: host double [H] or NULL.
 * 0 <= n_high <= H; low_bits 4 or 8.  A non-finite score returns
 * KVQ_ERR_NONFINITE and writes nothing.
 */
KVQ_API kvq_status kvq_allocate_head_bits(const double* k_stats, const double* v_stats, int32_t H,
                                  int32_t n_high, int32_t low_bits, int8_t* head_bits, double* score);

/*
 * kvq_prefill_attention_varlen -- kvq_prefill_attention over a batch of
 * sequences of different lengths, padded to S.
 *
 * seq_lens: device int32 [B], sequence b's length L_b (0 <= L_b <= S; a value
 *   outside that range reports KVQ_ERR_INVALID_ARG in dev_status and is
 *   clamped).  Rows i < L_b of q, k, v hold the sequence; rows L_b .. S-1 are
 *   padding and are never read into the result (they may hold anything,
 *   non-finite values included).
 * Cache positions 0 .. L_b-1 get the codes kvq_quantize would write;
 * positions from L_b to the end of its 128-token tile are cleared (codes and
 * scale/zero words 0); positions past that keep their contents.  Output rows
 * i < L_b are the attention of query i over keys j <= i (causal == 1) or
 * j < L_b (causal == 0), with the tile mask as in kvq_prefill_attention;
 * rows L_b .. S-1 of out are written as zeros.  Query tiles wholly past L_b
 * cost one store of zeros.  Other arguments, layouts and errors as in
 * kvq_prefill_attention.
 */
KVQ_API kvq_status kvq_prefill_attention_varlen(const void* q, const void* k, const void* v,
                                        int32_t B, int32_t Hq, int32_t Hkv, int32_t S, int32_t D,
                                        const int32_t* seq_lens, int32_t causal, float softmax_scale,
                                        const uint8_t* tile_mask, int32_t tile,
                                        const kvq_cache* k_cache, const kvq_cache* v_cache,
                                        void* out, int32_t out_dtype,
                                        int32_t* dev_status, void* stream);

/*
 * kvq_build_tile_mask -- a block-sparse tile mask for kvq_prefill_attention
 * (P4 §2.3: tiles judged unnecessary are skipped, the skipped share capped so
 * that no query block is starved), built on the GPU.
 *
 * mask: device uint8 [nT][nT], written whole.  For query tile qt the
 *   candidates are key tiles kt in [1, qt); the row skips
 *   floor(max(qt - 1, 0) * skip_num / skip_den) of them (0 <= skip_num <=
 *   skip_den; integer arithmetic, so each row's cap is exact): those with the
 *   smallest keys SplitMix64(seed, qt * nT + kt + 1) -- output number
 *   qt * nT + kt + 1 of the SplitMix64 generator (Steele, Lea and Flood,
 *   2014) seeded with `seed` -- ties to the smaller kt.  Entries are 1 for kept
 *   tiles, key tile 0 and the diagonal, 0 for skipped tiles and above the
 *   diagonal.  1 <= nT <= 16384.  One launch on `stream`.
 */
KVQ_API kvq_status kvq_build_tile_mask(uint8_t* mask, int32_t nT, int32_t skip_num, int32_t skip_den,
                                       uint64_t seed, void* stream);

/*
 * kvq_decode_attention_noalloc -- kvq_decode_attention for callers that may
 * not allocate device memory (for example code running inside another
 * framework's memory pool, or a plugin whose host forbids cudaMalloc at call
 * time).  The source pages have no counterpart to this call.
 *
 * Arguments and results are those of kvq_decode_attention, minus the
 * workspace: the split scratch is a fixed array of 4 MiB compiled into the
 * library, present on every GPU that loads it until the process exits.  A
 * shape whose kvq_decode_workspace_bytes() exceeds 4 MiB returns
 * KVQ_ERR_WORKSPACE and launches nothing.  The call allocates nothing; it
 * clears the array's arrival counters with an asynchronous memset on `stream`
 * before the decode launch.
 *
 * The first call on each device looks up the array's device address (with
 * that device current); make that first call before any stream capture.
 * Every call on a device shares the one array, so calls whose executions
 * overlap on the GPU (different streams, no ordering between them) race and
 * give wrong results; order them.
 */
KVQ_API kvq_status kvq_decode_attention_noalloc(const void* q, const kvq_cache* k, const kvq_cache* v,
                                                const int32_t* seq_lens, int32_t Hq, float softmax_scale,
                                                void* out, int32_t out_dtype,
                                                int32_t* dev_status, void* stream);

/*
 * kvq_decode_step -- one step of a decode loop over the quantised cache (the
 * decode phase of P4 §1.3: each new token's K/V is quantised on write, then
 * the new query attends the cache with dequantisation inside the read).
 *
 * Appends the new token of every (sequence b, KV head) to both caches at
 * position seq_lens[b] - 1, quantised exactly as kvq_quantize writes it, then
 * computes kvq_decode_attention over positions 0 .. seq_lens[b] - 1.
 *
 * k_new, v_new: device bf16 [B][Hkv][D], contiguous, 16-byte aligned.
 * seq_lens: device int32 [B], each length INCLUDING the new token.  A length
 *           outside [1, Tcap] reports KVQ_ERR_INVALID_ARG in dev_status and
 *           that sequence appends nothing (decode then treats the length as
 *           kvq_decode_attention does).
 * q, k, v, Hq, softmax_scale, out, out_dtype, workspace, dev_status, stream:
 *           as kvq_decode_attention; the workspace is required.
 * Two launches on `stream`: the append kernel (K and V together) and the
 * decode kernel, whose prologue overlaps the append kernel's end
 * (programmatic dependent launch); the decode waits for the append before
 * reading memory.  All arguments are checked before the first launch.
 */
KVQ_API kvq_status kvq_decode_step(const void* q, const void* k_new, const void* v_new,
                                   const kvq_cache* k, const kvq_cache* v, const int32_t* seq_lens,
                                   int32_t Hq, float softmax_scale, void* out, int32_t out_dtype,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   void* stream);

/*
 * Device staging bytes kvq_decode_step_host needs: q, k_new, v_new and the
 * output, each rounded up to 256 bytes.  0 on invalid shape.
 */
KVQ_API size_t kvq_decode_step_staging_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t out_dtype);

/*
 * kvq_decode_step_host -- kvq_decode_step with the step's inputs and output in
 * HOST memory: q_host bf16 [B][Hq][D], k_new_host / v_new_host bf16
 * [B][Hkv][D], out_host [B][Hq][D] of out_dtype, all 16-byte aligned.
 * When all four host buffers are pinned (page-locked, so mapped into the
 * GPU's address space) the call makes no copy calls: the append launch reads
 * the new K/V rows in place over the host link and stages q in `staging`,
 * and the decode launch writes the output straight into out_host.  Otherwise
 * it enqueues three host-to-device copies into `staging`, the two launches of
 * kvq_decode_step and a device-to-host copy of the output (with pageable
 * memory the copies may block the host).  Either way everything goes to
 * `stream` and the call returns once it is enqueued; out_host holds the
 * result after the caller synchronises the stream, and the host inputs and
 * `staging` must stay untouched until then.
 * Repeated steps (pinned buffers): the second call whose arguments all match
 * an earlier call's -- every pointer and size, Hq, softmax_scale, out_dtype,
 * both caches' fields and per-head bit widths, the current device -- captures
 * the two launches into a CUDA graph on an internal stream, and every later
 * matching call launches that graph on `stream` (one launch call, no
 * tensor-map encoding).  The kernels read the lengths, the new rows and the
 * caches at run time, so those may change between calls.  Up to 16 graphs
 * are kept for the life of the process; other steps launch directly, and so
 * does any call on a stream that is being captured.
 * staging: device scratch of >= kvq_decode_step_staging_bytes(B, Hq, Hkv, D,
 * out_dtype) bytes, 256-byte aligned.  The caches, seq_lens, workspace and
 * dev_status are device memory as in kvq_decode_step.
 */
KVQ_API kvq_status kvq_decode_step_host(const void* q_host, const void* k_new_host, const void* v_new_host,
                                        const kvq_cache* k, const kvq_cache* v, const int32_t* seq_lens,
                                        int32_t Hq, float softmax_scale, void* out_host, int32_t out_dtype,
                                        void* staging, size_t staging_bytes,
                                        void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                        void* stream);

/*
 * Paged caches: the block-table layout of the serving systems the pages
 * compare against (PagedAttention with an INT8 cache), here for the
 * group-quantised cache.  A page POOL is a kvq_cache whose B counts pages and
 * whose Tcap is KVQ_TILE_TOKENS (64): page p holds 64 consecutive tokens of
 * one sequence, in every head's code plane and in the scale/zero words, in
 * exactly the kvq_cache layout.  A block table maps sequence b's token t to
 * page pages[b * max_pages + t / 64], slot t % 64.  Pages are the caller's to
 * allocate; two sequences may share a page only while no call writes it.
 */
typedef struct kvq_block_table {
  const int32_t* pages;   /* device int32 [B][max_pages], 4-byte aligned */
  int32_t B;              /* sequences */
  int32_t max_pages;      /* pages per sequence: capacity max_pages * 64 tokens */
} kvq_block_table;

/*
 * kvq_quantize into a page pool: x's rows are (sequence b < table->B, KV
 * head, position t0 + t) with the strides of kvq_quantize, and each row is
 * written to its page and slot, quantised exactly as kvq_quantize does.
 * t0 + nt <= max_pages * 64.  A page id outside [0, pool->B) reports
 * KVQ_ERR_INVALID_ARG in dev_status and that row is not written.
 */
KVQ_API kvq_status kvq_quantize_paged(const void* x, int64_t sx_b, int64_t sx_h, int64_t sx_t,
                                      int32_t t0, int32_t nt, const kvq_cache* pool,
                                      const kvq_block_table* table, int32_t* dev_status, void* stream);

/*
 * kvq_decode_attention over page pools: q [table->B][Hq][D]; sequence b
 * attends its tokens 0 .. seq_lens[b] - 1 through the block table
 * (seq_lens[b] <= max_pages * 64, else KVQ_ERR_INVALID_ARG in dev_status and
 * the length is clamped).  A page id outside the pool reports
 * KVQ_ERR_INVALID_ARG and that tile reads page 0 instead.  The workspace is
 * kvq_decode_workspace_bytes(table->B, Hq, Hkv, D).  Other arguments as
 * kvq_decode_attention.
 */
KVQ_API kvq_status kvq_decode_attention_paged(const void* q, const kvq_cache* k_pool, const kvq_cache* v_pool,
                                              const kvq_block_table* table, const int32_t* seq_lens,
                                              int32_t Hq, float softmax_scale, void* out, int32_t out_dtype,
                                              void* workspace, size_t workspace_bytes,
                                              int32_t* dev_status, void* stream);

/*
 * kvq_decode_step over page pools: the new token of sequence b goes to page
 * pages[b * max_pages + (seq_lens[b] - 1) / 64], slot (seq_lens[b] - 1) % 64,
 * then kvq_decode_attention_paged.  A length outside [1, max_pages * 64] or a
 * page id outside the pool reports KVQ_ERR_INVALID_ARG and that sequence
 * appends nothing.
 */
KVQ_API kvq_status kvq_decode_step_paged(const void* q, const void* k_new, const void* v_new,
                                         const kvq_cache* k_pool, const kvq_cache* v_pool,
                                         const kvq_block_table* table, const int32_t* seq_lens,
                                         int32_t Hq, float softmax_scale, void* out, int32_t out_dtype,
                                         void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                         void* stream);

/*
 * kvq_policy -- per-call settings for the two phases (P4 §5.3: prefill and
 * decode want different settings -- prefill has no history to re-read and is
 * compute-bound, so its tile mask may skip more; decode re-reads the whole
 * cache for every token and is memory-bound, so it gains from fetching the
 * cache further ahead).  The prefill phase's sparsity is its tile mask
 * (kvq_build_tile_mask's skip ratio); the decode phase's prefetch width is
 * set here.  kvq_policy_default() fills the values every other call uses.
 *
 *   decode_ring_tiles     64-token tiles of K and V that each decode CTA keeps
 *                         in flight into shared memory, 2 or 4 (default 4).
 *   decode_l2_warm_tiles  tiles per CTA requested into L2 before the decode
 *                         waits for the previous kernel in the stream to
 *                         finish, 0 .. 16 (default 5).
 *   wait_limit_us         every bounded wait inside the decode, prefill and
 *                         chunk attention kernels gives up after this long
 *                         and reports KVQ_ERR_TIMEOUT in dev_status,
 *                         1 .. 60,000,000 (default 2,000,000 = 2 s).
 *   test_issue_limit      FOR TESTS OF THE TIMEOUT PATH ONLY; negative (the
 *                         default) = off.  Decode: each CTA's copy issuer
 *                         streams only its first test_issue_limit tiles, so
 *                         the waits for the rest run out.  Prefill: 0
 *                         withholds the query load, so every role's first
 *                         wait runs out (other values: no effect).  Chunk
 *                         attention: each CTA makes only the queries of its
 *                         first test_issue_limit pieces of work ready.
 *                         Nothing is left in flight; the call reports
 *                         KVQ_ERR_TIMEOUT and its outputs are unspecified.
 * An out-of-range field returns KVQ_ERR_INVALID_ARG and launches nothing.
 */
typedef struct kvq_policy {
  int32_t decode_ring_tiles;
  int32_t decode_l2_warm_tiles;
  uint32_t wait_limit_us;
  int32_t test_issue_limit;
} kvq_policy;

KVQ_API void kvq_policy_default(kvq_policy* policy);

/* kvq_decode_attention with a policy (NULL = kvq_policy_default). */
KVQ_API kvq_status kvq_decode_attention_ex(const void* q, const kvq_cache* k, const kvq_cache* v,
                                           const int32_t* seq_lens, int32_t Hq, float softmax_scale,
                                           void* out, int32_t out_dtype,
                                           void* workspace, size_t workspace_bytes,
                                           const kvq_policy* policy, int32_t* dev_status, void* stream);

/* kvq_prefill_attention_varlen with a policy (NULL = kvq_policy_default);
 * seq_lens may be NULL (every sequence S long, as kvq_prefill_attention). */
KVQ_API kvq_status kvq_prefill_attention_ex(const void* q, const void* k, const void* v,
                                            int32_t B, int32_t Hq, int32_t Hkv, int32_t S, int32_t D,
                                            const int32_t* seq_lens, int32_t causal, float softmax_scale,
                                            const uint8_t* tile_mask, int32_t tile,
                                            const kvq_cache* k_cache, const kvq_cache* v_cache,
                                            void* out, int32_t out_dtype, const kvq_policy* policy,
                                            int32_t* dev_status, void* stream);

/*
 * kvq_chunk -- a ragged batch of new tokens, packed: sequence b's n_b =
 * start[b + 1] - start[b] new tokens are rows start[b] .. start[b + 1] - 1 of
 * the caller's row buffers and cache positions seq_lens[b] - n_b ..
 * seq_lens[b] - 1, in order (as in kvq_decode_step, a length INCLUDES the new
 * tokens).  start[0] .. start[B] ascend from 0 to at most `rows`; a sequence
 * may have no new token.  The calls that take a chunk read both arrays on the
 * device.  A sequence with start[b] < 0, start[b + 1] < start[b],
 * start[b + 1] > rows, n_b > max_chunk, seq_lens[b] < n_b or seq_lens[b]
 * beyond the cache's capacity reports KVQ_ERR_INVALID_ARG in dev_status and is
 * left out: nothing of it is read or written.  Where the starts descend, chunk
 * attention leaves the whole call out, and the append and the read-back may
 * leave out any of its sequences.
 * Rows that belong to no sequence (from start[B] on) or to one that is left out
 * are left as they are; with KVQ_OUT_ZERO_REST or-ed to out_dtype the read-back
 * and chunk attention write them as zeros.  A call with rows == 0 does nothing
 * and needs no row buffers.  Capacities of 2^31 - 256 tokens and more are
 * KVQ_ERR_UNSUPPORTED.
 */
typedef struct kvq_chunk {
  const int32_t* start;      /* device int32 [B + 1], 4-byte aligned */
  const int32_t* seq_lens;   /* device int32 [B], 4-byte aligned */
  int32_t B;                 /* sequences, 1 .. 4096; the cache's B, or the block table's */
  int32_t rows;              /* rows of the caller's packed buffers; KVQ_ERR_UNSUPPORTED from 2^31 - 257 on */
  int32_t max_chunk;         /* most new tokens of one sequence; 0 = rows.  Chunk attention chooses its kernel by it. */
} kvq_chunk;

/*
 * kvq_append_chunk -- quantise-on-write of a chunk (several new tokens per
 * sequence, each sequence at its own position), K and V in one launch; each
 * row is quantised exactly as kvq_quantize does it.
 *
 * k_new, v_new: device bf16, channel d of (row r, KV head h) at
 *   x[r * s_row + h * s_head + d] (element strides, multiples of 8; channels
 *   contiguous; 16-byte aligned base), the same strides for both -- rows of a
 *   fused projection's output can be passed in place.
 * k, v: caches with identical B, Hkv, Tcap, D and head_bits.
 * Positions other than the chunk's keep their contents.  Non-finite input as
 * in kvq_quantize.  No two rows of a call may share a position (through pages
 * that two sequences share).
 */
KVQ_API kvq_status kvq_append_chunk(const void* k_new, const void* v_new, int64_t s_row, int64_t s_head,
                                    const kvq_chunk* chunk, const kvq_cache* k, const kvq_cache* v,
                                    int32_t* dev_status, void* stream);
/* The same into page pools; a row whose page id lies outside the pool reports
 * KVQ_ERR_INVALID_ARG and is not written. */
KVQ_API kvq_status kvq_append_chunk_paged(const void* k_new, const void* v_new, int64_t s_row, int64_t s_head,
                                          const kvq_chunk* chunk, const kvq_cache* k_pool, const kvq_cache* v_pool,
                                          const kvq_block_table* table, int32_t* dev_status, void* stream);

/*
 * kvq_dequantize -- the cache read back: row r of the chunk description gets
 * the stored values (c - z) * s of its cache position (the difference is
 * exact; one rounding, to out's type), for every KV head.  With start the
 * running sum of seq_lens it reads whole sequences.
 * out: device [rows][Hkv][D], contiguous, 16-byte aligned, fp32 or bf16
 *   (KVQ_OUT_ZERO_REST: see kvq_chunk).
 */
KVQ_API kvq_status kvq_dequantize(const kvq_cache* src, const kvq_chunk* chunk, void* out, int32_t out_dtype,
                                  int32_t* dev_status, void* stream);
/* The same from a page pool; a row whose page id lies outside the pool reports
 * KVQ_ERR_INVALID_ARG and is written as zeros. */
KVQ_API kvq_status kvq_dequantize_paged(const kvq_cache* pool, const kvq_chunk* chunk, const kvq_block_table* table,
                                        void* out, int32_t out_dtype, int32_t* dev_status, void* stream);

/*
 * kvq_chunk_attention -- attention of a chunk of new tokens over caches that
 * already hold them (kvq_append_chunk or kvq_quantize before it on the same
 * stream): prompt chunks, verification of several drafted tokens, or a batch
 * that mixes both with single tokens.  The query of row r, at cache position
 * p, attends its sequence's tokens j <= p; with window > 0 only those with
 * j > p - window or j < sinks (the last `window` tokens, itself among them,
 * and the first `sinks` ones).
 *
 * q: device bf16, channel d of (row r, query head h) at
 *   q[r * sq_row + h * sq_head + d] (element strides, multiples of 8; channels
 *   contiguous; 16-byte aligned base; |q| < 65504, as kvq_decode_attention).
 * Hq % Hkv == 0, Hq / Hkv <= 128.  window >= 0 (0: none), sinks >= 0.
 * out: device [rows][Hq][D], contiguous, 16-byte aligned, fp32 or bf16
 *   (KVQ_OUT_ZERO_REST: see kvq_chunk).
 * workspace: device scratch of >= kvq_chunk_workspace_bytes(rows, B, Hq, Hkv,
 *   D) bytes, with kvq_decode_attention's rules (16-byte aligned, zero-filled
 *   once before its first use, calls that share it ordered on the GPU).  One
 *   workspace serves chunk calls of every shape that fits it; it is not shared
 *   with other kinds of calls.
 * Cache tokens that no query of the call sees are not read into the result
 * (they may hold anything).  The values of the others have to be finite in
 * fp16, as the operands are (K_hat, V_hat and the weights are rounded to fp16 as
 * in kvq_prefill_attention; scores, sums and outputs are fp32): a token that some
 * query sees, with a group whose scale s and zero point z can stand for 65520 or
 * more (s * max(z, qmax - z)), reports KVQ_ERR_NONFINITE in dev_status, and the
 * outputs of its sequence are then unspecified (kvq_decode_attention takes such
 * values: its scales stay fp32).  A call whose work list of 128-token tiles could reach
 * 2^31 entries per KV head is KVQ_ERR_UNSUPPORTED.  The result depends on
 * neither the order of the CTAs nor the call's place in a program: equal calls
 * on equal devices give equal bits.  Errors and other arguments as
 * kvq_decode_attention.
 */
KVQ_API size_t kvq_chunk_workspace_bytes(int32_t rows, int32_t B, int32_t Hq, int32_t Hkv, int32_t D);
KVQ_API kvq_status kvq_chunk_attention(const void* q, int64_t sq_row, int64_t sq_head, const kvq_chunk* chunk,
                                       const kvq_cache* k, const kvq_cache* v, int32_t Hq, float softmax_scale,
                                       int32_t window, int32_t sinks, void* out, int32_t out_dtype,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);
/* The same over page pools.  Pages that hold no visible token may be anything;
 * a visible one outside the pool reports KVQ_ERR_INVALID_ARG and page 0 is
 * read instead. */
KVQ_API kvq_status kvq_chunk_attention_paged(const void* q, int64_t sq_row, int64_t sq_head, const kvq_chunk* chunk,
                                             const kvq_cache* k_pool, const kvq_cache* v_pool,
                                             const kvq_block_table* table, int32_t Hq, float softmax_scale,
                                             int32_t window, int32_t sinks, void* out, int32_t out_dtype,
                                             void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                             void* stream);

/* kvq_chunk_attention (table NULL) or kvq_chunk_attention_paged with a policy
 * (NULL = kvq_policy_default; its decode fields have no effect here). */
KVQ_API kvq_status kvq_chunk_attention_ex(const void* q, int64_t sq_row, int64_t sq_head, const kvq_chunk* chunk,
                                          const kvq_cache* k, const kvq_cache* v, const kvq_block_table* table,
                                          int32_t Hq, float softmax_scale, int32_t window, int32_t sinks, void* out,
                                          int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                          const kvq_policy* policy, int32_t* dev_status, void* stream);

/*
 * kvq_decode_attention_window -- kvq_decode_attention with a sliding window:
 * sequence b's query, at position len_b - 1, attends tokens j >= len_b -
 * window and j < min(sinks, len_b).  Only the 64-token tiles that hold such
 * tokens are read; tokens outside them may hold anything.  window == 0: every
 * token (kvq_decode_attention).  window, sinks >= 0.  Other arguments, the
 * workspace and errors as kvq_decode_attention, Hq / Hkv <= 8 among them: with
 * more query heads per KV head, kvq_chunk_attention computes the same from one
 * row per sequence (start 0 .. B).
 */
KVQ_API kvq_status kvq_decode_attention_window(const void* q, const kvq_cache* k, const kvq_cache* v,
                                               const int32_t* seq_lens, int32_t Hq, float softmax_scale,
                                               int32_t window, int32_t sinks, void* out, int32_t out_dtype,
                                               void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                               void* stream);
/* The same over page pools (kvq_decode_attention_paged); block-table entries
 * of tiles without a visible token are not used. */
KVQ_API kvq_status kvq_decode_attention_window_paged(const void* q, const kvq_cache* k_pool, const kvq_cache* v_pool,
                                                     const kvq_block_table* table, const int32_t* seq_lens,
                                                     int32_t Hq, float softmax_scale, int32_t window, int32_t sinks,
                                                     void* out, int32_t out_dtype, void* workspace,
                                                     size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * kvq_rotation -- what a model does to the projected queries and keys of every
 * head before they meet: a root-mean-square norm with weights, and a rotation
 * of channel pairs by the row's cache position.
 */
typedef struct kvq_rotation {
  const float* table;       /* device fp32 [positions][rot_dim], 16-byte aligned: row p holds position p's rot_dim / 2
                               cosines, then as many sines.  NULL: no rotation. */
  const void* q_weight;     /* device bf16 [D], 16-byte aligned; NULL: queries are not normed */
  const void* k_weight;     /* the same for keys */
  int32_t positions;        /* rows of the table */
  int32_t rot_dim;          /* channels 0 .. rot_dim - 1 turn, the others stay: a multiple of 16, 16 .. D */
  int32_t interleaved;      /* pair i is channels 2i and 2i + 1 (1), or i and i + rot_dim / 2 (0) */
  float eps;                /* 1e-12 .. 1, looked at where a weight is given */
} kvq_rotation;

/*
 * kvq_rotate_append -- from the projections' rows to the cache in one pass:
 * queries normed and rotated into q_out, keys normed, rotated and quantised
 * into k's cache, values quantised into v's (positions as kvq_append_chunk).
 *
 * For a row x[D] of a head, all arithmetic IEEE fp32 with one rounding an
 * operation unless said otherwise:
 *   with a weight w:  m = the exact mean of x^2, rounded once;
 *                     r = 1 / sqrt(m + eps);  y = (x * r) * w     (else y = x)
 *   with a table:     pair (a, b) -> (a * cos - b * sin, b * cos + a * sin)
 * then rounded to bf16.  Keys are quantised from that bf16 value exactly as
 * kvq_quantize does it, so the codes are a function of the inputs.  (m is
 * within 2^-38 of the exact mean before its rounding.)
 *
 * q: device bf16, channel d of (row r, query head h) at
 *   q[r * sq_row + h * sq_head + d]; k_new, v_new as kvq_append_chunk (the
 *   same strides for both); element strides, multiples of 8; 16-byte aligned.
 * q_out: device bf16 [rows][Hq][D], contiguous, 16-byte aligned; it may be q
 *   itself where q is laid out so, and overlaps no other input.
 * out_dtype: KVQ_OUT_BF16 (KVQ_OUT_ZERO_REST: see kvq_chunk).
 * Hq >= 1; rows * (Hq + 2 Hkv) below 2^31.  A row whose position is not below
 * `positions` (with a table) reports KVQ_ERR_INVALID_ARG and is left out like
 * the rows of an unusable sequence.  Non-finite keys and values as in
 * kvq_quantize (a key that the norm makes non-finite among them); non-finite
 * queries are not reported.
 */
KVQ_API kvq_status kvq_rotate_append(const void* q, int64_t sq_row, int64_t sq_head, const void* k_new,
                                     const void* v_new, int64_t s_row, int64_t s_head, const kvq_chunk* chunk,
                                     const kvq_rotation* rotation, int32_t Hq, const kvq_cache* k, const kvq_cache* v,
                                     void* q_out, int32_t out_dtype, int32_t* dev_status, void* stream);
/* The same into page pools; a row whose page id lies outside the pool reports
 * KVQ_ERR_INVALID_ARG, its key and value are not written, its query is. */
KVQ_API kvq_status kvq_rotate_append_paged(const void* q, int64_t sq_row, int64_t sq_head, const void* k_new,
                                           const void* v_new, int64_t s_row, int64_t s_head, const kvq_chunk* chunk,
                                           const kvq_rotation* rotation, int32_t Hq, const kvq_cache* k_pool,
                                           const kvq_cache* v_pool, const kvq_block_table* table, void* q_out,
                                           int32_t out_dtype, int32_t* dev_status, void* stream);

/*
 * Attention over selected blocks: a cache's tokens are looked at in blocks of
 * 64 (its tiles; a pool's pages).  Beside K's cache a caller keeps each
 * block's bounds -- per channel the least and greatest stored value -- in 8
 * bits, from which a cheap score tells which blocks a query needs.
 *
 * kvq_bounds -- bounds of every storage block of a K cache (block index
 * b * Tcap / 64 + i of sequence b's tokens 64 i .. 64 i + 63, or a pool's page
 * id), NB = B * Tcap / 64 of them:
 *   codes:  int8 [Hkv][NB][D / 32][2][32]: of each group of 32 channels the
 *           greatest values' codes, then the least values'.  16-byte aligned.
 *   scales: fp32 [Hkv][NB][D / 32].  16-byte aligned.
 * A code c stands for c * scale.  Per block and group, in IEEE fp32, over the
 * block's tokens below its sequence's length:
 *   a = max |stored value|, s = a / 127, codes ceil(greatest / s) and
 *   floor(least / s), clamped to +-127; a == 0: s = 0, codes 0
 * so that (to the rounding of s) no stored value lies outside.
 */
typedef struct kvq_bounds {
  int8_t* codes;
  float* scales;
} kvq_bounds;

/* Bytes of a cache's bounds: the codes (0) or the scales (1); -1 on invalid shape. */
KVQ_API int64_t kvq_bounds_bytes(const kvq_cache* k, int32_t which);

/*
 * kvq_block_bounds -- (re)computes the bounds of the blocks that hold a
 * chunk's positions, from the stored codes: call it after the append, on the
 * same stream.  With start the running sum of seq_lens it does whole
 * sequences.  Other blocks' bounds keep their contents.  A block with a
 * non-finite stored value reports KVQ_ERR_NONFINITE; its bounds are then
 * unspecified.
 */
KVQ_API kvq_status kvq_block_bounds(const kvq_cache* k, const kvq_chunk* chunk, const kvq_bounds* bounds,
                                    int32_t* dev_status, void* stream);
/* The same from a page pool; a page id outside the pool reports
 * KVQ_ERR_INVALID_ARG and is skipped. */
KVQ_API kvq_status kvq_block_bounds_paged(const kvq_cache* k_pool, const kvq_chunk* chunk,
                                          const kvq_block_table* table, const kvq_bounds* bounds, int32_t* dev_status,
                                          void* stream);

/*
 * kvq_bounds_values -- the bounds of n listed storage blocks as values:
 * out fp32 [Hkv][n][2][D] (greatest, then least), 16-byte aligned; blocks:
 * device int32 [n].  An index outside [0, NB) reports KVQ_ERR_INVALID_ARG and
 * gives zeros.  n == 0 does nothing.
 */
KVQ_API kvq_status kvq_bounds_values(const kvq_cache* k, const kvq_bounds* bounds, const int32_t* blocks, int32_t n,
                                     float* out, int32_t* dev_status, void* stream);

/*
 * kvq_select_blocks -- for each query row and KV head, the blocks of its
 * sequence that its queries (all of the head's group) need most.
 *
 * q: device bf16 [rows][Hq][D], contiguous, 16-byte aligned; Hq % Hkv == 0,
 *   Hq / Hkv <= 8.
 * row_seq: device int32 [rows], the sequence of each row, or NULL: row r is
 *   sequence r.  row_lens: device int32 [rows], the tokens that the row sees
 *   (a decode step's seq_lens; for drafted tokens, each one's position + 1).
 *   A row with a sequence outside the cache's (or the table's), or a length
 *   outside [0, capacity], reports KVQ_ERR_INVALID_ARG and counts as length 0.
 * The score of a block, all in IEEE fp32, one rounding an operation, per group
 * g of 32 channels with qp[d], qn[d] = the sums of max(q, 0) and of min(q, 0)
 * over the group's query heads in order:
 *   u = max(qp, -qn over g) / 127, cp = rne(qp / u), cn = rne(qn / u) (u == 0:
 *   0); n = sum of cp * greatest code + cn * least code, a whole number;
 *   t_g = (u * scale_g) * n; the score is ((t_0 + t_1) + t_2) + t_3
 * -- an upper bound of the summed q.k of any of the block's tokens, but for
 * the rounding of q to 8 bits.
 * Of a row's ceil(len / 64) blocks the first `first` and the last `last` are
 * always taken (first, last >= 0, first + last <= n_select); the rest are
 * those of the highest scores, ties to the lower index.  NaN scores (a
 * non-finite query reports KVQ_ERR_NONFINITE) select blocks of the sequence,
 * unspecified which.
 * blocks: device int32 [rows][Hkv][n_select], ascending, then -1 where the
 *   sequence has fewer.  1 <= n_select <= 65536.
 * workspace: device, >= kvq_select_workspace_bytes(rows, Hkv, capacity) bytes
 *   (capacity: tokens a sequence may have: Tcap, or 64 * max_pages), with
 *   kvq_decode_attention's rules (16-byte aligned, zero-filled once before its
 *   first use, calls that share it ordered on the GPU).  One workspace serves
 *   selections of every shape that fits it, and nothing else.
 * rows <= 4096; capacities above 2^29 tokens are KVQ_ERR_UNSUPPORTED.
 */
KVQ_API size_t kvq_select_workspace_bytes(int32_t rows, int32_t Hkv, int32_t capacity);
KVQ_API kvq_status kvq_select_blocks(const void* q, const kvq_cache* k, const kvq_bounds* bounds,
                                     const int32_t* row_seq, const int32_t* row_lens, int32_t rows, int32_t Hq,
                                     int32_t n_select, int32_t first, int32_t last, int32_t* blocks, void* workspace,
                                     size_t workspace_bytes, int32_t* dev_status, void* stream);
/* The same over a page pool; a block whose page id lies outside the pool
 * reports KVQ_ERR_INVALID_ARG and scores as page 0. */
KVQ_API kvq_status kvq_select_blocks_paged(const void* q, const kvq_cache* k_pool, const kvq_bounds* bounds,
                                           const kvq_block_table* table, const int32_t* row_seq,
                                           const int32_t* row_lens, int32_t rows, int32_t Hq, int32_t n_select,
                                           int32_t first, int32_t last, int32_t* blocks, void* workspace,
                                           size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * kvq_decode_attention_blocks -- kvq_decode_attention over listed blocks: the
 * query of row r and KV head h attends the tokens below row_lens[r] of its
 * sequence's blocks blocks[r][h][0 .. n - 1], n = min(n_select, ceil(len /
 * 64)), each KV head its own.  rows, row_seq, row_lens as kvq_select_blocks;
 * the list ascends, -1 (at its end) stands for no block.  An entry that does
 * not ascend, or lies outside the sequence, reports KVQ_ERR_INVALID_ARG and is
 * left out (the entry after it is compared with it all the same).  A row
 * without a token gives zeros.  Blocks that are not listed may hold anything.
 * q, out: [rows][Hq][D]; workspace: kvq_decode_workspace_bytes(rows, Hq, Hkv,
 * D) bytes, for calls of one rows, Hq, Hkv and D (its counters' place depends on
 * them: zero-fill it again before calls of another shape).  Other arguments and
 * errors as kvq_decode_attention.
 */
KVQ_API kvq_status kvq_decode_attention_blocks(const void* q, const kvq_cache* k, const kvq_cache* v,
                                               const int32_t* blocks, int32_t n_select, const int32_t* row_seq,
                                               const int32_t* row_lens, int32_t rows, int32_t Hq, float softmax_scale,
                                               void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                               int32_t* dev_status, void* stream);
/* The same over page pools (page ids as kvq_decode_attention_paged). */
KVQ_API kvq_status kvq_decode_attention_blocks_paged(const void* q, const kvq_cache* k_pool, const kvq_cache* v_pool,
                                                     const kvq_block_table* table, const int32_t* blocks,
                                                     int32_t n_select, const int32_t* row_seq,
                                                     const int32_t* row_lens, int32_t rows, int32_t Hq,
                                                     float softmax_scale, void* out, int32_t out_dtype,
                                                     void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                                     void* stream);

/*
 * kvq_page_table -- the pages of a pool and who has them, kept on the device:
 * every call below changes it in place, in the order of the stream, so that a
 * scheduler's loop needs no copies to the host.  Slot s is a sequence of
 * seq_lens[s] tokens in pages table[s][0 .. ceil(len / 64) - 1] (later entries
 * mean nothing and keep their contents); refs[p] counts the entries that are
 * page p, 0: free.  (table and seq_lens are what the block table and the chunk
 * of the other calls take.)  Pages are handed out lowest free page first.
 * No call shortens a sequence.  A program may lower a length itself (drafted
 * tokens that were rejected), within the last page, length > 64 * (pages - 1),
 * and where that page's count is 1: new tokens go into it, and a page that a
 * fork shares would change for the others too.  Lowered further, the pages past
 * the new end are in no used entry, but their counts stay: the program has to
 * lower those as well (refs[p] by one for each entry given up), or the pages
 * are lost until the table is made anew.
 */
typedef struct kvq_page_table {
  int32_t* refs;       /* device int32 [n_pages] */
  int32_t* table;      /* device int32 [slots][max_pages] */
  int32_t* seq_lens;   /* device int32 [slots] */
  int32_t n_pages;     /* 1 .. 2^24 */
  int32_t slots;       /* 1 .. 65536 */
  int32_t max_pages;   /* pages a slot may have; slots * max_pages and 64 * max_pages below 2^31 */
} kvq_page_table;

/* Device scratch of the calls that take a workspace (16-byte aligned, no
 * initial contents; calls that share it ordered on the GPU). 0 on invalid sizes. */
KVQ_API size_t kvq_pages_workspace_bytes(int32_t n_pages, int32_t slots);

/*
 * kvq_pages_reserve -- room for add[s] >= 0 more tokens in every slot: the
 * pages that the new length needs beyond those it has, handed out in the order
 * of the slots, and the length itself (the new tokens' rows can then be
 * appended).  Where the pages run out, the slots from the first one that they
 * do not suffice for get none: their lengths stay, KVQ_ERR_NO_PAGES is
 * reported (slots that need no new page are served all the same).  A negative
 * add, a length outside [0, 64 * max_pages] or one that would pass it reports
 * KVQ_ERR_INVALID_ARG and leaves the slot alone.
 * add: device int32 [slots].
 */
KVQ_API kvq_status kvq_pages_reserve(const kvq_page_table* pages, const int32_t* add, void* workspace,
                                     size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * kvq_pages_fork -- slot to[i] becomes a copy of slot from[i], i < n: it
 * shares the full pages (their counts rise) and gets its own copy of a last
 * page that is partly filled, in both pools and in `bounds` (NULL: none kept).
 * A slot may be forked into several.  to[i] has to be empty (length 0) and no
 * other pair's to; a pair that breaks this, names a slot outside [0, slots) or
 * whose from has a length outside [0, 64 * max_pages], reports
 * KVQ_ERR_INVALID_ARG and does nothing (of pairs with the same to, the first
 * is served).  Lengths are those before the call.  A pair that finds no page
 * for its copy, and those after it that need one, report KVQ_ERR_NO_PAGES and
 * do nothing.  A page id outside the pool in a used entry is copied as it
 * stands and reported as KVQ_ERR_INVALID_ARG; a partly filled last page with
 * such an id takes no page for to[i].
 * k_pool, v_pool: the pools, B = n_pages, Tcap = 64, of equal shape and bits.
 * from, to: device int32 [n]; n <= slots, n == 0 does nothing.
 */
KVQ_API kvq_status kvq_pages_fork(const kvq_page_table* pages, const kvq_cache* k_pool, const kvq_cache* v_pool,
                                  const kvq_bounds* bounds, const int32_t* from, const int32_t* to, int32_t n,
                                  void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * kvq_pages_free -- slots which[i], i < n, let their pages go (the counts
 * fall) and are empty.  A slot outside [0, slots), a length outside [0, 64 *
 * max_pages] or a page that is outside the pool or free already reports
 * KVQ_ERR_INVALID_ARG and is passed over (such a length becomes 0); a slot
 * listed twice is let go once.  n == 0 does nothing.
 */
KVQ_API kvq_status kvq_pages_free(const kvq_page_table* pages, const int32_t* which, int32_t n, int32_t* dev_status,
                                  void* stream);

/*
 * kvq_pages_compact -- the live pages (refs > 0) become pages 0 .. n_live - 1:
 * the live ones from n_live on move, in order, into the free ones before it,
 * in order; their data in both pools and `bounds` (NULL: none kept), their
 * counts and every table entry in use follow.  n_live (device int32 [1], NULL:
 * not wanted) gets the number of live pages.  Pages that became free keep
 * their data.
 */
KVQ_API kvq_status kvq_pages_compact(const kvq_page_table* pages, const kvq_cache* k_pool, const kvq_cache* v_pool,
                                     const kvq_bounds* bounds, int32_t* n_live, void* workspace,
                                     size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * kvq_copy_pages -- page dst[i] of both pools (and `bounds`, NULL: none kept)
 * becomes a copy of page src[i], i < n.  A pair with a negative index is
 * skipped; one beyond the pool reports KVQ_ERR_INVALID_ARG and is skipped.  A
 * page may be the source of several pairs, but a destination is no other
 * pair's source or destination.  src, dst: device int32 [n]; n == 0 does
 * nothing.
 */
KVQ_API kvq_status kvq_copy_pages(const kvq_cache* k_pool, const kvq_cache* v_pool, const kvq_bounds* bounds,
                                  const int32_t* src, const int32_t* dst, int32_t n, int32_t* dev_status,
                                  void* stream);

/* Static, human-readable name of a status code. */
KVQ_API const char* kvq_status_str(kvq_status status);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_H */
