/*
 * mxfp4.h -- C ABI of the MXFP4 (microscaled 4-bit floating point) operators
 * of libnvfp4fc2.so: quantisation, the block-scaled product, a paged KV cache
 * held in 4 bits, and attention over it, on one GB300 (sm_103a).
 *
 *   x (BF16/FP16/FP32)  --mxfp4_quantize-------> MXFP4 matrix
 *   MXFP4 matrix        --mxfp4_dequantize-----> BF16/FP16/FP32
 *   MXFP4 x MXFP4       --mxfp4_gemm-----------> BF16/FP16/FP32 (FP32 accumulation)
 *   x, MXFP4 weight     --mxfp4_linear---------> quantise the rows of x, then the product
 *   k, v, slots         --mxfp4_cache_write----> codes and scales in the paged cache
 *   cache, block table  --mxfp4_cache_read-----> k, v of whole sequences
 *   q, cache            --mxfp4_cache_attention> softmax(scale q k^T + mask) v
 *   q, cache, groups    --mxfp4_cache_attention_shared> the same, what a group shares read once
 *   q, k, positions     --head_norm_rotary-----> normed and rotated heads
 *   q, k, v, positions  --mxfp4_cache_write_rotary> rotated q; codes and scales of rotated k, and of v
 *   refs, table, lens   --mxfp4_pages_*--------> pages of rows: grown, forked, freed, made compact
 *   cache, page pairs   --mxfp4_cache_copy-----> copies of pages
 *
 * MXFP4 recipe (32 consecutive elements of a row share one scale):
 *   E     = clamp(floor(log2 max|x|) - 2 + 127, 0, 254), 0 for an all-zero block
 *   scale = 2^(E - 127)                               (E8M0)
 *   code  = RNE_E2M1_satfinite(x * 2^(127 - E))       (sign of zero kept)
 * All of it is exact but the one rounding of the element.  A block that holds
 * an infinity or a NaN gets E = 255 and zero codes, and reads back as NaN.
 * Against the NVFP4 of nvfp4_fc2.h there is no global scale, hence one pass.
 *
 * Layout of a matrix [rows, cols], cols_pad = ceil(cols / 128) * 128:
 *   QDATA   [rows, cols_pad / 2] uint8; byte j of a row = code(2j) | code(2j+1) << 4;
 *           elements in cols .. cols_pad - 1 are zero codes.
 *   scales  uint8, tiles of 128 rows x 4 scale columns (a scale column = 32
 *           elements): scale (r, c) at
 *           ((r/128)*(cols_pad/128) + c/4)*512 + (r%32)*16 + ((r/32)%4)*4 + c%4,
 *           for ceil(rows / 128) * 128 rows.  Scale columns past cols are 0;
 *           bytes of rows >= rows are never written and never matter.
 *
 * Layout of a KV cache of `pages` pages of `page_size` tokens:
 *   k_codes, v_codes    [pages, kv_heads, page_size, dim / 2] uint8
 *   k_scales, v_scales  [pages, kv_heads, page_size, dim / 32] uint8
 * Token t of sequence b lies in page table[b][t / page_size], at t % page_size.
 * Bytes that no token was written to may hold anything.
 *
 * Conventions (ownership, threads, streams, errors) are those of nvfp4_fc2.h:
 * the caller owns every buffer, all work is enqueued on `stream`, argument
 * errors are returned before anything is enqueued, and kernels with bounded
 * pipeline waits report NVFP4_ETIMEOUT in `dev_status` (device uint32 or
 * NULL; never cleared by the library).  Results do not depend on timing: the
 * same call on the same inputs gives the same bits.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stdint.h>
#include "nvfp4_fc2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the tensors outside the 4-bit format. */
enum { MXFP4_BF16 = 0, MXFP4_FP16 = 1, MXFP4_FP32 = 2 };

/* ceil(cols / 128) * 128 (0 for cols <= 0). */
int64_t mxfp4_padded_cols(int64_t cols);
/* Bytes of QDATA of a [rows, cols] matrix: rows * cols_pad / 2. */
int64_t mxfp4_qdata_bytes(int64_t rows, int64_t cols);
/* Bytes of the tiled scales: ceil(rows/128)*128 * cols_pad / 32. */
int64_t mxfp4_scale_bytes(int64_t rows, int64_t cols);
/* Byte offset of scale (r, c), c = column / 32. */
int64_t mxfp4_scale_offset(int64_t r, int64_t c, int64_t cols);

/* One-pass MXFP4 of x [rows, cols], row stride ld >= cols elements.
 *   dtype   MXFP4_BF16, _FP16 or _FP32; x aligned to its element, any ld
 *   rows, cols >= 1, cols <= 2^24, rows * cols_pad < 2^40
 *   qdata, scales  16-byte aligned, sizes as above */
nvfp4_status mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void* qdata,
                            void* scales, nvfp4_stream_t stream);

/* The values of an MXFP4 matrix, out [rows, cols], row stride ld >= cols:
 * exact in BF16 and FP32, rounded once (to nearest even, to infinity past
 * 65504) in FP16.  NaN blocks give NaN. */
nvfp4_status mxfp4_dequantize(const void* qdata, const void* scales, int64_t rows, int64_t cols, void* out,
                              int32_t dtype, int64_t ld, nvfp4_stream_t stream);

/* out[i, j] = round(sum_k A[i,k] W[j,k]), i < m, j < n: block-scaled FP4
 * tensor-core product with FP32 accumulation, rounded once to `dtype`.
 *   a_q, a_s  MXFP4 [m, k];  w_q, w_s  MXFP4 [n, k]  (16-byte aligned)
 *   m, n, k >= 1; k <= 2^24, m and n <= 2^30
 *   out       row stride ldo >= n, aligned to its element; elements outside
 *             [m, n] are not touched
 * The order of the sum depends on m, n and k only. */
nvfp4_status mxfp4_gemm(const void* a_q, const void* a_s, const void* w_q, const void* w_s, int64_t m, int64_t n,
                        int64_t k, void* out, int32_t dtype, int64_t ldo, uint32_t* dev_status,
                        nvfp4_stream_t stream);

/* Bytes of the workspace of mxfp4_linear for m rows of k elements. */
int64_t mxfp4_linear_workspace_bytes(int64_t m, int64_t k);

/* out = mxfp4(x) W^T: the rows of x [m, k] (row stride ldx, element type
 * x_dtype) are quantised and multiplied with an MXFP4 weight [n, k], as
 * mxfp4_quantize and mxfp4_gemm would.  workspace: 16-byte aligned, at least
 * mxfp4_linear_workspace_bytes(m, k) bytes (0 for few rows, which need none:
 * NULL then); its contents before and after do
 * not matter. */
nvfp4_status mxfp4_linear(const void* x, int32_t x_dtype, int64_t m, int64_t ldx, const void* w_q, const void* w_s,
                          int64_t n, int64_t k, void* out, int32_t dtype, int64_t ldo, void* workspace,
                          int64_t workspace_bytes, uint32_t* dev_status, nvfp4_stream_t stream);

/* A paged KV cache in device memory (layout above), every pointer 16-byte
 * aligned.  page_size: a power of two, 16 .. 256; dim: 64, 128 or 256;
 * kv_heads 1 .. 65535; pages 1 .. 2^31 - 1 with pages * kv_heads < 2^31. */
typedef struct {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  int64_t pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t dim;
  int32_t reserved;
} mxfp4_cache;

/* Quantises k and v of `tokens` tokens into their slots.
 *   k, v   [tokens, kv_heads, dim] of `dtype`, unit stride along dim, strides
 *          in elements along tokens (k_st, v_st) and heads (k_sh, v_sh)
 *   slots  device int64 [tokens]: page * page_size + offset; a slot below 0
 *          or past the cache is skipped.  The others have to differ: tokens of
 *          one slot leave a mixture of their codes and scales there
 * tokens may be 0. */
nvfp4_status mxfp4_cache_write(const mxfp4_cache* cache, const void* k, const void* v, int32_t dtype, int64_t tokens,
                               int64_t k_st, int64_t k_sh, int64_t v_st, int64_t v_sh, const int64_t* slots,
                               nvfp4_stream_t stream);

/* Reads whole sequences back: for every sequence b and t < starts[b+1] -
 * starts[b], row starts[b] + t of k and v [total, kv_heads, dim] (contiguous,
 * `dtype`) gets the token's values (NaN where its block holds E = 255).
 *   table   device int32 [seqs, table_ld]; ids outside the cache are clamped to it
 *   starts  device int32 [seqs + 1], starts[0] = 0, not decreasing, last = total
 * total may be 0. */
nvfp4_status mxfp4_cache_read(const mxfp4_cache* cache, const int32_t* table, int64_t table_ld, int64_t seqs,
                              const int32_t* starts, int64_t total, void* k, void* v, int32_t dtype,
                              nvfp4_stream_t stream);

/* Attention of new tokens over the cache.  Sequence b has lens[b] tokens in
 * the cache (its new ones among them) and n_b = q_starts[b+1] - q_starts[b]
 * queries, rows q_starts[b] .. of q; query i stands at position
 * p = lens[b] - n_b + i and sees key j iff
 *   0 <= j < lens[b],  j <= p where causal,
 *   and, where window > 0, j > p - window or j < sinks.
 * out = softmax(scale * q k^T) v over the keys it sees, zeros (and lse =
 * -inf) where it sees none; query head h reads kv head h / (q_heads/kv_heads).
 * Bytes of keys that a query does not see do not reach its result, NaN
 * scales among them.
 * Precision: scores, sums and outputs are binary32, rounded once to `dtype`;
 * for the product with the values the weights are rounded to 11 bits.  Beside
 * much larger ones small keys and values count as rounded, too: keys to 2^-40
 * of the largest of the 64 around them, values to 2^-16 of the largest that
 * the query sees in their block of 32 columns (2^-24 where all queries of the
 * call see that one).  Where queries of a call see very different ones, each
 * is worked out by itself, slowly, so that this holds for what each of them
 * sees.
 *   q       [total_q, q_heads, dim] of `dtype` (BF16 or FP16), strides q_st,
 *           q_sh in elements (unit along dim)
 *   out     as q, strides o_st, o_sh;  lse  float32 [total_q, q_heads] or NULL
 *           (natural logarithm of the sum of exponentials)
 *   q_starts device int32 [seqs + 1], not decreasing, or NULL: one query a
 *           sequence; what lies outside 0 .. total_q counts as its ends
 *   max_queries  an upper bound of n_b known to the host (1 for NULL);
 *           max_queries * q_heads / kv_heads <= 2^24, table_ld * page_size <= 2^31,
 *           lens[b] <= table_ld * page_size and < 2^31 - 2^25
 *   workspace    16-byte aligned, mxfp4_attention_workspace_bytes() bytes */
typedef struct {
  const void* q;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* q_starts;
  void* workspace;
  uint32_t* dev_status;
  int64_t q_st, q_sh, o_st, o_sh;
  int64_t table_ld;
  int64_t workspace_bytes;
  int32_t seqs;
  int32_t total_q;
  int32_t max_queries;
  int32_t q_heads;
  int32_t dtype;
  int32_t causal;
  int32_t window;
  int32_t sinks;
  float scale;
  int32_t reserved;
} mxfp4_attention;

/* Bytes of workspace that mxfp4_cache_attention needs on the current device
 * for these head counts (it does not depend on the lengths). */
int64_t mxfp4_attention_workspace_bytes(int32_t kv_heads, int32_t q_heads, int32_t dim, int32_t max_queries);

nvfp4_status mxfp4_cache_attention(const mxfp4_cache* cache, const mxfp4_attention* args, nvfp4_stream_t stream);

/* Attention of sequences that share a prefix: the result of
 * mxfp4_cache_attention (causal or not, without a window) on the same
 * arguments, but tokens that the sequences of a group have in common are read
 * once for all of them.  Sequences groups[g] .. groups[g+1] - 1 share their
 * first shared[g] tokens: what their block tables name there holds the same
 * bytes, as after mxfp4_pages_select, and is read through any one's.  Whole
 * pages of them are shared, and only as many as lie before every query of the
 * group (not causal: as every sequence has); the others are read by each
 * sequence.  Sequences before groups[0] and from groups[count] on share nothing.
 *   groups    device int32 [count + 1], not decreasing; what lies outside
 *             0 .. seqs counts as its ends
 *   shared    device int32 [count]
 *   max_group an upper bound of the queries of a group known to the host; the
 *             estimate below takes count * max_group queries, if there are as
 *             many, for those that share
 *   always    0: every sequence reads for itself where that is estimated to be
 *             as fast, from the sizes and as if the block tables were full (for
 *             short prefixes in tables of long ones mxfp4_cache_attention is the
 *             quicker call); 1: never
 *   args      as above, window and sinks 0, workspace_bytes of either query below
 * Precision: as above for each part; the parts are binary32 and joined in it. */
typedef struct {
  const int32_t* groups;
  const int32_t* shared;
  int32_t count;
  int32_t max_group;
  int32_t always;
  int32_t reserved;
} mxfp4_shared;

/* Bytes of workspace that mxfp4_cache_attention_shared needs at the most, whatever
 * page_size and `always` are. */
int64_t mxfp4_attention_shared_workspace_bytes(int32_t kv_heads, int32_t q_heads, int32_t dim, int32_t total_q,
                                               int32_t max_queries, int32_t seqs, int64_t table_ld, int32_t count,
                                               int32_t max_group);
/* Bytes that it needs for these arguments (from the sizes among them; no pointer in
 * them is followed): those of mxfp4_cache_attention where nothing is shared, while the
 * parts take two binary32 outputs. */
int64_t mxfp4_attention_shared_call_workspace_bytes(const mxfp4_cache* cache, const mxfp4_attention* args,
                                                    const mxfp4_shared* shared);

nvfp4_status mxfp4_cache_attention_shared(const mxfp4_cache* cache, const mxfp4_attention* args,
                                          const mxfp4_shared* shared, nvfp4_stream_t stream);

/* Heads of tokens: x [tokens, heads, dim], unit stride along dim, strides in
 * elements along tokens (st) and heads (sh); out alike (o_st, o_sh), and may be
 * x itself with the same strides, but shares memory with no other heads of the
 * call.  weight [dim] of the norm, or NULL for none. */
typedef struct {
  const void* x;
  void* out;
  const void* weight;
  int64_t st, sh, o_st, o_sh;
  int32_t heads;
  int32_t reserved;
} mxfp4_heads;

/* Rotary positions.  The first 2 * pairs elements of a head are pairs, the
 * others stay as they are.  Pair i is elements 2i and 2i + 1 (interleaved) or i
 * and i + pairs, and turns by position * frequency:
 *   (a, b) -> (a cos t - b sin t, b cos t + a sin t)
 *   t = 2 pi 2^-64 (positions[token, axis[i]] * turns[i] mod 2^64)
 *   turns      device int64 [pairs]: frequency / 2 pi in units of 2^-64
 *   axis       device int32 [pairs], or NULL for 0; clamped to 0 .. axes - 1
 *   positions  device int32 [tokens, axes]
 *   pairs      a multiple of 8, 2 * pairs <= dim; 0: no rotation */
typedef struct {
  const int64_t* turns;
  const int32_t* axis;
  const int32_t* positions;
  int32_t pairs;
  int32_t axes;
  int32_t interleaved;
  int32_t reserved;
} mxfp4_rotary;

/* out = rotation(norm(x)) for the heads of q, and of k unless it is NULL, with
 * norm(x) = x / sqrt(mean(x^2) + eps) * weight over each head.  Binary32, the
 * result rounded once.
 *   dtype         of x and out; weight_dtype: the same, or MXFP4_FP32
 *   dim           a multiple of 16 up to 256;  eps 1e-12 .. 1
 * tokens may be 0. */
nvfp4_status head_norm_rotary(const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_rotary* rotary, int32_t dtype,
                              int32_t weight_dtype, int64_t tokens, int32_t dim, float eps, nvfp4_stream_t stream);

/* head_norm_rotary of q into its out, and of k into its slots of the cache in
 * MXFP4 (quantised from binary32), where v goes as mxfp4_cache_write would put
 * it.  dtype BF16 or FP16; k->out and v->out are not used, v->weight is NULL;
 * slots as for mxfp4_cache_write (a token without one still has its q). */
nvfp4_status mxfp4_cache_write_rotary(const mxfp4_cache* cache, const mxfp4_heads* q, const mxfp4_heads* k,
                                      const mxfp4_heads* v, const int64_t* slots, const mxfp4_rotary* rotary,
                                      int32_t dtype, int32_t weight_dtype, int64_t tokens, float eps,
                                      nvfp4_stream_t stream);

/* The pages of a cache (of the caches of all layers that share a block table),
 * held on the device:
 *   refs   int32 [pages]: how many rows hold the page; 0 for a free one
 *   table  int32 [rows, table_ld]: row b of lens[b] tokens holds its first
 *          ceil(lens[b] / page_size) pages, each once
 *   lens   int32 [rows]
 * The functions change all three in place, in stream order, and touch no
 * cache.  Rows, lengths and page ids outside their ranges count as their ends
 * (lengths) or as no page.  Page ids come out the same for the same state.
 *   pages 1 .. 2^30, rows 1 .. 2^20, table_ld * page_size <= 2^31 - 2^25,
 *   page_size as for a cache; rows * table_ld <= 2^31 */
typedef struct {
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int64_t pages;
  int64_t table_ld;
  int32_t rows;
  int32_t page_size;
} mxfp4_pages;

/* Bytes of workspace (16-byte aligned) that each of the three needs. */
int64_t mxfp4_pages_workspace_bytes(const mxfp4_pages* pages);

/* Every row becomes what row sources[b] was before the call, its pages then
 * held by both; -1 (or no row): empty.  sources[b] = b leaves a row alone.
 * Table entries behind a row's pages stay as they were.
 *   sources  device int32 [rows] */
nvfp4_status mxfp4_pages_select(const mxfp4_pages* pages, const int32_t* sources, void* workspace,
                                int64_t workspace_bytes, nvfp4_stream_t stream);

/* Pages for counts[b] more tokens of every row, which its length then counts.
 * New pages are the free ones of the lowest ids, row by row.  Where a row's
 * next token goes into a page that holds some and other rows hold it too, the
 * row gets a copy of its own: copies[b] = (that page, new page), which
 * mxfp4_cache_copy has to copy in every cache before new tokens are written;
 * (-1, -1) elsewhere.  If all the rows that hold a page go on in it, the first
 * of them keeps it.
 *   counts   device int32 [rows]; below 0 counts as 0
 *   slots    device int64 [total]: the new tokens' slots, row by row; -1 behind
 *            the last one
 *   copies   device int32 [rows, 2]
 *   missing  device int32 [1]: 0; or the free pages that are lacking; or -1 if
 *            a row of the table is too short, or `total`: then slots and copies
 *            are -1 and nothing has changed */
nvfp4_status mxfp4_pages_extend(const mxfp4_pages* pages, const int32_t* counts, int64_t total, int64_t* slots,
                                int32_t* copies, int32_t* missing, void* workspace, int64_t workspace_bytes,
                                nvfp4_stream_t stream);

/* Moves the pages that are held to the ids 0 .. used - 1: those from `used` on,
 * in their order, to the free ids below it.
 *   moves  device int32 [pages / 2, 2]: (from, to) for mxfp4_cache_copy, which
 *          has to be called for every cache; (-1, -1) behind the last one
 *   used   device int32 [1] */
nvfp4_status mxfp4_pages_compact(const mxfp4_pages* pages, int32_t* moves, int32_t* used, void* workspace,
                                 int64_t workspace_bytes, nvfp4_stream_t stream);

/* Copies pages: page pairs[i][0] of `source` to page pairs[i][1] of `cache`
 * (which may be the same).  Pairs with an id outside of its cache are skipped.
 * No page is the target of two pairs, nor the target of one and the source of
 * another in the same cache.
 *   pairs  device int32 [count, 2]; count may be 0
 *   source has the cache's page_size, kv_heads and dim */
nvfp4_status mxfp4_cache_copy(const mxfp4_cache* cache, const mxfp4_cache* source, const int32_t* pairs,
                              int64_t count, nvfp4_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MXFP4_H */
