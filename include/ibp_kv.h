/*
 * ibp_kv.h -- C ABI of libibp_kv, an 8-bit KV page cache with the attention
 * that reads it, on AMD Instinct MI355X (gfx950).
 *
 * The page that libibp follows keeps the keys and values of offloaded LLM
 * inference as compressed 16-bit pages in host memory ("Reducing the GPU
 * Memory Bottleneck with Lossless Compression for ML -- Extended", Kamath,
 * Krishnamurthy, Canini, Peter, section "System integration").  This library
 * is the other end of that path: the pages a GPU attends over while it
 * decodes, in 8 bits, with the three operations of a decoding step.
 *
 *   ibp_kv_append     16-bit keys and values of new tokens into the pages
 *   ibp_kv_attention  attention of the new tokens' queries over the pages,
 *                     with the attention weight that each page received
 *   ibp_kv_evict      each head keeps its heaviest pages
 *
 * Pages
 * -----
 * A page holds page_tokens (16, 32 or 64) consecutive tokens of one
 * key/value head: head_dim (64, 128, 192 or 256) e4m3 codes a token for the
 * keys, as many for the values, and one 32-bit scale for each.  Page p is at
 * byte p * page_tokens * head_dim of k_codes and of v_codes; its scales are
 * k_scales[p] and v_scales[p]; a value is code * scale.  e4m3: sign, 4
 * exponent bits (bias 7), 3 mantissa bits, largest 448, no infinities, NaN =
 * 0x7F and 0xFF.
 *
 * A page is a run of page_tokens / 16 tiles of 16 tokens.  In a key tile,
 * token t, dim 64 j + 16 g + b (g < 4, b < 16) is byte
 *     1024 j + 256 g + 16 t + b
 * and in a value tile, token 4 g + r, dim 64 h + 16 c + i (g, r, c < 4,
 * i < 16) is byte
 *     1024 h + 256 g + 16 i + 4 c + r
 * so that lane l of a wave finds the operands of its matrix instructions in
 * the 16 bytes at 1024 j + 16 l.
 *
 * Tables
 * ------
 * Row (s, h) of `pages` lists the pages of sequence s, head h in token
 * order: max_pages ids at pages + (s * kv_heads + h) * max_pages.
 * lengths[s * kv_heads + h] counts the row's tokens ONCE THE NEW ONES ARE
 * IN: a step advances the lengths first, then appends, then attends.  A
 * length below 0 counts as 0, one above max_pages * page_tokens as that.  An
 * id outside [0, n_pages) is a hole: appending to it writes nothing, and its
 * tokens take no part in attention.  Two entries of the tables may name the
 * same page as long as no append writes to it.
 *
 * New tokens
 * ----------
 * A call brings up to n_new tokens a sequence; with `counts` (device int32,
 * one a sequence, clamped to [0, n_new]) sequence s brings its first
 * counts[s], without it n_new.  Token i of them is at position
 * length - count + i of every row of its sequence; a token whose position is
 * negative does not exist.
 *
 * Memory, streams, errors
 * -----------------------
 * As in ibp.h: the caller owns every buffer (all of it device memory here),
 * every call only enqueues kernels on `stream` (no allocation, no memset, no
 * synchronisation; a caller may capture it in a HIP graph), arguments are
 * checked on the host before anything is enqueued, statuses are those of
 * ibp.h, and a HIP error that is pending at entry is returned and left
 * pending.  The buffers and the stream are the current device's.  Device data (ids, lengths, counts, scales) is not checked on the
 * host; no value of it makes a kernel read or write outside the buffers.
 * A call whose rows need more threads than a launch has (2^32: some 2^24 rows
 * of an eviction or of attention, 2^22 rows of 1025-16384 pages of an eviction)
 * is an invalid argument.
 * Buffers that a call writes must not overlap what it reads, except where
 * said.  Equal inputs give equal bytes.
 */
#ifndef IBP_KV_H_
#define IBP_KV_H_

#include <stdint.h>

#include "ibp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of keys, values, queries and outputs. */
#define IBP_KV_BF16 0u
#define IBP_KV_FP16 1u

/* The pool of pages.  k_codes and v_codes: n_pages * page_tokens * head_dim
 * bytes, 16-byte aligned; k_scales and v_scales: n_pages floats. */
typedef struct ibp_kv_cache {
  uint64_t n_pages;
  uint32_t page_tokens;
  uint32_t head_dim;
  uint8_t *k_codes;
  float *k_scales;
  uint8_t *v_codes;
  float *v_scales;
} ibp_kv_cache;

/* Which pages hold which head of which sequence.  max_pages * page_tokens
 * must be below 2^31. */
typedef struct ibp_kv_table {
  uint64_t n_seqs;
  uint64_t kv_heads;
  uint64_t max_pages;
  const int32_t *pages;   /* [n_seqs][kv_heads][max_pages] */
  const int32_t *lengths; /* [n_seqs][kv_heads] */
} ibp_kv_table;

/* A 16-bit tensor [n_seqs][n_new][heads][head_dim]: element (s, i, h, d) is
 * at data + s * seq_stride + i * token_stride + h * head_stride + d, strides
 * in elements, any sign, 0 for a broadcast input; rows of an output must not lie
 * on each other.  Rows whose address and strides are multiples of 16 bytes are
 * moved 16 bytes at a time, others element by element. */
typedef struct ibp_kv_tensor {
  void *data;
  int64_t seq_stride;
  int64_t token_stride;
  int64_t head_stride;
} ibp_kv_tensor;

/*
 * Appends the new tokens' keys and values (kv_heads heads) to their pages.
 *
 * A page's scale is 2^e with the smallest e in [-126, 119] for which every
 * finite new value of the page is at most 448 * 2^e in magnitude; a page
 * that held tokens before keeps its scale if that is larger, else its codes
 * are brought to the new scale (which is exact until a code becomes
 * subnormal).  Codes are rounded to nearest, ties to even, and saturate at
 * 448; a value that is not finite becomes the code 0x7F and does not count
 * for the scale.  Bytes of the page past the row's length are cleared.
 * Appending the same tokens again changes nothing.
 */
int ibp_kv_append(const ibp_kv_cache *cache, const ibp_kv_table *table, uint32_t dtype,
                  uint64_t n_new, const ibp_kv_tensor *k, const ibp_kv_tensor *v,
                  const int32_t *counts, void *stream);

/* Bytes of workspace that ibp_kv_attention needs for these arguments; 0 when
 * it needs none or when they are not valid.  with_weights: whether weights
 * are asked for. */
uint64_t ibp_kv_attention_workspace_bytes(const ibp_kv_cache *cache, const ibp_kv_table *table,
                                          uint64_t q_heads, uint64_t n_new, int with_weights);

/*
 * Attention of the new tokens' queries (q_heads = group * kv_heads heads;
 * query head x reads key/value head x / group) over the row's pages: the
 * query at position p sees the tokens at positions 0..p of its row.
 *
 *     s_j = scale * (q . k_j),  w_j = exp(s_j) / sum_i exp(s_i),
 *     out = sum_j w_j v_j       (rounded once, to dtype)
 *
 * A query that sees nothing (its position is negative, every page is a hole,
 * every score is minus infinity), and one past its sequence's count, gets
 * zeros.  Scores, statistics and sums are held in 32 bits, the sums up to 2^8
 * times their normalised value for each token of the row: values above about
 * 2^119 / (tokens of the row) may overflow.  The w_j enter the second product
 * with 16 bits, and a page's share of them is the exponential of a difference of
 * 32-bit logarithms (a relative error of about 2^-23 times the largest score).
 * What a query may not see does not reach it, NaN included.  Values whose scale
 * is not finite are NaN.
 *
 * weights, weights_out (both or neither; float, [n_seqs][kv_heads][max_pages];
 * they may be the same buffer): weights_out = weights + the w_j that the
 * page's tokens received from all queries of the row.
 *
 * workspace: 16-byte aligned device memory of at least
 * ibp_kv_attention_workspace_bytes; its content does not matter and calls
 * that do not run at the same time may share it.
 */
int ibp_kv_attention(const ibp_kv_cache *cache, const ibp_kv_table *table, uint32_t dtype,
                     uint64_t q_heads, uint64_t n_new, const ibp_kv_tensor *q,
                     const ibp_kv_tensor *out, const int32_t *counts, float scale,
                     const float *weights, float *weights_out, void *workspace,
                     uint64_t workspace_bytes, void *stream);

/*
 * Every row keeps at most keep_pages pages: its first sink_pages, its last
 * recent_pages (at least 1: the last page may be partly filled) and, of the
 * pages between, those of the largest weight, the lower position first among
 * equals (-0 equals 0; NaN is above all numbers).  keep_pages must be at
 * least sink_pages + recent_pages.
 *
 * pages_out lists the kept pages in their order, then the evicted ones in
 * theirs, then the row's other entries as they were: the pages past the new
 * length are spare, for the tokens that come.  weights_out follows its page;
 * an evicted page's weight is 0.  lengths_out counts the tokens left.  No
 * page is touched.  The outputs must not overlap the inputs or each other.
 */
int ibp_kv_evict(const ibp_kv_table *table, uint32_t page_tokens, uint64_t keep_pages,
                 uint64_t sink_pages, uint64_t recent_pages, const float *weights,
                 int32_t *pages_out, float *weights_out, int32_t *lengths_out, void *stream);

/* Static description of a status code of this library. */
const char *ibp_kv_status_string(int status);

/* hipError_t behind the calling thread's last IBP_ERR_HIP from this library. */
int ibp_kv_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* IBP_KV_H_ */
