/*
 * ibp_kv_long.h -- C ABI of libibp_kv_long, long and shared contexts over the
 * 8-bit KV pages of ibp_kv.h, on AMD Instinct MI355X (gfx950).
 *
 *   ibp_kv_append_rotated    as ibp_kv_append, with the keys' position rotation
 *                            applied on the way, and that of the step's queries
 *   ibp_kv_outline           what bounds the keys of a page, in 8 bits
 *   ibp_kv_select            each row's pages whose outlines promise the largest
 *                            scores, as a table that ibp_kv_attention reads
 *   ibp_kv_attention_shared  attention of sequences that share a prefix, whose
 *                            pages are read once for all of them
 *
 * Pages, tables, new tokens and tensors are those of ibp_kv.h, and so are the
 * rules on memory, streams and errors; statuses have the text of
 * ibp_kv_status_string.
 */
#ifndef IBP_KV_LONG_H_
#define IBP_KV_LONG_H_

#include <stdint.h>

#include "ibp_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rotation of the first rotary_dim dims (a multiple of 16, at most head_dim) of
 * keys and queries.  Pair i of them, i < rotary_dim / 2, is dims i and i +
 * rotary_dim / 2, or with `interleaved` dims 2 i and 2 i + 1; at position p
 *     (x, y) -> (x * cos[p][i] - y * sin[p][i], y * cos[p][i] + x * sin[p][i]),
 * each product and each sum rounded to 32 bits.  cos, sin: float
 * [n_positions][rotary_dim / 2], 16-byte aligned.  positions: int32
 * [n_seqs][n_new], the positions of the new tokens; null: their places in their
 * rows (which are others once pages have been evicted, and where rows are a
 * sequence's own behind a shared prefix).  At a position outside [0, n_positions)
 * the rotated dims are NaN. */
typedef struct ibp_kv_rotation {
  uint64_t n_positions;
  uint32_t rotary_dim;
  uint32_t interleaved;
  const float *cos;
  const float *sin;
  const int32_t *positions;
} ibp_kv_rotation;

/* Outlines of the pool's pages: codes int8 [n_pages][2][head_dim], 16-byte
 * aligned, scales float [n_pages].  With u = 2^e the smallest power of two, e >=
 * -15, for which no number of the page's key codes is above 127 u, codes hold
 * for each dim the largest number in units of u, rounded up, and the smallest,
 * rounded down, and the scale is the keys' scale * u: a key of the page is at
 * most codes[0] * scale and at least codes[1] * scale.  The outline of a page
 * with a NaN code, or whose keys' scale is not finite, is zeros with the scale
 * NaN. */
typedef struct ibp_kv_outlines {
  int8_t *codes;
  float *scales;
} ibp_kv_outlines;

/*
 * ibp_kv_append of the keys after the rotation.  Scales and codes come from the
 * rotated numbers in 32 bits (one that is not finite becomes the code 0x7F), which
 * are not rounded to 16 bits between.
 *
 * q, q_out (both or neither; q_heads heads, a multiple of kv_heads): the new
 * tokens' queries are rotated too, and rounded once to dtype; those of a token that
 * does not exist (past its sequence's count, at a place below 0) become zeros.
 * q_out may be q with the same strides, and must not overlap it otherwise.
 *
 * outlines (may be null): those of the pages that receive new tokens are brought
 * up to date, as by ibp_kv_outline.
 */
int ibp_kv_append_rotated(const ibp_kv_cache *cache, const ibp_kv_table *table, uint32_t dtype,
                          uint64_t n_new, const ibp_kv_tensor *k, const ibp_kv_tensor *v,
                          const int32_t *counts, const ibp_kv_rotation *rotation, uint64_t q_heads,
                          const ibp_kv_tensor *q, const ibp_kv_tensor *q_out,
                          const ibp_kv_outlines *outlines, void *stream);

/* Outlines of the pages that hold the last tokens of each row, n_new of them or,
 * with counts, counts[s] (clamped to [0, n_new]): of the tokens that a page
 * holds, old ones and new ones.  Rows that name the same page must hold the same
 * number of its tokens. */
int ibp_kv_outline(const ibp_kv_cache *cache, const ibp_kv_outlines *outlines,
                   const ibp_kv_table *table, uint64_t n_new, const int32_t *counts, void *stream);

/* Bytes of workspace that ibp_kv_select needs; 0 when it needs none or when the
 * arguments are not valid. */
uint64_t ibp_kv_select_workspace_bytes(const ibp_kv_cache *cache, const ibp_kv_table *table);

/*
 * Every row keeps at most keep_pages pages for its new tokens' queries (q_heads =
 * group * kv_heads heads): its first sink_pages, its last recent_pages and, of
 * the pages between, those with the largest scores, the lower position first
 * among equals.  keep_pages must be at least sink_pages + recent_pages, and
 * recent_pages cover the new tokens wherever their first page begins:
 * (n_new + page_tokens - 2) / page_tokens + 1.
 *
 * A page's score is the largest that a query q of the row (a query of a token
 * that exists; one with a number that is not finite takes no part) could give to
 * a key within the outline: with q rounded to whole numbers of t, the smallest
 * power of two (2^-126 or more) of which 127 * 128 are at least the largest
 * magnitude of q (1 for zeros),
 *     S = sum over d of  (q_d > 0 ? q_d * codes[0][d] : q_d * codes[1][d]),
 * which is exact, rounded once to 32 bits, times t; the largest of these
 * (minus infinity without queries) times the outline's scale.  Holes have the score
 * minus infinity; NaN is above all numbers; -0 equals 0.  (A bound on attention's scores for a scale
 * above 0, but for the rounding of q.)
 *
 * pages_out, places_out: int32 [n_seqs][kv_heads][keep_pages], the ids of the
 * kept pages in table order and their places in the row's table, -1 past them.
 * lengths_out: tokens of the kept pages.  With these as its table
 * ibp_kv_attention attends over the selected pages.  The outputs must not overlap
 * the inputs or each other.
 */
int ibp_kv_select(const ibp_kv_cache *cache, const ibp_kv_outlines *outlines,
                  const ibp_kv_table *table, uint32_t dtype, uint64_t q_heads, uint64_t n_new,
                  const ibp_kv_tensor *q, const int32_t *counts, uint64_t keep_pages,
                  uint64_t sink_pages, uint64_t recent_pages, int32_t *pages_out,
                  int32_t *lengths_out, int32_t *places_out, void *workspace,
                  uint64_t workspace_bytes, void *stream);

/* Bytes of workspace that ibp_kv_attention_shared needs; 0 when it needs none or
 * when the arguments are not valid. */
uint64_t ibp_kv_attention_shared_workspace_bytes(const ibp_kv_cache *cache,
                                                 const ibp_kv_table *prefix,
                                                 const ibp_kv_table *table, uint64_t q_heads,
                                                 uint64_t n_new);

/*
 * ibp_kv_attention where all sequences begin with the same tokens: `prefix` is a
 * table of one sequence, of the same kv_heads, with the pages and lengths of
 * these.  Pages, lengths and positions of `table` are those of a sequence's own
 * tokens, without the prefix: the query at position p sees the whole prefix and the
 * own tokens at positions 0..p.  (ibp_kv_append_rotated takes the positions behind
 * the prefix as `positions`.)  A query of a token that does not exist gets zeros;
 * one that sees neither a token of the prefix nor an own one gets zeros.
 * Scores, statistics, sums, what a query may not see, and scales that are not
 * finite are as for ibp_kv_attention.  So are the weights in the second product, 16
 * bits each, but for one case: with more than 32 query rows to a head over all
 * sequences (n_seqs * n_new * group) and outputs of bf16, which have 8 bits, a weight
 * of the prefix may be off by half a step of 11 bits (2^-11 of itself) or by 2^-24
 * of the row's largest, whichever is more; a sequence's result may differ by that
 * with the batch it is in.  No weights are counted.
 *
 * workspace: as for ibp_kv_attention; about head_dim * 4 bytes for each query row
 * and part, of the prefix and of the rows.
 */
int ibp_kv_attention_shared(const ibp_kv_cache *cache, const ibp_kv_table *prefix,
                            const ibp_kv_table *table, uint32_t dtype, uint64_t q_heads,
                            uint64_t n_new, const ibp_kv_tensor *q, const ibp_kv_tensor *out,
                            const int32_t *counts, float scale, void *workspace,
                            uint64_t workspace_bytes, void *stream);

/* hipError_t behind the calling thread's last IBP_ERR_HIP from this library. */
int ibp_kv_long_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* IBP_KV_LONG_H_ */
