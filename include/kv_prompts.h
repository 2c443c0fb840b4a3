/*
 * kv_prompts.h - C ABI of what prompts, and the hypotheses or requests that share them, need over the paged 8-bit
 * K/V cache of kv_pages.h: coding new rows with the position rotation applied on the way, attention of whole prompts
 * (or chunks of them), and verify attention that reads pages which several sequences share once.  Same library,
 * conventions, pool, sequences and status codes as kv_pages.h; the pages of the sources have no counterpart.
 *
 * Packed rows
 *   The rows of all sequences of a call lie in one array of n_tokens rows.
 *   first_row     int32 [n_seqs]: sequence b's live rows are rows first_row[b] .. first_row[b] + n_live[b] - 1; row r of
 *                 them sits at position lens[b] - n_live[b] + r.  No two sequences' rows overlap.  Rows that belong to
 *                 none may lie between, before and behind them; what a call writes leaves them as they were.  (Rows
 *                 of the padded layout of kv_pages.h, [n_seqs][n_rows], are first_row[b] = b n_rows.)  Of a sequence
 *                 without live rows it is not looked at.
 *   n_live        int32 [n_seqs]: 0..n_tokens
 * A sequence whose rows do not lie within the array (VA_DEV_BAD_COUNT) counts as empty.
 */
#ifndef KV_PROMPTS_H
#define KV_PROMPTS_H

#include "kv_pages.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VA_MAX_TOKENS 16777216    /* packed rows of one call */
#define VA_DEV_BEYOND_TABLE 2048  /* a position past the end of the rotation's table */
#define VA_DEV_VALUE_SCALE 4096   /* a value scale, not 0, outside 2^-60..2^60 */

/*
 * kv_page_append_rope_b8 - rotate the live rows' queries and keys by their positions, and code the keys and the
 * values into the pages of their sequences.
 *   q, q_out      device [n_tokens][n_kv_heads * group][128] bf16, or both NULL (keys and values alone); q_out may be q
 *                 itself, but not overlap it otherwise.  q_out's rows that belong to no sequence stay as they were.
 *   k_new, v_new  device [n_tokens][n_kv_heads][128] bf16
 *   n_tokens      1..VA_MAX_TOKENS; n_seqs 1..VA_PAGED_MAX_SEQS; group 1..VA_PAGED_MAX_GROUP
 *   cos_sin       device float [n_positions][rot_dim], 16-byte aligned: row p holds the cosines of position p, then
 *                 its sines, rot_dim / 2 each
 *   rot_dim       16, 32, .. 128: dimensions 0..rot_dim-1 are rotated, the others pass
 *   interleaved   0: dimensions (i, i + rot_dim / 2) are pair i; 1: dimensions (2 i, 2 i + 1) are
 *   codes, scales one layer's pool, updated in place
 * A pair (a, b) becomes (a c - b s, b c + a s) in fp32, each product and each sum rounded once; queries are rounded
 * once more, to bf16; keys are coded from the fp32 values, by the rule of kv_page_append_b8 (which also holds for
 * rotated keys that are infinite or no number).
 *   dev_status    as for kv_page_append_b8, and VA_DEV_BEYOND_TABLE (lens above n_positions): nothing of that
 *                 sequence is written; a page that is none (VA_DEV_BAD_PAGE) is not written, its queries are
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED (a pool of more than 2^31 - 1 rows) or VA_CUDA_ERROR.
 */
VA_API va_status kv_page_append_rope_b8(const va_bf16 *q, const va_bf16 *k_new, const va_bf16 *v_new, int n_seqs,
                                        int n_tokens, int n_kv_heads, int group, const int32_t *first_row,
                                        const int32_t *n_live, const int32_t *lens, const int32_t *table, int max_pages,
                                        const float *cos_sin, int n_positions, int rot_dim, int interleaved,
                                        void *k_codes, void *v_codes, float *k_scale, float *v_scale, int n_pages,
                                        int format, va_bf16 *q_out, int32_t *dev_status, va_stream stream);

/*
 * prompt_attn_paged_b8 - attention of every sequence's live rows, any number of them, over its pages: a whole prompt,
 * a chunk of one behind what the cache holds already, or single tokens.  A row at p sees keys 0..p, or with a window W
 * keys max(0, p - W + 1)..p.
 *   q, out        device [n_tokens][n_kv_heads * group][128] bf16 (out must not overlap q); out's rows that belong to
 *                 no sequence stay as they were
 *   out_lse       optional device float [n_tokens][n_kv_heads * group]: log-sum-exp of the scores and the sink
 *   n_tokens      1..VA_MAX_TOKENS; n_seqs 1..VA_PAGED_MAX_SEQS; group 1..VA_PAGED_MAX_GROUP
 *   window, scale, sink, workspace  as for verify_attn_paged_b8; va_prompt_workspace_bytes bytes
 * What is rounded of a key is its weight times its value scale: to 11 bits, and where that is below 2^-17 of the row's
 * largest such product, to 2^-28 of the largest.  Next to a key of a larger scale, one of equal weight and a scale 2^-17 or
 * less of it so loses digits, and from 2^-28 on all of them: 448 x 2^-28 of the larger product at most, where the larger
 * key's own codes are steps of 2^-9 of it or more.  (verify_attn_paged_b8 computes scales so far apart in fp32.)  Value
 * scales below 2^-60 count as 2^-60, those above 2^60 may cost accuracy (VA_DEV_VALUE_SCALE tells of either), as may a
 * head's value scales that lie more than 2^100 apart.
 * A needed table entry that is no page sets VA_DEV_BAD_PAGE and its positions count as masked (a row that sees
 * nothing: out 0, out_lse the sink, or -inf).
 *   dev_status    VA_DEV_BAD_PAGE; VA_DEV_BAD_COUNT, VA_DEV_BEYOND_CACHE: that sequence's rows stay as they were (all
 *                 sequences' where the counts add up to more than n_tokens: VA_DEV_BAD_COUNT);
 *                 VA_DEV_VALUE_SCALE: a page that is read has a value scale (of a position that the sequence has)
 *                 beyond the range above;
 *                 VA_DEV_TIMEOUT: a wait took more than a second, the output is void
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED (a pool of more than 2^31 - 1 rows) or VA_CUDA_ERROR.
 */
VA_API va_status prompt_attn_paged_b8(const va_bf16 *q, int n_seqs, int n_tokens, int n_kv_heads, int group,
                                      const int32_t *first_row, const int32_t *n_live, const int32_t *lens,
                                      const int32_t *table, int max_pages, const void *k_codes, const void *v_codes,
                                      const float *k_scale, const float *v_scale, int n_pages, int format, int window,
                                      float scale, const float *sink, void *workspace, size_t workspace_bytes,
                                      va_bf16 *out, float *out_lse, int32_t *dev_status, va_stream stream);

/* Bytes of the workspace of prompt_attn_paged_b8; 0 for arguments out of range. */
VA_API size_t va_prompt_workspace_bytes(int n_seqs, int n_tokens, int n_kv_heads, int group);

/*
 * verify_attn_shared_b8 - verify_attn_paged_b8 for slots in groups that share their leading pages (hypotheses that
 * kv_page_reorder forked, requests behind the same instructions): such pages are read once for the group.
 *   share         slots per group (0: one group of all); n_seqs is a multiple of it
 * The leading entries that all of a group's table rows (but those of slots without live rows) have in common are found
 * on the device; of them those pages are shared that every live row sees to their end.  Nothing has to be in common:
 * of a group that shares no page each slot is attended by itself, by the same kernels, which takes up to 2.4 times as long
 * as verify_attn_paged_b8 where slots have few (row, query head) pairs and long histories; that is the call for slots
 * that are known to share nothing.  Where the sizes given (max_pages and the window for the lengths) say that little is
 * read twice, small calls and few rows in groups of two or three, the call is handed to verify_attn_paged_b8 whole.
 *   All other arguments, results and status bits are as for verify_attn_paged_b8, the workspace is of
 * va_shared_workspace_bytes bytes.  Roundings and the limits of value scales are those of prompt_attn_paged_b8, and
 * VA_DEV_VALUE_SCALE tells of scales beyond the limits, but in calls that are handed on, which round as
 * verify_attn_paged_b8 does and have no such limits.  out and out_lse must not overlap q.
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED (a pool of more than 2^31 - 1 rows) or VA_CUDA_ERROR.
 */
VA_API va_status verify_attn_shared_b8(const va_bf16 *q, int n_seqs, int n_rows, int n_kv_heads, int group, int share,
                                       const int32_t *n_live, const int32_t *lens, const int32_t *table, int max_pages,
                                       const void *k_codes, const void *v_codes, const float *k_scale,
                                       const float *v_scale, int n_pages, int format, int window, float scale,
                                       const float *sink, void *workspace, size_t workspace_bytes, va_bf16 *out,
                                       float *out_lse, int32_t *dev_status, va_stream stream);

/* Bytes of the workspace of verify_attn_shared_b8; 0 for arguments out of range. */
VA_API size_t va_shared_workspace_bytes(int n_seqs, int n_rows, int n_kv_heads, int group);

#ifdef __cplusplus
}
#endif

#endif /* KV_PROMPTS_H */
