/*
 * kv_pages.h - C ABI of a paged 8-bit K/V cache that many sequences share: coding new rows into pages,
 * verify attention of a whole batch over its pages, and the operations on the pages themselves (room for new
 * tokens with copy on write, forking, freeing and reordering, copying, compaction).
 * Same library, conventions and status codes as verify_attn.h: every call is asynchronous on `stream`,
 * allocates and synchronises nothing, and keeps every per-step value (lengths, live rows, page tables,
 * reference counts, parents) in device memory, so that a step can be captured in a CUDA graph.  The pages of
 * the sources have no counterpart to these entry points: the sources serve one request over a dense cache;
 * this is that cache for several requests, with its sliding windows, sinks and verify rows.
 *
 * Pool of one layer
 *   page          VA_TILE (64) consecutive positions of one sequence, every KV head
 *   codes         [n_pages][n_kv_heads][64][128] bytes, keys and values apart, 16-byte aligned
 *   scales        [n_pages][n_kv_heads][4] fp32, one per block of VA_B8_BLOCK (16) positions and head
 *   format        VA_B8_E4M3 (codes are E4M3, the largest 448) or VA_B8_INT8 (codes are int8 in -127..127),
 *                 for keys and values alike.  An element stands for scale x code.  (The append writes no
 *                 NaN code.)
 * Sequences
 *   table         int32 [n_seqs][max_pages]: entry x is the page of positions 64 x .. 64 x + 63, -1 = none;
 *                 max_pages 1..2^25 - 1
 *   lens          int32 [n_seqs]: positions of the sequence, its live rows among them
 *   n_live        int32 [n_seqs]: live rows of the call, 0..n_rows; row r sits at position
 *                 lens - n_live + r.  Rows past n_live are padding.
 *   refs          int32 [n_pages]: how many table entries name the page; 0 = free.  This is the whole state of
 *                 the allocator.  A new page is always the lowest-numbered free one.
 * What a call finds wrong on the device is OR-ed into the optional word dev_status (VA_DEV_* bits): a sequence
 * whose count or length is out of range counts as empty, a page number outside 0..n_pages-1 as no page.
 * kv_page_append_b8 and the page operations expect that the pages they write belong to one sequence only;
 * kv_page_extend sees to that.
 */
#ifndef KV_PAGES_H
#define KV_PAGES_H

#include "verify_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VA_B8_E4M3 0
#define VA_B8_INT8 1
#define VA_B8_BLOCK 16            /* positions that share a scale */
#define VA_PAGED_MAX_SEQS 1024    /* sequences of one call */
#define VA_PAGED_MAX_KV_HEADS 64
#define VA_PAGED_MAX_GROUP 8      /* query heads per KV head */

/* device status bits of these calls (next to those of verify_attn.h) */
#define VA_DEV_BAD_PAGE 128       /* a table entry that is needed is no page of the pool */
#define VA_DEV_NO_PAGES 256       /* not enough free pages: the call changed nothing */
#define VA_DEV_NONFINITE 512      /* a new row holds an infinity or NaN (coded as stated there) */
#define VA_DEV_BAD_COUNT 1024     /* a count or source index out of range */

/*
 * kv_page_append_b8 - code the live rows' K and V into the pages of their sequences, before they are read.
 *   k_new, v_new  device [n_seqs][n_rows][n_kv_heads][128] bf16; n_rows 1..2^24 (a step's rows or a whole
 *                 prompt)
 *   codes, scales one layer's pool, updated in place
 * Per block of 16 positions and head that receives rows, in fp32 with one rounding to nearest per operation:
 *   s' = max|x| / C over the new rows (C = 448 or 127); s = max(s', s_old) where the block holds older rows of
 *   the sequence, else s'; if s > s_old the older codes become rn((c s_old) / s); the new codes are rn(x / s),
 *   ties to even; s = 0 gives codes 0.  A block's scale therefore only grows until its first position is
 *   written again.  rn of a value that is no zero may be -0 (E4M3).
 *   An infinity takes no part in max|x| and becomes the largest code of its sign (code 0 if s = 0), a NaN
 *   becomes 0; VA_DEV_NONFINITE tells of either.
 *   dev_status    also VA_DEV_BAD_COUNT (n_live outside 0..n_rows or above lens), VA_DEV_BEYOND_CACHE (lens
 *                 above 64 max_pages): nothing of that sequence is written; VA_DEV_BAD_PAGE: that page is not
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED (a pool of more than 2^31 - 1 rows) or VA_CUDA_ERROR.
 */
VA_API va_status kv_page_append_b8(const va_bf16 *k_new, const va_bf16 *v_new, int n_seqs, int n_rows,
                                   int n_kv_heads, const int32_t *n_live, const int32_t *lens,
                                   const int32_t *table, int max_pages, void *k_codes, void *v_codes,
                                   float *k_scale, float *v_scale, int n_pages, int format, int32_t *dev_status,
                                   va_stream stream);

/*
 * verify_attn_paged_b8 - verify attention of every sequence's live rows over its pages, sink and all.
 *   q             device [n_seqs][n_rows][n_kv_heads * group][128] bf16; query head h reads KV head h / group
 *   n_seqs        1..VA_PAGED_MAX_SEQS; n_rows 1..VA_MAX_ROWS; group 1..VA_PAGED_MAX_GROUP
 *   window        0 (a row at p sees keys 0..p) or W >= 1 (keys max(0, p - W + 1)..p)
 *   scale         softmax scale applied to q.k (finite)
 *   sink          device float [n_kv_heads * group] or NULL: logit of a zero-value key, post-scale
 *   workspace     device memory, 16-byte aligned, va_paged_workspace_bytes bytes (contents do not matter).
 *                 Calls that may run at the same time need workspaces of their own.
 *   out           device, as q: the attention output rounded once to bf16; padding rows 0
 *   out_lse       optional device float [n_seqs][n_rows][n_kv_heads * group]: log-sum-exp of the scores and the
 *                 sink; -inf for padding rows
 * Weights are rounded to 11 bits.  Where a head's seen V scales lie more than 2^9 apart (0 aside) or pass 2^89, those parts
 * of the history are computed in fp32 instead, which takes twenty to forty times as long.
 * Only pages that hold a visible position are read, so entries below every row's window may be -1; a page's
 * positions past the sequence's end may hold anything.  A needed entry that is no page sets VA_DEV_BAD_PAGE and
 * its positions count as masked (a row that sees nothing: out 0, out_lse the sink, or -inf).
 *   dev_status    VA_DEV_BAD_PAGE; VA_DEV_BAD_COUNT, VA_DEV_BEYOND_CACHE: as in kv_page_append_b8, that sequence's
 *                 rows are padding; VA_DEV_TIMEOUT: a load did not arrive within a second, the output is void
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED (a pool of more than 2^31 - 1 rows) or VA_CUDA_ERROR.
 */
VA_API va_status verify_attn_paged_b8(const va_bf16 *q, int n_seqs, int n_rows, int n_kv_heads, int group,
                                      const int32_t *n_live, const int32_t *lens, const int32_t *table,
                                      int max_pages, const void *k_codes, const void *v_codes,
                                      const float *k_scale, const float *v_scale, int n_pages, int format,
                                      int window, float scale, const float *sink, void *workspace,
                                      size_t workspace_bytes, va_bf16 *out, float *out_lse, int32_t *dev_status,
                                      va_stream stream);

/* Bytes of the workspace of verify_attn_paged_b8; 0 for arguments out of range. */
VA_API size_t va_paged_workspace_bytes(int n_seqs, int n_rows, int n_kv_heads, int group);

/*
 * kv_page_extend - room for n_new[b] more tokens of every sequence: afterwards the pages of positions
 * lens[b] .. lens[b] + n_new[b] - 1 are there and belong to the sequence alone, and lens[b] has grown by
 * n_new[b].  Call it before kv_page_append_b8 (whose n_live is then n_new).
 *   n_new         device int32 [n_seqs]; 0 leaves a sequence as it is
 *   A table entry of those pages that is -1 gets a new page.  One whose page other entries name too (refs > 1)
 *   gets a new page as well, and where the sequence has positions in it already (they are below lens[b]) the
 *   page is copied first, in all layers; if all of a page's refs are among the pages to be written by this
 *   call, the lowest slot keeps it.  The new pages are the lowest-numbered free ones, in order of (slot, entry).
 *   codes, scales the pools of all layers: [n_layers][n_pages]... in one piece
 *   workspace     device memory, 16-byte aligned, va_page_ops_workspace_bytes bytes (contents do not matter);
 *                 calls that may run at the same time need their own
 *   dev_status    VA_DEV_NO_PAGES, VA_DEV_BAD_COUNT (n_new < 0 or lens < 0), VA_DEV_BEYOND_CACHE
 *                 (lens + n_new > 64 max_pages) or VA_DEV_BAD_PAGE (an entry that is neither -1 nor a page with
 *                 refs >= 1): the call then changes nothing
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED or VA_CUDA_ERROR.
 */
VA_API va_status kv_page_extend(int32_t *table, int32_t *lens, const int32_t *n_new, int n_seqs, int max_pages,
                                int32_t *refs, int n_pages, int n_layers, int n_kv_heads, void *k_codes,
                                void *v_codes, float *k_scale, float *v_scale, void *workspace,
                                size_t workspace_bytes, int32_t *dev_status, va_stream stream);

/*
 * kv_page_reorder - slot j takes the sequence of slot src[j], all at once: table row, length and references.
 * src[j] = j keeps a sequence, another slot's number forks that slot's (the pages are shared, none is copied
 * until kv_page_extend has to), -1 frees slot j.  With the parents of va_beam_select it reorders the hypotheses
 * of a beam search.
 *   src           device int32 [n_seqs], counted from the first slot of j's group
 *   group         slots per group (0: one group of all); n_seqs is a multiple of it
 *   dev_status    VA_DEV_BAD_COUNT (src outside -1..group-1: the slot keeps its sequence), VA_DEV_BAD_PAGE (an
 *                 entry that is neither -1 nor a page: it is moved but not counted)
 * Returns VA_OK, VA_INVALID_ARG or VA_CUDA_ERROR.
 */
VA_API va_status kv_page_reorder(int32_t *table, int32_t *lens, int n_seqs, int max_pages, const int32_t *src,
                                 int group, int32_t *refs, int n_pages, int32_t *dev_status, va_stream stream);

/*
 * kv_page_copy - page dst[i] becomes a copy of page src[i] (codes and scales, all layers), i < n_pairs.
 *   src, dst      device int32 [n_pairs], n_pairs 0..n_pages; no page may be a destination twice, or a source and a
 *                 destination
 *   dev_status    VA_DEV_BAD_PAGE: a pair that names no page is skipped
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED or VA_CUDA_ERROR.
 */
VA_API va_status kv_page_copy(const int32_t *src, const int32_t *dst, int n_pairs, int n_pages, int n_layers,
                              int n_kv_heads, void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                              int32_t *dev_status, va_stream stream);

/*
 * kv_page_compact - move the live pages (refs > 0) to the lowest numbers: with n live pages, the i-th live page
 * numbered n or higher moves to the i-th free page below n, in all layers; table and refs follow.
 *   table         every table whose entries refs counts, as one [n_seqs][max_pages]
 *   moved_to      device int32 [n_pages]: each live page's new number, -1 for a page that was free
 *   n_live_pages  device int32: n
 *   workspace     as for kv_page_extend
 *   dev_status    VA_DEV_BAD_PAGE: an entry that is neither -1 nor a live page (it becomes -1)
 * Returns VA_OK, VA_INVALID_ARG, VA_UNSUPPORTED or VA_CUDA_ERROR.
 */
VA_API va_status kv_page_compact(int32_t *table, int n_seqs, int max_pages, int32_t *refs, int n_pages,
                                 int n_layers, int n_kv_heads, void *k_codes, void *v_codes, float *k_scale,
                                 float *v_scale, int32_t *moved_to, int32_t *n_live_pages, void *workspace,
                                 size_t workspace_bytes, int32_t *dev_status, va_stream stream);

/* Bytes of the workspace of kv_page_extend and kv_page_compact; 0 for arguments out of range. */
VA_API size_t va_page_ops_workspace_bytes(int n_seqs, int max_pages, int n_pages);

#ifdef __cplusplus
}
#endif

#endif /* KV_PAGES_H */
