/*
 * beam_select.h - C ABI of beam search's selection: the best hypotheses over beams and vocabulary.  Same library,
 * conventions and status codes as verify_attn.h; the candidates of a row are ranked as in spec_sample.h.
 * kv_page_reorder (kv_pages.h) then moves the hypotheses' caches to their new slots.
 */
#ifndef BEAM_SELECT_H
#define BEAM_SELECT_H

#include "spec_sample.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VA_LOGITS_F32 0
#define VA_LOGITS_BF16 1
#define VA_BEAM_MAX_BEAMS 32
#define VA_BEAM_MAX_GROUPS 1024

/*
 * va_beam_select - for each of n_groups requests the n_out best continuations of its n_beams hypotheses.
 * Hypothesis i of a request continues with token t at the score
 *     scores[i] + l[t] - log sum_t' exp(l[t'])
 * with l its row of logits; a finished hypothesis continues with end_token alone, at scores[i].  The scores are
 * sums of 64 bits (the log-sum-exp's exponentials are summed in 32), so that near candidates of different
 * hypotheses keep their order; they are rounded once, at the end.  Equal scores: the lower hypothesis first, and
 * of one hypothesis the candidate order of spec_sample.h (larger logit, then lower token).  A logit of -inf or NaN
 * is no candidate; where a row holds +inf, its +inf logits share the probability.
 *   logits        device [n_groups * n_beams] rows of `vocab` entries, row_stride entries apart: fp32 (format
 *                 VA_LOGITS_F32; 16-byte aligned, row_stride a multiple of 4) or bf16 (VA_LOGITS_BF16; a multiple
 *                 of 8; a single row's is not looked at).  vocab 1..VA_SAMPLE_MAX_VOCAB, any; the entries between rows
 *                 are not used.  Rows of an odd vocabulary so need padding between them.
 *   scores        device float [n_groups * n_beams]; -inf: no hypothesis
 *   finished      optional device int32 [n_groups * n_beams], not 0 = finished; end_token then in 0..vocab-1
 *   n_beams       1..VA_BEAM_MAX_BEAMS; n_out 1..VA_SAMPLE_MAX_K; n_groups 1..VA_BEAM_MAX_GROUPS
 *   parents, tokens  device int32 [n_groups][n_out]: hypothesis (0..n_beams-1) and token, best first; -1 and
 *                 -1 past the candidates there are
 *   out_scores    device float [n_groups][n_out]; -inf past the candidates there are (not the memory of `scores`)
 *   workspace     device memory of va_beam_workspace_bytes bytes, 16-byte aligned, zeroed once before its first
 *                 use; every call leaves its counters at zero, so that it serves calls of any smaller shape.
 *                 Calls that may run at the same time need their own.
 * Returns VA_OK, VA_INVALID_ARG or VA_CUDA_ERROR.
 */
VA_API va_status va_beam_select(const void *logits, int format, int64_t row_stride, int n_groups, int n_beams,
                                int vocab, const float *scores, const int32_t *finished, int end_token, int n_out,
                                int32_t *parents, int32_t *tokens, float *out_scores, void *workspace,
                                size_t workspace_bytes, va_stream stream);

/* Bytes of the workspace of va_beam_select; 0 for arguments out of range. */
VA_API size_t va_beam_workspace_bytes(int n_groups, int n_beams, int vocab, int n_out);

#ifdef __cplusplus
}
#endif

#endif /* BEAM_SELECT_H */
