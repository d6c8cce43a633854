/*
 * ccv_logits.h -- C ABI of what stands between a model's logits and the choice
 * of tokens (spec_verify of ccv_layer.h), in the same library (libccv.so).  The
 * conventions of ccv.h hold.
 */
#ifndef CCV_LOGITS_H_
#define CCV_LOGITS_H_

#include "ccv_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The arguments of logits_process.  For row b, position i and token v of the
 * vocabulary, with x the logit:
 *     x = x / r where x > 0, x r elsewhere     if v was seen before position i
 *     x = x - f n - p [n > 0]                  n: how often v was said before it
 *     x = x + the sum of v's entries in the bias list, in its order
 *     x = -inf                                 if the position's mask excludes v
 * in fp32, rounded once to the output's type.  What was seen is the row's
 * history and drafts 0 .. i-1; what was said is the history from the prompt's
 * end on and those drafts.
 *
 * logits, out   (batch, num_positions, vocab <= 2^30), vocab stride 1, bf16 or
 *               (logits_fp32, out_fp32) fp32.  out may be logits itself (same
 *               pointer, type and strides); without a mask a logit that nothing
 *               changes is then neither read nor written, with one it may be
 *               written once more as it is.  Otherwise out must not overlap an
 *               input.  out's rows must lie apart (CCV_ERR_STRIDE).
 * history       int32 (num_lines, history_size >= 0), stride 1 along a line: the
 *               tokens of a request, its prompt first; NULL: none (then
 *               history_lengths and prompt_lengths are not read).  Row b has
 *               line history_indices[b] (line b when NULL); a line equal to
 *               pad_slot_id skips the row (out untouched), a line outside the
 *               pool is counted in err_count and skips it, too.
 * history_lengths, prompt_lengths  int32 [num_lines]: tokens of the line, and
 *               how many of them are prompt (NULL: none).  A length outside
 *               [0, history_size] is counted and taken as the nearer bound.
 * draft_tokens  int32 (batch, num_positions - 1) or NULL (none): the token that
 *               each position but the first follows.
 * Tokens outside [0, vocab) in the history, the drafts and the bias list are
 * passed over; those above it are counted in err_count.
 * repetition, frequency, presence  fp32 [batch] or NULL (1, 0, 0); repetition
 *               above 0.
 * bias_ids, bias  int32 and fp32 (batch, bias_size), stride 1 along a row, one
 *               row stride; or NULL.  Meant for up to some hundred entries:
 *               the time grows with their square.  Many tokens are better
 *               excluded by the mask.
 * mask          int32 (batch, num_positions, (vocab + 31) / 32), stride 1 along
 *               the last: bit v % 32 of word v / 32 is 1 where v may follow; NULL:
 *               everything may.
 */
typedef struct ccv_logits_args {
    const void *logits;
    int64_t l_stride_b, l_stride_pos;
    void *out;
    int64_t o_stride_b, o_stride_pos;
    const int32_t *history;
    int64_t h_stride_line;
    const int32_t *history_indices, *history_lengths, *prompt_lengths;
    const int32_t *draft_tokens;
    int64_t d_stride_b, d_stride_pos;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_ids;
    const float *bias;
    int64_t b_stride_b;
    const int32_t *mask;
    int64_t m_stride_b, m_stride_pos;
    int logits_fp32, out_fp32;
    int batch, num_positions, vocab, num_lines, history_size, bias_size, pad_slot_id;
} ccv_logits_args;

int logits_process(const ccv_logits_args *args, int *err_count, ccv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CCV_LOGITS_H_ */
