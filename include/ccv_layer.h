/*
 * ccv_layer.h -- C ABI of the operators that a linear-attention layer runs
 * next to the causal convolution of ccv.h, in the same library (libccv.so):
 * the gated delta rule over a pool of states, the norms around it, and the
 * verification of drafted tokens whose counts ccv_update_spec and gdr_update
 * take.  The conventions of ccv.h hold: device pointers, element strides
 * >= 0, no allocation, no synchronisation, grids from the integer sizes alone
 * (so every call can be captured), status codes, err_count, and programmatic
 * stream serialization.  Forward only, as the rest of the library.
 */
#ifndef CCV_LAYER_H_
#define CCV_LAYER_H_

#include "ccv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum ccv_layer_status {
    CCV_ERR_DIM = -10,      /* a head dimension or row length the operator does not support */
    CCV_ERR_HEADS = -11,    /* value heads are not a multiple of key heads */
    CCV_ERR_WORKSPACE = -12 /* the workspace is missing, too small or misaligned */
};

/* A bf16 tensor (tokens or rows, heads, dim) for the delta rule; rows is the
 * batch row of gdr_update (unused by gdr_fwd, whose tokens are flat). */
typedef struct ccv_heads_view {
    const void *data;
    int64_t stride_row;
    int64_t stride_tok;
    int64_t stride_head;
    int64_t stride_dim;
} ccv_heads_view;

/*
 * The tensors of a gated delta rule call.  For value head h with key head
 * h / (num_v_heads / num_k_heads), per token, with the state S of shape
 * (dim_v, dim_k) in fp32:
 *     S <- a S + b (v - a S k) k^T        o = S q
 * q and k are first divided by sqrt(sum of squares + 1e-6) when qk_l2norm is
 * set, and q is multiplied by scale.  a = exp(g) and b = beta.
 *
 * q, k          (.., num_k_heads, dim_k) bf16; v (.., num_v_heads, dim_v) bf16;
 *               out as v, written, must not overlap an input.
 * g, beta       (.., num_v_heads), gate_stride_row / _tok / _head shared by
 *               both.  a_log == dt_bias == NULL: fp32, the decay's logarithm
 *               (<= 0; -inf clears the state) and the write strength.
 *               Otherwise bf16 projections x and y with fp32 a_log and
 *               dt_bias of num_v_heads: g = -exp(a_log) softplus(x + dt_bias),
 *               b = 1 / (1 + exp(-y)).
 * state         pool (num_lines, num_v_heads, dim_v, dim_k) fp32.
 * dim_k <= 256 and dim_v <= 1024 (CCV_ERR_DIM).
 */
typedef struct ccv_gdr_args {
    ccv_heads_view q, k, v, out;
    const void *g, *beta;
    int64_t gate_stride_row, gate_stride_tok, gate_stride_head;
    const float *a_log, *dt_bias;
    float *state;
    int64_t s_stride_line, s_stride_head, s_stride_v, s_stride_k;
    int num_lines;
    int num_k_heads, num_v_heads, dim_k, dim_v;
    float scale;
    int qk_l2norm;
    int pad_slot_id;
} ccv_gdr_args;

/*
 * gdr_fwd -- gated delta rule over varlen sequences (prefill).
 * query_start_loc, cache_indices, has_initial_state mean what they mean for
 * ccv_fwd: sequence i owns tokens [qsl[i], qsl[i+1]) and state line
 * cache_indices[i] (line i when NULL); a line equal to pad_slot_id skips the
 * sequence; without an initial state the state starts at zero, and the final
 * state is written to the line either way.  args->state may be NULL (zero
 * start, no write-back; then has_initial_state must be NULL:
 * CCV_ERR_ARGUMENT).  A sequence of no tokens writes nothing.  Offsets must not
 * decrease: a sequence whose own offsets do, or leave [0, total_tokens], is
 * skipped and counted in err_count, and the other sequences' results are then
 * undefined.
 * With dim_k <= 128 and more than 8 tokens a sequence on average the call runs
 * in chunks of 64 tokens on the tensor cores, and where sequences and heads are
 * too few to fill the card also cuts sequences into segments that run side by
 * side; otherwise token by token.  On finite inputs the forms differ in
 * rounding alone.  A value, key, gate or state row that is not finite makes
 * the outputs of the rows it reaches, from its token on, and their final state
 * not finite (a query: its own token's), in every form; tokens before it, other
 * rows and other sequences are as without it.  Finite inputs whose sums leave
 * fp32's range can in the chunked form also reach the tokens before them in
 * their 64-token chunk.
 * The choice of form follows from the integer sizes, and so from the average
 * length: one long sequence among many short or empty ones runs as the average
 * would.  The environment variables CCV_GDR_PATH=chunked or =recurrent and
 * CCV_GDR_SEGMENT=<chunks of a segment, 0: none>, read at each call, force it
 * (for testing and tuning).
 * Where q, k, v and out have a contiguous dim axis of a multiple of 8 elements,
 * and strides and addresses that are multiples of 16 bytes, the chunked form
 * copies whole tiles; otherwise (the (dim, tokens) layout, say) it copies
 * elements, several times as slow.
 * A wait inside a kernel that runs out (2 s, on work of the same block) is
 * counted in err_count, and what its block should have written is NaN.
 * workspace     gdr_fwd_workspace(...) bytes, 128-byte aligned, not shared
 *               with another call in flight.
 */
int gdr_fwd(const ccv_gdr_args *args, const int32_t *query_start_loc, int batch,
            const int32_t *cache_indices, const uint8_t *has_initial_state, int total_tokens,
            void *workspace, int64_t workspace_bytes, int *err_count, ccv_stream_t stream);

/* Bytes of workspace gdr_fwd needs for these sizes (0: none).  The chunked
 * form takes 42240 for each 64 tokens and value head, and batch times that in
 * all for sequences' ends: 2.85 GB for 131072 tokens of 32 heads. */
int64_t gdr_fwd_workspace(int total_tokens, int batch, int num_k_heads, int num_v_heads,
                          int dim_k, int dim_v);

/*
 * gdr_update -- gated delta rule over `seqlen` new tokens of each of `batch`
 * rows (decode, speculative verify).
 * state_indices int32 [batch] or NULL (line b for row b); a line equal to
 *               pad_slot_id skips the row (out and states untouched).
 * output_state_indices  int32 (batch, oidx_steps >= seqlen) or NULL: the state
 *               after token t is written to that line when the entry is >= 0,
 *               and the row's own line is not written.  NULL: the state after
 *               the last token replaces the row's line.  Written lines must
 *               not be lines that other rows of the call read or write.
 * num_accepted_tokens  int32 [batch] or NULL; needs output_state_indices
 *               (CCV_ERR_ARGUMENT).  Row b starts from line
 *               output_state_indices[b, num_accepted_tokens[b] - 1], the state
 *               after the last token that the previous step kept; a count
 *               outside [1, oidx_steps] or a line outside the pool skips the
 *               row and is counted in err_count.
 */
int gdr_update(const ccv_gdr_args *args, const int32_t *state_indices,
               const int32_t *num_accepted_tokens, const int32_t *output_state_indices,
               int64_t oi_stride_b, int64_t oi_stride_step, int oidx_steps, int batch, int seqlen,
               int *err_count, ccv_stream_t stream);

/*
 * gated_rms_norm -- the norm of a block's heads with its gate, bf16:
 *   norm_before_gate != 0:  out = x rsqrt(mean(x^2) + eps) weight act(gate)
 *   norm_before_gate == 0:  u = x act(gate), out = u rsqrt(mean(u^2) + eps) weight
 * over the last dimension of (tokens, heads, dim).  activation: 0 none
 * (act(z) = z), 1 SiLU, 2 sigmoid.  weight [dim], contiguous.  out may be x or
 * gate itself (same pointer and strides) or must not overlap them.
 * dim <= 32768 (CCV_ERR_DIM).
 */
int gated_rms_norm(const ccv_heads_view *x, const ccv_heads_view *gate, const void *weight,
                   const ccv_heads_view *out, int tokens, int heads, int dim, float eps,
                   int activation, int norm_before_gate, ccv_stream_t stream);

/*
 * residual_rms_norm -- what lies between two blocks, in one pass over the rows:
 *   t = x [rsqrt(mean(x^2) + eps) (post_weight + weight_offset)] [gate]
 *   h = residual + scale t                           -> residual_out
 *   out = h rsqrt(mean(h^2) + eps) (weight + weight_offset)
 * x, out        (tokens, dim) bf16; residual and residual_out bf16, or fp32
 *               when residual_fp32 is set.  h is normalised before it is
 *               rounded.  residual_out may be residual itself and out may be x
 *               itself (same pointer and strides); otherwise no output
 *               overlaps an input.
 * weight, post_weight  [dim] bf16, contiguous; post_weight NULL: no norm of x.
 * gate          bf16, strides (tok, dim), stride_tok 0 for one gate a channel;
 *               NULL: none.
 * dim <= 32768 (CCV_ERR_DIM).
 */
int residual_rms_norm(const void *x, int64_t x_stride_tok, int64_t x_stride_dim,
                      const void *residual, int64_t r_stride_tok, int64_t r_stride_dim,
                      int residual_fp32, const void *weight, const void *post_weight,
                      const void *gate, int64_t g_stride_tok, int64_t g_stride_dim,
                      void *out, int64_t out_stride_tok, int64_t out_stride_dim,
                      void *residual_out, int64_t ro_stride_tok, int64_t ro_stride_dim,
                      int tokens, int dim, float scale, float eps, float weight_offset,
                      ccv_stream_t stream);

/*
 * spec_verify -- accepts or rejects drafted tokens against the target model's
 * probabilities, from given random numbers.
 * target_logits (batch, num_positions = drafts + 1, vocab <= 2^30), stride 1,
 *               bf16 or (logits_fp32) fp32: position i predicts the token
 *               after draft i-1.  p_i = softmax(logits_i / temperature).
 *               -inf and NaN logits have probability 0; +inf counts as the
 *               largest finite value.
 * draft_tokens  int32 (batch, drafts).  draft_probs fp32 (batch, drafts,
 *               vocab), vocab stride 1, the distributions they were drawn
 *               from, or NULL when each was certain (q = 1 at the token).
 * num_drafts    int32 [batch] or NULL (all `drafts`): the row's drafts, at
 *               most `drafts`; negative: a padded row, which gets count 0 and
 *               tokens -1.
 * temperature   fp32 [batch] or NULL (1).  0 (or anything else that is not
 *               above 0): greedy, p is 1 at the largest logit (the lowest
 *               index on ties).
 * uniform       fp32 (batch, drafts) in [0, 1); noise fp32 (batch, vocab),
 *               vocab stride 1, > 0, exponentially distributed.
 * Draft i is kept while every earlier one is and uniform_i q_i(x_i) <
 * p_i(x_i).  At the first that is not, the next token is drawn from
 * r = max(p_i - q_i, 0); with all kept, from r = p of the following position:
 * it is the index of the largest r_v / noise_v, the lowest on ties, or -1 when
 * no r_v is above 0.  Greedy rows take the largest logit of that position.
 * out_tokens    int32 (batch, drafts + 1), contiguous: the kept drafts, the
 *               next token, then -1.
 * num_accepted  int32 [batch]: kept drafts + 1, what num_accepted_tokens of
 *               ccv_update_spec and gdr_update takes for the next step.
 * A draft token outside [0, vocab) is rejected; the first one met is counted in
 * err_count.
 * workspace     spec_verify_workspace(...) bytes, 16-byte aligned.
 */
int spec_verify(const void *target_logits, int logits_fp32, int64_t t_stride_b, int64_t t_stride_pos,
                const int32_t *draft_tokens, int64_t d_stride_b, int64_t d_stride_pos,
                const float *draft_probs, int64_t p_stride_b, int64_t p_stride_pos,
                const int32_t *num_drafts, const float *temperature,
                const float *uniform, int64_t u_stride_b, int64_t u_stride_pos,
                const float *noise, int64_t n_stride_b,
                int32_t *out_tokens, int32_t *num_accepted,
                int batch, int drafts, int vocab, void *workspace, int64_t workspace_bytes,
                int *err_count, ccv_stream_t stream);

/* Bytes of workspace spec_verify needs for these sizes (0: sizes that it
 * refuses). */
int64_t spec_verify_workspace(int batch, int drafts, int vocab);

#ifdef __cplusplus
}
#endif

#endif /* CCV_LAYER_H_ */
