/*
 * ccv_ssm.h -- C ABI of the selective state space scan that Mamba-style layers
 * run on the causal convolution's output, in the same library (libccv.so): over
 * prompts (ssm_fwd) and over the new tokens of each row (ssm_update).  The
 * conventions of ccv.h and ccv_layer.h hold: device pointers, element strides
 * >= 0, no allocation, no synchronisation, grids from the integer sizes alone
 * (so every call can be captured), status codes, err_count, and programmatic
 * stream serialization.  Forward only, as the rest of the library.
 */
#ifndef CCV_SSM_H_
#define CCV_SSM_H_

#include "ccv_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * The tensors of a call.  For head h of group h / (num_heads / num_groups),
 * per token, with the state S of shape (head_dim, dim_state) in fp32:
 *     d = dt + dt_bias;  d = log(1 + exp(d)) when dt_softplus is set
 *     d = min(max(d, dt_min), dt_max)
 *     S <- exp(d A) S + d x B^T        y = S C + D x
 *     out = y, or y z / (1 + exp(-z)) with a gate z
 * Layers whose channels each have their own step are heads of head_dim 1.
 *
 * x, z, out     (.., num_heads, head_dim) bf16; z.data NULL: no gate.  out must
 *               not overlap an input.  The elements of out, and those of state,
 *               lie apart, each axis past those of smaller strides
 *               (CCV_ERR_STRIDE).
 * B, C          (.., num_groups, dim_state) bf16.
 * dt            (.., num_heads) bf16, or fp32 when dt_fp32 is set.
 * A             fp32, contiguous: [num_heads], or (a_per_state)
 *               [num_heads, dim_state].  Decays are meant to be at most 1
 *               (A <= 0 and d >= 0); larger ones hold until fp32 overflows.  Minus
 *               infinity counts as fp32's lowest number: a step of 0 leaves the
 *               state, and one above 1e-36 nothing of it.
 * D, dt_bias    fp32 [num_heads] or NULL (0).
 * dt_min, dt_max  bounds of d (-inf and inf: none; 0 and inf are usual).
 * state         pool (num_lines, num_heads, head_dim, dim_state) fp32.
 * head_dim <= 1024 and dim_state <= 256 (CCV_ERR_DIM); num_heads is a multiple
 * of num_groups (CCV_ERR_HEADS).
 */
typedef struct ccv_ssm_args {
    ccv_heads_view x, z, out, B, C;
    const void *dt;
    int64_t dt_stride_row, dt_stride_tok, dt_stride_head;
    const float *A, *D, *dt_bias;
    float *state;
    int64_t s_stride_line, s_stride_head, s_stride_dim, s_stride_state;
    float dt_min, dt_max;
    int dt_fp32, dt_softplus, a_per_state;
    int num_lines, num_heads, num_groups, head_dim, dim_state, pad_slot_id;
} ccv_ssm_args;

/*
 * ssm_fwd -- the scan over varlen sequences (prefill).
 * query_start_loc, cache_indices, has_initial_state and state mean what they
 * mean for gdr_fwd: sequence i owns tokens [qsl[i], qsl[i+1]) and state line
 * cache_indices[i] (line i when NULL); a line equal to pad_slot_id skips the
 * sequence; without an initial state the state starts at zero, and the final
 * state is written to the line either way.  args->state may be NULL (zero
 * start, no write-back; then has_initial_state must be NULL:
 * CCV_ERR_ARGUMENT).  A sequence of no tokens writes nothing.  Offsets must not
 * decrease: a sequence whose own offsets do, or leave [0, total_tokens], is
 * skipped and counted in err_count, and the other sequences' results are then
 * undefined.  Tokens past the last sequence are not written.
 * Values that are not finite stay where the formulas carry them: to later
 * tokens of the same sequence and head, for x to the same channel alone, for B
 * and C to their group's heads; C and z to their own token.
 * Three forms, chosen from the integer sizes: token by token with the state in
 * registers (up to 8 tokens a sequence on average); 128 tokens a step on the
 * tensor cores (one decay a head, dim_state <= 128, head_dim >= 8), where
 * what makes the state keeps 24 bits and what makes outputs alone 16; a scan of
 * tiles of tokens (the others).  The last two cut sequences into segments where that pays.
 * CCV_SSM_PATH=recurrent, =chunked or =scan and CCV_SSM_SEGMENT (128s of
 * tokens, 0: whole sequences) in the environment force a choice where it can
 * run; they are read at each call and by ssm_fwd_workspace.
 * A wait inside the chunked kernel that does not end within two seconds ends
 * the call instead: outputs and states it did not reach are NaN, and err_count
 * is raised.
 * workspace     ssm_fwd_workspace(...) bytes, 128-byte aligned, not shared
 *               with another call in flight.
 */
int ssm_fwd(const ccv_ssm_args *args, const int32_t *query_start_loc, int batch,
            const int32_t *cache_indices, const uint8_t *has_initial_state, int total_tokens,
            void *workspace, int64_t workspace_bytes, int *err_count, ccv_stream_t stream);

/* Bytes of workspace ssm_fwd needs for these sizes (0: none, or sizes that it
 * refuses).  copies: whether x, B or C have to be copied for the chunked form,
 * which reads rows of 16-byte pieces: they need not where each has stride_dim 1,
 * its address on 16 bytes, and strides of tokens and (of more than one) heads
 * that are multiples of 8 and above 0. */
int64_t ssm_fwd_workspace(int total_tokens, int batch, int num_heads, int num_groups, int head_dim,
                          int dim_state, int a_per_state, int copies);

/*
 * ssm_update -- the scan over `seqlen` new tokens of each of `batch` rows
 * (decode, speculative verify).  state_indices, num_accepted_tokens and
 * output_state_indices mean what they mean for gdr_update: a row's line is
 * state_indices[b] (line b when NULL; pad_slot_id skips the row) and is updated
 * in place; with output_state_indices (batch, oidx_steps >= seqlen) the state
 * after token t goes to that line when the entry is >= 0 instead, and with
 * num_accepted_tokens row b starts from line output_state_indices[b,
 * num_accepted_tokens[b] - 1].  Written lines must not be lines that other rows
 * of the call read or write.
 */
int ssm_update(const ccv_ssm_args *args, const int32_t *state_indices,
               const int32_t *num_accepted_tokens, const int32_t *output_state_indices,
               int64_t oi_stride_b, int64_t oi_stride_step, int oidx_steps, int batch, int seqlen,
               int *err_count, ccv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CCV_SSM_H_ */
