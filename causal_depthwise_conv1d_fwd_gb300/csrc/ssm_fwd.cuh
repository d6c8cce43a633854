// What ssm_fwd's forms share: a call's arguments, and the forms' launches.
#pragma once

#include "ssm_common.cuh"

namespace ccv {

struct SsmFwd {
    ccv_ssm_args a;
    const int32_t *query_start_loc, *cache_indices;
    const uint8_t *has_initial_state;
    int batch, total_tokens;
    int *err_count;
    int seg_chunks;     // chunks of 128 tokens of a segment; 0: sequences are not cut
    float *seg_state;   // a segment's final state from zero, then its first state
    float *seg_decay;   // what a segment multiplies its first state by (chunked), or the sums of its steps (scan)
};

// The chunked form: one decay a head, dim_state up to 128, x, B and C as tensor maps take them.
bool ssm_chunked_dims(int dim_state, int a_per_state);
int64_t ssm_chunked_workspace(int total_tokens, int batch, int num_heads, int head_dim, int seg_chunks);
int ssm_chunked_segments(int total_tokens, int batch, int num_heads, int head_dim);
int ssm_launch_chunked(const SsmFwd &p, void *workspace, cudaStream_t stream);

// The scan: any sizes and strides.
int64_t ssm_scan_workspace(int total_tokens, int batch, int num_heads, int head_dim, int dim_state, int seg_units);
int ssm_scan_segments(int total_tokens, int batch, int num_heads, int num_groups, int head_dim, int dim_state);
int ssm_launch_scan(const SsmFwd &p, void *workspace, cudaStream_t stream);

}  // namespace ccv
