// Selective state space scan over varlen sequences (prefill).
#include "ssm_common.cuh"

extern "C" int64_t ssm_fwd_workspace(int total_tokens, int batch, int num_heads, int num_groups, int head_dim, int dim_state,
                                     int a_per_state) {
    return 0;
}

extern "C" int ssm_fwd(const ccv_ssm_args *args, const int32_t *query_start_loc, int batch, const int32_t *cache_indices,
                       const uint8_t *has_initial_state, int total_tokens, void *workspace, int64_t workspace_bytes, int *err_count,
                       ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || total_tokens < 0 || total_tokens > (1 << 30)) return CCV_ERR_SIZE;
    const int status = ssm_check(args, 1, total_tokens);
    if (status != CCV_OK) return status;
    if (args->state == nullptr && has_initial_state != nullptr) return CCV_ERR_ARGUMENT;
    if (batch == 0 || total_tokens == 0 || args->num_heads == 0 || args->head_dim == 0 || args->dim_state == 0) return CCV_OK;
    if (query_start_loc == nullptr) return CCV_ERR_NULL_POINTER;
    const SsmRows rows{query_start_loc, cache_indices, has_initial_state, nullptr, nullptr, 0, 0, 0, batch, 0, total_tokens, err_count};
    return ssm_launch_recurrent(*args, rows, stream);
}
