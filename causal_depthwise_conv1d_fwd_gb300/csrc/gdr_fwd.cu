// Gated delta rule over varlen sequences (prefill).
#include "gdr_common.cuh"

extern "C" int64_t gdr_fwd_workspace(int total_tokens, int batch, int num_k_heads, int num_v_heads, int dim_k, int dim_v) {
    return 0;
}

extern "C" int gdr_fwd(const ccv_gdr_args *args, const int32_t *query_start_loc, int batch, const int32_t *cache_indices,
                       const uint8_t *has_initial_state, int total_tokens, void *workspace, int64_t workspace_bytes,
                       int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || total_tokens < 0) return CCV_ERR_SIZE;
    const int status = gdr_check(args, 1, total_tokens);
    if (status != CCV_OK) return status;
    if (has_initial_state != nullptr && args->state == nullptr) return CCV_ERR_ARGUMENT;
    if (batch == 0 || total_tokens == 0 || args->num_v_heads == 0 || args->dim_v == 0 || args->dim_k == 0) return CCV_OK;
    if (query_start_loc == nullptr) return CCV_ERR_NULL_POINTER;
    const GdrRows rows{query_start_loc, cache_indices, has_initial_state, nullptr, nullptr, 0, 0, 0, batch, 0,
                       total_tokens, err_count};
    return gdr_launch_recurrent(*args, rows, stream);
}
