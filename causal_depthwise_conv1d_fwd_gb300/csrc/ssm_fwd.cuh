// What ssm_fwd's forms share: a call's arguments, and the forms' launches.
#pragma once

#include "ccv_math2.cuh"
#include "ssm_common.cuh"

namespace ccv {

// log(1 + e^x) = max(x, 0) + log1p(e^{-|x|}) of a pair, the latter as t times a polynomial in t = e^{-|x|} (least largest relative
// error on [0, 1], 3e-8; with its own rounding 2.3e-7).  A step's relative error is what counts, however small the step is.
__device__ __forceinline__ f32x2 softplus2(f32x2 x) {
    float x0, x1;
    unpack2(x, x0, x1);
    const f32x2 t = pack2(ex2_approx(-1.4426950408889634f * fabsf(x0)), ex2_approx(-1.4426950408889634f * fabsf(x1)));
    const auto both = [](float c) { return pack2(c, c); };
    f32x2 q = fma2(both(0.005232623778283596f), t, both(-0.029504956677556038f));
    q = fma2(q, t, both(0.07822549343109131f));
    q = fma2(q, t, both(-0.1366320699453354f));
    q = fma2(q, t, both(0.1910598874092102f));
    q = fma2(q, t, both(-0.2484297752380371f));
    q = fma2(q, t, both(0.3331909477710724f));
    q = fma2(q, t, both(-0.4999949336051941f));
    q = fma2(q, t, both(0.9999999403953552f));
    return fma2(q, t, pack2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
}

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
int ssm_chunked_segments(int total_tokens, int batch, int num_heads, int num_groups, int head_dim);
int ssm_launch_chunked(const SsmFwd &p, void *workspace, cudaStream_t stream);

// The scan: any sizes and strides.
int64_t ssm_scan_workspace(int total_tokens, int batch, int num_heads, int head_dim, int dim_state, int seg_units);
int ssm_scan_segments(int total_tokens, int batch, int num_heads, int num_groups, int head_dim, int dim_state);
int ssm_launch_scan(const SsmFwd &p, void *workspace, cudaStream_t stream);

}  // namespace ccv
