// What the gated delta rule's kernels share: gates, the host's argument checks, and the recurrent kernel's launch.
#pragma once

#include <cmath>

#include "ccv_common.cuh"
#include "ccv_layer.h"

namespace ccv {

constexpr float kGdrNormEps = 1e-6f;
constexpr int kGdrMaxDk = 256;
constexpr int kGdrMaxDv = 1024;

// The decay's logarithm and the write strength of one (token, value head), as they are in memory.  Raw projections are
// bf16; expf and log1pf rather than the approximations, since the logarithm is summed over a chunk and the decay
// multiplies an fp32 state.
struct GdrGates {
    uint32_t g, beta;  // bits
    float bias, a_log;
    __device__ __forceinline__ void load(const ccv_gdr_args &a, int64_t off, int h) {
        if (a.a_log != nullptr) {
            g = static_cast<const uint16_t *>(a.g)[off];
            beta = static_cast<const uint16_t *>(a.beta)[off];
            bias = a.dt_bias[h];
            a_log = a.a_log[h];
        } else {
            g = static_cast<const uint32_t *>(a.g)[off];
            beta = static_cast<const uint32_t *>(a.beta)[off];
        }
    }
    __device__ __forceinline__ void get(bool raw, float &decay, float &strength) const {
        if (raw) {
            const float x = bf16_bits(static_cast<uint16_t>(g)) + bias;
            const float y = bf16_bits(static_cast<uint16_t>(beta));
            const float softplus = x > 20.0f ? x : log1pf(expf(x));
            decay = -expf(a_log) * softplus;
            strength = 1.0f / (1.0f + expf(-y));
        } else {
            decay = __uint_as_float(g);
            strength = __uint_as_float(beta);
        }
    }
};
__device__ __forceinline__ void gdr_gates(const ccv_gdr_args &a, int64_t off, int h, float &g, float &beta) {
    GdrGates gates;
    gates.load(a, off, h);
    gates.get(a.a_log != nullptr, g, beta);
}

// ------------------------------------------------------------ host side ----

inline bool gdr_stride_ok(const ccv_heads_view &v) {
    return v.stride_row >= 0 && v.stride_tok >= 0 && v.stride_head >= 0 && v.stride_dim >= 0;
}

inline Extent gdr_extent(const ccv_heads_view &v, int64_t rows, int64_t toks, int64_t heads, int64_t dim, int size = 2) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(v.data);
    const int64_t last = (rows - 1) * v.stride_row + (toks - 1) * v.stride_tok + (heads - 1) * v.stride_head +
                         (dim - 1) * v.stride_dim;
    return Extent{base, base + static_cast<uintptr_t>(last) * size + size - 1};
}

// Sizes, strides, pointers and overlaps of a call over `rows` x `toks` tokens.
inline int gdr_check(const ccv_gdr_args *a, int64_t rows, int64_t toks) {
    if (a == nullptr) return CCV_ERR_NULL_POINTER;
    if (a->num_k_heads < 0 || a->num_v_heads < 0 || a->dim_k < 0 || a->dim_v < 0 || a->num_lines < 0)
        return CCV_ERR_SIZE;
    if (a->dim_k > kGdrMaxDk || a->dim_v > kGdrMaxDv) return CCV_ERR_DIM;
    if (a->num_v_heads > 0 && (a->num_k_heads == 0 || a->num_v_heads % a->num_k_heads != 0)) return CCV_ERR_HEADS;
    if (!gdr_stride_ok(a->q) || !gdr_stride_ok(a->k) || !gdr_stride_ok(a->v) || !gdr_stride_ok(a->out) ||
        a->gate_stride_row < 0 || a->gate_stride_tok < 0 || a->gate_stride_head < 0 || a->s_stride_line < 0 ||
        a->s_stride_head < 0 || a->s_stride_v < 0 || a->s_stride_k < 0)
        return CCV_ERR_STRIDE;
    if (rows == 0 || toks == 0 || a->num_v_heads == 0 || a->dim_v == 0 || a->dim_k == 0) return CCV_OK;
    if (a->q.data == nullptr || a->k.data == nullptr || a->v.data == nullptr || a->out.data == nullptr ||
        a->g == nullptr || a->beta == nullptr || (a->a_log == nullptr) != (a->dt_bias == nullptr))
        return CCV_ERR_NULL_POINTER;
    const Extent eo = gdr_extent(a->out, rows, toks, a->num_v_heads, a->dim_v);
    const ccv_heads_view gv{a->g, a->gate_stride_row, a->gate_stride_tok, a->gate_stride_head, 0};
    const ccv_heads_view bv{a->beta, a->gate_stride_row, a->gate_stride_tok, a->gate_stride_head, 0};
    const int gsize = a->a_log != nullptr ? 2 : 4;
    if (overlaps(eo, gdr_extent(a->q, rows, toks, a->num_k_heads, a->dim_k)) ||
        overlaps(eo, gdr_extent(a->k, rows, toks, a->num_k_heads, a->dim_k)) ||
        overlaps(eo, gdr_extent(a->v, rows, toks, a->num_v_heads, a->dim_v)) ||
        overlaps(eo, gdr_extent(gv, rows, toks, a->num_v_heads, 1, gsize)) ||
        overlaps(eo, gdr_extent(bv, rows, toks, a->num_v_heads, 1, gsize)))
        return CCV_ERR_ALIAS;
    if (a->state != nullptr && a->num_lines > 0) {
        const ccv_heads_view sv{a->state, a->s_stride_line, a->s_stride_head, a->s_stride_v, a->s_stride_k};
        const Extent es = gdr_extent(sv, a->num_lines, a->num_v_heads, a->dim_v, a->dim_k, 4);
        if (overlaps(es, eo)) return CCV_ERR_ALIAS;
    }
    return CCV_OK;
}

// Which tokens and state lines the recurrent kernel's rows use: `seqlen` tokens of a batch row, or a varlen sequence
// when query_start_loc is set.
struct GdrRows {
    const int32_t *query_start_loc;
    const int32_t *state_indices;
    const uint8_t *has_initial_state;
    const int32_t *num_accepted;
    const int32_t *out_indices;
    int64_t oi_stride_b, oi_stride_step;
    int oidx_steps;
    int batch, seqlen, total_tokens;
    int *err_count;
};

int gdr_launch_recurrent(const ccv_gdr_args &a, const GdrRows &rows, cudaStream_t stream);

}  // namespace ccv
