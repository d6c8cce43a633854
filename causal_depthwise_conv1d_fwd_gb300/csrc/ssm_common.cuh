// What the kernels of the selective state space scan share: steps, the host's argument checks, and the recurrent kernel's
// launch.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "ccv_common.cuh"
#include "ccv_math2.cuh"
#include "ccv_ssm.h"

namespace ccv {

constexpr int kSsmMaxStates = 256;
constexpr int kSsmMaxDim = 1024;
constexpr float kLog2e = 1.4426950408889634f;

// log(1 + e^x) = max(x, 0) + log1p(e^{-|x|}) of a pair, the latter as t times a polynomial in t = e^{-|x|} (least largest relative
// error on [0, 1], 3e-8).  A step's relative error is what counts, however small the step is: with all roundings 2.4e-7 above -2;
// below, the exponent's rounding grows with it, 5.2e-7 to -10 (2e-7 on average) and 1.7e-6 to -32.
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

// The step d of one (token, head), from its input with the bias.  A step that is not a number stays one.
__device__ __forceinline__ float ssm_step(float raw, float bias, const ccv_ssm_args &a) {
    float d = raw + bias, unused;
    if (a.dt_softplus) unpack2(softplus2(pack2(d, d)), d, unused);
    return d < a.dt_min ? a.dt_min : d > a.dt_max ? a.dt_max : d;
}
__device__ __forceinline__ float ssm_raw_step(const ccv_ssm_args &a, int64_t off) {
    return a.dt_fp32 ? static_cast<const float *>(a.dt)[off] : bf16_bits(static_cast<const uint16_t *>(a.dt)[off]);
}

// A rate, or a multiple of one, with fp32's lowest number for minus infinity: a step of 0, as tokens past a tile's end have, then
// leaves the state (0 times infinity is NaN), and larger ones leave nothing of it.  NaN stays.
__device__ __forceinline__ float bounded_rate(float a) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(-FLT_MAX));
    return a;
}

// ------------------------------------------------------------ host side ----

inline bool ssm_view_ok(const ccv_heads_view &v) {
    return v.stride_row >= 0 && v.stride_tok >= 0 && v.stride_head >= 0 && v.stride_dim >= 0;
}
inline Extent ssm_extent(const ccv_heads_view &v, int64_t rows, int64_t toks, int64_t heads, int64_t dim, int size = 2) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(v.data);
    const int64_t last = (rows - 1) * v.stride_row + (toks - 1) * v.stride_tok + (heads - 1) * v.stride_head +
                         (dim - 1) * v.stride_dim;
    return Extent{base, base + static_cast<uintptr_t>(last) * size + size - 1};
}

// Whether each element of a written view has a place of its own: each axis steps over all of those with smaller strides.
inline bool ssm_apart(const ccv_heads_view &v, int64_t rows, int64_t toks, int64_t heads, int64_t dim) {
    struct Axis {
        int64_t stride, count;
    } axes[4] = {{v.stride_row, rows}, {v.stride_tok, toks}, {v.stride_head, heads}, {v.stride_dim, dim}};
    std::sort(axes, axes + 4, [](const Axis &a, const Axis &b) { return a.stride < b.stride; });
    int64_t span = 1;
    for (const Axis &a : axes) {
        if (a.count <= 1) continue;
        if (a.stride < span) return false;
        span += (a.count - 1) * a.stride;
    }
    return true;
}

// Sizes, strides, pointers and overlaps of a call over `rows` x `toks` tokens.
inline int ssm_check(const ccv_ssm_args *a, int64_t rows, int64_t toks) {
    if (a == nullptr) return CCV_ERR_NULL_POINTER;
    if (a->num_heads < 0 || a->num_groups < 0 || a->head_dim < 0 || a->dim_state < 0 || a->num_lines < 0) return CCV_ERR_SIZE;
    if (a->head_dim > kSsmMaxDim || a->dim_state > kSsmMaxStates) return CCV_ERR_DIM;
    if (a->num_heads > 0 && (a->num_groups == 0 || a->num_heads % a->num_groups != 0)) return CCV_ERR_HEADS;
    if (static_cast<int64_t>(a->num_heads) * a->head_dim > (1 << 30)) return CCV_ERR_SIZE;
    for (const ccv_heads_view *v : {&a->x, &a->z, &a->out, &a->B, &a->C})
        if (!ssm_view_ok(*v)) return CCV_ERR_STRIDE;
    if (a->dt_stride_row < 0 || a->dt_stride_tok < 0 || a->dt_stride_head < 0 || a->s_stride_line < 0 || a->s_stride_head < 0 ||
        a->s_stride_dim < 0 || a->s_stride_state < 0)
        return CCV_ERR_STRIDE;
    if (rows == 0 || toks == 0 || a->num_heads == 0 || a->head_dim == 0 || a->dim_state == 0) return CCV_OK;
    if (a->x.data == nullptr || a->out.data == nullptr || a->B.data == nullptr || a->C.data == nullptr || a->dt == nullptr ||
        a->A == nullptr)
        return CCV_ERR_NULL_POINTER;
    const int64_t h = a->num_heads, g = a->num_groups, p = a->head_dim, n = a->dim_state;
    const Extent eo = ssm_extent(a->out, rows, toks, h, p);
    auto flat = [](const float *q, int64_t count) {
        const uintptr_t base = reinterpret_cast<uintptr_t>(q);
        return Extent{base, base + static_cast<uintptr_t>(count) * 4u - 1u};
    };
    const ccv_heads_view dv{a->dt, a->dt_stride_row, a->dt_stride_tok, a->dt_stride_head, 0};
    if (overlaps(eo, ssm_extent(a->x, rows, toks, h, p)) || overlaps(eo, ssm_extent(a->B, rows, toks, g, n)) ||
        overlaps(eo, ssm_extent(a->C, rows, toks, g, n)) || overlaps(eo, ssm_extent(dv, rows, toks, h, 1, a->dt_fp32 ? 4 : 2)) ||
        overlaps(eo, flat(a->A, a->a_per_state ? h * n : h)) || (a->D != nullptr && overlaps(eo, flat(a->D, h))) ||
        (a->dt_bias != nullptr && overlaps(eo, flat(a->dt_bias, h))) ||
        (a->z.data != nullptr && overlaps(eo, ssm_extent(a->z, rows, toks, h, p))))
        return CCV_ERR_ALIAS;
    if (a->state != nullptr && a->num_lines > 0) {
        const ccv_heads_view sv{a->state, a->s_stride_line, a->s_stride_head, a->s_stride_dim, a->s_stride_state};
        if (overlaps(ssm_extent(sv, a->num_lines, h, p, n, 4), eo)) return CCV_ERR_ALIAS;
    }
    return CCV_OK;
}

// That of a call's written tensors, once ssm_check has passed it.
inline int ssm_check_written(const ccv_ssm_args &a, int64_t rows, int64_t toks) {
    const ccv_heads_view state{a.state, a.s_stride_line, a.s_stride_head, a.s_stride_dim, a.s_stride_state};
    const bool apart = ssm_apart(a.out, rows, toks, a.num_heads, a.head_dim) &&
                       (a.state == nullptr || ssm_apart(state, a.num_lines, a.num_heads, a.head_dim, a.dim_state));
    return apart ? CCV_OK : CCV_ERR_STRIDE;
}

// The arguments with limits that do not cross: min(max(d, lo), hi) is hi throughout where lo is above hi, and the kernels compare
// with lo first.
inline ccv_ssm_args ssm_ordered(const ccv_ssm_args &args) {
    ccv_ssm_args a = args;
    if (a.dt_min > a.dt_max) a.dt_min = a.dt_max;
    return a;
}

// Which tokens and state lines the recurrent kernel's rows use: `seqlen` tokens of a batch row, or a varlen sequence
// when query_start_loc is set.
struct SsmRows {
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

int ssm_launch_recurrent(const ccv_ssm_args &a, const SsmRows &rows, cudaStream_t stream);

}  // namespace ccv
