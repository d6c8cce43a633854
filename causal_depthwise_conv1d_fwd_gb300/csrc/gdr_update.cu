// Gated delta rule, recurrent form: decode rows, speculative-verify rows, and short varlen sequences.
//
// One token of one value head is
//     p = S k,  r = S q                                  (dim_v dot products each, over dim_k)
//     d = b (v - a p),  o = a r + d (k.q),  S <- a S + d k^T
// so both products come out of one pass over the old state, which then stays in registers for the next token.  The
// state dominates the traffic: 4 dim_k dim_v bytes read and written per head against 2 (2 dim_k + 2 dim_v) for the
// rest, so the kernel is bound by HBM for more than a few rows (256 rows of 32 heads of 128 x 128: 167 to 177 us on
// different cards, 6.1 to 6.45 TB/s, and of 256 x 128: 350 us, 6.2 TB/s; 64 rows of 4 tokens with a state stored after each:
// 107 to 110 us, 6.2 to 6.3 TB/s) and by one memory round trip below that.
//
// A row of S (dim_k values, contiguous) belongs to 8 lanes, each holding every eighth group of 4 values: a warp's load
// of 4 rows covers whole 128-byte lines, the dot products take 3 shuffles, and no shared memory or barrier is needed.
#include "gdr_common.cuh"

namespace ccv {
namespace {

constexpr int kGdrThreads = 128;
constexpr int kLanes = 8;  // lanes that share a row of the state

// 4 values at d..d+3 of a row of `dim`, zeros past its end.  V: one aligned vector load.
template <bool V>
__device__ __forceinline__ void load_state4(const float *p, int64_t stride, int d, int dim, float (&f)[4]) {
    if constexpr (V) {
        const float4 x = d < dim ? __ldcs(reinterpret_cast<const float4 *>(p + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = d + i < dim ? p[(d + i) * stride] : 0.0f;
    }
}
template <bool V>
__device__ __forceinline__ void store_state4(float *p, int64_t stride, int d, int dim, const float (&f)[4]) {
    if constexpr (V) {
        if (d < dim) __stcs(reinterpret_cast<float4 *>(p + d), make_float4(f[0], f[1], f[2], f[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (d + i < dim) p[(d + i) * stride] = f[i];
    }
}
template <bool V>
__device__ __forceinline__ void load_bf16x4(const uint16_t *p, int64_t stride, int d, int dim, float (&f)[4]) {
    if constexpr (V) {
        const uint2 x = d < dim ? *reinterpret_cast<const uint2 *>(p + d) : make_uint2(0u, 0u);
        f[0] = bf16_lo(x.x); f[1] = bf16_hi(x.x); f[2] = bf16_lo(x.y); f[3] = bf16_hi(x.y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = d + i < dim ? bf16_bits(p[(d + i) * stride]) : 0.0f;
    }
}

__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) x += __shfl_xor_sync(kFullMask, x, m);
    return x;
}

// DK: dim_k rounded up to 64, 128 or 256.  R: rows of S per group of 8 lanes.  V: dim_k and every stride and pointer
// allow 16-byte vectors of the state and 8-byte vectors of q and k.
template <int DK, int R, bool V>
__global__ void __launch_bounds__(kGdrThreads) gdr_recurrent_kernel(const __grid_constant__ ccv_gdr_args a,
                                                                    const __grid_constant__ GdrRows rw, int slices) {
    constexpr int NV = DK / (4 * kLanes);                      // groups of 4 values a lane holds of a row
    constexpr int kRowsPerBlock = kGdrThreads / kLanes * R;
    wait_prior_grid();
    release_next_grid();
    const int slice = blockIdx.x % slices;
    const int bh = blockIdx.x / slices;
    const int h = bh % a.num_v_heads, b = bh / a.num_v_heads;
    const int hk = h / (a.num_v_heads / a.num_k_heads);
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const bool first = threadIdx.x == 0 && slice == 0 && h == 0;  // counts a row's error once

    int64_t t0 = 0, row = b;
    int n = rw.seqlen;
    if (rw.query_start_loc != nullptr) {
        const int s = rw.query_start_loc[b], e = rw.query_start_loc[b + 1];
        if (s < 0 || e < s || e > rw.total_tokens) {
            if (first) count_error(rw.err_count);
            return;
        }
        t0 = s;
        n = e - s;
        row = 0;
    }
    if (n == 0) return;
    int line = rw.state_indices != nullptr ? rw.state_indices[b] : b;
    if (line == a.pad_slot_id) return;
    bool fresh = a.state == nullptr || (rw.query_start_loc != nullptr &&
                                        (rw.has_initial_state == nullptr || rw.has_initial_state[b] == 0));
    bool good = a.state == nullptr || (line >= 0 && line < a.num_lines);
    int64_t from = line;
    if (rw.num_accepted != nullptr) {
        const int kept = rw.num_accepted[b];
        if (kept >= 1 && kept <= rw.oidx_steps) {
            from = rw.out_indices[b * rw.oi_stride_b + (kept - 1) * rw.oi_stride_step];
            good = from >= 0 && from < a.num_lines;
        } else {
            good = false;
        }
    }
    if (!good) {
        if (first) count_error(rw.err_count);
        return;
    }

    const int64_t head_off = h * a.s_stride_head;
    float s[R][NV][4];
    int vr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        vr[r] = slice * kRowsPerBlock + r * (kGdrThreads / kLanes) + group;
        const bool use = !fresh && vr[r] < a.dim_v;
        const float *p = use ? a.state + from * a.s_stride_line + head_off + vr[r] * a.s_stride_v : a.state;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            load_state4<V>(p, a.s_stride_k, j * 4 * kLanes + lane * 4, use ? a.dim_k : 0, s[r][j]);
    }

    const uint16_t *qp = static_cast<const uint16_t *>(a.q.data) + row * a.q.stride_row + t0 * a.q.stride_tok + hk * a.q.stride_head;
    const uint16_t *kp = static_cast<const uint16_t *>(a.k.data) + row * a.k.stride_row + t0 * a.k.stride_tok + hk * a.k.stride_head;
    const uint16_t *vp = static_cast<const uint16_t *>(a.v.data) + row * a.v.stride_row + t0 * a.v.stride_tok + h * a.v.stride_head;
    uint16_t *op = static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + row * a.out.stride_row + t0 * a.out.stride_tok + h * a.out.stride_head;
    int64_t gate = row * a.gate_stride_row + t0 * a.gate_stride_tok + h * a.gate_stride_head;

    for (int t = 0; t < n; ++t) {
        float k[NV][4], q[NV][4];
        float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = j * 4 * kLanes + lane * 4;
            load_bf16x4<V>(kp, a.k.stride_dim, d, a.dim_k, k[j]);
            load_bf16x4<V>(qp, a.q.stride_dim, d, a.dim_k, q[j]);
        }
        float v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = vr[r] < a.dim_v ? bf16_bits(vp[vr[r] * a.v.stride_dim]) : 0.0f;
        float g, beta;
        gdr_gates(a, gate, h, g, beta);
        const float alpha = expf(g);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kk += k[j][i] * k[j][i];
                qq += q[j][i] * q[j][i];
            }
        float rk = 1.0f, rq = a.scale;
        if (a.qk_l2norm) {
            rk = rsqrtf(group_sum(kk) + kGdrNormEps);
            rq = rsqrtf(group_sum(qq) + kGdrNormEps) * a.scale;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                k[j][i] *= rk;
                q[j][i] *= rq;
                kq += k[j][i] * q[j][i];
            }
        kq = group_sum(kq);
        float p[R], o[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            p[r] = 0.0f;
            o[r] = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[r] = fmaf(s[r][j][i], k[j][i], p[r]);
                    o[r] = fmaf(s[r][j][i], q[j][i], o[r]);
                }
        }
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                p[r] += __shfl_xor_sync(kFullMask, p[r], m);
                o[r] += __shfl_xor_sync(kFullMask, o[r], m);
            }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float d = beta * (v[r] - alpha * p[r]);
            o[r] = alpha * o[r] + d * kq;
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][j][i] = fmaf(alpha, s[r][j][i], d * k[j][i]);
            if (lane == 0 && vr[r] < a.dim_v) op[vr[r] * a.out.stride_dim] = round_bf16(o[r]);
        }
        if (rw.out_indices != nullptr) {
            const int64_t to = rw.out_indices[b * rw.oi_stride_b + t * rw.oi_stride_step];
            if (to >= a.num_lines) {
                if (first) count_error(rw.err_count);
            } else if (to >= 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float *w = a.state + to * a.s_stride_line + head_off + vr[r] * a.s_stride_v;
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        store_state4<V>(w, a.s_stride_k, j * 4 * kLanes + lane * 4, vr[r] < a.dim_v ? a.dim_k : 0, s[r][j]);
                }
            }
        }
        kp += a.k.stride_tok;
        qp += a.q.stride_tok;
        vp += a.v.stride_tok;
        op += a.out.stride_tok;
        gate += a.gate_stride_tok;
    }
    if (rw.out_indices == nullptr && a.state != nullptr) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float *w = a.state + line * a.s_stride_line + head_off + vr[r] * a.s_stride_v;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                store_state4<V>(w, a.s_stride_k, j * 4 * kLanes + lane * 4, vr[r] < a.dim_v ? a.dim_k : 0, s[r][j]);
        }
    }
}

template <int DK, int R, bool V>
int launch(const ccv_gdr_args &a, const GdrRows &rows, cudaStream_t stream) {
    constexpr int kRows = kGdrThreads / kLanes * R;
    const int slices = (a.dim_v + kRows - 1) / kRows;
    const int64_t blocks = static_cast<int64_t>(slices) * a.num_v_heads * rows.batch;
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    return launch_pdl(gdr_recurrent_kernel<DK, R, V>, dim3(static_cast<unsigned>(blocks)), dim3(kGdrThreads), 0, stream, a,
                      rows, slices);
}

bool vector_ok(const ccv_gdr_args &a) {
    auto bf = [](const ccv_heads_view &v) {
        return (reinterpret_cast<uintptr_t>(v.data) & 7u) == 0 && v.stride_dim == 1 && v.stride_row % 4 == 0 &&
               v.stride_tok % 4 == 0 && v.stride_head % 4 == 0;
    };
    if (a.dim_k % 4 != 0 || !bf(a.q) || !bf(a.k)) return false;
    return a.state == nullptr || (aligned16(a.state) && a.s_stride_k == 1 && a.s_stride_line % 4 == 0 &&
                                  a.s_stride_head % 4 == 0 && a.s_stride_v % 4 == 0);
}

}  // namespace

int gdr_launch_recurrent(const ccv_gdr_args &a, const GdrRows &rows, cudaStream_t stream) {
    const bool vec = vector_ok(a);
    if (a.dim_k <= 64) return vec ? launch<64, 2, true>(a, rows, stream) : launch<64, 2, false>(a, rows, stream);
    if (a.dim_k <= 128) return vec ? launch<128, 2, true>(a, rows, stream) : launch<128, 2, false>(a, rows, stream);
    return vec ? launch<256, 2, true>(a, rows, stream) : launch<256, 2, false>(a, rows, stream);
}

}  // namespace ccv

extern "C" int gdr_update(const ccv_gdr_args *args, const int32_t *state_indices, const int32_t *num_accepted_tokens,
                          const int32_t *output_state_indices, int64_t oi_stride_b, int64_t oi_stride_step,
                          int oidx_steps, int batch, int seqlen, int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || seqlen < 0) return CCV_ERR_SIZE;
    const int status = gdr_check(args, batch, seqlen);
    if (status != CCV_OK) return status;
    if (oi_stride_b < 0 || oi_stride_step < 0) return CCV_ERR_STRIDE;
    if (num_accepted_tokens != nullptr && output_state_indices == nullptr) return CCV_ERR_ARGUMENT;
    if (output_state_indices != nullptr && oidx_steps < seqlen) return CCV_ERR_CAPACITY;
    if (batch == 0 || seqlen == 0 || args->num_v_heads == 0 || args->dim_v == 0 || args->dim_k == 0) return CCV_OK;
    if (args->state == nullptr) return CCV_ERR_NULL_POINTER;
    const GdrRows rows{nullptr,     state_indices,  nullptr,    num_accepted_tokens, output_state_indices,
                       oi_stride_b, oi_stride_step, oidx_steps, batch,               seqlen,
                       0,           err_count};
    return gdr_launch_recurrent(*args, rows, stream);
}
