// Selective state space scan, recurrent form: decode rows, speculative-verify rows, and short varlen sequences.
//
// One token of one row of the state (head h, channel p) is
//     s <- exp(d A) s + (d x) B,   y = s . C
// over dim_state values.  The state dominates the traffic: 8 bytes a value read and written against 2 for x, z and out over
// a whole row of it, so the kernel is bound by HBM for more than a few rows and by one memory round trip below that.
//
// A row of S (contiguous) belongs to LANES lanes, each holding every LANES-th group of 4 values: a warp's load covers whole
// 128-byte lines, and no shared memory or barrier is needed.  A group of lanes has R rows next to each other; what goes by the row
// (x, the step, the decay where a head has one, the output) is one lane's work and reaches the others by shuffles, and the sums
// over the lanes are taken for all rows at once, so that each ends with the lane that its row belongs to.
//
// 256 rows of 128 heads of 64 channels with 128 states take 344 us (6.3 TB/s), 64 rows of 4 tokens with every state kept 204, one
// row 4.  256 rows of 8192 channels with 16 states and a decay for each take 68 (4.2 TB/s): there instructions (61 % of the slots)
// and latency count as well.
#include <algorithm>

#include "ssm_common.cuh"

namespace ccv {
namespace {

constexpr int kSsmThreads = 128;

// 4 values at d..d+3 of a row of `dim`, zeros past its end.  V: one aligned vector load.
template <bool V>
__device__ __forceinline__ void load4(const float *p, int64_t stride, int d, int dim, float (&f)[4]) {
    if constexpr (V) {
        const float4 x = d < dim ? __ldcs(reinterpret_cast<const float4 *>(p + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = d + i < dim ? p[(d + i) * stride] : 0.0f;
    }
}
template <bool V>
__device__ __forceinline__ void store4(float *p, int64_t stride, int d, int dim, const float (&f)[4]) {
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

// LANES x NV x 4: dim_state rounded up.  R: rows of the state a group of lanes has.  PER: A has a value a state.
// V: dim_state and every stride and pointer allow 16-byte vectors of the state and 8-byte vectors of B and C.
template <int LANES, int NV, int R, bool PER, bool V>
__global__ void __launch_bounds__(kSsmThreads, !V || NV > 4 ? 1 : PER ? 5 : R == 1 ? 8 : 6) ssm_recurrent_kernel(const __grid_constant__ ccv_ssm_args a,
                                                                    const __grid_constant__ SsmRows rw, int slices, int per) {
    constexpr int kGroups = kSsmThreads / LANES;
    wait_prior_grid();
    release_next_grid();
    const int part = blockIdx.x / static_cast<unsigned>(slices), slice = blockIdx.x - part * slices;
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const bool first = threadIdx.x == 0 && slice == 0;  // counts a row's error once

    const int rows = a.num_heads * a.head_dim, rep = a.num_heads / a.num_groups;
    const int first_row = (slice * kGroups + group) * R;
    float decay[PER ? R : 1][PER ? NV : 1][PER ? 4 : 1];
    int64_t off[R];  // of the row in a state line
    int grp[R];
    const int own_row = first_row + lane % R;  // the lane's
    const bool own = lane < R && own_row < rows;
    int own_h = 0, own_ch = 0;
    const auto find_rows = [&] {
        // one division for the first row; the others follow it
        int h = min(first_row, rows - 1), ch = 0, g = 0;
        if (a.head_dim != 1) {
            ch = h;
            h /= a.head_dim;
            ch -= h * a.head_dim;
        }
        if (a.num_groups != 1) g = h / rep;
        int in_group = h - g * rep;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            off[r] = h * a.s_stride_head + ch * a.s_stride_dim;
            grp[r] = g;
            if (lane % R == r) {
                own_h = h;
                own_ch = ch;
            }
            if constexpr (PER) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const float *rates = a.A + static_cast<int64_t>(h) * a.dim_state;
                    const int d = (j * LANES + lane) * 4;
                    if constexpr (V) {
                        const float4 f = d < a.dim_state ? __ldg(reinterpret_cast<const float4 *>(rates + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
                        decay[r][j][0] = f.x; decay[r][j][1] = f.y; decay[r][j][2] = f.z; decay[r][j][3] = f.w;
                    } else {
                        load4<false>(rates, 1, d, a.dim_state, decay[r][j]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) decay[r][j][i] = bounded_rate(decay[r][j][i] * kLog2e);
                }
            }
            if (first_row + r + 1 < rows && ++ch == a.head_dim) {
                ch = 0;
                ++h;
                if (++in_group == rep) {
                    in_group = 0;
                    ++g;
                }
            }
        }
    };
    if (PER) find_rows();
    const int end = PER ? min((part + 1) * per, rw.batch) : part + 1;
    for (int b = PER ? part * per : part; b < end; ++b) {
        int64_t t0 = 0, row = b;
        int n = rw.seqlen;
        if (rw.query_start_loc != nullptr) {
            const int s = rw.query_start_loc[b], e = rw.query_start_loc[b + 1];
            if (s < 0 || e < s || e > rw.total_tokens) {
                if (first) count_error(rw.err_count);
                continue;
            }
            t0 = s;
            n = e - s;
            row = 0;
        }
        if (n == 0) continue;
        const int line = rw.state_indices != nullptr ? rw.state_indices[b] : b;
        if (line == a.pad_slot_id) continue;
        const bool fresh = a.state == nullptr || (rw.query_start_loc != nullptr &&
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
            continue;
        }

        if (!PER) find_rows();
        float s[R][NV][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                load4<V>(fresh ? a.A : a.state + from * a.s_stride_line + off[r], a.s_stride_state, (j * LANES + lane) * 4,
                         first_row + r < rows && !fresh ? a.dim_state : 0, s[r][j]);
        const int h = own_h, ch = own_ch;
        const float bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f, skip = a.D != nullptr ? a.D[h] : 0.0f;
        const float rate = PER ? 0.0f : bounded_rate(a.A[h] * kLog2e);

        const auto at = [&](const ccv_heads_view &v, int64_t head, int64_t dim) {
            return static_cast<const uint16_t *>(v.data) + row * v.stride_row + t0 * v.stride_tok + head * v.stride_head + dim * v.stride_dim;
        };
        const uint16_t *xp = at(a.x, h, ch), *zp = at(a.z, h, ch), *bp = at(a.B, 0, 0), *cp = at(a.C, 0, 0);
        uint16_t *op = const_cast<uint16_t *>(at(a.out, h, ch));
        int64_t step = row * a.dt_stride_row + t0 * a.dt_stride_tok + h * a.dt_stride_head;

        for (int t = 0; t < n; ++t) {
            const float x = bf16_bits(*xp), d = ssm_step(ssm_raw_step(a, step), bias, a);
            const float z = a.z.data != nullptr ? bf16_bits(*zp) : 0.0f;
            const float dx = d * x, same = PER ? d : ex2_approx(d * rate);
            float y[R], bv[NV][4], cv[NV][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float e_or_d = __shfl_sync(kFullMask, same, r, LANES), w = __shfl_sync(kFullMask, dx, r, LANES);
                if (r == 0 || grp[r] != grp[r - 1]) {
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        load_bf16x4<V>(bp + grp[r] * a.B.stride_head, a.B.stride_dim, (j * LANES + lane) * 4, a.dim_state, bv[j]);
                        load_bf16x4<V>(cp + grp[r] * a.C.stride_head, a.C.stride_dim, (j * LANES + lane) * 4, a.dim_state, cv[j]);
                    }
                }
                y[r] = 0.0f;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = PER ? ex2_approx(e_or_d * decay[PER ? r : 0][PER ? j : 0][PER ? i : 0]) : e_or_d;
                        s[r][j][i] = fmaf(e, s[r][j][i], w * bv[j][i]);
                        y[r] = fmaf(s[r][j][i], cv[j][i], y[r]);
                    }
            }
            // halving: after the steps that the rows' count allows each lane has one row's sum over some lanes, then over all
#pragma unroll
            for (int m = R / 2; m > 0; m >>= 1)
#pragma unroll
                for (int r = 0; r < m; ++r) {
                    const bool upper = (lane & m) != 0;
                    const float keep = upper ? y[r + m] : y[r], give = upper ? y[r] : y[r + m];
                    y[r] = keep + __shfl_xor_sync(kFullMask, give, m);
                }
#pragma unroll
            for (int m = R; m < LANES; m <<= 1) y[0] += __shfl_xor_sync(kFullMask, y[0], m);
            if (own) {
                float o = fmaf(skip, x, y[0]);
                if (a.z.data != nullptr) o *= silu(z);
                *op = round_bf16(o);
            }
            if (rw.out_indices != nullptr) {
                const int64_t to = rw.out_indices[b * rw.oi_stride_b + t * rw.oi_stride_step];
                if (to >= a.num_lines) {
                    if (first) count_error(rw.err_count);
                } else if (to >= 0) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int j = 0; j < NV; ++j)
                            store4<V>(a.state + to * a.s_stride_line + off[r], a.s_stride_state, (j * LANES + lane) * 4,
                                      first_row + r < rows ? a.dim_state : 0, s[r][j]);
                }
            }
            xp += a.x.stride_tok;
            zp += a.z.stride_tok;
            bp += a.B.stride_tok;
            cp += a.C.stride_tok;
            op += a.out.stride_tok;
            step += a.dt_stride_tok;
        }
        if (rw.out_indices == nullptr && a.state != nullptr) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    store4<V>(a.state + line * a.s_stride_line + off[r], a.s_stride_state, (j * LANES + lane) * 4,
                              first_row + r < rows ? a.dim_state : 0, s[r][j]);
        }
    }
}

template <int LANES, int NV, int R, bool PER, bool V>
int launch(const ccv_ssm_args &a, const SsmRows &rows, cudaStream_t stream) {
    constexpr int kRows = kSsmThreads / LANES * R;
    const int slices = (a.num_heads * a.head_dim + kRows - 1) / kRows;
    // With a decay a state the block's rates are as large as its rows of the state, and it keeps them for up to 6 of the batch's
    // rows, as long as two waves of blocks are left (5 an SM of 152).  A row a block takes for 64, 128, 256 and 512 rows of 8192
    // channels 22, 41, 85 and 162 us, and this 20, 36, 70 and 132; for 16 rows 7.2, and two rows a block 8.0.
    int per = 1;
    if (PER) {
        per = static_cast<int>(std::min<int64_t>(6, std::max<int64_t>(1, static_cast<int64_t>(slices) * rows.batch / (2 * 5 * 152))));
        const int parts = (rows.batch + per - 1) / per;
        per = (rows.batch + parts - 1) / parts;
    }
    const int64_t blocks = static_cast<int64_t>(slices) * ((rows.batch + per - 1) / per);
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    return launch_pdl(ssm_recurrent_kernel<LANES, NV, R, PER, V>, dim3(static_cast<unsigned>(blocks)), dim3(kSsmThreads), 0, stream,
                      a, rows, slices, per);
}

// Lanes, groups of 4 values a lane, and rows of a group of lanes.  256 rows of 8192 channels with 16 states: 68 us, with 2 rows 93;
// with 15 states (single elements) 179, with 2 rows 276; but one decay a head, 128 rows of 64 heads of 64 with 15 states, 37 with
// 2 rows, 47 with 4.  128 rows of 64 heads of 64 channels with 64 states: 54 us (4 rows 58, 16 lanes 62), with 63 states 179 (one
// row 203), with 128 states 88 (2 rows 122, 16 lanes with 2 rows 105), with 256 states 170 (8 lanes 195, 2 rows 233, 32 lanes 276).
template <bool PER, bool V>
int launch_states(const ccv_ssm_args &a, const SsmRows &rows, cudaStream_t stream) {
    if (a.dim_state <= 16) return launch<4, 1, V || PER ? 4 : 2, PER, V>(a, rows, stream);
    if (a.dim_state <= 32) return launch<8, 1, V || PER ? 4 : 2, PER, V>(a, rows, stream);
    if (a.dim_state <= 64) return launch<8, 2, 2, PER, V>(a, rows, stream);
    if (a.dim_state <= 128) return launch<8, 4, 1, PER, V>(a, rows, stream);
    return launch<16, 4, 1, PER, V>(a, rows, stream);
}

bool vector_ok(const ccv_ssm_args &a) {
    auto bf = [](const ccv_heads_view &v) {
        return (reinterpret_cast<uintptr_t>(v.data) & 7u) == 0 && v.stride_dim == 1 && v.stride_row % 4 == 0 &&
               v.stride_tok % 4 == 0 && v.stride_head % 4 == 0;
    };
    if (a.dim_state % 4 != 0 || !bf(a.B) || !bf(a.C) || (a.a_per_state && !aligned16(a.A))) return false;
    return a.state == nullptr || (aligned16(a.state) && a.s_stride_state == 1 && a.s_stride_line % 4 == 0 &&
                                  a.s_stride_head % 4 == 0 && a.s_stride_dim % 4 == 0);
}

}  // namespace

int ssm_launch_recurrent(const ccv_ssm_args &a, const SsmRows &rows, cudaStream_t stream) {
    const bool vec = vector_ok(a);
    if (a.a_per_state) return vec ? launch_states<true, true>(a, rows, stream) : launch_states<true, false>(a, rows, stream);
    return vec ? launch_states<false, true>(a, rows, stream) : launch_states<false, false>(a, rows, stream);
}

}  // namespace ccv

extern "C" int ssm_update(const ccv_ssm_args *args, const int32_t *state_indices, const int32_t *num_accepted_tokens,
                          const int32_t *output_state_indices, int64_t oi_stride_b, int64_t oi_stride_step, int oidx_steps,
                          int batch, int seqlen, int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || seqlen < 0) return CCV_ERR_SIZE;
    int status = ssm_check(args, batch, seqlen);
    if (status != CCV_OK) return status;
    if (oi_stride_b < 0 || oi_stride_step < 0) return CCV_ERR_STRIDE;
    if (num_accepted_tokens != nullptr && output_state_indices == nullptr) return CCV_ERR_ARGUMENT;
    if (output_state_indices != nullptr && oidx_steps < seqlen) return CCV_ERR_CAPACITY;
    if (batch == 0 || seqlen == 0 || args->num_heads == 0 || args->head_dim == 0 || args->dim_state == 0) return CCV_OK;
    if (args->state == nullptr) return CCV_ERR_NULL_POINTER;
    if ((status = ssm_check_written(*args, batch, seqlen)) != CCV_OK) return status;
    const SsmRows rows{nullptr,     state_indices,  nullptr,    num_accepted_tokens, output_state_indices,
                       oi_stride_b, oi_stride_step, oidx_steps, batch,               seqlen,
                       0,           err_count};
    return ssm_launch_recurrent(ssm_ordered(*args), rows, stream);
}
