// The norms around a block: gated_rms_norm (of its heads, with the gate) and residual_rms_norm (its output's norm, gate
// and scale, the residual addition, and the norm that opens the next block).
//
// Both read each element once, keep the row in registers in fp32, reduce it, and write once: 6 bytes an element for the
// first, 8 to 14 for the second.  Rows that allow 16-byte vectors are bound by HBM up to 16384 elements where they fill the
// card (16384 x 32 x 128 with gate: 66 us, 6.1 TB/s; 8191 x 4096 with a post norm, channel gate and fp32 residual: 65 us,
// 6.2 TB/s), and by one launch's latency below.  Above 16384 a block of 1024 threads has the SM to itself and waits on its
// loads (1677 x 20000: gated 64 us, 3.1 TB/s).  Rows that go element by element (a length that is not a multiple of 8, other
// strides, an address off 16 bytes) are bound by the count of loads and stores: 8191 x 2500 takes 74 us plain and 122 with
// post norm, token gate and fp32 residual (2.2 and 2.3 TB/s), gated 83 (1.5); 8191 x 4096 one element off 16 bytes, gated, 98
// against 36 on it.
// A row belongs to LPR lanes: within a warp the reductions are shuffles; longer rows reduce over the block's warps.
#include "ccv_common.cuh"
#include "ccv_layer.h"

namespace ccv {
namespace {

constexpr int kMaxRow = 32768;
constexpr int kNormThreads = 128;  // threads of a block when a row needs no more

constexpr int norm_threads(int lanes) { return lanes > kNormThreads ? lanes : kNormThreads; }

// A thread with up to 8 single elements or 2 vectors of a row has both operands' in flight at once and in registers.  With
// more, two operands and their addresses pass the 64 registers that a thread of 1024 may have: it keeps one, and reads the
// other after the sum, a few at a time.  (The bf16 residual's 4 vectors wait unwidened and fit: 1023 rows of 32768 take 46 us
// so and 57 the other way; gated rows of that length, 48 us, took 177 with both.)
constexpr bool holds_both(int vec, int count) { return count <= (vec == 1 ? 8 : 2); }
template <int VEC>
__device__ __forceinline__ void pause_loads(int j, float &used) {  // later loads come after `used` is there, and after stores
    if ((j + 1) * VEC % 8 == 0) asm volatile("" : "+f"(used)::"memory");
}

// Sum over the LPR lanes of a row; the block is one row when LPR > 32.
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float *warp_sums) {
#pragma unroll
    for (int m = 1; m < (LPR < 32 ? LPR : 32); m <<= 1) x += __shfl_xor_sync(kFullMask, x, m);
    if constexpr (LPR > 32) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        if (lane == 0) warp_sums[warp] = x;
        __syncthreads();
        x = lane < LPR / 32 ? warp_sums[lane] : 0.0f;
#pragma unroll
        for (int m = 1; m < LPR / 32; m <<= 1) x += __shfl_xor_sync(kFullMask, x, m);
        x = __shfl_sync(kFullMask, x, 0);
        __syncthreads();
    }
    return x;
}

template <int VEC>
__device__ __forceinline__ void load_row(const uint16_t *p, int64_t stride, int d, int dim, float (&f)[VEC]) {
    Raw<VEC> r;
    r.zero();
    if (d < dim) r = load_plain<VEC>(p + (VEC == 8 ? d : d * stride));
    r.to_float(f);
}
template <int VEC>
__device__ __forceinline__ void load_row(const float *p, int64_t stride, int d, int dim, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = d < dim ? *reinterpret_cast<const float4 *>(p + d) : z;
        const float4 b = d < dim ? *reinterpret_cast<const float4 *>(p + d + 4) : z;
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        f[0] = d < dim ? p[d * stride] : 0.0f;
    }
}
template <int VEC>
__device__ __forceinline__ void store_row(uint16_t *p, int64_t stride, int d, int dim, const float (&f)[VEC]) {
    Raw<VEC> r;
    r.from_float(f);
    if (d < dim) store_stream<VEC>(p + (VEC == 8 ? d : d * stride), r);
}
template <int VEC>
__device__ __forceinline__ void store_row(float *p, int64_t stride, int d, int dim, const float (&f)[VEC]) {
    if (d >= dim) return;
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4 *>(p + d) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + d + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        p[d * stride] = f[0];
    }
}

__device__ __forceinline__ float gate_act(float z, int activation) {
    if (activation == 0) return z;
    const float s = rcp_approx(1.0f + __expf(-z));
    return activation == 1 ? z * s : s;
}

struct GatedArgs {
    ccv_heads_view x, gate, out;
    const uint16_t *weight;
    int64_t rows;
    int heads, dim;
    float eps;
    int activation, before;
};

// R: rows a thread has in flight at once.  One row of 128 values is 32 bytes a lane, x and gate together; with two, 16384 x 32
// rows take 67 us (6.0 TB/s) instead of 75, with four 73 (registers).
template <int LPR, int VEC, int NV, int R>
__global__ void __launch_bounds__(norm_threads(LPR), LPR == 1024 ? 1 : 0) gated_rms_norm_kernel(const __grid_constant__ GatedArgs a) {
    __shared__ float warp_sums[32];
    wait_prior_grid();
    release_next_grid();
    constexpr int kThreads = norm_threads(LPR);
    constexpr int kRows = kThreads / LPR;  // rows of a block's pass
    const int lane = threadIdx.x % LPR;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kRows * R) + threadIdx.x / LPR;
    constexpr bool kBoth = holds_both(VEC, NV);
    float x[R][NV][VEC], z[R][kBoth ? NV : 1][VEC];
    const uint16_t *gp[R];
    uint16_t *op[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = first + r * kRows;
        const bool live = row < a.rows;
        unsigned tok = live ? static_cast<unsigned>(row) : 0u, head = 0;
        if (a.heads > 1) {
            head = tok % a.heads;
            tok /= a.heads;
        }
        const int dim = live ? a.dim : 0;
        const uint16_t *xp = static_cast<const uint16_t *>(a.x.data) + tok * a.x.stride_tok + head * a.x.stride_head;
        gp[r] = static_cast<const uint16_t *>(a.gate.data) + tok * a.gate.stride_tok + head * a.gate.stride_head;
        op[r] = live ? static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + tok * a.out.stride_tok + head * a.out.stride_head
                     : nullptr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = (j * LPR + lane) * VEC;
            load_row<VEC>(xp, a.x.stride_dim, d, dim, x[r][j]);
            if constexpr (kBoth) load_row<VEC>(gp[r], a.gate.stride_dim, d, dim, z[r][j]);
        }
    }
    float w[kBoth ? NV : 1][VEC];
#pragma unroll
    for (int j = 0; j < NV && kBoth; ++j) load_row<VEC>(a.weight, 1, (j * LPR + lane) * VEC, a.dim, w[j]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int dim = op[r] != nullptr ? a.dim : 0;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float(&gate)[VEC] = z[r][kBoth ? j : 0];
            if constexpr (!kBoth)
                if (!a.before) load_row<VEC>(gp[r], a.gate.stride_dim, (j * LPR + lane) * VEC, dim, gate);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (kBoth || !a.before) gate[i] = gate_act(gate[i], a.activation);
                if (!a.before) {  // past the row's end x is 0 and the gate finite
                    x[r][j][i] *= gate[i];
                    gate[i] = 1.0f;
                }
                sum = fmaf(x[r][j][i], x[r][j][i], sum);
            }
            if constexpr (!kBoth) pause_loads<VEC>(j, sum);
        }
        const float scale = rsqrtf(row_sum<LPR>(sum, warp_sums) / a.dim + a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int d = (j * LPR + lane) * VEC;
            float(&gate)[VEC] = z[r][kBoth ? j : 0], (&weight)[VEC] = w[kBoth ? j : 0];
            if constexpr (!kBoth) {
                load_row<VEC>(a.weight, 1, d, a.dim, weight);
                if (a.before) load_row<VEC>(gp[r], a.gate.stride_dim, d, dim, gate);
            }
            float y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (!kBoth) gate[i] = a.before ? gate_act(gate[i], a.activation) : 1.0f;
                y[i] = x[r][j][i] * scale * weight[i] * gate[i];
            }
            store_row<VEC>(op[r], a.out.stride_dim, d, dim, y);
            if constexpr (!kBoth) pause_loads<VEC>(j, x[r][j][0]);
        }
    }
}

struct ResidualArgs {
    const uint16_t *x;
    const void *residual;
    const uint16_t *weight, *post_weight, *gate;
    uint16_t *out;
    void *residual_out;
    int64_t xt, xd, rt, rd, gt, gd, ot, od, rot, rod;
    int tokens, dim;
    float scale, eps, offset;
};

template <int LPR, int VEC, int NV, typename Res>
__global__ void __launch_bounds__(norm_threads(LPR), LPR == 1024 ? 1 : 0) residual_rms_norm_kernel(const __grid_constant__ ResidualArgs a) {
    __shared__ float warp_sums[32];
    wait_prior_grid();
    release_next_grid();
    constexpr int kThreads = norm_threads(LPR);
    const int lane = threadIdx.x % LPR;
    int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / LPR) + threadIdx.x / LPR;
    const int dim = row < a.tokens ? a.dim : 0;
    if (row >= a.tokens) row = 0;
    const uint16_t *xp = a.x + row * a.xt;
    const Res *rp = static_cast<const Res *>(a.residual) + row * a.rt;
    constexpr bool kBoth = holds_both(VEC, NV) || (VEC == 8 && sizeof(Res) == 2);
    float x[NV][VEC], residual[kBoth ? NV : 1][VEC];  // x, then h
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = (j * LPR + lane) * VEC;
        load_row<VEC>(xp, a.xd, d, dim, x[j]);
        if constexpr (kBoth) load_row<VEC>(rp, a.rd, d, dim, residual[j]);
    }
    float post = a.scale;
    if (a.post_weight != nullptr) {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum = fmaf(x[j][i], x[j][i], sum);
        post *= rsqrtf(row_sum<LPR>(sum, warp_sums) / a.dim + a.eps);
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = (j * LPR + lane) * VEC;
        float f[VEC];
        if (a.post_weight != nullptr) {
            load_row<VEC>(a.post_weight, 1, d, dim, f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] *= f[i] + a.offset;
        }
        if (a.gate != nullptr) {
            load_row<VEC>(a.gate + row * a.gt, a.gd, d, dim, f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[j][i] *= f[i];
        }
        float(&res)[VEC] = residual[kBoth ? j : 0];
        if constexpr (!kBoth) load_row<VEC>(rp, a.rd, d, dim, res);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            x[j][i] = fmaf(post, x[j][i], res[i]);
            sum = fmaf(x[j][i], x[j][i], sum);
        }
        if constexpr (!kBoth) pause_loads<VEC>(j, sum);
    }
    const float scale = rsqrtf(row_sum<LPR>(sum, warp_sums) / a.dim + a.eps);
    Res *hp = static_cast<Res *>(a.residual_out) + row * a.rot;
    uint16_t *op = a.out + row * a.ot;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int d = (j * LPR + lane) * VEC;
        store_row<VEC>(hp, a.rod, d, dim, x[j]);
        float w[VEC];
        load_row<VEC>(a.weight, 1, d, dim, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = x[j][i] * scale * (w[i] + a.offset);
        store_row<VEC>(op, a.od, d, dim, w);
        if constexpr (!kBoth) pause_loads<VEC>(j, x[j][0]);
    }
}

// Calls f.template operator()<LPR, VEC, NV>() with the least lanes a row of `dim` elements needs.  With vectors of 8 a
// lane holds 1 vector up to 256 elements (a warp's 32 lanes), 2 vectors a lane up to 512, then whole blocks with 2 or 4.
// Single elements (a length that is not a multiple of 8, a stride, or an address off 16 bytes) go 8 to a lane up to a
// block's 1024 lanes, then 16 and 32.
template <typename F>
int for_row(int dim, bool vec, F f) {
    if (vec) {
        if (dim <= 64) return f.template operator()<8, 8, 1>();
        if (dim <= 128) return f.template operator()<16, 8, 1>();
        if (dim <= 256) return f.template operator()<32, 8, 1>();
        if (dim <= 512) return f.template operator()<32, 8, 2>();
        if (dim <= 2048) return f.template operator()<128, 8, 2>();
        if (dim <= 4096) return f.template operator()<256, 8, 2>();
        if (dim <= 8192) return f.template operator()<512, 8, 2>();
        if (dim <= 16384) return f.template operator()<1024, 8, 2>();
        return f.template operator()<1024, 8, 4>();
    }
    if (dim <= 256) return f.template operator()<32, 1, 8>();
    if (dim <= 2048) return f.template operator()<256, 1, 8>();
    if (dim <= 4096) return f.template operator()<512, 1, 8>();
    if (dim <= 8192) return f.template operator()<1024, 1, 8>();
    if (dim <= 16384) return f.template operator()<1024, 1, 16>();
    return f.template operator()<1024, 1, 32>();
}

unsigned row_blocks(int64_t rows, int lanes) {
    const int per = lanes > kNormThreads ? 1 : kNormThreads / lanes;
    return static_cast<unsigned>((rows + per - 1) / per);
}

struct GatedLaunch {
    GatedArgs a;
    cudaStream_t stream;
    template <int LPR, int VEC, int NV>
    int operator()() const {
        // Two rows a thread once there are enough rows for every SM's threads to have two: below that one row each spreads
        // the call over more SMs.
        if constexpr (LPR <= 32 && VEC == 8 && NV == 1) {
            if (a.rows * LPR >= 2ll * 2048 * current_device_sms())
                return launch_pdl(gated_rms_norm_kernel<LPR, VEC, NV, 2>, dim3(row_blocks((a.rows + 1) / 2, LPR)),
                                  dim3(kNormThreads), 0, stream, a);
        }
        return launch_pdl(gated_rms_norm_kernel<LPR, VEC, NV, 1>, dim3(row_blocks(a.rows, LPR)),
                          dim3(norm_threads(LPR)), 0, stream, a);
    }
};

template <typename Res>
struct ResidualLaunch {
    ResidualArgs a;
    cudaStream_t stream;
    template <int LPR, int VEC, int NV>
    int operator()() const {
        return launch_pdl(residual_rms_norm_kernel<LPR, VEC, NV, Res>, dim3(row_blocks(a.tokens, LPR)),
                          dim3(norm_threads(LPR)), 0, stream, a);
    }
};

Extent extent2(const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int size) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(p);
    const int64_t last = (n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2;
    return Extent{base, base + static_cast<uintptr_t>(last) * size + size - 1};
}

bool vec_view(const void *p, int64_t s0, int64_t s1, int64_t sd) {
    return aligned16(p) && sd == 1 && s0 % 8 == 0 && s1 % 8 == 0;
}

}  // namespace
}  // namespace ccv

extern "C" int gated_rms_norm(const ccv_heads_view *x, const ccv_heads_view *gate, const void *weight,
                              const ccv_heads_view *out, int tokens, int heads, int dim, float eps, int activation,
                              int norm_before_gate, ccv_stream_t stream) {
    using namespace ccv;
    if (x == nullptr || gate == nullptr || out == nullptr) return CCV_ERR_NULL_POINTER;
    if (tokens < 0 || heads < 0 || dim < 0) return CCV_ERR_SIZE;
    if (activation < 0 || activation > 2) return CCV_ERR_ARGUMENT;
    if (dim > kMaxRow) return CCV_ERR_DIM;
    for (const ccv_heads_view *v : {x, gate, out})
        if (v->stride_tok < 0 || v->stride_head < 0 || v->stride_dim < 0) return CCV_ERR_STRIDE;
    if (tokens == 0 || heads == 0 || dim == 0) return CCV_OK;
    if (x->data == nullptr || gate->data == nullptr || weight == nullptr || out->data == nullptr) return CCV_ERR_NULL_POINTER;
    auto extent = [&](const ccv_heads_view *v) {
        return extent2(v->data, tokens, v->stride_tok, heads, v->stride_head, dim, v->stride_dim, 2);
    };
    for (const ccv_heads_view *v : {x, gate}) {
        const bool same = v->data == out->data && v->stride_tok == out->stride_tok && v->stride_head == out->stride_head &&
                          v->stride_dim == out->stride_dim;
        if (!same && overlaps(extent(v), extent(out))) return CCV_ERR_ALIAS;
    }
    if (overlaps(extent2(weight, 1, 0, 1, 0, dim, 1, 2), extent(out))) return CCV_ERR_ALIAS;
    const int64_t rows = static_cast<int64_t>(tokens) * heads;
    if (rows > 0x7fffffff) return CCV_ERR_SIZE;
    bool vec = dim % 8 == 0 && aligned16(weight);
    for (const ccv_heads_view *v : {x, gate, out}) vec = vec && vec_view(v->data, v->stride_tok, v->stride_head, v->stride_dim);
    // Heads that follow each other like tokens do are rows of one axis: no division in the kernel.
    GatedArgs a{*x, *gate, *out, static_cast<const uint16_t *>(weight), rows, heads, dim, eps, activation, norm_before_gate};
    bool flat = true;
    for (const ccv_heads_view *v : {x, gate, out}) flat = flat && v->stride_tok == heads * v->stride_head;
    if (flat) {
        a.heads = 1;
        for (ccv_heads_view *v : {&a.x, &a.gate, &a.out}) v->stride_tok = v->stride_head;
    }
    return for_row(dim, vec, GatedLaunch{a, stream});
}

extern "C" int residual_rms_norm(const void *x, int64_t x_stride_tok, int64_t x_stride_dim, const void *residual,
                                 int64_t r_stride_tok, int64_t r_stride_dim, int residual_fp32, const void *weight,
                                 const void *post_weight, const void *gate, int64_t g_stride_tok, int64_t g_stride_dim,
                                 void *out, int64_t out_stride_tok, int64_t out_stride_dim, void *residual_out,
                                 int64_t ro_stride_tok, int64_t ro_stride_dim, int tokens, int dim, float scale, float eps,
                                 float weight_offset, ccv_stream_t stream) {
    using namespace ccv;
    if (tokens < 0 || dim < 0) return CCV_ERR_SIZE;
    if (dim > kMaxRow) return CCV_ERR_DIM;
    for (int64_t s : {x_stride_tok, x_stride_dim, r_stride_tok, r_stride_dim, g_stride_tok, g_stride_dim, out_stride_tok,
                      out_stride_dim, ro_stride_tok, ro_stride_dim})
        if (s < 0) return CCV_ERR_STRIDE;
    if (tokens == 0 || dim == 0) return CCV_OK;
    if (x == nullptr || residual == nullptr || weight == nullptr || out == nullptr || residual_out == nullptr)
        return CCV_ERR_NULL_POINTER;
    const int rsize = residual_fp32 ? 4 : 2;
    const Extent ex = extent2(x, tokens, x_stride_tok, dim, x_stride_dim, 1, 0, 2);
    const Extent er = extent2(residual, tokens, r_stride_tok, dim, r_stride_dim, 1, 0, rsize);
    const Extent eo = extent2(out, tokens, out_stride_tok, dim, out_stride_dim, 1, 0, 2);
    const Extent ero = extent2(residual_out, tokens, ro_stride_tok, dim, ro_stride_dim, 1, 0, rsize);
    const Extent ew = extent2(weight, 1, 0, dim, 1, 1, 0, 2);
    const bool out_is_x = out == x && out_stride_tok == x_stride_tok && out_stride_dim == x_stride_dim;
    const bool in_place = residual_out == residual && ro_stride_tok == r_stride_tok && ro_stride_dim == r_stride_dim;
    if ((!out_is_x && overlaps(eo, ex)) || (!in_place && overlaps(ero, er)) || overlaps(eo, er) || overlaps(ero, ex) ||
        overlaps(eo, ero) || overlaps(ew, eo) || overlaps(ew, ero))
        return CCV_ERR_ALIAS;
    if (post_weight != nullptr) {
        const Extent ep = extent2(post_weight, 1, 0, dim, 1, 1, 0, 2);
        if (overlaps(ep, eo) || overlaps(ep, ero)) return CCV_ERR_ALIAS;
    }
    if (gate != nullptr) {
        const Extent eg = extent2(gate, tokens, g_stride_tok, dim, g_stride_dim, 1, 0, 2);
        if (overlaps(eg, eo) || overlaps(eg, ero)) return CCV_ERR_ALIAS;
    }
    auto vec_res = [&](const void *p, int64_t st, int64_t sd) {
        return aligned16(p) && sd == 1 && st % (residual_fp32 ? 4 : 8) == 0;
    };
    const bool vec = dim % 8 == 0 && aligned16(weight) && (post_weight == nullptr || aligned16(post_weight)) &&
                     vec_view(x, x_stride_tok, 0, x_stride_dim) && vec_view(out, out_stride_tok, 0, out_stride_dim) &&
                     vec_res(residual, r_stride_tok, r_stride_dim) && vec_res(residual_out, ro_stride_tok, ro_stride_dim) &&
                     (gate == nullptr || vec_view(gate, g_stride_tok, 0, g_stride_dim));
    const ResidualArgs a{static_cast<const uint16_t *>(x), residual, static_cast<const uint16_t *>(weight),
                         static_cast<const uint16_t *>(post_weight), static_cast<const uint16_t *>(gate),
                         static_cast<uint16_t *>(out), residual_out, x_stride_tok, x_stride_dim, r_stride_tok, r_stride_dim,
                         g_stride_tok, g_stride_dim, out_stride_tok, out_stride_dim, ro_stride_tok, ro_stride_dim,
                         tokens, dim, scale, eps, weight_offset};
    return residual_fp32 ? for_row(dim, vec, ResidualLaunch<float>{a, stream})
                         : for_row(dim, vec, ResidualLaunch<uint16_t>{a, stream});
}
