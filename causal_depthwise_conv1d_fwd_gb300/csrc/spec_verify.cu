// Verification of drafted tokens: softmax statistics of every position, then acceptance and the draw of the next token.
//
// The probabilities are never written: position i's are exp((l - m) / T) / z with the position's maximum m and sum z.
// The draw is a race (the largest r_v / noise_v) and not a walk along cumulative sums, so the answer does not depend on
// the order in which any sum is formed and every split of the vocabulary gives the same token.
#include <cfloat>

#include "ccv_common.cuh"
#include "ccv_layer.h"

namespace ccv {
namespace {

constexpr int kVerifyThreads = 512;

struct VerifyArgs {
    const void *logits;
    int logits_fp32;
    int64_t tb, tp;
    const int32_t *tokens;
    int64_t db, dp;
    const float *probs;
    int64_t pb, pp;
    const int32_t *num_drafts;
    const float *temperature;
    const float *uniform;
    int64_t ub, up;
    const float *noise;
    int64_t nb;
    int32_t *out_tokens, *num_accepted;
    int batch, drafts, vocab;
    float *stats;  // (batch, drafts + 1, 4): maximum, its index's bits, sum of exponentials
    int *err_count;
};

// A logit: NaN is masked like -inf, +inf is the largest finite value.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float logit(const VerifyArgs &a, int64_t off) {
    return clean(a.logits_fp32 ? static_cast<const float *>(a.logits)[off]
                               : bf16_bits(static_cast<const uint16_t *>(a.logits)[off]));
}

// The larger value, and of equal ones the lower index.
__device__ __forceinline__ void take_best(float &v, int &i, float ov, int oi) {
    if (ov > v || (ov == v && oi < i)) {
        v = ov;
        i = oi;
    }
}

template <int kThreads>
__device__ __forceinline__ void block_best(float &v, int &i, float *sv, int *si) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) take_best(v, i, __shfl_xor_sync(kFullMask, v, m), __shfl_xor_sync(kFullMask, i, m));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
        sv[warp] = v;
        si[warp] = i;
    }
    __syncthreads();
    v = lane < kThreads / 32 ? sv[lane] : -INFINITY;
    i = lane < kThreads / 32 ? si[lane] : INT32_MAX;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) take_best(v, i, __shfl_xor_sync(kFullMask, v, m), __shfl_xor_sync(kFullMask, i, m));
    __syncthreads();
}

// e^((x - best) / temp) for x <= best; 0 where x is masked, whatever best is.
__device__ __forceinline__ float weight_of(float x, float best, float inv_temp) {
    return x == -INFINITY ? 0.0f : expf((x - best) * inv_temp);
}

__global__ void __launch_bounds__(kVerifyThreads) verify_stats_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ float sv[32];
    __shared__ int si[32];
    wait_prior_grid();
    const int pos = blockIdx.x % (a.drafts + 1), b = blockIdx.x / (a.drafts + 1);
    const int n = a.num_drafts != nullptr ? a.num_drafts[b] : a.drafts;
    if (pos > n) return;
    const float temp = a.temperature != nullptr ? a.temperature[b] : 1.0f;
    const float inv = temp > 0.0f ? 1.0f / temp : 1.0f;
    const int64_t at = b * a.tb + pos * a.tp;
    float best = -INFINITY, sum = 0.0f;
    int index = INT32_MAX;
    for (int v = threadIdx.x; v < a.vocab; v += kVerifyThreads) {
        const float x = logit(a, at + v);
        if (x > best) {
            sum = sum * weight_of(best, x, inv) + 1.0f;
            best = x;
            index = v;
        } else {
            sum += weight_of(x, best, inv);
        }
    }
    const float mine = best;
    block_best<kVerifyThreads>(best, index, sv, si);
    sum *= weight_of(mine, best, inv);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
    if (threadIdx.x % 32 == 0) sv[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        float z = 0.0f;
        for (int w = 0; w < kVerifyThreads / 32; ++w) z += sv[w];
        float *out = a.stats + static_cast<int64_t>(blockIdx.x) * 4;
        out[0] = best;
        out[1] = __int_as_float(index);
        out[2] = z;
    }
}

__global__ void __launch_bounds__(kVerifyThreads) verify_pick_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ float sv[32];
    __shared__ int si[32];
    __shared__ int s_kept;
    wait_prior_grid();
    const int b = blockIdx.x;
    int n = a.num_drafts != nullptr ? a.num_drafts[b] : a.drafts;
    int32_t *out = a.out_tokens + static_cast<int64_t>(b) * (a.drafts + 1);
    if (n < 0) {
        for (int i = threadIdx.x; i <= a.drafts; i += kVerifyThreads) out[i] = -1;
        if (threadIdx.x == 0) a.num_accepted[b] = 0;
        return;
    }
    if (n > a.drafts) n = a.drafts;
    const float temp = a.temperature != nullptr ? a.temperature[b] : 1.0f;
    const bool greedy = !(temp > 0.0f);
    const float inv = greedy ? 1.0f : 1.0f / temp;
    const float *stats = a.stats + static_cast<int64_t>(b) * (a.drafts + 1) * 4;
    if (threadIdx.x == 0) {
        int kept = 0;
        for (; kept < n; ++kept) {
            const int token = a.tokens[b * a.db + kept * a.dp];
            if (token < 0 || token >= a.vocab) {
                count_error(a.err_count);
                break;
            }
            const float *st = stats + kept * 4;
            float p;
            if (greedy) p = st[0] > -INFINITY && token == __float_as_int(st[1]) ? 1.0f : 0.0f;
            else p = st[2] > 0.0f ? weight_of(logit(a, b * a.tb + kept * a.tp + token), st[0], inv) / st[2] : 0.0f;
            const float q = a.probs != nullptr ? a.probs[b * a.pb + kept * a.pp + token] : 1.0f;
            if (!(a.uniform[b * a.ub + kept * a.up] * q < p)) break;
        }
        s_kept = kept;
    }
    __syncthreads();
    const int kept = s_kept;
    const float best = stats[kept * 4], z = stats[kept * 4 + 2];
    float top = 0.0f;  // a score has to be above 0
    int index = INT32_MAX;
    if (greedy) {
        if (best > -INFINITY) {
            top = 1.0f;
            index = __float_as_int(stats[kept * 4 + 1]);
        }
    } else if (z > 0.0f) {
        const int64_t at = b * a.tb + kept * a.tp;
        const float *q = kept < n && a.probs != nullptr ? a.probs + b * a.pb + kept * a.pp : nullptr;
        const int sure = kept < n && a.probs == nullptr ? a.tokens[b * a.db + kept * a.dp] : -1;
        for (int v = threadIdx.x; v < a.vocab; v += kVerifyThreads) {
            float r = weight_of(logit(a, at + v), best, inv) / z;
            if (q != nullptr) r -= q[v];
            if (v == sure) r = 0.0f;
            const float score = r / a.noise[b * a.nb + v];
            if (r > 0.0f && score > top) {
                top = score;
                index = v;
            }
        }
        block_best<kVerifyThreads>(top, index, sv, si);
    }
    for (int i = threadIdx.x; i <= a.drafts; i += kVerifyThreads)
        out[i] = i < kept ? a.tokens[b * a.db + i * a.dp] : i == kept && index != INT32_MAX ? index : -1;
    if (threadIdx.x == 0) a.num_accepted[b] = kept + 1;
}

}  // namespace
}  // namespace ccv

extern "C" int64_t spec_verify_workspace(int batch, int drafts, int vocab) {
    if (batch <= 0 || drafts < 0 || vocab <= 0) return 0;
    return static_cast<int64_t>(batch) * (drafts + 1) * 16;
}

extern "C" int spec_verify(const void *target_logits, int logits_fp32, int64_t t_stride_b, int64_t t_stride_pos,
                           const int32_t *draft_tokens, int64_t d_stride_b, int64_t d_stride_pos, const float *draft_probs,
                           int64_t p_stride_b, int64_t p_stride_pos, const int32_t *num_drafts, const float *temperature,
                           const float *uniform, int64_t u_stride_b, int64_t u_stride_pos, const float *noise,
                           int64_t n_stride_b, int32_t *out_tokens, int32_t *num_accepted, int batch, int drafts, int vocab,
                           void *workspace, int64_t workspace_bytes, int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || drafts < 0 || vocab < 0) return CCV_ERR_SIZE;
    for (int64_t s : {t_stride_b, t_stride_pos, d_stride_b, d_stride_pos, p_stride_b, p_stride_pos, u_stride_b, u_stride_pos,
                      n_stride_b})
        if (s < 0) return CCV_ERR_STRIDE;
    if (batch == 0) return CCV_OK;
    if (vocab == 0 || static_cast<int64_t>(batch) * (drafts + 1) > 0x7fffffff) return CCV_ERR_SIZE;
    if (target_logits == nullptr || noise == nullptr || out_tokens == nullptr || num_accepted == nullptr ||
        (drafts > 0 && (draft_tokens == nullptr || uniform == nullptr)))
        return CCV_ERR_NULL_POINTER;
    if (workspace == nullptr || workspace_bytes < spec_verify_workspace(batch, drafts, vocab) || !aligned16(workspace))
        return CCV_ERR_WORKSPACE;
    auto extent = [](const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        return Extent{lo, lo + static_cast<uintptr_t>((n0 - 1) * s0 + (n1 - 1) * s1) * 4u + 3u};
    };
    const Extent et = extent(out_tokens, batch, drafts + 1, drafts + 1, 1), ea = extent(num_accepted, batch, 1, 1, 0);
    if (overlaps(et, ea) ||
        (drafts > 0 && (overlaps(et, extent(draft_tokens, batch, d_stride_b, drafts, d_stride_pos)) ||
                        overlaps(ea, extent(draft_tokens, batch, d_stride_b, drafts, d_stride_pos)))) ||
        (num_drafts != nullptr &&
         (overlaps(et, extent(num_drafts, batch, 1, 1, 0)) || overlaps(ea, extent(num_drafts, batch, 1, 1, 0)))))
        return CCV_ERR_ALIAS;
    const VerifyArgs a{target_logits, logits_fp32, t_stride_b, t_stride_pos, draft_tokens, d_stride_b, d_stride_pos,
                       draft_probs, p_stride_b, p_stride_pos, num_drafts, temperature, uniform, u_stride_b, u_stride_pos,
                       noise, n_stride_b, out_tokens, num_accepted, batch, drafts, vocab,
                       static_cast<float *>(workspace), err_count};
    const int status = launch_pdl(verify_stats_kernel, dim3(static_cast<unsigned>(batch * (drafts + 1))),
                                  dim3(kVerifyThreads), 0, stream, a);
    if (status != CCV_OK) return status;
    return launch_pdl(verify_pick_kernel, dim3(static_cast<unsigned>(batch)), dim3(kVerifyThreads), 0, stream, a);
}
