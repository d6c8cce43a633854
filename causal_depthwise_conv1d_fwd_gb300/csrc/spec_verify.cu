// Verification of drafted tokens: softmax statistics of every position, then acceptance and the draw of the next token.
//
// The probabilities are never written: position i's are exp((l - m) / T) / z with the position's maximum m and sum z.
// The draw is a race (the largest r_v / noise_v) and not a walk along cumulative sums, so the answer does not depend on
// the order in which any sum is formed and every split of the vocabulary gives the same token.
#include <algorithm>
#include <cfloat>

#include "ccv_common.cuh"
#include "ccv_layer.h"

namespace ccv {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kStep = kVerifyThreads * 8;  // logits of one pass of a block, 8 a thread
constexpr int kVectors = 4;                // passes that a thread has in flight
constexpr int kShare = kVectors * kStep;   // a block's share of a row in the draw, and in the statistics of small calls
constexpr int kLongShare = 2 * kShare;     // in the statistics of large ones
constexpr int kPickBlocks = 4, kPickBlocks32 = 3;  // blocks an SM of the draw, for bf16 and fp32 logits (2, 3, 5, 6 were slower)

struct VerifyArgs {
    const void *logits;
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
    int share, splits;  // logits of a block of the statistics, and such blocks a row
    int shares, rounds;  // blocks a row of the draw, and how often each takes kShare logits
    float4 *stats;     // (batch, drafts + 1, splits): maximum, its index's bits, sum of exponentials
    float2 *best;      // (batch, shares): a share's best score and its index's bits
    unsigned *done;    // (batch): shares finished
    int *err_count;
};

// A logit: NaN is masked like -inf, +inf is the largest finite value.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }
__device__ __forceinline__ float widen(uint16_t x) { return bf16_bits(x); }
__device__ __forceinline__ float widen(float x) { return x; }

// 8 logits from row[i..] as they are in memory, of which those in [0, end) are real; the others are -inf.  row + i is on a
// 16-byte boundary.
template <typename T> struct Logits;
template <> struct Logits<uint16_t> {
    Raw<8> r;
    __device__ __forceinline__ void load(const uint16_t *row, int i, int end) {
        if (i >= 0 && i + 8 <= end) {
            r.v = *reinterpret_cast<const uint4 *>(row + i);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) r.set_elem(k, i + k >= 0 && i + k < end ? row[i + k] : uint16_t(0xff80));
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { r.to_float(f); }
};
template <> struct Logits<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *row, int i, int end) {
        if (i >= 0 && i + 8 <= end) {
            a = *reinterpret_cast<const float4 *>(row + i);
            b = *reinterpret_cast<const float4 *>(row + i + 4);
        } else {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = i + k >= 0 && i + k < end ? row[i + k] : -INFINITY;
            a = make_float4(f[0], f[1], f[2], f[3]);
            b = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};
template <typename T>
__device__ __forceinline__ void load8(const T *row, int i, int end, float (&f)[8]) {
    Logits<T> l;
    l.load(row, i, end);
    l.get(f);
}
__device__ __forceinline__ void load8_plain(const float *row, int i, int end, bool aligned, float (&f)[8]) {
    if (aligned && i + 8 <= end) {
        const float4 x = *reinterpret_cast<const float4 *>(row + i), y = *reinterpret_cast<const float4 *>(row + i + 4);
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w; f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = i + k >= 0 && i + k < end ? row[i + k] : 1.0f;
    }
}

// The larger value, and of equal ones the lower index.
__device__ __forceinline__ void take_best(float &v, int &i, float ov, int oi) {
    if (ov > v || (ov == v && oi < i)) {
        v = ov;
        i = oi;
    }
}
__device__ __forceinline__ void warp_best(float &v, int &i) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) take_best(v, i, __shfl_xor_sync(kFullMask, v, m), __shfl_xor_sync(kFullMask, i, m));
}
__device__ __forceinline__ void block_best(float &v, int &i, float *sv, int *si) {
    warp_best(v, i);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
        sv[warp] = v;
        si[warp] = i;
    }
    __syncthreads();
    v = lane < kVerifyThreads / 32 ? sv[lane] : -INFINITY;
    i = lane < kVerifyThreads / 32 ? si[lane] : INT32_MAX;
    warp_best(v, i);
    __syncthreads();
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^((x - best) / temp) as 2^((x - best) rate), rate = log2(e) / temp.  A masked x gives 0, also when best is -inf.
struct Weigh {
    float rate, best;
    __device__ __forceinline__ Weigh(float rate_, float best_) : rate(rate_), best(best_ == -INFINITY ? 0.0f : best_) {}
    __device__ __forceinline__ float operator()(float x) const { return ex2((x - best) * rate); }
};
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float rate_of(const VerifyArgs &a, int b) {
    const float t = a.temperature != nullptr ? a.temperature[b] : 1.0f;
    // 0 marks a greedy row.  Any other rate stays finite and above 0: 0 * infinity is NaN, for the largest logit with a
    // temperature below 4.3e-39 and for masked logits with an infinite one.
    return t > 0.0f ? fminf(fmaxf(kLog2e / t, __int_as_float(1)), FLT_MAX) : 0.0f;
}

// Maximum, its first index and the sum of exponentials of one share of one position.  Rows may start at any element: the
// shares count from the 16-byte boundary at or before the row's start, so that all but the edges are whole vectors.  Each
// thread keeps a running maximum and sum, one more exponential for every 8 logits, so nothing waits for the block until the
// end and the next vectors are always on their way: 64 x 5 rows of 131072 bf16 logits take 23 us (3.6 TB/s; the exponentials
// and the arithmetic around them are the bound) against 33 with a block-wide maximum first.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, sizeof(T) == 2 ? 5 : 2) verify_stats_kernel(const __grid_constant__ VerifyArgs a) {
    constexpr int kWarps = kVerifyThreads / 32;
    __shared__ float sv[kWarps], ss[kWarps];
    __shared__ int si[kWarps];
    wait_prior_grid();
    release_next_grid();
    const int split = blockIdx.x % a.splits, row = blockIdx.x / a.splits;
    const int pos = row % (a.drafts + 1), b = row / (a.drafts + 1);
    if (pos == 0 && split == 0 && threadIdx.x == 0) a.done[b] = 0;
    const int n = a.num_drafts != nullptr ? a.num_drafts[b] : a.drafts;
    if (pos > n) return;
    const float rate = rate_of(a, b);
    const T *logits = static_cast<const T *>(a.logits) + b * a.tb + pos * a.tp;
    const int before = static_cast<int>(reinterpret_cast<uintptr_t>(logits) % 16 / sizeof(T));
    const int first = split * a.share - before, end = min(a.vocab, first + a.share);
    float best = -INFINITY, sum = 0.0f;
    int where = 0;  // the vector that holds `best`
    auto take = [&](const float (&x)[8], int at) {
        float m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        if (m > best) {
            if (rate > 0.0f) sum *= Weigh(rate, m)(best);
            best = m;
            where = at;
        }
        if (rate > 0.0f) {
            const Weigh weigh(rate, best);
            float part[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 8; ++k) part[k & 1] += weigh(x[k]);
            sum += part[0] + part[1];
        }
    };
    const int mine = first + static_cast<int>(threadIdx.x) * 8;
    Logits<T> now[kVectors], next[kVectors];
#pragma unroll
    for (int j = 0; j < kVectors; ++j) now[j].load(logits, mine + j * kStep, end);
    for (int v0 = mine; v0 < end; v0 += kVectors * kStep) {
        const int v1 = v0 + kVectors * kStep;
        if (v1 < end) {
#pragma unroll
            for (int j = 0; j < kVectors; ++j) next[j].load(logits, v1 + j * kStep, end);
        }
#pragma unroll
        for (int j = 0; j < kVectors; ++j) {
            float x[8];
            now[j].get(x);
            take(x, v0 + j * kStep);
            now[j] = next[j];
        }
    }
    if (!(sum < INFINITY) || best == INFINITY) {  // a NaN or +inf among them: once more, cleaned
        best = -INFINITY;
        sum = 0.0f;
        for (int v0 = mine; v0 < end; v0 += kStep) {
            float x[8];
            load8(logits, v0, end, x);
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = clean(x[k]);
            take(x, v0);
        }
    }
    int index = INT32_MAX;
    const float top = best;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) best = fmaxf(best, __shfl_xor_sync(kFullMask, best, m));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) sv[warp] = best;
    __syncthreads();
    best = sv[lane % kWarps];
#pragma unroll
    for (int m = kWarps / 2; m > 0; m >>= 1) best = fmaxf(best, __shfl_xor_sync(kFullMask, best, m));
    if (top == best && best > -INFINITY) {
        float x[8];
        load8(logits, where, end, x);
#pragma unroll
        for (int k = 7; k >= 0; --k)
            if (clean(x[k]) == best) index = where + k;
    }
    sum *= Weigh(rate, best)(top);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
    index = __reduce_min_sync(kFullMask, index);
    if (lane == 0) {
        ss[warp] = sum;
        si[warp] = index;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float z = 0.0f;
        for (int w = 0; w < kWarps; ++w) {
            z += ss[w];
            index = min(index, si[w]);
        }
        a.stats[blockIdx.x] = make_float4(best, __int_as_float(index), z, 0.0f);
    }
}

// Every block of a row repeats the acceptance (a few values), then races its part of the vocabulary; the block that ends
// last joins them.  Bound by HBM and by the chain around the race (sums, decision, logits, join): 20 us for 84 MB at
// 64 x 131072, with all blocks on the card at once; 24 with a block for every 8192 logits.
template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, sizeof(T) == 2 ? kPickBlocks : kPickBlocks32) verify_pick_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ float sv[32];
    __shared__ int si[32];
    constexpr int kWarps = kVerifyThreads / 32;
    __shared__ float s_best[kWarps], s_z[kWarps];
    __shared__ int s_top[kWarps];
    __shared__ bool s_keep[kWarps], s_last;
    // The statistics kernel lets this one start only after its own wait for what came before, so the caller's inputs are there
    // already: the drafts' values are on their way while it ends.
    const int split = blockIdx.x % a.shares, b = blockIdx.x / a.shares;
    const int n = min(a.num_drafts != nullptr ? a.num_drafts[b] : a.drafts, a.drafts);
    int32_t *out = a.out_tokens + static_cast<int64_t>(b) * (a.drafts + 1);
    if (n < 0) {
        wait_prior_grid();
        release_next_grid();
        if (split == 0) {
            for (int i = threadIdx.x; i <= a.drafts; i += kVerifyThreads) out[i] = -1;
            if (threadIdx.x == 0) a.num_accepted[b] = 0;
        }
        return;
    }
    const float rate = rate_of(a, b);
    const bool greedy = rate == 0.0f;
    const T *row = static_cast<const T *>(a.logits) + b * a.tb;
    const float *noise = a.noise + b * a.nb;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // What the decision on a draft takes beside the sums.
    int token = -1;
    float logit = -INFINITY, q_token = 1.0f, u = 0.0f;
    auto draft = [&](int i) {
        token = -1;
        if (i >= n) return;
        token = a.tokens[b * a.db + i * a.dp];
        u = a.uniform[b * a.ub + i * a.up];
        if (token >= 0 && token < a.vocab) {
            logit = clean(widen(row[i * a.tp + token]));
            if (a.probs != nullptr) q_token = a.probs[b * a.pb + i * a.pp + token];
        }
    };
    draft(warp);
    wait_prior_grid();
    release_next_grid();
    int kept = 0;
    float best, z;
    int first;  // of the largest logits of position `kept`
    for (int i0 = 0;; i0 += kWarps) {  // a warp a position; the last one (n) has no draft and ends the search
        const int i = i0 + warp;
        if (i <= n) {
            if (i0 > 0) draft(i);
            const float4 *st = a.stats + (static_cast<int64_t>(b) * (a.drafts + 1) + i) * a.splits;
            float m = -INFINITY, sum = 0.0f;
            int at = INT32_MAX;
            for (int k = lane; k < a.splits; k += 32) {
                const float4 x = st[k];
                if (x.x > m) {
                    sum *= Weigh(rate, x.x)(m);
                    m = x.x;
                    at = __float_as_int(x.y);
                }
                sum += x.z * Weigh(rate, m)(x.x);
            }
            const float mine = m;
            warp_best(m, at);
            sum *= Weigh(rate, m)(mine);
#pragma unroll
            for (int j = 16; j > 0; j >>= 1) sum += __shfl_xor_sync(kFullMask, sum, j);
            if (lane == 0) {
                bool keep = false;
                if (token >= 0 && token < a.vocab) {
                    float p = greedy && token == at && m > -INFINITY ? 1.0f : 0.0f;
                    if (!greedy && sum > 0.0f) p = Weigh(rate, m)(logit) / sum;
                    keep = u * q_token < p;
                }
                s_best[warp] = m;
                s_z[warp] = sum;
                s_top[warp] = at;
                s_keep[warp] = keep;
            }
        }
        __syncthreads();
        int w = 0;
        while (w < kWarps && i0 + w < n && s_keep[w]) ++w;
        kept = i0 + w;
        if (w < kWarps) {
            best = s_best[w];
            z = s_z[w];
            first = s_top[w];
            break;
        }
        __syncthreads();
    }
    if (split == 0 && threadIdx.x == 0 && kept < n) {
        const int token = a.tokens[b * a.db + kept * a.dp];
        if (token < 0 || token >= a.vocab) count_error(a.err_count);
    }
    float top = 0.0f;  // a score has to be above 0
    int index = INT32_MAX;
    const bool race = !greedy && z > 0.0f;
    if (race) {
        const T *logits = row + kept * a.tp;
        const float *q = kept < n && a.probs != nullptr ? a.probs + b * a.pb + kept * a.pp : nullptr;
        const int sure = kept < n && a.probs == nullptr ? a.tokens[b * a.db + kept * a.dp] : -1;
        // whole vectors where all three rows allow them
        const int before = static_cast<int>(reinterpret_cast<uintptr_t>(logits) % 16 / sizeof(T));
        const int start = split * a.rounds * kShare - before;
        const Weigh weigh(rate, best);
        const float inv_z = 1.0f / z;
        const bool vn = reinterpret_cast<uintptr_t>(noise + start) % 16 == 0;
        const bool vq = q != nullptr && reinterpret_cast<uintptr_t>(q + start) % 16 == 0;
        for (int round = 0; round < a.rounds; ++round) {
#pragma unroll
            for (int j = 0; j < kVectors; ++j) {
                const int v0 = start + (round * kVectors + j) * kStep + threadIdx.x * 8;
                float x[8], w[8], y[8] = {};
                load8(logits, v0, a.vocab, x);
                load8_plain(noise, v0, a.vocab, vn && v0 >= 0, w);
                if (q != nullptr) load8_plain(q, v0, a.vocab, vq && v0 >= 0, y);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float r = fmaf(weigh(clean(x[k])), inv_z, -y[k]);
                    if (v0 + k == sure) r = 0.0f;
                    const float score = r * rcp_approx(w[k]);
                    if (score > top) {  // never so for r <= 0
                        top = score;
                        index = v0 + k;
                    }
                }
            }
        }
        block_best(top, index, sv, si);
        if (threadIdx.x == 0) {
            a.best[static_cast<int64_t>(b) * a.shares + split] = make_float2(top, __int_as_float(index));
            __threadfence();
            s_last = atomicAdd(a.done + b, 1u) == static_cast<unsigned>(a.shares) - 1;
        }
        __syncthreads();
        if (!s_last) return;
        __threadfence();
        top = 0.0f;
        index = INT32_MAX;
        for (int k = threadIdx.x % 32; k < a.shares; k += 32) {
            const float2 x = __ldcg(a.best + static_cast<int64_t>(b) * a.shares + k);
            take_best(top, index, x.x, __float_as_int(x.y));
        }
        warp_best(top, index);
    } else {
        if (split != 0) return;
        if (greedy && best > -INFINITY) index = first;
    }
    for (int i = threadIdx.x; i <= a.drafts; i += kVerifyThreads)
        out[i] = i < kept ? a.tokens[b * a.db + i * a.dp] : i == kept && index != INT32_MAX ? index : -1;
    if (threadIdx.x == 0) a.num_accepted[b] = kept + 1;
}

// Shares of a row: its logits and what is before them up to a 16-byte boundary (see verify_stats_kernel), `before` at most.
int64_t shares_of(int vocab, int64_t share, int before = 7) { return (static_cast<int64_t>(vocab) + before + share - 1) / share; }

// A block of the statistics takes a long share once that still fills the card (8 blocks on each of its 152 SMs): each thread then loads its
// second 4 vectors under the first 4's arithmetic.  Below that, shorter shares spread a row over more SMs.
int stats_share(int64_t rows, int vocab) { return rows * shares_of(vocab, kLongShare) >= 8 * 152 ? kLongShare : kShare; }

// How often a block of the draw takes kShare logits: as often as keeps all rows' blocks on the card at once, since each repeats
// the chain up to the race.
int64_t pick_rounds(int batch, int64_t shares, int resident) {
    const int64_t blocks = std::max<int64_t>(1, resident * 152 / batch);
    return (shares + blocks - 1) / blocks;
}

// Rows of logits, or -1 where their blocks would pass a grid's limit.
int64_t logit_rows(int batch, int drafts, int vocab) {
    const int64_t positions = static_cast<int64_t>(drafts) + 1, shares = shares_of(vocab, kShare);
    return vocab > (1 << 30) || positions > 0x7fffffff / batch || batch * positions > 0x7fffffff / shares ? -1 : batch * positions;
}

int64_t stats_blocks(int64_t rows, int vocab) {
    return rows * shares_of(vocab, stats_share(rows, vocab));
}

template <typename T>
int launch_verify(const VerifyArgs &a, cudaStream_t stream) {
    const int status = launch_pdl(verify_stats_kernel<T>, dim3(static_cast<unsigned>(a.batch * (a.drafts + 1)) * a.splits),
                                  dim3(kVerifyThreads), 0, stream, a);
    if (status != CCV_OK) return status;
    return launch_pdl(verify_pick_kernel<T>, dim3(static_cast<unsigned>(a.batch) * a.shares), dim3(kVerifyThreads), 0, stream, a);
}

}  // namespace
}  // namespace ccv

extern "C" int64_t spec_verify_workspace(int batch, int drafts, int vocab) {
    if (batch <= 0 || drafts < 0 || vocab <= 0) return 0;
    const int64_t rows = ccv::logit_rows(batch, drafts, vocab);
    if (rows < 0) return 0;
    return ccv::stats_blocks(rows, vocab) * 16 + batch * ccv::shares_of(vocab, ccv::kShare) * 8 + static_cast<int64_t>(batch) * 4;
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
    const int64_t rows = vocab > 0 ? logit_rows(batch, drafts, vocab) : -1;
    if (rows < 0) return CCV_ERR_SIZE;
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
    const int share = stats_share(rows, vocab);
    const int size = logits_fp32 ? 4 : 2;
    const int before = aligned16(target_logits) && t_stride_b * size % 16 == 0 && t_stride_pos * size % 16 == 0 ? 0 : 7;
    const int64_t rounds = pick_rounds(batch, shares_of(vocab, kShare, before), logits_fp32 ? kPickBlocks32 : kPickBlocks);
    const int64_t shares = shares_of(vocab, rounds * kShare, before), splits = shares_of(vocab, share, before);
    uint8_t *space = static_cast<uint8_t *>(workspace), *best = space + stats_blocks(rows, vocab) * 16;
    const VerifyArgs a{target_logits, t_stride_b, t_stride_pos, draft_tokens, d_stride_b, d_stride_pos, draft_probs, p_stride_b,
                       p_stride_pos, num_drafts, temperature, uniform, u_stride_b, u_stride_pos, noise, n_stride_b, out_tokens,
                       num_accepted, batch, drafts, vocab, share, static_cast<int>(splits),
                       static_cast<int>(shares), static_cast<int>(rounds), reinterpret_cast<float4 *>(space), reinterpret_cast<float2 *>(best),
                       reinterpret_cast<unsigned *>(best + batch * shares * 8), err_count};
    return logits_fp32 ? launch_verify<float>(a, stream) : launch_verify<uint16_t>(a, stream);
}
