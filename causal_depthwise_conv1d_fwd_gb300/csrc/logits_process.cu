// Adjustment of logits before tokens are chosen: penalties for what a request has said, a bias list, a grammar's mask.
//
// A block has a share of one row's vocabulary for all of the row's positions.  It counts the share's tokens in the history into
// a table in shared memory (a word a token: how often it was said, whether it is in the prompt, whether it has a bias), then
// goes through the positions, adding the draft that each one follows.  A row's history is read by all of its blocks, from L2
// after the first.
#include "ccv_common.cuh"
#include "ccv_logits.h"

namespace ccv {
namespace {

constexpr int kLogitsThreads = 256;
constexpr int kShare = 8192;  // tokens of a block's table: 32 KB
constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

struct Penalties {
    float repetition, frequency, presence;
};

// One logit's penalties and bias.  `bias` are the row's entries.
__device__ __forceinline__ float adjust(float x, uint32_t entry, int token, const Penalties &p, const int32_t *ids, const float *bias,
                                        int size) {
    const float n = static_cast<float>(entry & kCount);
    if ((entry & (kPrompt | kCount)) != 0) {
        x = x > 0.0f ? x / p.repetition : x * p.repetition;
        if (n > 0.0f) x = x - p.frequency * n - p.presence;
    }
    if (entry & kBiased) {
        float sum = 0.0f;
        for (int i = 0; i < size; ++i)
            if (ids[i] == token) sum += bias[i];
        x += sum;
    }
    return x;
}

template <bool F32>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (F32) return static_cast<const float *>(p)[i];
    else return bf16_bits(static_cast<const uint16_t *>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store_logit(void *p, int64_t i, float x) {
    if constexpr (F32) static_cast<float *>(p)[i] = x;
    else static_cast<uint16_t *>(p)[i] = round_bf16(x);
}

// IN, OUT: fp32 logits and results.  PLACE: out is logits.
template <bool IN, bool OUT, bool PLACE>
__global__ void __launch_bounds__(kLogitsThreads) logits_kernel(const __grid_constant__ ccv_logits_args a, int shares, int *err_count) {
    __shared__ uint32_t table[kShare];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / shares, first = (blockIdx.x % shares) * kShare, n = min(kShare, a.vocab - first);
    for (int i = tid; i < kShare; i += kLogitsThreads) table[i] = 0;
    wait_prior_grid();
    release_next_grid();
    const int line = a.history_indices != nullptr ? a.history_indices[b] : b;
    if (a.history_indices != nullptr && line == a.pad_slot_id) return;
    if (a.history != nullptr && (line < 0 || line >= a.num_lines)) {
        if (tid == 0) count_error(err_count);
        return;
    }
    __syncthreads();
    bool odd = false;
    auto add = [&](int token, bool said) {
        odd |= token >= a.vocab;
        const unsigned at = static_cast<unsigned>(token - first);
        if (token >= 0 && at < static_cast<unsigned>(n)) {
            if (said) atomicAdd(&table[at], 1u);
            else atomicOr(&table[at], kPrompt);
        }
    };
    if (a.history != nullptr) {
        int told = a.history_lengths[line], prompt = a.prompt_lengths != nullptr ? a.prompt_lengths[line] : 0;
        odd |= told < 0 || told > a.history_size || prompt < 0 || prompt > a.history_size;
        told = min(max(told, 0), a.history_size);
        prompt = min(max(prompt, 0), a.history_size);
        const int32_t *ids = a.history + line * a.h_stride_line;
        for (int i = tid; i < told; i += kLogitsThreads) add(ids[i], i >= prompt);
    }
    const int32_t *bias_ids = a.bias_ids + b * a.b_stride_b;
    const float *bias = a.bias + b * a.b_stride_b;
    for (int i = tid; i < a.bias_size; i += kLogitsThreads) {
        const int token = bias_ids[i];
        odd |= token >= a.vocab;
        const unsigned at = static_cast<unsigned>(token - first);
        if (token >= 0 && at < static_cast<unsigned>(n)) atomicOr(&table[at], kBiased);
    }
    const Penalties p{a.repetition != nullptr ? a.repetition[b] : 1.0f, a.frequency != nullptr ? a.frequency[b] : 0.0f,
                      a.presence != nullptr ? a.presence[b] : 0.0f};
    for (int pos = 0; pos < a.num_positions; ++pos) {
        if (pos > 0 && a.draft_tokens != nullptr && tid == 0) add(a.draft_tokens[b * a.d_stride_b + (pos - 1) * a.d_stride_pos], true);
        __syncthreads();
        const int64_t from = b * a.l_stride_b + pos * a.l_stride_pos + first, to = b * a.o_stride_b + pos * a.o_stride_pos + first;
        const int32_t *mask = a.mask != nullptr ? a.mask + b * a.m_stride_b + pos * a.m_stride_pos + first / 32 : nullptr;
        for (int i = tid; i < n; i += kLogitsThreads) {
            const uint32_t entry = table[i];
            const bool may = mask == nullptr || ((static_cast<uint32_t>(mask[i / 32]) >> (i & 31)) & 1u) != 0;
            if (PLACE && may && entry == 0) continue;
            float x = -INFINITY;
            if (may) x = adjust(load_logit<IN>(a.logits, from + i), entry, first + i, p, bias_ids, bias, a.bias_size);
            store_logit<OUT>(a.out, to + i, x);
        }
        __syncthreads();
    }
    if (odd) count_error(err_count);
}

int check(const ccv_logits_args *a) {
    if (a == nullptr) return CCV_ERR_NULL_POINTER;
    if (a->batch < 0 || a->num_positions < 0 || a->vocab < 0 || a->vocab > (1 << 30) || a->num_lines < 0 || a->history_size < 0 ||
        a->bias_size < 0 || a->history_size >= (1 << 29) || a->num_positions >= (1 << 29))
        return CCV_ERR_SIZE;
    for (int64_t s : {a->l_stride_b, a->l_stride_pos, a->o_stride_b, a->o_stride_pos, a->h_stride_line, a->d_stride_b, a->d_stride_pos,
                      a->b_stride_b, a->m_stride_b, a->m_stride_pos})
        if (s < 0) return CCV_ERR_STRIDE;
    if (a->batch == 0 || a->num_positions == 0 || a->vocab == 0) return CCV_OK;
    if (a->logits == nullptr || a->out == nullptr) return CCV_ERR_NULL_POINTER;
    if (a->history != nullptr && a->history_lengths == nullptr) return CCV_ERR_NULL_POINTER;
    if (a->bias_size > 0 && (a->bias_ids == nullptr || a->bias == nullptr)) return CCV_ERR_NULL_POINTER;
    auto range = [](const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int size) {
        const uintptr_t base = reinterpret_cast<uintptr_t>(p);
        return Extent{base, base + static_cast<uintptr_t>((n0 - 1) * s0 + (n1 - 1) * s1 + n2) * size - 1};
    };
    const int64_t b = a->batch, n = a->num_positions, v = a->vocab;
    const Extent out = range(a->out, b, a->o_stride_b, n, a->o_stride_pos, v, a->out_fp32 ? 4 : 2);
    const bool place = a->out == a->logits && a->out_fp32 == a->logits_fp32 && a->o_stride_b == a->l_stride_b && a->o_stride_pos == a->l_stride_pos;
    if (!place && overlaps(out, range(a->logits, b, a->l_stride_b, n, a->l_stride_pos, v, a->logits_fp32 ? 4 : 2))) return CCV_ERR_ALIAS;
    auto bad = [&](const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2) {
        return p != nullptr && n0 > 0 && n1 > 0 && n2 > 0 && overlaps(out, range(p, n0, s0, n1, s1, n2, 4));
    };
    if (bad(a->history, a->num_lines, a->h_stride_line, 1, 0, a->history_size) || bad(a->history_indices, 1, 0, 1, 0, b) ||
        bad(a->history_lengths, 1, 0, 1, 0, a->num_lines) || bad(a->prompt_lengths, 1, 0, 1, 0, a->num_lines) ||
        bad(a->draft_tokens, b, a->d_stride_b, n - 1, a->d_stride_pos, 1) || bad(a->repetition, 1, 0, 1, 0, b) ||
        bad(a->frequency, 1, 0, 1, 0, b) || bad(a->presence, 1, 0, 1, 0, b) || bad(a->bias_ids, b, a->b_stride_b, 1, 0, a->bias_size) ||
        bad(a->bias, b, a->b_stride_b, 1, 0, a->bias_size) || bad(a->mask, b, a->m_stride_b, n, a->m_stride_pos, (v + 31) / 32))
        return CCV_ERR_ALIAS;
    return CCV_OK;
}

}  // namespace
}  // namespace ccv

extern "C" int logits_process(const ccv_logits_args *args, int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    const int status = check(args);
    if (status != CCV_OK) return status;
    if (args->batch == 0 || args->num_positions == 0 || args->vocab == 0) return CCV_OK;
    const int shares = (args->vocab + kShare - 1) / kShare;
    const int64_t blocks = static_cast<int64_t>(shares) * args->batch;
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kLogitsThreads);
    const bool place = args->out == args->logits;
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, stream, *args, shares, err_count); };
    if (args->logits_fp32) {
        if (place) return go(logits_kernel<true, true, true>);
        return args->out_fp32 ? go(logits_kernel<true, true, false>) : go(logits_kernel<true, false, false>);
    }
    if (place) return go(logits_kernel<false, false, true>);
    return args->out_fp32 ? go(logits_kernel<false, true, false>) : go(logits_kernel<false, false, false>);
}
