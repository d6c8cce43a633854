// Adjustment of logits before tokens are chosen: penalties for what a request has said, a bias list, a grammar's mask.
//
// A block has a share of one row's vocabulary for all of the row's positions.  It counts the share's tokens in the history into
// a table in shared memory (a word a token: how often it was said, whether it is in the prompt, whether it has a bias) and notes
// them in a bitmap, then goes through the positions, adding the draft that each one follows, eight logits at a time.  Where no
// lane of a warp has more than two bits they are stored once more, one by one; else all of the warp's logits go through the
// penalties' arithmetic, which has no branches.  A row's history is read by all of its blocks, from L2 after the first.
// 64 rows of 5 positions of 131072 bf16 logits with histories of 4000 tokens and a mask take 55 us (3.1 TB/s of what has to be
// moved): 9 for the histories, 12 for the adjustments, the rest the latency of 1024 blocks at 4 an SM.  A share of 8192 tokens is
// a table of 32 KB; with 4096 every history is read twice as often, and it took no less.  256 rows of one position, histories of
// 3000: bf16 44 us (floor 20), fp32 78 (40); with a mask 53 and 91, in place 54 and 98.  Every block reads its row's history: 64 x 5
// positions with 32768 tokens take 74 us, with 100000 128.  A bias list is searched for each of its tokens: 64 rows of fp32 with 30
// entries take 21 us, with 300 68, with 3000 1500.
//
// In place and without a mask only the tokens that were seen matter.  Where they are few enough for a hash table in shared memory
// a block takes a whole row: it counts the history there and goes through the table's slots at each position.
// 256 rows of 131072 fp32 logits with up to 4000 tokens take 21 us (by shares 61): two waves of a block's latency.  It is the
// pool's width that the table has to hold, since lengths are not known to the host: from 12289 tokens a line on it is shares.
#include <algorithm>

#include "ccv_common.cuh"
#include "ccv_logits.h"

namespace ccv {
namespace {

constexpr int kLogitsThreads = 256;
constexpr int kShare = 8192;  // tokens of a block's table: 32 KB
constexpr int kAhead = 8;     // history tokens that a thread has in flight
constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

struct Penalties {
    float repetition, inverse, frequency, presence;  // the quotient is a product with 1 / repetition: 2 units of fp32 off at most
    const int32_t *ids;  // the row's bias list
    const float *bias;
    int size;
};

// One logit's penalties and bias.
__device__ __forceinline__ float adjust(float x, uint32_t entry, int token, const Penalties &p) {
    const float n = static_cast<float>(entry & kCount);
    x = (entry & (kPrompt | kCount)) != 0u ? x * (x > 0.0f ? p.inverse : p.repetition) : x;
    x = n > 0.0f ? fmaf(-p.frequency, n, x) - p.presence : x;
    if (entry & kBiased) {
        float sum = 0.0f;
        for (int i = 0; i < p.size; ++i)
            if (p.ids[i] == token) sum += p.bias[i];
        x += sum;
    }
    return x;
}

// Eight logits as they are in memory: 16 bytes of bf16, or 32 of fp32.
template <bool F32> struct Eight;
template <> struct Eight<false> {
    uint4 v;
    __device__ __forceinline__ void load(const void *p, int64_t i) { v = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i)); }
    __device__ __forceinline__ void store(void *p, int64_t i) const { __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i), v); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        Raw<8> r;
        r.v = v;
        r.to_float(f);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        Raw<8> r;
        r.from_float(f);
        v = r.v;
    }
    __device__ __forceinline__ float one(int i) const { return bf16_bits(Raw<8>{v}.elem(i)); }
    // -inf where a bit of `may` is not set
    __device__ __forceinline__ void mask(uint32_t may) {
        const auto half = [&](int i, uint32_t w) {
            const uint32_t keep = ((may >> (2 * i)) & 1u) * 0xffffu + ((may >> (2 * i + 1)) & 1u) * 0xffff0000u;
            return (w & keep) | (0xff80ff80u & ~keep);
        };
        v = make_uint4(half(0, v.x), half(1, v.y), half(2, v.z), half(3, v.w));
    }
};
template <> struct Eight<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        a = __ldcs(q);
        b = __ldcs(q + 1);
    }
    __device__ __forceinline__ void store(void *p, int64_t i) const {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        __stcs(q, a);
        __stcs(q + 1, b);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ float one(int i) const {
        const float4 h = i < 4 ? a : b;
        return (i & 3) == 0 ? h.x : (i & 3) == 1 ? h.y : (i & 3) == 2 ? h.z : h.w;
    }
    __device__ __forceinline__ void mask(uint32_t may) {
        const auto one = [&](int i, float x) { return ((may >> i) & 1u) != 0u ? x : -INFINITY; };
        a = make_float4(one(0, a.x), one(1, a.y), one(2, a.z), one(3, a.w));
        b = make_float4(one(4, b.x), one(5, b.y), one(6, b.z), one(7, b.w));
    }
};
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
// Elements from address p on to the next 16-byte boundary.
template <bool F32>
__device__ __forceinline__ int to_boundary(const void *p, int64_t i) {
    constexpr int kSize = F32 ? 4 : 2;
    return static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) + i * kSize) % 16) % 16 / kSize);
}

// IN, OUT: fp32 logits and results.  PLACE: out is logits.
template <bool IN, bool OUT, bool PLACE>
__global__ void __launch_bounds__(kLogitsThreads, IN ? 1 : 4) logits_kernel(const __grid_constant__ ccv_logits_args a, int shares, int *err_count) {
    __shared__ __align__(16) uint32_t table[kShare];
    __shared__ uint32_t touched[kShare / 32 + 1];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / shares, first = (blockIdx.x % shares) * kShare, n = min(kShare, a.vocab - first);
    for (int i = tid; i < kShare / 4; i += kLogitsThreads) reinterpret_cast<uint4 *>(table)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = tid; i < kShare / 32 + 1; i += kLogitsThreads) touched[i] = 0u;
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
    const auto note = [&](int token, uint32_t flag) {  // flag 0: said
        odd |= token >= a.vocab;
        const unsigned at = static_cast<unsigned>(token) - static_cast<unsigned>(first);
        if (at >= static_cast<unsigned>(n)) return;
        if (flag == 0u) atomicAdd(&table[at], 1u);
        else atomicOr(&table[at], flag);
        atomicOr(&touched[at / 32], 1u << (at % 32));
    };
    if (a.history != nullptr) {
        int told = a.history_lengths[line], prompt = a.prompt_lengths != nullptr ? a.prompt_lengths[line] : 0;
        odd |= told < 0 || told > a.history_size || prompt < 0 || prompt > a.history_size;
        told = min(max(told, 0), a.history_size);
        prompt = min(max(prompt, 0), a.history_size);
        const int32_t *ids = a.history + line * a.h_stride_line;
        for (int i0 = tid; i0 < told; i0 += kLogitsThreads * kAhead) {
            int token[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) token[j] = i0 + j * kLogitsThreads < told ? __ldg(ids + i0 + j * kLogitsThreads) : -1;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) note(token[j], i0 + j * kLogitsThreads < prompt ? kPrompt : 0u);
        }
    }
    const float repetition = a.repetition != nullptr ? a.repetition[b] : 1.0f;
    const Penalties p{repetition,
                      1.0f / repetition,
                      a.frequency != nullptr ? a.frequency[b] : 0.0f,
                      a.presence != nullptr ? a.presence[b] : 0.0f,
                      a.bias_ids + b * a.b_stride_b,
                      a.bias + b * a.b_stride_b,
                      a.bias_size};
    for (int i = tid; i < p.size; i += kLogitsThreads) note(p.ids[i], kBiased);

    for (int pos = 0; pos < a.num_positions; ++pos) {
        if (pos > 0 && a.draft_tokens != nullptr) {
            __syncthreads();  // the last position's threads are done with the table
            if (tid == 0) note(a.draft_tokens[b * a.d_stride_b + (pos - 1) * a.d_stride_pos], 0u);
        }
        const int64_t from = b * a.l_stride_b + pos * a.l_stride_pos + first, to = b * a.o_stride_b + pos * a.o_stride_pos + first;
        const int32_t *mask = a.mask != nullptr ? a.mask + b * a.m_stride_b + pos * a.m_stride_pos + first / 32 : nullptr;
        const int words = (n + 31) / 32;
        // Elements up to 16 bytes' boundary and past the last vector go one by one; all do where input and output never meet one.
        int head = to_boundary<IN>(a.logits, from);
        if (to_boundary<OUT>(a.out, to + head) != 0) head = n;
        head = min(head, n);
        const int vectors = (n - head) / 8, rest = n - head - vectors * 8;
        constexpr int kVectors = kShare / 8 / kLogitsThreads;
        if (!PLACE || mask != nullptr) {
            uint32_t may[kVectors];  // eight bits each
            Eight<IN> x[PLACE ? 1 : kVectors];
#pragma unroll
            for (int j = 0; j < kVectors; ++j) {
                const int at = head + (tid + j * kLogitsThreads) * 8;
                may[j] = 0xffu;
                if (tid + j * kLogitsThreads >= vectors) continue;
                if constexpr (!PLACE) x[j].load(a.logits, from + at);
                if (mask != nullptr)
                    may[j] = __funnelshift_r(__ldg(mask + at / 32), at / 32 + 1 < words ? __ldg(mask + at / 32 + 1) : 0, at % 32) & 0xffu;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kVectors; ++j) {
                const int at = head + (tid + j * kLogitsThreads) * 8;
                const bool mine = tid + j * kLogitsThreads < vectors;
                const uint32_t bits = mine ? __funnelshift_r(touched[at / 32], touched[at / 32 + 1], at % 32) & may[j] : 0u;
                Eight<IN> in;
                if constexpr (PLACE) {
                    if (mine && may[j] != 0u && (may[j] != 0xffu || bits != 0u)) in.load(a.logits, from + at);
                } else {
                    in = x[j];
                }
                const bool many = __any_sync(kFullMask, __popc(bits) > 2);
                if (!mine || (PLACE && may[j] == 0xffu && bits == 0u)) continue;
                Eight<OUT> result;
                if (many || IN != OUT) {
                    float f[8];
                    in.get(f);
                    if (many) {
                        uint32_t entry[8];
                        if (head % 4 == 0) {
                            const uint4 e0 = *reinterpret_cast<const uint4 *>(&table[at]), e1 = *reinterpret_cast<const uint4 *>(&table[at + 4]);
                            entry[0] = e0.x; entry[1] = e0.y; entry[2] = e0.z; entry[3] = e0.w;
                            entry[4] = e1.x; entry[5] = e1.y; entry[6] = e1.z; entry[7] = e1.w;
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) entry[i] = table[at + i];
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = adjust(f[i], entry[i], first + at + i, p);
                    }
                    result.set(f);
                } else if constexpr (IN == OUT) {
                    result = in;
                }
                if (mask != nullptr) result.mask(may[j]);
                result.store(a.out, to + at);
                if (many) continue;
                for (uint32_t left = bits; left != 0u; left &= left - 1u) {
                    const int i = __ffs(left) - 1;
                    store_logit<OUT>(a.out, to + at + i, adjust(in.one(i), table[at + i], first + at + i, p));
                }
            }
            for (int k = tid; k < head + rest; k += kLogitsThreads) {
                const int at = k < head ? k : k + vectors * 8;
                const uint32_t entry = table[at];
                const bool can = mask == nullptr || ((static_cast<uint32_t>(mask[at / 32]) >> (at % 32)) & 1u) != 0;
                if (PLACE && can && entry == 0u) continue;
                store_logit<OUT>(a.out, to + at, can ? adjust(load_logit<IN>(a.logits, from + at), entry, first + at, p) : -INFINITY);
            }
        } else {
            __syncthreads();
            for (int word = tid; word < words; word += kLogitsThreads)
                for (uint32_t bits = touched[word]; bits != 0u;) {
                    int at[4];
                    float f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        at[i] = bits != 0u ? word * 32 + __ffs(bits) - 1 : -1;
                        bits &= bits - 1u;
                        f[i] = at[i] >= 0 ? load_logit<IN>(a.logits, from + at[i]) : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (at[i] >= 0) store_logit<OUT>(a.out, to + at[i], adjust(f[i], table[at[i]], first + at[i], p));
                }
        }
    }
    if (__syncthreads_or(odd) && tid == 0) count_error(err_count);
}

constexpr int kMaxSlots = 16384;
constexpr uint32_t kNone = 0xffffffffu;

// Slots of the hash table: a quarter stays empty even if all of a row's tokens differ; 0 where they are too many for it.
int hash_slots(const ccv_logits_args &a) {
    const int64_t tokens = static_cast<int64_t>(a.history != nullptr ? a.history_size : 0) + (a.draft_tokens != nullptr ? a.num_positions - 1 : 0) + a.bias_size;
    int slots = 1024;
    while (3 * static_cast<int64_t>(slots) < 4 * tokens && slots <= kMaxSlots) slots *= 2;
    return slots <= kMaxSlots ? slots : 0;
}
size_t hash_bytes(int slots) { return static_cast<size_t>(slots) * 8; }  // key and entry

// A block a row, in place and without a mask.  slots: a power of two, at most three quarters of them used.
template <bool F32, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logits_row_kernel(const __grid_constant__ ccv_logits_args a, int slots, int parts, int *err_count) {
    extern __shared__ __align__(16) uint32_t hash[];
    uint32_t *key = hash, *entry = hash + slots;
    const int tid = threadIdx.x, b = blockIdx.x / parts, part = blockIdx.x % parts, shift = 32 - (31 - __clz(slots));
    for (int i = tid; i < slots / 4; i += THREADS) {
        reinterpret_cast<uint4 *>(key)[i] = make_uint4(kNone, kNone, kNone, kNone);
        reinterpret_cast<uint4 *>(entry)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    wait_prior_grid();
    release_next_grid();
    const int line = a.history_indices != nullptr ? a.history_indices[b] : b;
    if (a.history_indices != nullptr && line == a.pad_slot_id) return;
    if (a.history != nullptr && (line < 0 || line >= a.num_lines)) {
        if (tid == 0 && part == 0) count_error(err_count);
        return;
    }
    __syncthreads();
    bool odd = false;
    const auto note = [&](int token, uint32_t flag) {  // flag 0: said
        odd |= token >= a.vocab;
        if (static_cast<unsigned>(token) >= static_cast<unsigned>(a.vocab)) return;
        uint32_t at = (static_cast<uint32_t>(token) * 2654435769u) >> shift;  // multiplicative hashing (Knuth)
        for (;; at = (at + 1) & (slots - 1)) {  // some slots stay empty, so it ends
            const uint32_t old = atomicCAS(&key[at], kNone, static_cast<uint32_t>(token));
            if (old == kNone || old == static_cast<uint32_t>(token)) break;
        }
        if (flag == 0u) atomicAdd(&entry[at], 1u);
        else atomicOr(&entry[at], flag);
    };
    if (a.history != nullptr) {
        int told = a.history_lengths[line], prompt = a.prompt_lengths != nullptr ? a.prompt_lengths[line] : 0;
        odd |= told < 0 || told > a.history_size || prompt < 0 || prompt > a.history_size;
        told = min(max(told, 0), a.history_size);
        prompt = min(max(prompt, 0), a.history_size);
        const int32_t *ids = a.history + line * a.h_stride_line;
        for (int i0 = tid; i0 < told; i0 += THREADS * kAhead) {
            int token[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) token[j] = i0 + j * THREADS < told ? __ldg(ids + i0 + j * THREADS) : -1;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) note(token[j], i0 + j * THREADS < prompt ? kPrompt : 0u);
        }
    }
    const float repetition = a.repetition != nullptr ? a.repetition[b] : 1.0f;
    const Penalties p{repetition,
                      1.0f / repetition,
                      a.frequency != nullptr ? a.frequency[b] : 0.0f,
                      a.presence != nullptr ? a.presence[b] : 0.0f,
                      a.bias_ids + b * a.b_stride_b,
                      a.bias + b * a.b_stride_b,
                      a.bias_size};
    for (int i = tid; i < p.size; i += THREADS) note(p.ids[i], kBiased);
    // The part's positions, and the drafts before them; the last part has seen them all.
    const int first_pos = parts > 1 ? part : 0, end_pos = parts > 1 ? part + 1 : a.num_positions;
    if (a.draft_tokens != nullptr)
        for (int i = tid; i < first_pos; i += THREADS) note(a.draft_tokens[b * a.d_stride_b + i * a.d_stride_pos], 0u);
    for (int pos = first_pos; pos < end_pos; ++pos) {
        if (pos > first_pos && a.draft_tokens != nullptr) {
            __syncthreads();  // the last position's threads are done with the table
            if (tid == 0) note(a.draft_tokens[b * a.d_stride_b + (pos - 1) * a.d_stride_pos], 0u);
        }
        __syncthreads();
        const int64_t from = b * a.l_stride_b + pos * a.l_stride_pos;
        // eight slots a thread at once: their logits' loads are in flight together
        for (int i0 = tid; i0 < slots; i0 += THREADS * 8) {
            uint32_t token[8];
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = i0 + j * THREADS;
                token[j] = i < slots ? key[i] : kNone;
                f[j] = token[j] != kNone ? load_logit<F32>(a.logits, from + token[j]) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (token[j] != kNone) store_logit<F32>(a.out, from + token[j], adjust(f[j], entry[i0 + j * THREADS], static_cast<int>(token[j]), p));
        }
    }
    if (__syncthreads_or(odd) && tid == 0 && part == parts - 1) count_error(err_count);
}

template <bool F32, int THREADS>
int launch_row_blocks(const ccv_logits_args &a, int slots, int *err_count, cudaStream_t stream) {
    int dev = 0;
    current_device_sms(&dev);
    cudaError_t err;
    if (resident_blocks<logits_row_kernel<F32, THREADS>>(THREADS, hash_bytes(kMaxSlots), dev, &err) == 0) return static_cast<int>(err);
    // A block a position where that takes less time by waves of blocks: a table takes about as long as a position, and a block a row
    // makes one table for n positions.  5 positions with 4000 tokens: 8 rows 10 us, in a block a row 23; 30 rows 11 and 24; 64 rows
    // in a block a row 30; with 900 tokens 64 rows 9 and 12.
    const int64_t room = 152 * (1024 / THREADS), n = a.num_positions;
    const auto waves = [&](int64_t blocks) { return (blocks + room - 1) / room; };
    const int parts = 2 * waves(a.batch * n) < waves(a.batch) * (1 + n) && a.batch * n < (1 << 30) ? static_cast<int>(n) : 1;
    return launch_pdl(logits_row_kernel<F32, THREADS>, dim3(static_cast<unsigned>(a.batch) * parts), dim3(THREADS), hash_bytes(slots), stream, a,
                      slots, parts, err_count);
}

// Two blocks of 512 threads fit an SM, and up to 4096 slots are little work: 256 rows of 131072 logits with 300, 900 and 2000
// tokens take 4.7, 7.0 and 11 us so, with 1024 threads 7.9, 9.9 and 14; with 4000 (8192 slots) 25 and 21.
template <bool F32>
int launch_rows(const ccv_logits_args &a, int slots, int *err_count, cudaStream_t stream) {
    return slots <= 4096 ? launch_row_blocks<F32, 512>(a, slots, err_count, stream) : launch_row_blocks<F32, 1024>(a, slots, err_count, stream);
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
    // The output's rows lie apart: positions inside batch rows, or the other way round.
    const int64_t ob = b > 1 ? a->o_stride_b : 0, op = n > 1 ? a->o_stride_pos : 0;
    const bool inside = (n == 1 || op >= v) && (b == 1 || ob >= (n - 1) * op + v);
    const bool around = (b == 1 || ob >= v) && (n == 1 || op >= (b - 1) * ob + v);
    return inside || around ? CCV_OK : CCV_ERR_STRIDE;
}

}  // namespace
}  // namespace ccv

extern "C" int logits_process(const ccv_logits_args *args, int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    const int status = check(args);
    if (status != CCV_OK) return status;
    if (args->batch == 0 || args->num_positions == 0 || args->vocab == 0) return CCV_OK;
    const bool place = args->out == args->logits;
    if (const int slots = place && args->mask == nullptr ? hash_slots(*args) : 0)
        return args->logits_fp32 ? launch_rows<true>(*args, slots, err_count, stream) : launch_rows<false>(*args, slots, err_count, stream);
    const int shares = (args->vocab + kShare - 1) / kShare;
    const int64_t blocks = static_cast<int64_t>(shares) * args->batch;
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kLogitsThreads);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, block, 0, stream, *args, shares, err_count); };
    if (args->logits_fp32) {
        if (place) return go(logits_kernel<true, true, true>);
        return args->out_fp32 ? go(logits_kernel<true, true, false>) : go(logits_kernel<true, false, false>);
    }
    if (place) return go(logits_kernel<false, false, true>);
    return args->out_fp32 ? go(logits_kernel<false, true, false>) : go(logits_kernel<false, false, false>);
}
