// Selective state space scan over varlen sequences (prefill), chunked form on the tensor cores, for one decay a head.
//
// A chunk holds Q = 128 tokens.  With d_j the step of token j and G the running sum of d A inside the chunk, unrolling the
// recurrence gives, for a head's x (tokens, 64), B and C (tokens, 128) and state S (128, 64) at the chunk's start,
//     y_i = e^{G_i} C_i S + sum_{j <= i} M_ij x_j,   M_ij = (C_i . B_j) e^{G_i - G_j} d_j
//     S  <- e^{G_Q} S + sum_j B_j^T (e^{G_Q - G_j} d_j x_j)
// and C B^T is the same for all heads of a group.  Nothing but S is sequential, and S only by its own multiply-add, so all
// products of a chunk run beside those of its neighbours.  A block has a head of one sequence (or segment) and goes through its
// chunks with four warpgroups that all run the same code on a quarter each:
//   the state in registers (thread n has 16 channels of row n), its parts to shared memory for C S, and its multiply-add;
//   the weighted tokens' parts for the state's sum; M from C B^T (tensor memory to tensor memory), 32 of its columns; and the
//   outputs, 16 channels.
// Three more warps copy tiles, sum the steps, and issue the products.  Heads wider than 64 are cut into panels of 64.
//
// What bounds it: 700 instructions a warp and chunk, on four warps a scheduler (46 % of the issue slots while a block runs); no warp
// waits for a product any more.  4 x 4096 tokens of 128 heads with 128 states take 360 us, 0.30 of the tensor cores' cycles, where
// the bytes take 96; 11027 tokens of 32 heads in segments 122 (15); 232 tokens in 4 prompts 11.  On the way here, still with two
// parts of the weighted tokens: a role a warpgroup took 1097 us (the hot instructions were twice as many and missed the instruction
// cache), two heads a block 424 (registers), one with the copies and the steps in one warp 396, with a barrier for every hand-over
// 383, without either 346.  Three parts with two stages of x and of B took 398, since x came late.
//
// Precision.  What is not bf16 from the start enters the tensor cores in bf16 parts; the other factors, x, B and C, are exact.  The
// weighted tokens, which make the state, have three parts, all 24 bits: with two the state is 2.6e-6 of itself off, with three
// 2e-7, as much as the steps are off (the forms that multiply it by a decay a token are 1e-6 off after 1000).  M and the state in C S reach the outputs alone, which are rounded to 8 bits, and have two parts
// (2^-17 of each term).  Sums and the state are fp32: the tensor cores' accumulators within a chunk, a multiply-add from chunk to
// chunk.  Smaller parts are added first, since the tensor cores' sums truncate.  G is summed in pairs of floats, and so are its
// differences.
//
// What is not finite.  A sum over a chunk takes zeros for the tokens after its own, and 0 * NaN is NaN.  So an x that is not
// finite is left out of the products, and its channel is NaN from that token on, the final state too; a step that is not
// finite, or whose rate is NaN, makes M's rows from its own on, and the state, NaN by itself; so do B and C, whose products are
// masked and not multiplied by zero.  Rows of the last tile that belong to the next sequence are zeroed.
#include <climits>
#include <cstdlib>
#include <cstring>

#include "ccv_varlen.cuh"
#include "ssm_fwd.cuh"

namespace ccv {
namespace {

constexpr int Q = 128;              // tokens of a chunk
constexpr int kTile = Q * 128;      // bytes of 128 rows of 64 bf16 values
constexpr int kCompute = 16;  // warps that compute; the others:
constexpr int kCopyWarp = kCompute, kStepWarp = kCompute + 1, kIssueWarp = kCompute + 2;
constexpr int kThreads = (kCompute + 3) * 32;
// Columns of tensor memory: C B^T; M in two halves of 64 tokens, each in two parts; M x; C S; the sum for the state.
constexpr uint32_t kColCB = 0, kColM = 128, kColMX = 256, kColCS = 320, kColSum = 448;  // C S twice
constexpr int kStateFloats = 128 * 64;  // of a head's panel in the workspace

struct Maps {
    CUtensorMap x, b, c;
};

struct Gates {  // of a chunk's tokens: G log2(e) as a pair of floats, the steps, and e^{G_Q - G_j} d_j
    float hi[Q], lo[Q], d[Q], weight[Q];
};

struct Smem {
    uint8_t x[3][kTile];        // stage; the outputs are written over it
    uint8_t b[2][kTile];        // panel of 64 states
    uint8_t c[2][kTile];        // panel
    uint8_t w[3][kTile];        // part: weighted tokens
    uint8_t s[2][kTile];        // part: the state
    Gates gates[2];             // stage
    float since[4][Q];          // 32 rows of M: G of the tokens up to them, counted from the rows' first
    // Whoever waits for a chunk's last products has all of what it made for the chunk free again, and one warp issues all products
    // in order: what is not made ahead needs no barrier for its way back.
    uint64_t in_full[3], x_free[3], b_full[2], b_free[2], c_full, c_free, gates_free[2];  // in: x and the steps
    uint64_t parts_full, m_full, cb_full, sum_full, mx_full, drain;            // parts: of the weighted tokens and the state
    int first_bad[64];          // channel: the first of the block's tokens whose x is not finite
    int any_bad;
    int seq, start, end, abort;
    uint32_t tmem;
};
constexpr size_t kSmemBytes = sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "");

// mbar_wait for a whole warp whose lanes stay together.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, volatile int *abort) {
    uint64_t start = 0;
    for (int i = 1; !__all_sync(kFullMask, mbar_try_wait(bar, parity)); ++i) {
        if ((i & 63) != 0) continue;
        const uint64_t now = timer_ns();
        if (start == 0) start = now;
        if (__any_sync(kFullMask, *abort != 0 || now - start > kMaxWaitNs)) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// Quarters (32 tokens) of a chunk with `rows` tokens from its start on to the sequence's end; the others are left out.
__device__ __forceinline__ int quarters_of(int rows) { return min(4, (rows + 31) / 32); }

// The warp's own arrival, after all its lanes are done.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// Sums of pairs of floats (hi, lo) with |lo| within half a unit of hi: good to 2^-44 or so.
__device__ __forceinline__ float2 add_pairs(float2 a, float2 b) {
    const float s = a.x + b.x, t = s - a.x;
    const float e = ((a.x - (s - t)) + (b.x - t)) + (a.y + b.y);
    const float hi = s + e;
    return make_float2(hi, e - (hi - s));
}

// Four steps from their inputs with the bias, and the logarithms (base 2) of their decays.
__device__ __forceinline__ void steps_of(float (&d)[4], float2 (&g)[4], float bias, float scale, int real, const ccv_ssm_args &a) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        f32x2 x = add2(pack2(d[i], d[i + 1]), pack2(bias, bias));
        if (a.dt_softplus) x = softplus2(x);
        unpack2(x, d[i], d[i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        d[i] = i >= real ? 0.0f : d[i] < a.dt_min ? a.dt_min : d[i] > a.dt_max ? a.dt_max : d[i];
        constexpr float kHi = 1.4426950216293335f, kLo = 1.9259629911266175e-8f;  // log2(e)
        float u = d[i] * scale, rest = fmaf(d[i], scale, -u);
        // e^-200 is 0 in fp32 and e^1000 infinite
        if (!(u >= -200.0f && u <= 1000.0f)) {
            u = u < -200.0f ? -200.0f : u > 1000.0f ? 1000.0f : 0.0f;
            rest = 0.0f;
        }
        g[i].x = u * kHi;
        g[i].y = fmaf(u, kHi, -g[i].x) + fmaf(u, kLo, rest * kHi);
        if (!(fabsf(d[i]) < INFINITY)) d[i] = NAN;
    }
}

__device__ __forceinline__ f32x2 same2(float x) { return pack2(x, x); }

// FULL: outputs and the sequences' final states; otherwise segments' own states for the join.
// NP: panels of 64 states.  GATED: with z.  vec_out: rows of out (and z) allow 16-byte vectors.
template <bool FULL, int NP, bool GATED>
__global__ void __launch_bounds__(kThreads, 1) ssm_chunk_kernel(const __grid_constant__ SsmFwd p, const __grid_constant__ Maps maps, int vec_out) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const ccv_ssm_args &a = p.a;
    const int tid = threadIdx.x, warp = __shfl_sync(kFullMask, tid >> 5, 0), lane = tid & 31;
    const int panels = (a.head_dim + 63) / 64, all = a.num_heads * panels;
    const int unit = blockIdx.x / all, v = blockIdx.x % all;  // panel among all panels of all heads
    const int h = v / panels, panel = v % panels, group = h / (a.num_heads / a.num_groups);
    wait_prior_grid();
    release_next_grid();
    if ((smem_u32(smem_raw) & 1023u) != 0) {  // swizzled tiles need it
        if (tid == 0) count_error(p.err_count);
        return;
    }

    // The block's sequence, and its tokens of it.
    int seq = unit, s, e, segment = 0, segments = 1;
    const int unit_tokens = p.seg_chunks * Q;
    if (p.seg_chunks > 0) {
        if (warp == 0) {
            int i, f, t;
            find_sequence(p.query_start_loc, p.batch, unit, unit_tokens, lane, i, f, t);
            if (lane == 0) {
                sm.seq = i;
                sm.start = f;
                sm.end = t;
            }
        }
        __syncthreads();
        seq = sm.seq;
        s = sm.start;
        e = sm.end;
    } else {
        s = p.query_start_loc[seq];
        e = p.query_start_loc[seq + 1];
    }
    const bool told = tid == 0 && v == 0 && FULL;  // counts a sequence's error
    if (!sequence_ok(s, e, p.total_tokens)) {
        if (told) count_error(p.err_count);
        return;
    }
    if (s == e) return;
    if (p.seg_chunks > 0) {
        segment = unit - first_slot(s, seq, unit_tokens);
        segments = (e - s + unit_tokens - 1) / unit_tokens;
        if (segment < 0 || segment >= segments) return;
    }
    const int line = p.cache_indices != nullptr ? p.cache_indices[seq] : seq;
    if (line == a.pad_slot_id) return;
    if (a.state != nullptr && (line < 0 || line >= a.num_lines)) {
        if (told && segment == 0) count_error(p.err_count);
        return;
    }
    const bool last = segment == segments - 1;
    if (!FULL && last) return;
    if (p.seg_chunks > 0) {
        s += segment * unit_tokens;
        if (!last) e = s + unit_tokens;
    }
    const int chunks = (e - s + Q - 1) / Q;

    if (tid == 0) {
        sm.abort = sm.any_bad = 0;
        const auto init = [](uint64_t &b, int n) { mbar_init(&b, n); };
        for (int i = 0; i < 3; ++i) {
            init(sm.in_full[i], 2);  // the copy and the steps
            init(sm.x_free[i], kCompute);
        }
        for (int i = 0; i < 2; ++i) {
            init(sm.gates_free[i], kCompute);
            init(sm.b_full[i], 1);
            init(sm.b_free[i], 1);
        }
        init(sm.parts_full, kCompute);
        init(sm.m_full, kCompute);
        for (uint64_t *bar : {&sm.c_full, &sm.c_free, &sm.cb_full, &sm.sum_full, &sm.mx_full, &sm.drain}) init(*bar, 1);
        mbar_init_fence();
    }
    if (tid < 64) sm.first_bad[tid] = INT_MAX;
    if (warp == kCopyWarp) tmem_alloc<512>(&sm.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, sm.tmem, 0);
    volatile int *abort = &sm.abort;
    // Stages of B: the states alone have no use for C's place, and are done with a chunk sooner.
    constexpr int kStages = FULL ? 1 : 2;
    const auto tile_b = [&](int c, int i) { return c % kStages == 0 ? sm.b[i] : sm.c[i]; };

    if (warp == kCopyWarp) {
        int issued = 0, issued_b = 0, issued_c = 0, c = 0;
        for (; c < chunks; ++c) {
            const int t0 = s + c * Q;
            if (c >= 3 && !wait_all(&sm.x_free[c % 3], (c / 3 - 1) & 1, abort)) break;
            if (lane == 0) {
                mbar_expect_tx(&sm.in_full[c % 3], kTile);
                tensor_load(sm.x[c % 3], &maps.x, panel * 64, h, t0, &sm.in_full[c % 3]);
            }
            __syncwarp();
            issued = c + 1;
            // C is free before B, and both early enough: C B^T of the next chunk is wanted a chunk's time later.
            if constexpr (FULL) {
                if (c >= 1 && !wait_all(&sm.c_free, (c - 1) & 1, abort)) break;
                if (lane == 0) {
                    mbar_expect_tx(&sm.c_full, NP * kTile);
                    for (int i = 0; i < NP; ++i) tensor_load(sm.c[i], &maps.c, i * 64, group, t0, &sm.c_full);
                }
                __syncwarp();
                issued_c = c + 1;
            }
            if (c >= kStages && !wait_all(&sm.b_free[c % kStages], (c / kStages - 1) & 1, abort)) break;
            if (lane == 0) {
                mbar_expect_tx(&sm.b_full[c % kStages], 2 * kTile);
                for (int i = 0; i < 2; ++i) tensor_load(tile_b(c, i), &maps.b, i * 64, group, t0, &sm.b_full[c % kStages]);
            }
            __syncwarp();
            issued_b = c + 1;
        }
        if (c < chunks) {  // gave up: let the copies land before the shared memory goes
            int quiet = 0;
            for (int i = max(0, issued - 3); i < issued; ++i) wait_all(&sm.in_full[i % 3], (i / 3) & 1, &quiet);
            for (int i = max(0, issued_b - kStages); i < issued_b; ++i) wait_all(&sm.b_full[i % kStages], (i / kStages) & 1, &quiet);
            if (issued_c > 0) wait_all(&sm.c_full, (issued_c - 1) & 1, &quiet);
        }
    } else if (warp == kStepWarp) {
        // A chunk's steps and their sums, four tokens a lane.  What it loads it converts a chunk later.
        uint32_t raw[4];
        const int shift = a.dt_fp32 ? 0 : 16;
        const float scale = bounded_rate(a.A[h]);
        const float bias = scale != scale ? NAN : a.dt_bias != nullptr ? a.dt_bias[h] : 0.0f;  // a rate that is NaN shows in the steps
        const auto fetch = [&](int chunk) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = s + chunk * Q + lane * 4 + i;
                const int64_t at = t * a.dt_stride_tok + h * a.dt_stride_head;
                raw[i] = t >= e ? 0u : a.dt_fp32 ? static_cast<const uint32_t *>(a.dt)[at] : static_cast<const uint16_t *>(a.dt)[at];
            }
        };
        fetch(0);
        for (int c = 0; c < chunks; ++c) {
            const int st = c & 1;
            float d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = __uint_as_float(raw[i] << shift);
            if (c + 1 < chunks) fetch(c + 1);
            float2 sum[4];
            steps_of(d, sum, bias, scale, e - s - c * Q - lane * 4, a);
#pragma unroll
            for (int i = 1; i < 4; ++i) sum[i] = add_pairs(sum[i - 1], sum[i]);
            float2 total = sum[3];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float2 o = make_float2(__shfl_up_sync(kFullMask, total.x, m), __shfl_up_sync(kFullMask, total.y, m));
                if (lane >= m) total = add_pairs(o, total);
            }
            const float2 end = make_float2(__shfl_sync(kFullMask, total.x, 31), __shfl_sync(kFullMask, total.y, 31));
            float2 before = make_float2(__shfl_up_sync(kFullMask, total.x, 1), __shfl_up_sync(kFullMask, total.y, 1));
            if (lane == 0) before = make_float2(0.0f, 0.0f);
            float weight[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum[i] = i < 3 ? add_pairs(before, sum[i]) : total;
                weight[i] = d[i] * ex2_approx((end.x - sum[i].x) + (end.y - sum[i].y));
            }
            if (c >= 2 && !wait_all(&sm.gates_free[st], (c / 2 - 1) & 1, abort)) break;
            Gates &g = sm.gates[st];
            *reinterpret_cast<float4 *>(g.hi + lane * 4) = make_float4(sum[0].x, sum[1].x, sum[2].x, sum[3].x);
            *reinterpret_cast<float4 *>(g.lo + lane * 4) = make_float4(sum[0].y, sum[1].y, sum[2].y, sum[3].y);
            *reinterpret_cast<float4 *>(g.d + lane * 4) = make_float4(d[0], d[1], d[2], d[3]);
            *reinterpret_cast<float4 *>(g.weight + lane * 4) = make_float4(weight[0], weight[1], weight[2], weight[3]);
            warp_arrive(&sm.in_full[c % 3], lane);
        }
    } else if (warp == kIssueWarp) {
        const uint32_t el = elect_lane(), w = desc_low(smem_u32(sm.w[0])), cc = desc_low(smem_u32(sm.c[0])), s0 = desc_low(smem_u32(sm.s[0]));
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) {
            const int rows = e - s - c * Q, quarters = quarters_of(rows);
            const uint32_t b = desc_low(smem_u32(tile_b(c, 0))), x = desc_low(smem_u32(sm.x[c % 3]));
            if (!(ok = wait_all(&sm.b_full[c % kStages], (c / kStages) & 1, abort))) break;
            if constexpr (FULL) {  // C B^T
                if (!(ok = wait_all(&sm.c_full, c & 1, abort))) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4 * NP; ++ks) {
                    const uint32_t at = ((ks / 4) * kTile + (ks % 4) * 32) / 16;
                    mma_ss(tmem + kColCB, cc + at, b + at, mma_desc(128, 128, false), ks > 0, el);
                }
                mma_commit(&sm.cb_full, el);
            }
            if (!(ok = wait_all(&sm.parts_full, c & 1, abort))) break;
            tc_fence_after();
            if constexpr (FULL) {  // C S: all warps have left the outputs before the last behind them
#pragma unroll
                for (int part = 1; part >= 0; --part)
#pragma unroll
                    for (int ks = 0; ks < 4 * NP; ++ks)
                        mma_ss(tmem + kColCS + (c & 1) * 64, cc + ((ks / 4) * kTile + (ks % 4) * 32) / 16,
                               s0 + (part * kTile + ks * 2048) / 16, mma_desc(128, 64, true), part < 1 || ks > 0, el);
                mma_commit(&sm.c_free, el);
            }
            // the chunk's sum for the state; B is MN-major here, its panels are kTile apart
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half * 64 < rows)
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
                            mma_ss(tmem + kColSum, (b | ((kTile / 16) << 16)) + ks * 2048 / 16, w + (part * kTile + ks * 2048) / 16,
                                   mma_desc(128, 64, true) | (1u << 15), half > 0 || part < 2 || ks > 0, el);
            mma_commit(&sm.sum_full, el);
            mma_commit(&sm.b_free[c % kStages], el);
            if constexpr (FULL) {  // M x
                if (!(ok = wait_all(&sm.m_full, c & 1, abort) && wait_all(&sm.in_full[c % 3], (c / 3) & 1, abort))) break;
                tc_fence_after();
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            if (half * 4 + ks < 2 * quarters)
                                mma_ts(tmem + kColMX, tmem + kColM + half * 64 + part * 32 + ks * 8, x + (half * 4 + ks) * 2048 / 16,
                                       mma_desc(128, 64, true), half + (1 - part) + ks > 0, el);
                mma_commit(&sm.mx_full, el);
            }
        }
        if (!ok) {  // gave up: let the products end before their memories go
            if (el) count_error(p.err_count);
            int quiet = 0;
            mma_commit(&sm.drain, el);
            wait_all(&sm.drain, 0, &quiet);
        }
    } else if (warp < kCompute) {
        // Thread i of a warpgroup has token i and row i of the state; the warpgroup has 16 channels, and 32 of M's columns.
        const int qd = warp >> 2, w = warp & 3, i = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        const uint32_t col_m = lanes + kColM + (qd >> 1) * 64 + (qd & 1) * 16;
        const int first = panel * 64 + qd * 16, width = max(0, min(16, a.head_dim - first));  // channels of the head
        float *pool = a.state != nullptr ? a.state + line * a.s_stride_line + h * a.s_stride_head + first * a.s_stride_dim + i * a.s_stride_state
                                         : nullptr;
        float *slot = p.seg_chunks > 0 ? p.seg_state + (unit * static_cast<int64_t>(all) + v) * kStateFloats + qd * 16 * 128 + i : nullptr;
        f32x2 st2[8];  // two channels each
        {
            const bool kept = FULL && segments > 1, init = a.state != nullptr && p.has_initial_state != nullptr && p.has_initial_state[seq] != 0;
            const float *from = kept ? slot : pool;
            const int64_t step = kept ? 128 : a.s_stride_dim;
            const int count = kept ? 16 : FULL && init && i < a.dim_state ? width : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f[2];
#pragma unroll
                for (int l = 0; l < 2; ++l) f[l] = 2 * j + l < count ? from[(2 * j + l) * step] : 0.0f;
                st2[j] = pack2(f[0], f[1]);
            }
        }
        const float skip = FULL && a.D != nullptr ? a.D[h] : 0.0f;
        uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + h * a.out.stride_head + first * a.out.stride_dim;
        const uint16_t *z = static_cast<const uint16_t *>(a.z.data) + h * a.z.stride_head + first * a.z.stride_dim;
        // M's columns of tokens after a warp's own are zero, and nothing writes them again.
        if (FULL && qd > w) {
            const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_store(col_m + (j & 1) * 32 + (j >> 1) * 8, none);
            tmem_wait_store();
        }
        float whole = 1.0f;  // decay over all tokens
        bool ok = true;
        int c;
        const int piece = tid & 7;
        // The next chunk's weighted tokens and state are made while M x runs; -1 makes the first's.
        for (c = -1; c < chunks; ++c) {
            const int stage = c & 1, rows = e - s - c * Q, quarters = quarters_of(rows), next = c + 1;
            const Gates &g = sm.gates[stage];
            uint8_t *xt = sm.x[(c + 3) % 3];
            float row_decay = 0.0f;
            bool bad = false;
            if (c >= 0) {
                if constexpr (FULL) {
                    // M's columns of 32 tokens, from C B^T: times d_j and e^{G_i - G_j}, G counted from the first token of the warp's
                    // rows (where the decays are weak that is as exact as it needs, and where they are strong the difference is large).
                    const float ghi = g.hi[i], glo = g.lo[i];
                    row_decay = ex2_approx(ghi + glo);
                    const bool mine = qd <= w && qd < quarters;
                    float own = 0.0f;
                    if (mine) {
                        const float base_hi = w > 0 ? g.hi[w * 32 - 1] : 0.0f, base_lo = w > 0 ? g.lo[w * 32 - 1] : 0.0f;
                        own = (ghi - base_hi) + (glo - base_lo);
                        const int j = qd * 32 + lane;
                        sm.since[w][j] = (g.hi[j] - base_hi) + (g.lo[j] - base_lo);
                    }
                    __syncwarp();
                    if (!(ok = wait_all(&sm.cb_full, c & 1, abort))) break;
                    tc_fence_after();
                    if (mine) {
                        // Unrolled, like the issuing warp's loops.  With rolled loops around tensor memory's instructions, whose
                        // operands then went by the loop's counter, an early form stopped with a misaligned address.  All of its
                        // accesses to vectors were checked and none was misaligned; the cause is not known.  What is known to
                        // differ: its warps' numbers came straight from threadIdx, so to the compiler those operands could differ
                        // from lane to lane, which these instructions do not allow.
                        const float *since = sm.since[w] + qd * 32, *steps = g.d + qd * 32;
#pragma unroll
                        for (int j0 = 0; j0 < 32; j0 += 16) {
                            float f[16];
                            tmem_load(lanes + kColCB + qd * 32 + j0, f);
                            tmem_wait_load();
                            uint32_t hi[8], mid[8];
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float4 gj = *reinterpret_cast<const float4 *>(since + j0 + j);
                                const ulonglong2 dj = *reinterpret_cast<const ulonglong2 *>(steps + j0 + j);
                                const float at[4] = {gj.x, gj.y, gj.z, gj.w};
                                float m[4];
#pragma unroll
                                for (int l = 0; l < 4; ++l) m[l] = ex2_approx(own - at[l]);
                                unpack2(mul2(mul2(pack2(m[0], m[1]), dj.x), pack2(f[j], f[j + 1])), m[0], m[1]);
                                unpack2(mul2(mul2(pack2(m[2], m[3]), dj.y), pack2(f[j + 2], f[j + 3])), m[2], m[3]);
                                if (qd == w) {  // a branch: without the masks the other warps have a quarter fewer instructions
#pragma unroll
                                    for (int l = 0; l < 4; ++l) m[l] = j0 + j + l <= lane ? m[l] : 0.0f;
                                }
                                split_bf16x2(pack2(m[0], m[1]), hi[j / 2], mid[j / 2]);
                                split_bf16x2(pack2(m[2], m[3]), hi[j / 2 + 1], mid[j / 2 + 1]);
                            }
                            tmem_store(col_m + j0 / 2, hi);
                            tmem_store(col_m + 32 + j0 / 2, mid);
                        }
                        tmem_wait_store();
                    }
                    tc_fence_before();
                    warp_arrive(&sm.m_full, lane);
                }
                const float gamma = ex2_approx(g.hi[Q - 1] + g.lo[Q - 1]);
                warp_arrive(&sm.gates_free[stage], lane);

                // S <- e^{G_Q} S + the chunk's sum
                if (!(ok = wait_all(&sm.sum_full, c & 1, abort))) break;  // and C S is done with the state's parts
                tc_fence_after();
                const f32x2 g2 = same2(gamma);
                {
                    float f[16];
                    tmem_load(lanes + kColSum + qd * 16, f);
                    tmem_wait_load();
#pragma unroll
                    for (int j = 0; j < 8; ++j) st2[j] = fma2(g2, st2[j], pack2(f[2 * j], f[2 * j + 1]));
                }
                tc_fence_before();
                whole *= gamma;
                // What this chunk has is noted before sum_full.  Another warp may be noting the next chunk's meanwhile, so the lanes
                // vote: those of a row store it together below.
                bad = __any_sync(kFullMask, sm.any_bad != 0);
                if (bad) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float f[2];
                        unpack2(st2[j], f[0], f[1]);
#pragma unroll
                        for (int l = 0; l < 2; ++l) f[l] = sm.first_bad[qd * 16 + 2 * j + l] < (c + 1) * Q ? NAN : f[l];
                        st2[j] = pack2(f[0], f[1]);
                    }
                }
            }
            if (next < chunks) {
                const int ns = next & 1, left = e - s - next * Q;
                if (!(ok = wait_all(&sm.in_full[next % 3], (next / 3) & 1, abort))) break;
                if (left < Q && !(ok = wait_all(&sm.b_full[next % kStages], (next / kStages) & 1, abort))) break;  // its other rows become zeros here
                uint8_t *nx = sm.x[next % 3];
                if constexpr (FULL) {  // the state's parts for C S
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t hi[4], mid[4];
#pragma unroll
                        for (int l = 0; l < 4; ++l) split_bf16x2(st2[4 * j + l], hi[l], mid[l]);
                        const int at = i * 128 + (((qd * 2 + j) ^ (i & 7)) << 4);
                        *reinterpret_cast<uint4 *>(sm.s[0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(sm.s[1] + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    }
                }
                // The weighted tokens' parts, and what is wrong with the tile: rows of another sequence, values that are not finite.
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = half * 64 + (tid >> 3), at = row * 128 + ((piece ^ (row & 7)) << 4);
                    if (half * 64 >= left) break;
                    uint4 x = *reinterpret_cast<const uint4 *>(nx + at);
                    const f32x2 wt = same2(sm.gates[ns].weight[row]);
                    if (row >= left) {
                        x = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(nx + at) = x;
                        *reinterpret_cast<uint4 *>(tile_b(next, 0) + at) = x;
                        *reinterpret_cast<uint4 *>(tile_b(next, 1) + at) = x;
                    }
                    uint32_t word[4] = {x.x, x.y, x.z, x.w};
                    f32x2 f[4], odd = 0ull;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        f[j] = pack2(bf16_lo(word[j]), bf16_hi(word[j]));
                        odd = fma2(f[j], 0ull, odd);
                    }
                    if ((odd & 0x7fffffff7fffffffull) != 0ull) {  // 0 x is NaN
                        sm.any_bad = 1;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t bits = (j & 1) ? word[j / 2] >> 16 : word[j / 2] & 0xffffu;
                            if ((bits & 0x7f80u) != 0x7f80u) continue;
                            atomicMin(&sm.first_bad[piece * 8 + j], next * Q + row);
                            word[j / 2] &= (j & 1) ? 0xffffu : 0xffff0000u;
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) f[j] = pack2(bf16_lo(word[j]), bf16_hi(word[j]));
                        *reinterpret_cast<uint4 *>(nx + at) = make_uint4(word[0], word[1], word[2], word[3]);
                    }
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) split_bf16x3(mul2(f[j], wt), hi[j], mid[j], lo[j]);
                    *reinterpret_cast<uint4 *>(sm.w[0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(sm.w[1] + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    *reinterpret_cast<uint4 *>(sm.w[2] + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_shared();
                warp_arrive(&sm.parts_full, lane);
                if (!FULL) warp_arrive(&sm.x_free[next % 3], lane);
            }
            if (c < 0) continue;

            // out_i = e^{G_i} (C S)_i + (M x)_i + D x_i, with the gate
            if constexpr (FULL) {
                if (!(ok = wait_all(&sm.mx_full, c & 1, abort))) break;
                tc_fence_after();
                const bool fast = vec_out && !bad;
                const int64_t t = s + c * Q + i;
                const f32x2 decay2 = same2(row_decay), skip2 = same2(skip);
                float mx[16], cs[16];
                __syncwarp();
                tmem_load(lanes + kColMX + qd * 16, mx);
                tmem_load(lanes + kColCS + (c & 1) * 64 + qd * 16, cs);
                tmem_wait_load();
                tc_fence_before();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int ch = half * 8;
                    uint4 *x = reinterpret_cast<uint4 *>(xt + i * 128 + (((qd * 2 + half) ^ (i & 7)) << 4));
                    const uint32_t word[4] = {x->x, x->y, x->z, x->w};
                    f32x2 y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = ch + 2 * j;
                        y[j] = fma2(decay2, pack2(cs[at], cs[at + 1]), pack2(mx[at], mx[at + 1]));
                        y[j] = fma2(skip2, pack2(bf16_lo(word[j]), bf16_hi(word[j])), y[j]);
                    }
                    if constexpr (GATED) {
                        if (i < rows && ch < width) {
                            if (vec_out) {
                                const uint4 zz = __ldg(reinterpret_cast<const uint4 *>(z + t * a.z.stride_tok + ch));
                                const uint32_t zw[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], silu2(pack2(bf16_lo(zw[j]), bf16_hi(zw[j]))));
                            } else {
                                const auto at = [&](int j) { return ch + j < width ? bf16_bits(z[t * a.z.stride_tok + (ch + j) * a.z.stride_dim]) : 0.0f; };
#pragma unroll
                                for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], silu2(pack2(at(2 * j), at(2 * j + 1))));
                            }
                        }
                    }
                    // over the thread's own values of x, which nothing reads any more
                    *x = make_uint4(f32x2_to_bf16x2(y[0]), f32x2_to_bf16x2(y[1]), f32x2_to_bf16x2(y[2]), f32x2_to_bf16x2(y[3]));
                }
                if (fast) {  // two lanes a row: with a whole row a lane a store takes more of L1's cycles
                    __syncwarp();
                    const int part = lane & 1;
#pragma unroll
                    for (int r16 = 0; r16 < 2; ++r16) {
                        const int tr = w * 32 + r16 * 16 + (lane >> 1);
                        const uint4 val = *reinterpret_cast<const uint4 *>(xt + tr * 128 + (((qd * 2 + part) ^ (tr & 7)) << 4));
                        if (tr < rows && part * 8 < width) *reinterpret_cast<uint4 *>(out + (t - i + tr) * a.out.stride_tok + part * 8) = val;
                    }
                } else {
#pragma unroll 1
                    for (int ch = 0; i < rows && ch < width; ++ch) {
                        uint16_t f = *reinterpret_cast<const uint16_t *>(xt + i * 128 + (((qd * 2 + (ch >> 3)) ^ (i & 7)) << 4) + (ch & 7) * 2);
                        if (bad && sm.first_bad[qd * 16 + ch] <= c * Q + i) f = 0x7fffu;
                        out[t * a.out.stride_tok + ch * a.out.stride_dim] = f;
                    }
                }
                fence_async_shared();
                warp_arrive(&sm.x_free[c % 3], lane);
            }
        }
        if (FULL && !ok)  // gave up
            for (c = max(c, 0); c < chunks; ++c)
                if (s + c * Q + i < e)
                    for (int ch = 0; ch < width; ++ch) out[(s + c * Q + i) * a.out.stride_tok + ch * a.out.stride_dim] = 0x7fffu;
        if (!FULL || (last && a.state != nullptr)) {
            float *to = FULL ? pool : slot;
            const int64_t step = FULL ? a.s_stride_dim : 128;
            const int count = !FULL ? 16 : i < a.dim_state ? width : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float f[2];
                unpack2(st2[j], f[0], f[1]);
#pragma unroll
                for (int l = 0; l < 2; ++l)
                    if (2 * j + l < count) to[(2 * j + l) * step] = ok ? f[l] : NAN;
            }
            if (!FULL && i == 0 && qd == 0) p.seg_decay[static_cast<int64_t>(unit) * all + v] = whole;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kCopyWarp) tmem_free<512>(tmem);
}

// The segments' first states, one after the other, from their own: F <- decay F + own.  A thread has four values of a head's
// panel; the first segment's is a copy of the pool's, whose line the last segment writes while the first may still start.
__global__ void __launch_bounds__(256) ssm_join_kernel(const __grid_constant__ SsmFwd p, int panels) {
    const ccv_ssm_args &a = p.a;
    wait_prior_grid();
    release_next_grid();
    constexpr int kBlocks = kStateFloats / (256 * 4);
    const int per_seq = a.num_heads * panels * kBlocks, seq = blockIdx.x / per_seq;
    const int v = blockIdx.x % per_seq / kBlocks, at = (blockIdx.x % kBlocks * 256 + threadIdx.x) * 4;
    const int s = p.query_start_loc[seq], e = p.query_start_loc[seq + 1], unit = p.seg_chunks * Q;
    if (!sequence_ok(s, e, p.total_tokens) || e - s <= unit) return;
    const int line = p.cache_indices != nullptr ? p.cache_indices[seq] : seq;
    if (line == a.pad_slot_id || (a.state != nullptr && (line < 0 || line >= a.num_lines))) return;
    const int segments = (e - s + unit - 1) / unit, h = v / panels, ch = v % panels * 64 + at / 128, n = at % 128;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state != nullptr && p.has_initial_state != nullptr && p.has_initial_state[seq] != 0 && ch < a.head_dim) {
        const float *pool = a.state + line * a.s_stride_line + h * a.s_stride_head + ch * a.s_stride_dim;
        if (n < a.dim_state) f.x = pool[n * a.s_stride_state];
        if (n + 1 < a.dim_state) f.y = pool[(n + 1) * a.s_stride_state];
        if (n + 2 < a.dim_state) f.z = pool[(n + 2) * a.s_stride_state];
        if (n + 3 < a.dim_state) f.w = pool[(n + 3) * a.s_stride_state];
    }
    const int64_t step = static_cast<int64_t>(a.num_heads) * panels, slot = first_slot(s, seq, unit) * step + v;
    float4 *to = reinterpret_cast<float4 *>(p.seg_state + slot * kStateFloats + at);
    const float *decay = p.seg_decay + slot;
    for (int i = 0; i < segments; ++i) {
        const float4 x = i + 1 < segments ? *to : f;
        const float d = i + 1 < segments ? *decay : 0.0f;
        *to = f;
        f = make_float4(fmaf(d, f.x, x.x), fmaf(d, f.y, x.y), fmaf(d, f.z, x.z), fmaf(d, f.w, x.w));
        to += step * (kStateFloats / 4);
        decay += step;
    }
}

int64_t segment_slots(int total_tokens, int batch, int seg_chunks) {
    return static_cast<int64_t>(total_tokens) / (static_cast<int64_t>(seg_chunks) * Q) + batch;
}

template <bool FULL, int NP, bool GATED>
int launch_chunks(const SsmFwd &p, const Maps &maps, int64_t units, int vec_out, cudaStream_t stream) {
    int dev = 0;
    current_device_sms(&dev);
    cudaError_t err;
    if (resident_blocks<ssm_chunk_kernel<FULL, NP, GATED>>(kThreads, kSmemBytes, dev, &err) == 0) return static_cast<int>(err);
    const int64_t blocks = units * p.a.num_heads * ((p.a.head_dim + 63) / 64);
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    return launch_pdl(ssm_chunk_kernel<FULL, NP, GATED>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), kSmemBytes, stream, p, maps, vec_out);
}

template <int NP, bool GATED>
int launch_all(const SsmFwd &p, const Maps &maps, int vec_out, cudaStream_t stream) {
    if (p.seg_chunks == 0) return launch_chunks<true, NP, GATED>(p, maps, p.batch, vec_out, stream);
    const int64_t units = segment_slots(p.total_tokens, p.batch, p.seg_chunks);
    int status = launch_chunks<false, 2, false>(p, maps, units, vec_out, stream);
    if (status != CCV_OK) return status;
    const int panels = (p.a.head_dim + 63) / 64;
    const int64_t joins = static_cast<int64_t>(p.batch) * p.a.num_heads * panels * (kStateFloats / 1024);
    if (joins > 0x7fffffff) return CCV_ERR_SIZE;
    status = launch_pdl(ssm_join_kernel, dim3(static_cast<unsigned>(joins)), dim3(256), 0, stream, p, panels);
    if (status != CCV_OK) return status;
    return launch_chunks<true, NP, GATED>(p, maps, units, vec_out, stream);
}

}  // namespace

bool ssm_chunked_dims(int dim_state, int a_per_state) { return !a_per_state && dim_state <= 128; }

// Chunks of a segment, or 0 to leave sequences whole, for sequences of equal lengths (their offsets are on the device).  In
// chunk times of a block (3 us): the first pass takes 0.6 of one a chunk, a block 0.8 to start and end, the two launches more 3.
// Each pass runs in waves of one block an SM.  11027 tokens of 32 heads take 122 us so and 232 whole, 30000 of 64 507 and 616;
// 2 x 4000 of 64 heads 137 in two segments and 92 whole.  Lengths that differ are not seen: 11000 tokens and 23 prompts of 40, 32
// heads, stay whole and take 233, in segments of 29 chunks 147.
int ssm_chunked_segments(int total_tokens, int batch, int num_heads, int head_dim) {
    const char *forced = std::getenv("CCV_SSM_SEGMENT");  // chunks of a segment (for testing and tuning)
    if (forced != nullptr) return std::atoi(forced) > 0 && std::atoi(forced) < (1 << 20) ? std::atoi(forced) : 0;
    constexpr int kSms = 152;  // a GB300's: the workspace's size may not depend on the device that is current
    const int64_t each = static_cast<int64_t>(batch) * Q;
    const int chunks = static_cast<int>((total_tokens + each - 1) / each);
    const int64_t blocks = static_cast<int64_t>(batch) * num_heads * ((head_dim + 63) / 64);
    auto waves = [](int64_t n) { return static_cast<double>((n + kSms - 1) / kSms); };
    double best = waves(blocks) * (chunks + 0.8);
    int choice = 0;
    for (int n = 2; n <= 64 && n <= chunks; ++n) {
        const int length = (chunks + n - 1) / n;
        const double cost = 3 + waves(blocks * (n - 1)) * (length * 0.6 + 0.8) + waves(blocks * n) * (length + 0.8);
        if (cost < best) {
            best = cost;
            choice = length;
        }
    }
    return choice;
}

int64_t ssm_chunked_workspace(int total_tokens, int batch, int num_heads, int head_dim, int seg_chunks) {
    if (seg_chunks == 0) return 0;
    const int64_t slots = segment_slots(total_tokens, batch, seg_chunks) * num_heads * ((head_dim + 63) / 64);
    return slots * kStateFloats * 4 + (slots * 4 + 127) / 128 * 128;
}

int ssm_launch_chunked(const SsmFwd &call, void *workspace, cudaStream_t stream) {
    SsmFwd p = call;
    const ccv_ssm_args &a = p.a;
    if (p.seg_chunks > 0) {
        const int64_t slots = segment_slots(p.total_tokens, p.batch, p.seg_chunks) * a.num_heads * ((a.head_dim + 63) / 64);
        p.seg_state = static_cast<float *>(workspace);
        p.seg_decay = p.seg_state + slots * kStateFloats;
    }
    Maps maps;
    if (!encode_heads_map(&maps.x, a.x, a.head_dim, a.num_heads, p.total_tokens, Q) ||
        !encode_heads_map(&maps.b, a.B, a.dim_state, a.num_groups, p.total_tokens, Q) ||
        !encode_heads_map(&maps.c, a.C, a.dim_state, a.num_groups, p.total_tokens, Q))
        return CCV_ERR_STRIDE;
    auto rows = [](const ccv_heads_view &v) {
        return aligned16(v.data) && v.stride_dim == 1 && v.stride_tok % 8 == 0 && v.stride_head % 8 == 0;
    };
    const int vec_out = a.head_dim % 8 == 0 && rows(a.out) && (a.z.data == nullptr || rows(a.z));
    if (a.z.data != nullptr)
        return a.dim_state <= 64 ? launch_all<1, true>(p, maps, vec_out, stream) : launch_all<2, true>(p, maps, vec_out, stream);
    return a.dim_state <= 64 ? launch_all<1, false>(p, maps, vec_out, stream) : launch_all<2, false>(p, maps, vec_out, stream);
}

}  // namespace ccv
