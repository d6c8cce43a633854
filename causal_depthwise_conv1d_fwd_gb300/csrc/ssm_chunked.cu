// Selective state space scan over varlen sequences (prefill), chunked form on the tensor cores, for one decay a head.
//
// A chunk holds Q = 128 tokens.  With d_j the step of token j and G the running sum of d A inside the chunk, unrolling the
// recurrence gives, for a head's x (tokens, 64), B and C (tokens, 128) and state S (128, 64) at the chunk's start,
//     y_i = e^{G_i} C_i S + sum_{j <= i} M_ij x_j,   M_ij = (C_i . B_j) e^{G_i - G_j} d_j
//     S  <- e^{G_Q} S + sum_j B_j^T (e^{G_Q - G_j} d_j x_j)
// and C B^T is the same for all heads of a group.  Nothing but S is sequential, and S only by its own multiply-add, so all
// products of a chunk run beside those of its neighbours.  A block has two heads of a group of one sequence (or segment) and
// goes through its chunks:
//   warpgroups 0, 1  a head each: M from C B^T (tensor memory to tensor memory), then the head's outputs
//   warpgroups 2, 3  a head each: the state in registers (thread n has row n), its parts to shared memory for C S, and the
//                    weighted tokens' parts for the state's sum
//   four warps       copies and steps; products C B^T and M x; products of the state's sum; products C S
// Heads wider than 64 are cut into panels of 64 that share steps and decays.
//
// Precision.  The state is fp32, so the operands of what reaches it keep 24 bits: B enters as its own bf16 values (exact), the
// weighted tokens as three bf16 parts, and the sum over chunks is an fp32 multiply-add.  Products that reach the output alone
// (M, S) keep 16 bits an operand, two parts; x and C are exact.  Smaller parts are added first, since the tensor cores' sums
// truncate.  G is summed in 64-bit fixed point, and differences of it are taken as pairs of floats.
//
// What is not finite.  A sum over a chunk takes zeros for the tokens after its own, and 0 * NaN is NaN.  So an x that is not
// finite is left out of the products, and its channel is NaN from that token on, the final state too; a step that is not finite
// makes M's rows from its own on, and the state, NaN by itself; so do B and C, whose products are masked and not multiplied by
// zero.  Rows of the last tile that belong to the next sequence are zeroed.
#include <climits>
#include <cstdlib>
#include <cstring>

#include "ccv_varlen.cuh"
#include "ssm_fwd.cuh"

namespace ccv {
namespace {

constexpr int Q = 128;              // tokens of a chunk
constexpr int kTile = Q * 128;      // bytes of 128 rows of 64 bf16 values
constexpr int kQuarter = kTile / 4; // of 32 rows
constexpr int kThreads = 640;
constexpr int kCopyWarp = 16, kOutWarp = 17, kSumWarp = 18, kStateWarp = 19;
// Columns of tensor memory: C B^T; M in two halves of 64 tokens, each in two parts; M x; C S; the heads' sums for the state.
constexpr uint32_t kColCB = 0, kColM = 128, kColMX = 256, kColCS = 320, kColSum = 384;
constexpr int kStateFloats = 128 * 64;  // of a head's panel in the workspace

struct Maps {
    CUtensorMap x, b, c;
};

struct Gates {  // of a chunk's tokens and a head: G log2(e) as a pair of floats, and the steps
    float hi[Q], lo[Q], d[Q];
};

struct Smem {
    uint8_t x[2][2][kTile];     // stage, head
    uint8_t b[2][2][kTile];     // stage, panel of 64 states
    uint8_t c[2][kTile];        // panel
    uint8_t w[2][3][kQuarter];  // head, part: weighted tokens
    uint8_t s[2][kTile];        // part: the state of the head whose turn it is
    Gates gates[2][2];          // stage, head
    float weight[2][Q];         // head: what tokens count for in the state's sum
    float factor[2][192];       // head: what the 32, 64, 96 tokens before warps 1, 2, 3 count for in their rows of M
    // A barrier's phase is waited for by the same threads each time, or by ones that know the phase before it to be over: a wait
    // tells a phase from the next one only.
    uint64_t xb_full[2], xb_free[2], c_full, c_free, gates_full[2], gates_free[2];
    uint64_t cb_full, cb_free, m_full[2], m_free[2], mx_full[2], mx_free, cs_full[2], cs_free, s_full, s_free[2];
    uint64_t w_full[2], w_free[2], sum_full[2], x_ok[2][2], together[2], cleared[2], drain[3];
    int first_bad[2][2][64];    // stage, head, channel: the first token whose x is not finite
    int any_bad[2][2];
    int seq, start, end, abort;
    uint32_t tmem;
};
constexpr size_t kSmemBytes = sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "");

// The warp's own arrival, after all its lanes are done.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ f32x2 same2(float x) { return pack2(x, x); }
__device__ __forceinline__ bool odd_bf16x2(uint32_t w) {  // either is not finite
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// FULL: outputs and the sequences' final states; otherwise segments' own states for the join.
// NP: panels of 64 states.  VO: rows of out (and z) allow 16-byte vectors.
template <bool FULL, int NP>
__global__ void __launch_bounds__(kThreads, 1) ssm_chunk_kernel(const __grid_constant__ SsmFwd p, const __grid_constant__ Maps maps, int vec_out) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    const ccv_ssm_args &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int panels = (a.head_dim + 63) / 64, rep = a.num_heads / a.num_groups;
    const int per_group = (rep * panels + 1) / 2, pairs = a.num_groups * per_group;
    const int unit = blockIdx.x / pairs, pair = blockIdx.x % pairs;
    const int group = pair / per_group, v0 = (pair % per_group) * 2;  // first panel of the pair, within the group
    const int nh = min(2, rep * panels - v0);
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
    const bool told = tid == 0 && pair == 0 && FULL;  // counts a sequence's error
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
        sm.abort = 0;
        const auto init = [](uint64_t &b, int n) { mbar_init(&b, n); };
        for (int i = 0; i < 2; ++i) {
            init(sm.xb_full[i], 1);
            init(sm.xb_free[i], FULL ? 2 + 4 * nh : 1);  // both issuers of products, and the outputs' warps
            init(sm.gates_full[i], 1);
            init(sm.gates_free[i], FULL ? 8 * nh : 4 * nh);
            init(sm.m_full[i], 4);
            init(sm.m_free[i], 1);
            init(sm.w_full[i], 4);
            init(sm.w_free[i], 1);
            init(sm.sum_full[i], 1);
            init(sm.mx_full[i], 1);
            init(sm.cs_full[i], 1);
            init(sm.s_free[i], 1);
            for (int k = 0; k < 2; ++k) init(sm.x_ok[i][k], 4);
            init(sm.together[i], 4);
            init(sm.cleared[i], 4);
        }
        init(sm.c_full, 1);
        init(sm.c_free, 2);
        init(sm.cb_full, 1);
        init(sm.cb_free, 4 * nh);
        init(sm.mx_free, 4);
        init(sm.cs_free, 4);
        init(sm.s_full, 4);
        for (uint64_t &b : sm.drain) init(b, 1);
        mbar_init_fence();
    }
    if (tid < 256) (&sm.first_bad[0][0][0])[tid] = INT_MAX;
    if (tid < 4) (&sm.any_bad[0][0])[tid] = 0;
    if (warp == kCopyWarp) tmem_alloc<512>(&sm.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, sm.tmem, 0);
    volatile int *abort = &sm.abort;

    if (warp == kCopyWarp) {
        // Copies of a chunk's tiles, then its steps and their sums; four tokens a lane.
        int issued = 0, c = 0;
        float raw[2][4], scale[2], bias[2];
        int head[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            head[k] = group * rep + min(v0 + k, rep * panels - 1) / panels;
            scale[k] = a.A[head[k]];
            bias[k] = a.dt_bias != nullptr ? a.dt_bias[head[k]] : 0.0f;
        }
        const auto fetch = [&](int chunk) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = s + chunk * Q + lane * 4 + i;
                    raw[k][i] = t < e && k < nh ? ssm_raw_step(a, t * a.dt_stride_tok + head[k] * a.dt_stride_head) : 0.0f;
                }
        };
        fetch(0);
        for (; c < chunks; ++c) {
            const int st = c & 1, t0 = s + c * Q;
            if (c >= 2 && !mbar_wait_warp(&sm.xb_free[st], (c / 2 - 1) & 1, abort)) break;
            if (lane == 0) {
                mbar_expect_tx(&sm.xb_full[st], (2 + nh) * kTile);
                for (int i = 0; i < 2; ++i) tensor_load(sm.b[st][i], &maps.b, i * 64, group, t0, &sm.xb_full[st]);
                for (int k = 0; k < nh; ++k) tensor_load(sm.x[st][k], &maps.x, ((v0 + k) % panels) * 64, head[k], t0, &sm.xb_full[st]);
            }
            issued = c + 1;
            if (c >= 2 && !mbar_wait_warp(&sm.gates_free[st], (c / 2 - 1) & 1, abort)) break;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k >= nh) break;
                float d[4];
                int64_t sum[4], run = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool real = t0 + lane * 4 + i < e;
                    d[i] = real ? ssm_step(raw[k][i], bias[k], a) : 0.0f;
                    // e^-200 is 0 in fp32 and e^1000 infinite: keeps the sums in range
                    float u = d[i] * scale[k];
                    u = u < -200.0f ? -200.0f : u > 1000.0f ? 1000.0f : u == u ? u : 0.0f;
                    if (!(fabsf(d[i]) < INFINITY)) d[i] = NAN;
                    constexpr float kOne = 1099511627776.0f;  // 2^40
                    run += real ? __float2ll_rn(u * 1.4426950408889634f * kOne) : 0ll;
                    sum[i] = run;
                }
                int64_t total = run;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const int64_t o = __shfl_up_sync(kFullMask, total, m);
                    if (lane >= m) total += o;
                }
                const int64_t before = total - run;
                Gates &g = sm.gates[st][k];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float hi = __ll2float_rn(sum[i] + before);
                    g.hi[lane * 4 + i] = hi * 0x1p-40f;
                    g.lo[lane * 4 + i] = __ll2float_rn(sum[i] + before - __float2ll_rn(hi)) * 0x1p-40f;
                    g.d[lane * 4 + i] = d[i];
                }
            }
            warp_arrive(&sm.gates_full[st], lane);
            if (c + 1 < chunks) fetch(c + 1);
            if constexpr (FULL) {
                if (c >= 1 && !mbar_wait_warp(&sm.c_free, (c - 1) & 1, abort)) break;
                if (lane == 0) {
                    mbar_expect_tx(&sm.c_full, NP * kTile);
                    for (int i = 0; i < NP; ++i) tensor_load(sm.c[i], &maps.c, i * 64, group, t0, &sm.c_full);
                }
            }
        }
        if (c < chunks) {  // gave up: let the copies land before the shared memory goes
            int quiet = 0;
            for (int i = max(0, issued - 2); i < issued; ++i) mbar_wait_warp(&sm.xb_full[i & 1], (i / 2) & 1, &quiet);
            if (FULL && c > 0) mbar_wait_warp(&sm.c_full, (c - 1) & 1, &quiet);
        }
    } else if (warp == kOutWarp) {
        if constexpr (FULL) {
            const uint32_t el = elect_lane();
            int c = 0, k = 0;
            for (; c < chunks; ++c) {
                const int st = c & 1;
                const uint32_t b = desc_low(smem_u32(sm.b[st][0])), cc = desc_low(smem_u32(sm.c[0]));
                if (!mbar_wait_warp(&sm.xb_full[st], (c / 2) & 1, abort) || !mbar_wait_warp(&sm.c_full, c & 1, abort)) break;
                if (c >= 1 && !mbar_wait_warp(&sm.cb_free, (c - 1) & 1, abort)) break;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < 4 * NP; ++ks) {
                    const uint32_t at = ((ks / 4) * kTile + (ks % 4) * 32) / 16;
                    mma_ss(tmem + kColCB, cc + at, b + at, mma_desc(128, 128, false), ks > 0, el);
                }
                mma_commit(&sm.cb_full, el);
                mma_commit(&sm.c_free, el);
                for (k = 0; k < nh; ++k) {
                    const int u = c * nh + k;
                    const uint32_t x = desc_low(smem_u32(sm.x[st][k]));
                    if (!mbar_wait_warp(&sm.x_ok[st][k], (c / 2) & 1, abort)) break;
                    if (u >= 1 && !mbar_wait_warp(&sm.mx_free, (u - 1) & 1, abort)) break;
                    int half = 0;
                    for (; half < 2; ++half) {
                        if (!mbar_wait_warp(&sm.m_full[half], u & 1, abort)) break;
                        tc_fence_after();
#pragma unroll
                        for (int part = 1; part >= 0; --part)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_ts(tmem + kColMX, tmem + kColM + half * 64 + part * 32 + ks * 8, x + (half * 4 + ks) * 2048 / 16,
                                       mma_desc(128, 64, true), half + (1 - part) + ks > 0, el);
                        mma_commit(&sm.m_free[half], el);
                    }
                    if (half < 2) break;
                    mma_commit(&sm.mx_full[k], el);
                }
                if (k < nh) break;
                mma_commit(&sm.xb_free[st], el);
            }
            if (c < chunks) {  // gave up: let the products end before their memories go
                if (el) count_error(p.err_count);
                int quiet = 0;
                mma_commit(&sm.drain[0], el);
                mbar_wait_warp(&sm.drain[0], 0, &quiet);
            }
        }
    } else if (warp == kSumWarp) {
        const uint32_t el = elect_lane();
        bool ok = true;
        for (int c = 0; ok && c < chunks; ++c) {
            const int st = c & 1;
            const uint32_t b = desc_low(smem_u32(sm.b[st][0])) | ((kTile / 16) << 16);  // MN-major: its panels are kTile apart
            if (!(ok = mbar_wait_warp(&sm.xb_full[st], (c / 2) & 1, abort))) break;
            for (int q = 0; ok && q < 4; ++q)
                for (int k = 0; k < nh; ++k) {
                    if (!(ok = mbar_wait_warp(&sm.w_full[k], q & 1, abort))) break;
                    tc_fence_after();
                    const uint32_t w = desc_low(smem_u32(sm.w[k][0]));
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
                            mma_ss(tmem + kColSum + k * 64, b + (q * 2 + ks) * 2048 / 16, w + (part * kQuarter + ks * 2048) / 16,
                                   mma_desc(128, 64, true) | (1u << 15), q > 0 || part < 2 || ks > 0, el);
                    mma_commit(&sm.w_free[k], el);
                    if (q == 3) mma_commit(&sm.sum_full[k], el);
                }
            if (ok) mma_commit(&sm.xb_free[st], el);
        }
        if (!ok) {
            if (el) count_error(p.err_count);
            int quiet = 0;
            mma_commit(&sm.drain[1], el);
            mbar_wait_warp(&sm.drain[1], 0, &quiet);
        }
    } else if (warp == kStateWarp) {
        if constexpr (FULL) {
            const uint32_t el = elect_lane();
            const uint32_t cc = desc_low(smem_u32(sm.c[0])), s0 = desc_low(smem_u32(sm.s[0]));
            bool ok = true;
            for (int c = 0; ok && c < chunks; ++c) {
                if (!(ok = mbar_wait_warp(&sm.c_full, c & 1, abort))) break;
                for (int k = 0; k < nh; ++k) {
                    const int u = c * nh + k;
                    if (!(ok = mbar_wait_warp(&sm.s_full, u & 1, abort))) break;
                    if (u >= 1 && !(ok = mbar_wait_warp(&sm.cs_free, (u - 1) & 1, abort))) break;
                    tc_fence_after();
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int ks = 0; ks < 4 * NP; ++ks)
                            mma_ss(tmem + kColCS, cc + ((ks / 4) * kTile + (ks % 4) * 32) / 16, s0 + (part * kTile + ks * 2048) / 16,
                                   mma_desc(128, 64, true), part < 1 || ks > 0, el);
                    mma_commit(&sm.cs_full[k], el);
                    mma_commit(&sm.s_free[k], el);
                }
                if (ok) mma_commit(&sm.c_free, el);
            }
            if (!ok) {
                if (el) count_error(p.err_count);
                int quiet = 0;
                mma_commit(&sm.drain[2], el);
                mbar_wait_warp(&sm.drain[2], 0, &quiet);
            }
        }
    } else if (warp >= 8) {
        // The state of one head: thread n has its row n.
        const int k = (warp >> 2) & 1, n = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        if (k < nh) {
            const int h = group * rep + (v0 + k) / panels, panel = (v0 + k) % panels, width = min(64, a.head_dim - panel * 64);
            const int64_t v = static_cast<int64_t>(group) * rep * panels + v0 + k;  // among all panels of all heads
            float *pool = a.state != nullptr ? a.state + line * a.s_stride_line + h * a.s_stride_head + panel * 64 * a.s_stride_dim +
                                                   n * a.s_stride_state
                                             : nullptr;
            float *slot = p.seg_chunks > 0 ? p.seg_state + (unit * static_cast<int64_t>(a.num_heads) * panels + v) * kStateFloats + n : nullptr;
            f32x2 st2[32];
            {
                const bool init = FULL && segments == 1 && a.state != nullptr && p.has_initial_state != nullptr && p.has_initial_state[seq] != 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int ch = 2 * i + j;
                        f[j] = 0.0f;
                        if (FULL && segments > 1) f[j] = slot[ch * 128];
                        else if (init && ch < width && n < a.dim_state) f[j] = pool[ch * a.s_stride_dim];
                    }
                    st2[i] = pack2(f[0], f[1]);
                }
            }
            float whole = 1.0f;  // decay over all tokens
            int cleared = 0;
            bool ok = true;
            for (int c = 0; c < chunks; ++c) {
                const int stage = c & 1, rows = min(Q, e - s - c * Q);
                if (!(ok = mbar_wait_warp(&sm.gates_full[stage], (c / 2) & 1, abort))) break;
                const Gates &g = sm.gates[stage][k];
                const float ghi = g.hi[Q - 1], glo = g.lo[Q - 1];
                const float gamma = ex2_approx(ghi + glo);
                sm.weight[k][n] = g.d[n] * ex2_approx((ghi - g.hi[n]) + (glo - g.lo[n]));
                warp_arrive(&sm.gates_free[stage], lane);
                if constexpr (FULL) {
                    // the state's parts for C S, once the other head's (or the last chunk's) are used
                    const int from = k == 0 ? nh - 1 : 0, turn = k == 0 ? c - 1 : c;
                    if (turn >= 0 && !(ok = mbar_wait_warp(&sm.s_free[from], turn & 1, abort))) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t hi[4], mid[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) split_bf16x2(st2[4 * i + j], hi[j], mid[j]);
                        const int at = n * 128 + ((i ^ (n & 7)) << 4);
                        *reinterpret_cast<uint4 *>(sm.s[0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(sm.s[1] + at) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    }
                    fence_async_shared();
                    warp_arrive(&sm.s_full, lane);
                }
                // the tokens' parts, and what is wrong with the tile: rows of another sequence, values that are not finite
                if (!(ok = mbar_wait_warp(&sm.xb_full[stage], (c / 2) & 1, abort))) break;
                const bool stale = sm.any_bad[stage][k] != 0;  // of two chunks ago, whose readers are done (the stage was free)
                warp_arrive(&sm.together[k], lane);            // the weights are there, and all have looked
                if (!(ok = mbar_wait_warp(&sm.together[k], c & 1, abort))) break;
                if (stale) {
                    if (n < 64) sm.first_bad[stage][k][n] = INT_MAX;
                    if (n == 64) sm.any_bad[stage][k] = 0;
                    warp_arrive(&sm.cleared[k], lane);
                    if (!(ok = mbar_wait_warp(&sm.cleared[k], cleared & 1, abort))) break;
                    ++cleared;
                }
                uint8_t *xt = sm.x[stage][k];
                const int piece = n & 7;
                for (int q = 0; q < 4; ++q) {
                    if ((c > 0 || q > 0) && !(ok = mbar_wait_warp(&sm.w_free[k], (q - 1) & 1, abort))) break;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int in = r * 16 + (n >> 3), row = q * 32 + in, sw = (piece ^ (row & 7)) << 4;
                        uint4 x = *reinterpret_cast<const uint4 *>(xt + row * 128 + sw);
                        if (row >= rows) {
                            x = make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4 *>(xt + row * 128 + sw) = x;
                            if (k == 0) {
                                *reinterpret_cast<uint4 *>(sm.b[stage][0] + row * 128 + sw) = x;
                                *reinterpret_cast<uint4 *>(sm.b[stage][1] + row * 128 + sw) = x;
                            }
                        }
                        uint32_t word[4] = {x.x, x.y, x.z, x.w};
                        if (odd_bf16x2(word[0]) || odd_bf16x2(word[1]) || odd_bf16x2(word[2]) || odd_bf16x2(word[3])) {
                            sm.any_bad[stage][k] = 1;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t bits = (j & 1) ? word[j / 2] >> 16 : word[j / 2] & 0xffffu;
                                if ((bits & 0x7f80u) != 0x7f80u) continue;
                                atomicMin(&sm.first_bad[stage][k][piece * 8 + j], row);
                                word[j / 2] &= (j & 1) ? 0xffffu : 0xffff0000u;
                            }
                            *reinterpret_cast<uint4 *>(xt + row * 128 + sw) = make_uint4(word[0], word[1], word[2], word[3]);
                        }
                        const f32x2 wt = same2(sm.weight[k][row]);
                        uint32_t part[3][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            split_bf16x3(mul2(pack2(bf16_lo(word[j]), bf16_hi(word[j])), wt), part[0][j], part[1][j], part[2][j]);
#pragma unroll
                        for (int i = 0; i < 3; ++i)
                            *reinterpret_cast<uint4 *>(sm.w[k][i] + in * 128 + sw) = make_uint4(part[i][0], part[i][1], part[i][2], part[i][3]);
                    }
                    fence_async_shared();
                    warp_arrive(&sm.w_full[k], lane);
                }
                if (!ok) break;
                warp_arrive(&sm.x_ok[stage][k], lane);
                if (!(ok = mbar_wait_warp(&sm.sum_full[k], c & 1, abort))) break;
                tc_fence_after();
                const f32x2 g2 = same2(gamma);
#pragma unroll
                for (int i0 = 0; i0 < 64; i0 += 16) {
                    float f[16];
                    tmem_load(lanes + kColSum + k * 64 + i0, f);
                    tmem_wait_load();
#pragma unroll
                    for (int i = 0; i < 8; ++i) st2[i0 / 2 + i] = fma2(g2, st2[i0 / 2 + i], pack2(f[2 * i], f[2 * i + 1]));
                }
                tc_fence_before();
                whole *= gamma;
                if (sm.any_bad[stage][k]) {  // all of the group's arrivals are before sum_full
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float f0, f1;
                        unpack2(st2[i], f0, f1);
                        if (sm.first_bad[stage][k][2 * i] < Q) f0 = NAN;
                        if (sm.first_bad[stage][k][2 * i + 1] < Q) f1 = NAN;
                        st2[i] = pack2(f0, f1);
                    }
                }
            }
            if (!FULL || (last && a.state != nullptr)) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float f[2];
                    unpack2(st2[i], f[0], f[1]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int ch = 2 * i + j;
                        const float x = ok ? f[j] : NAN;
                        if (!FULL) slot[ch * 128] = x;
                        else if (ch < width && n < a.dim_state) pool[ch * a.s_stride_dim] = x;
                    }
                }
                if (!FULL && n == 0) p.seg_decay[static_cast<int64_t>(unit) * a.num_heads * panels + v] = whole;
            }
        }
    } else if constexpr (FULL) {
        // M and the outputs of one head: thread i has token i.
        const int k = warp >> 2, i = tid & 127, w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        if (k < nh) {
            const int h = group * rep + (v0 + k) / panels, panel = (v0 + k) % panels, width = min(64, a.head_dim - panel * 64);
            const float skip = a.D != nullptr ? a.D[h] : 0.0f;
            uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + h * a.out.stride_head + panel * 64 * a.out.stride_dim;
            const uint16_t *z = static_cast<const uint16_t *>(a.z.data) + h * a.z.stride_head + panel * 64 * a.z.stride_dim;
            // The columns of tokens after a warp's own are zero in both halves, and nothing writes them again.
            const uint32_t none[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            if (k == 0)
                for (int blk = w + 1; blk < 4; ++blk)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int j = 0; j < 2; ++j) tmem_store(lanes + kColM + (blk >> 1) * 64 + part * 32 + (blk & 1) * 16 + j * 8, none);
            tmem_wait_store();
            int c = 0;
            for (; c < chunks; ++c) {
                const int stage = c & 1, u = c * nh + k, rows = min(Q, e - s - c * Q);
                if (!mbar_wait_warp(&sm.gates_full[stage], (c / 2) & 1, abort)) break;
                const Gates &g = sm.gates[stage][k];
                const float ghi = g.hi[i], glo = g.lo[i];
                const float base_hi = w > 0 ? g.hi[w * 32 - 1] : 0.0f, base_lo = w > 0 ? g.lo[w * 32 - 1] : 0.0f;
                const float own = (ghi - base_hi) + (glo - base_lo);  // since the warp's first token
                const float here = ex2_approx(own), row_decay = ex2_approx(ghi + glo);
                float *before = sm.factor[k] + 16 * w * (w - 1);
#pragma unroll
                for (int b = 0; b < 3; ++b)
                    if (b < w) {
                        const int j = b * 32 + lane;
                        before[j] = g.d[j] * ex2_approx((base_hi - g.hi[j]) + (base_lo - g.lo[j]));
                    }
                const float own_d = g.d[i];
                warp_arrive(&sm.gates_free[stage], lane);
                bool ok = mbar_wait_warp(&sm.cb_full, c & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const f32x2 here2 = same2(here);
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    if ((blk & 1) == 0 && u >= 1 && !(ok = mbar_wait_warp(&sm.m_free[blk >> 1], (u - 1) & 1, abort))) break;
                    if (blk <= w) {
#pragma unroll
                        for (int j0 = 0; j0 < 32; j0 += 16) {
                            float f[16];
                            tmem_load(lanes + kColCB + blk * 32 + j0, f);
                            tmem_wait_load();
                            uint32_t hi[8], mid[8];
                            if (blk < w) {
#pragma unroll
                                for (int j = 0; j < 16; j += 4) {
                                    const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(before + blk * 32 + j0 + j);
                                    split_bf16x2(mul2(mul2(pack2(f[j], f[j + 1]), b2.x), here2), hi[j / 2], mid[j / 2]);
                                    split_bf16x2(mul2(mul2(pack2(f[j + 2], f[j + 3]), b2.y), here2), hi[j / 2 + 1], mid[j / 2 + 1]);
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    float m[2];
#pragma unroll
                                    for (int l = 0; l < 2; ++l) {
                                        const int t = j0 + j + l;
                                        const float gj = __shfl_sync(kFullMask, own, t), dj = __shfl_sync(kFullMask, own_d, t);
                                        m[l] = t <= lane ? f[j + l] * (dj * ex2_approx(own - gj)) : 0.0f;
                                    }
                                    split_bf16x2(pack2(m[0], m[1]), hi[j / 2], mid[j / 2]);
                                }
                            }
                            const uint32_t to = lanes + kColM + (blk >> 1) * 64 + (blk & 1) * 16 + j0 / 2;
                            tmem_store(to, hi);
                            tmem_store(to + 32, mid);
                        }
                    }
                    if (blk & 1) {
                        tmem_wait_store();
                        tc_fence_before();
                        warp_arrive(&sm.m_full[blk >> 1], lane);
                    }
                }
                if (!ok) break;
                warp_arrive(&sm.cb_free, lane);

                // out_i = e^{G_i} (C S)_i + (M x)_i + D x_i, with the gate
                if (!mbar_wait_warp(&sm.xb_full[stage], (c / 2) & 1, abort) || !mbar_wait_warp(&sm.cs_full[k], c & 1, abort) ||
                    !mbar_wait_warp(&sm.mx_full[k], c & 1, abort))
                    break;
                tc_fence_after();
                const uint8_t *xt = sm.x[stage][k] + i * 128;
                const bool bad = sm.any_bad[stage][k] != 0;
                const int64_t t = s + c * Q + i;
                const f32x2 decay2 = same2(row_decay), skip2 = same2(skip);
#pragma unroll
                for (int j0 = 0; j0 < 64; j0 += 16) {
                    float mx[16], cs[16];
                    __syncwarp();
                    tmem_load(lanes + kColMX + j0, mx);
                    tmem_load(lanes + kColCS + j0, cs);
                    tmem_wait_load();
                    if (j0 == 48) {
                        tc_fence_before();
                        warp_arrive(&sm.mx_free, lane);
                        warp_arrive(&sm.cs_free, lane);
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int ch = j0 + half * 8;
                        const uint4 x = *reinterpret_cast<const uint4 *>(xt + (((ch >> 3) ^ (i & 7)) << 4));
                        const uint32_t word[4] = {x.x, x.y, x.z, x.w};
                        f32x2 y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = half * 8 + 2 * j;
                            y[j] = fma2(decay2, pack2(cs[at], cs[at + 1]), pack2(mx[at], mx[at + 1]));
                            y[j] = fma2(skip2, pack2(bf16_lo(word[j]), bf16_hi(word[j])), y[j]);
                        }
                        if (bad) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float f0, f1;
                                unpack2(y[j], f0, f1);
                                if (sm.first_bad[stage][k][ch + 2 * j] <= i) f0 = NAN;
                                if (sm.first_bad[stage][k][ch + 2 * j + 1] <= i) f1 = NAN;
                                y[j] = pack2(f0, f1);
                            }
                        }
                        if (i >= rows || ch >= width) {
                        } else if (vec_out) {
                            if (a.z.data != nullptr) {
                                const uint4 zz = __ldg(reinterpret_cast<const uint4 *>(z + t * a.z.stride_tok + ch));
                                const uint32_t zw[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], silu2(pack2(bf16_lo(zw[j]), bf16_hi(zw[j]))));
                            }
                            *reinterpret_cast<uint4 *>(out + t * a.out.stride_tok + ch) =
                                make_uint4(f32x2_to_bf16x2(y[0]), f32x2_to_bf16x2(y[1]), f32x2_to_bf16x2(y[2]), f32x2_to_bf16x2(y[3]));
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (ch + j >= width) continue;
                                float f0, f1;
                                unpack2(y[j / 2], f0, f1);
                                float f = (j & 1) ? f1 : f0;
                                if (a.z.data != nullptr) f *= silu(bf16_bits(z[t * a.z.stride_tok + (ch + j) * a.z.stride_dim]));
                                out[t * a.out.stride_tok + (ch + j) * a.out.stride_dim] = round_bf16(f);
                            }
                        }
                    }
                }
                warp_arrive(&sm.xb_free[stage], lane);
            }
            for (; c < chunks; ++c)  // gave up
                if (s + c * Q + i < e)
                    for (int ch = 0; ch < width; ++ch) out[(s + c * Q + i) * a.out.stride_tok + ch * a.out.stride_dim] = 0x7fffu;
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

template <bool FULL, int NP>
int launch_chunks(const SsmFwd &p, const Maps &maps, int64_t units, int vec_out, cudaStream_t stream) {
    int dev = 0;
    current_device_sms(&dev);
    cudaError_t err;
    if (resident_blocks<ssm_chunk_kernel<FULL, NP>>(kThreads, kSmemBytes, dev, &err) == 0) return static_cast<int>(err);
    const int panels = (p.a.head_dim + 63) / 64, rep = p.a.num_heads / p.a.num_groups;
    const int64_t blocks = units * p.a.num_groups * ((static_cast<int64_t>(rep) * panels + 1) / 2);
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    return launch_pdl(ssm_chunk_kernel<FULL, NP>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), kSmemBytes, stream, p, maps, vec_out);
}

template <int NP>
int launch_all(const SsmFwd &p, const Maps &maps, int vec_out, cudaStream_t stream) {
    if (p.seg_chunks == 0) return launch_chunks<true, NP>(p, maps, p.batch, vec_out, stream);
    const int64_t units = segment_slots(p.total_tokens, p.batch, p.seg_chunks);
    int status = launch_chunks<false, NP>(p, maps, units, vec_out, stream);
    if (status != CCV_OK) return status;
    const int panels = (p.a.head_dim + 63) / 64;
    const int64_t joins = static_cast<int64_t>(p.batch) * p.a.num_heads * panels * (kStateFloats / 1024);
    if (joins > 0x7fffffff) return CCV_ERR_SIZE;
    status = launch_pdl(ssm_join_kernel, dim3(static_cast<unsigned>(joins)), dim3(256), 0, stream, p, panels);
    if (status != CCV_OK) return status;
    return launch_chunks<true, NP>(p, maps, units, vec_out, stream);
}

}  // namespace

bool ssm_chunked_dims(int dim_state, int a_per_state) { return !a_per_state && dim_state <= 128; }

// Chunks of a segment, or 0 to leave sequences whole, for sequences of equal lengths (their offsets are on the device).  In
// chunk times of a block: the first pass takes 0.6 of one a chunk, the two launches more take 4.  Each pass runs in waves of
// one block an SM.
int ssm_chunked_segments(int total_tokens, int batch, int num_heads, int num_groups, int head_dim) {
    const char *forced = std::getenv("CCV_SSM_SEGMENT");  // chunks of a segment (for testing and tuning)
    if (forced != nullptr) return std::atoi(forced) > 0 && std::atoi(forced) < (1 << 20) ? std::atoi(forced) : 0;
    constexpr int kSms = 152;  // a GB300's: the workspace's size may not depend on the device that is current
    const int64_t each = static_cast<int64_t>(batch) * Q;
    const int chunks = static_cast<int>((total_tokens + each - 1) / each);
    const int64_t blocks = static_cast<int64_t>(batch) * num_groups * ((static_cast<int64_t>(num_heads / num_groups) * ((head_dim + 63) / 64) + 1) / 2);
    auto waves = [](int64_t n) { return static_cast<double>((n + kSms - 1) / kSms); };
    double best = waves(blocks) * chunks;
    int choice = 0;
    for (int n = 2; n <= 64 && n <= chunks; ++n) {
        const int length = (chunks + n - 1) / n;
        const double cost = 4 + waves(blocks * (n - 1)) * length * 0.6 + waves(blocks * n) * length;
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
    return a.dim_state <= 64 ? launch_all<1>(p, maps, vec_out, stream) : launch_all<2>(p, maps, vec_out, stream);
}

}  // namespace ccv
