// Selective state space scan over varlen sequences (prefill), token by token, for layers whose channels each have their own
// step and a decay for every state, and for whatever else the chunked form does not take.
//
// A row (head h, channel p) has dim_state states in the registers of LANES lanes; a block has 32 rows (16 above 64 states) of one
// group of one sequence (or segment), LANES threads each, and goes through its tokens in tiles of as many.  The tile's inputs come
// to registers while the one before is worked on; from there the steps (one a row and token, where the lanes would each repeat it)
// go to shared memory as pairs d, d x, and B and C as floats.  For a token a lane then needs
//     e = 2^{d A log2 e},   s <- e s + (d x) B,   y += s C
// for its own states: an exponential, two multiplications and two multiply-adds a state, in pairs.  The sums over the lanes are
// taken for LANES tokens at once, halving what each lane holds at every step, so that a lane ends with one token's output.
//
// 4 x 4096 tokens of 8192 channels with 16 states take 836 us, 1.2 TB/s of what has to be moved.  Nothing in it is at its limit
// alone: shared memory is busy for 72 % of the time (each lane reads a token's B, C and steps), instructions are issued in 64 % of
// the cycles, and the exponentials need 235 us of it (32 a cycle and SM).  More lanes a row, more rows a lane, and exponentials by
// polynomials on the multiply-add pipes were all slower.  At 16 states a thread has 72 registers for seven blocks an SM, and 28
// bytes (for the segments' own states 76) go to local memory.  The same for 1009 + 37 + 300 tokens of 2048 channels, in segments of
// 128: 56 us.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "ccv_varlen.cuh"
#include "ssm_fwd.cuh"

namespace ccv {
namespace {

constexpr int kUnit = 128;    // tokens of a segment's unit

template <int LANES, int NS, int ROWS, int TOKENS>
struct ScanSmem {
    static constexpr int rows = ROWS, states = LANES * NS, T = TOKENS, threads = LANES * ROWS;
    float2 step[T][rows];        // d, d x; two rows' pairs (16 bytes) are at place_of(row / 2)
    // A thread writes eight rows of a token, so the eight threads of a token write 64 bytes apart: the places' low bits spread
    // them over the banks, and leave the rows of a warp's loads side by side.
    static __device__ __forceinline__ int place_of(int pair) { return pair ^ ((pair >> 3) & (rows / 16 - 1)); }
    float b[T][states], c[T][states];
    uint16_t x[T][rows], z[T][rows];  // outputs take the place of x
    int seq, start, end;
};

// Which of a call's tensors have rows of 16-byte pieces for a block's channels.
struct ScanVec {
    bool x, z, out, dt, bc;
};

// Eight consecutive rows' values of one token, from row `r` of the group on, as bf16 bits; rows past `count` are zero.
__device__ __forceinline__ uint4 load8(const ccv_heads_view &v, int64_t tok, int head0, int dim, int r, int count, bool vec) {
    const uint16_t *src = static_cast<const uint16_t *>(v.data) + tok * v.stride_tok;
    if (vec && r + 8 <= count) {
        const int h = r / dim;
        return __ldg(reinterpret_cast<const uint4 *>(src + (head0 + h) * v.stride_head + (r - h * dim) * v.stride_dim));
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (r + i < count) {
            const int h = (r + i) / dim;
            w[i / 2] |= static_cast<uint32_t>(src[(head0 + h) * v.stride_head + (r + i - h * dim) * v.stride_dim]) << (16 * (i & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// FULL: outputs and the sequences' final states; otherwise segments' own states and the sums of their steps, for the join.
// LANES x NS: dim_state rounded up.  PER: A has a value a state.
template <int LANES, int NS, int ROWS, int TOKENS, bool PER, bool FULL>
__global__ void __launch_bounds__(LANES * ROWS, LANES == 4 ? 7 : 1) ssm_scan_kernel(const __grid_constant__ SsmFwd p, const __grid_constant__ ScanVec vec) {
    using S = ScanSmem<LANES, NS, ROWS, TOKENS>;
    constexpr int T = S::T, kRows = S::rows, kThreads = S::threads, kPieces = kRows / 8;
    constexpr int kLoads = (T * kPieces + kThreads - 1) / kThreads;              // groups of 8 rows that a thread brings
    constexpr int kQuads = T * S::states / 4 / kThreads;                         // and of 4 states
    static_assert(kPieces >= 1 && kThreads % kPieces == 0 && T % LANES == 0 && T * S::states / 4 % kThreads == 0, "");
    __shared__ S sm;
    const ccv_ssm_args &a = p.a;
    const int tid = threadIdx.x, lane = tid % 32 / (32 / LANES);
    const int row = tid / 32 * (32 / LANES) + tid % (32 / LANES);
    const int rep = a.num_heads / a.num_groups, group_rows = rep * a.head_dim;
    const int per_group = (group_rows + kRows - 1) / kRows, blocks = a.num_groups * per_group;
    const int unit = blockIdx.x / blocks, rest = blockIdx.x % blocks;
    const int group = rest / per_group, r0 = (rest % per_group) * kRows, head0 = group * rep;
    wait_prior_grid();
    release_next_grid();

    int seq = unit, s, e, segment = 0, segments = 1;
    const int unit_tokens = p.seg_chunks * kUnit;
    if (p.seg_chunks > 0) {
        if (tid < 32) {
            int i, f, t;
            find_sequence(p.query_start_loc, p.batch, unit, unit_tokens, tid, i, f, t);
            if (tid == 0) {
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
    const bool told = tid == 0 && rest == 0 && FULL;  // counts a sequence's error
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

    // The lane's states of its row: j * 4 LANES + 4 lane + i.
    const int all_rows = a.num_heads * a.head_dim;
    const int r = r0 + row, row_head = head0 + (r < group_rows ? r / a.head_dim : 0);
    const auto pool_at = [&] {
        const int h = r / a.head_dim;
        return a.state + line * a.s_stride_line + (head0 + h) * a.s_stride_head + (r - h * a.head_dim) * a.s_stride_dim;
    };
    const auto slot_at = [&] { return p.seg_state + (static_cast<int64_t>(unit) * all_rows + head0 * a.head_dim + r) * S::states; };
    f32x2 st[NS / 2], decay[PER ? NS / 2 : 1];
    const bool kept = FULL && segments > 1, init = FULL && a.state != nullptr && p.has_initial_state != nullptr && p.has_initial_state[seq] != 0;
    {
        const bool some = r < group_rows && (kept || init);
        const float *from = !some ? a.A : kept ? slot_at() : pool_at();
        const int64_t step = kept ? 1 : a.s_stride_state;
        const float *rates = a.A + static_cast<int64_t>(row_head) * (PER ? a.dim_state : 1);
#pragma unroll
        for (int j = 0; j < NS; j += 2) {
            const int n = (j / 4) * 4 * LANES + lane * 4 + (j & 3);
            st[j / 2] = pack2(some && n < a.dim_state ? from[n * step] : 0.0f, some && n + 1 < a.dim_state ? from[(n + 1) * step] : 0.0f);
            if (PER) decay[j / 2] = pack2(n < a.dim_state ? bounded_rate(rates[n] * kLog2e) : 0.0f, n + 1 < a.dim_state ? bounded_rate(rates[n + 1] * kLog2e) : 0.0f);
        }
        if (!PER) decay[0] = pack2(bounded_rate(rates[0] * kLog2e), bounded_rate(rates[0] * kLog2e));
    }
    const float skip = FULL && a.D != nullptr && r < group_rows ? a.D[row_head] : 0.0f;

    // The next tile's inputs: token tid / kPieces (+ ..), 8 rows.
    const int piece = tid % kPieces, tok = tid / kPieces, at = r0 + piece * 8;
    const auto loads = [&](int l) { return tok + l * (kThreads / kPieces) < T; };
    constexpr int kStep = kThreads / kPieces;  // tokens between a thread's loads
    uint4 xr[kLoads], zr[kLoads], dr[kLoads][2];
    uint2 br[kQuads], cr[kQuads];
    auto load_quad = [&](const ccv_heads_view &v, int64_t t, int n) {
        const uint16_t *src = static_cast<const uint16_t *>(v.data) + t * v.stride_tok + group * v.stride_head + n * v.stride_dim;
        if (vec.bc && n + 4 <= a.dim_state) return __ldg(reinterpret_cast<const uint2 *>(src));
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = n + i < a.dim_state ? src[i * v.stride_dim] : 0u;
        return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    };
    auto fetch = [&](int t0) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
            const int64_t t = t0 + tok + l * kStep;
            const bool in = loads(l) && t < e;
            xr[l] = zr[l] = dr[l][0] = dr[l][1] = make_uint4(0u, 0u, 0u, 0u);
            if (!in) continue;
            xr[l] = load8(a.x, t, head0, a.head_dim, at, group_rows, vec.x);
            if (FULL && a.z.data != nullptr) zr[l] = load8(a.z, t, head0, a.head_dim, at, group_rows, vec.z);
            const int64_t off = t * a.dt_stride_tok;
            if (vec.dt && at + 8 <= group_rows) {  // head_dim is 1
                if (a.dt_fp32) {
                    const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(a.dt) + off + head0 + at);
                    const float4 f = __ldg(src), g = __ldg(src + 1);
                    dr[l][0] = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
                    dr[l][1] = make_uint4(__float_as_uint(g.x), __float_as_uint(g.y), __float_as_uint(g.z), __float_as_uint(g.w));
                } else {
                    dr[l][0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.dt) + off + head0 + at));
                }
            } else {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[i] = 0u;
                    if (at + i < group_rows)
                        w[i] = __float_as_uint(ssm_raw_step(a, off + (head0 + (at + i) / a.head_dim) * a.dt_stride_head));
                }
                if (a.dt_fp32) {
                    dr[l][0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dr[l][1] = make_uint4(w[4], w[5], w[6], w[7]);
                } else {
                    dr[l][0] = make_uint4((w[0] >> 16) | w[1], (w[2] >> 16) | w[3], (w[4] >> 16) | w[5], (w[6] >> 16) | w[7]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int quad = tid + i * kThreads, n = quad % (S::states / 4) * 4;
            const int64_t t = t0 + quad / (S::states / 4);
            br[i] = t < e ? load_quad(a.B, t, n) : make_uint2(0u, 0u);
            if (FULL) cr[i] = t < e ? load_quad(a.C, t, n) : make_uint2(0u, 0u);
        }
    };
    f32x2 bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto of = [&](int r) { return a.dt_bias != nullptr && r < group_rows ? a.dt_bias[head0 + r / a.head_dim] : 0.0f; };
        bias[i] = pack2(of(at + 2 * i), of(at + 2 * i + 1));
    }
    const bool limits = a.dt_max < INFINITY || !(a.dt_min <= (a.dt_softplus ? 0.0f : -INFINITY));
    auto widen = [](uint2 w) { return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)); };
    float sum_d = 0.0f;  // of the row's steps
    const int row_at = 2 * S::place_of(row / 2) + (row & 1);

    fetch(s);
    for (int t0 = s; t0 < e; t0 += T) {
        const int n = min(T, e - t0);
        // what was fetched, to shared memory
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
            const int t = tok + l * kStep;
            if (!loads(l)) continue;
            const uint32_t xw[4] = {xr[l].x, xr[l].y, xr[l].z, xr[l].w};
            const uint32_t d0[4] = {dr[l][0].x, dr[l][0].y, dr[l][0].z, dr[l][0].w}, d1[4] = {dr[l][1].x, dr[l][1].y, dr[l][1].z, dr[l][1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x2 d = a.dt_fp32 ? pack2(__uint_as_float(i < 2 ? d0[2 * (i & 1)] : d1[2 * (i & 1)]),
                                            __uint_as_float(i < 2 ? d0[2 * (i & 1) + 1] : d1[2 * (i & 1) + 1]))
                                    : pack2(bf16_lo(d0[i]), bf16_hi(d0[i]));
                d = add2(d, bias[i]);
                if (a.dt_softplus) d = softplus2(d);
                float f0, f1, g0, g1;
                unpack2(d, f0, f1);
                if (limits) {
                    f0 = f0 < a.dt_min ? a.dt_min : f0 > a.dt_max ? a.dt_max : f0;
                    f1 = f1 < a.dt_min ? a.dt_min : f1 > a.dt_max ? a.dt_max : f1;
                    d = pack2(f0, f1);
                }
                unpack2(mul2(d, pack2(bf16_lo(xw[i]), bf16_hi(xw[i]))), g0, g1);
                *reinterpret_cast<float4 *>(&sm.step[t][2 * S::place_of(piece * 4 + i)]) =
                    t < n ? make_float4(f0, g0, f1, g1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            if (FULL) {
                *reinterpret_cast<uint4 *>(&sm.x[t][piece * 8]) = xr[l];
                if (a.z.data != nullptr) *reinterpret_cast<uint4 *>(&sm.z[t][piece * 8]) = zr[l];
            }
        }
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            const int quad = tid + i * kThreads, at_n = quad % (S::states / 4) * 4, t = quad / (S::states / 4);
            *reinterpret_cast<float4 *>(&sm.b[t][at_n]) = widen(br[i]);
            if (FULL) *reinterpret_cast<float4 *>(&sm.c[t][at_n]) = widen(cr[i]);
        }
        __syncthreads();
        if (t0 + T < e) fetch(t0 + T);

        // Sums first and outputs after them: a store to shared memory would keep the next tokens' loads behind it.
        float sums[T / LANES];
#pragma unroll
        for (int g = 0; g < T; g += LANES) {  // tokens whose sums are taken together
            float y[LANES];
#pragma unroll
            for (int l = 0; l < LANES; ++l) {
                const float2 step = sm.step[g + l][row_at];
                const f32x2 d2 = pack2(step.x, step.x), dx2 = pack2(step.y, step.y);
                f32x2 acc = 0ull, same = 0ull;
                if constexpr (!PER) {
                    float u0, u1;
                    unpack2(mul2(d2, decay[0]), u0, u1);
                    const float a1 = ex2_approx(u0);
                    same = pack2(a1, a1);
                }
                if (!FULL) sum_d += step.x;
#pragma unroll
                for (int j = 0; j < NS; j += 4) {
                    const ulonglong2 b2 = *reinterpret_cast<const ulonglong2 *>(&sm.b[g + l][j * LANES + lane * 4]);
                    ulonglong2 c2 = make_ulonglong2(0ull, 0ull);
                    if (FULL) c2 = *reinterpret_cast<const ulonglong2 *>(&sm.c[g + l][j * LANES + lane * 4]);
                    f32x2 e0 = same, e1 = same;
                    if constexpr (PER) {
                        float u0, u1, u2, u3;
                        unpack2(mul2(d2, decay[j / 2]), u0, u1);
                        unpack2(mul2(d2, decay[j / 2 + 1]), u2, u3);
                        e0 = pack2(ex2_approx(u0), ex2_approx(u1));
                        e1 = pack2(ex2_approx(u2), ex2_approx(u3));
                    }
                    st[j / 2] = fma2(e0, st[j / 2], mul2(dx2, b2.x));
                    st[j / 2 + 1] = fma2(e1, st[j / 2 + 1], mul2(dx2, b2.y));
                    if constexpr (FULL) {
                        acc = j == 0 ? mul2(st[0], c2.x) : fma2(st[j / 2], c2.x, acc);
                        acc = fma2(st[j / 2 + 1], c2.y, acc);
                    }
                }
                float lo, hi;
                unpack2(acc, lo, hi);
                y[l] = lo + hi;
            }
            if constexpr (FULL) {
                // y[i] summed over the lanes for lane i: at each step a lane keeps the half of the sums that has its bit
#pragma unroll
                for (int m = LANES / 2; m > 0; m >>= 1)
#pragma unroll
                    for (int l = 0; l < m; ++l) {
                        const bool upper = (lane & m) != 0;
                        const float keep = upper ? y[l + m] : y[l], give = upper ? y[l] : y[l + m];
                        y[l] = keep + __shfl_xor_sync(kFullMask, give, m * (32 / LANES));
                    }
                sums[g / LANES] = y[0];
            }
        }
        if constexpr (FULL) {
#pragma unroll
            for (int g = 0; g < T; g += LANES) {
                const int t = g + lane;
                float o = fmaf(skip, bf16_bits(sm.x[t][row]), sums[g / LANES]);
                if (a.z.data != nullptr) o *= silu(bf16_bits(sm.z[t][row]));
                sm.x[t][row] = round_bf16(o);
            }
        }
        __syncthreads();
        if constexpr (FULL) {
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                const int t = tok + l * kStep;
                if (!loads(l) || t >= n) continue;
                uint16_t *to = static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + (t0 + t) * a.out.stride_tok;
                if (vec.out && at + 8 <= group_rows) {
                    const int oh = at / a.head_dim;
                    *reinterpret_cast<uint4 *>(to + (head0 + oh) * a.out.stride_head + (at - oh * a.head_dim) * a.out.stride_dim) =
                        *reinterpret_cast<const uint4 *>(&sm.x[t][piece * 8]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (at + i < group_rows) {
                            const int oh = (at + i) / a.head_dim;
                            to[(head0 + oh) * a.out.stride_head + (at + i - oh * a.head_dim) * a.out.stride_dim] = sm.x[t][piece * 8 + i];
                        }
                }
            }
            // the same thread writes these places of x next
        }
    }

    if (r >= group_rows) return;
    if (!FULL || (last && a.state != nullptr)) {
        float *to = FULL ? pool_at() : slot_at();
        const int64_t step = FULL ? a.s_stride_state : 1;
#pragma unroll
        for (int j = 0; j < NS; j += 2) {
            const int n = (j / 4) * 4 * LANES + lane * 4 + (j & 3);
            float f0, f1;
            unpack2(st[j / 2], f0, f1);
            if (n < a.dim_state) to[n * step] = f0;
            if (n + 1 < a.dim_state) to[(n + 1) * step] = f1;
        }
    }
    if (!FULL && lane == 0) p.seg_decay[static_cast<int64_t>(unit) * all_rows + head0 * a.head_dim + r] = sum_d;
}

// The segments' first states, one after the other, from their own: F <- e^{A sum of d} F + own, a thread a row and state; the
// first segment's is a copy of the pool's, whose line the last segment writes while the first may still start.
__global__ void __launch_bounds__(256) ssm_scan_join_kernel(const __grid_constant__ SsmFwd p, int states) {
    const ccv_ssm_args &a = p.a;
    wait_prior_grid();
    release_next_grid();
    const int rows = a.num_heads * a.head_dim;
    const int64_t per_seq = (static_cast<int64_t>(rows) * a.dim_state + 255) / 256;
    const int seq = static_cast<int>(blockIdx.x / per_seq);
    const int64_t at = blockIdx.x % per_seq * 256 + threadIdx.x;
    const int s = p.query_start_loc[seq], e = p.query_start_loc[seq + 1], unit = p.seg_chunks * kUnit;
    if (at >= static_cast<int64_t>(rows) * a.dim_state || !sequence_ok(s, e, p.total_tokens) || e - s <= unit) return;
    const int line = p.cache_indices != nullptr ? p.cache_indices[seq] : seq;
    if (line == a.pad_slot_id || (a.state != nullptr && (line < 0 || line >= a.num_lines))) return;
    const int row = static_cast<int>(at / a.dim_state), n = static_cast<int>(at % a.dim_state), h = row / a.head_dim, ch = row % a.head_dim;
    const int segments = (e - s + unit - 1) / unit;
    const float rate = bounded_rate(a.A[a.a_per_state ? static_cast<int64_t>(h) * a.dim_state + n : h]);
    float f = 0.0f;
    if (a.state != nullptr && p.has_initial_state != nullptr && p.has_initial_state[seq] != 0)
        f = a.state[line * a.s_stride_line + h * a.s_stride_head + ch * a.s_stride_dim + n * a.s_stride_state];
    const int64_t slot = first_slot(s, seq, unit);
    float *to = p.seg_state + (slot * rows + row) * states + n;
    const float *sum = p.seg_decay + slot * rows + row;
    const int64_t next = static_cast<int64_t>(rows) * states;
    float own = *to, d = *sum;  // there are two segments at least; the last one's own are not wanted
    for (int i = 0; i < segments; ++i) {
        const bool more = i + 2 < segments;
        const float own1 = more ? to[next] : 0.0f, d1 = more ? sum[rows] : 0.0f;  // ahead of the store, behind which they would wait
        *to = f;
        f = fmaf(expf(d * rate), f, own);
        own = own1;
        d = d1;
        to += next;
        sum += rows;
    }
}

int64_t segment_slots(int total_tokens, int batch, int seg_units) {
    return static_cast<int64_t>(total_tokens) / (static_cast<int64_t>(seg_units) * kUnit) + batch;
}
// States that a row has room for.
int padded_states(int dim_state) { return dim_state <= 16 ? 16 : dim_state <= 32 ? 32 : dim_state <= 64 ? 64 : dim_state <= 128 ? 128 : 256; }

template <int LANES, int NS, int ROWS, int TOKENS, bool PER>
int launch_scan(const SsmFwd &p, const ScanVec &vec, cudaStream_t stream) {
    const int rows = ROWS, group_rows = p.a.num_heads / p.a.num_groups * p.a.head_dim;
    const int64_t blocks = static_cast<int64_t>(p.a.num_groups) * ((group_rows + rows - 1) / rows);
    const int64_t units = p.seg_chunks > 0 ? segment_slots(p.total_tokens, p.batch, p.seg_chunks) : p.batch;
    if (blocks * units > 0x7fffffff) return CCV_ERR_SIZE;
    const dim3 grid(static_cast<unsigned>(blocks * units)), block(LANES * ROWS);
    if (p.seg_chunks > 0) {
        int status = launch_pdl(ssm_scan_kernel<LANES, NS, ROWS, TOKENS, PER, false>, grid, block, 0, stream, p, vec);
        if (status != CCV_OK) return status;
        const int64_t joins = p.batch * ((static_cast<int64_t>(p.a.num_heads) * p.a.head_dim * p.a.dim_state + 255) / 256);
        if (joins > 0x7fffffff) return CCV_ERR_SIZE;
        status = launch_pdl(ssm_scan_join_kernel, dim3(static_cast<unsigned>(joins)), dim3(256), 0, stream, p, LANES * NS);
        if (status != CCV_OK) return status;
    }
    return launch_pdl(ssm_scan_kernel<LANES, NS, ROWS, TOKENS, PER, true>, grid, block, 0, stream, p, vec);
}

// Lanes a row, states a lane, rows and tokens a tile by what is fastest for 2 x 2048 ungated tokens of 4096 channels: 32 states 235 us (16
// rows 250, 4 x 8 lanes 329), 64 states 337 (16 rows 369, 16 x 4 lanes 508), 128 states 664 (16 x 8 lanes 717 to 1170, 32 tokens
// 850), 256 states 1330 (8 rows 2256).
template <bool PER>
int launch_states(const SsmFwd &p, const ScanVec &vec, cudaStream_t stream) {
    const int n = p.a.dim_state;
    if (n <= 16) return launch_scan<4, 4, 32, 32, PER>(p, vec, stream);
    if (n <= 32) return launch_scan<8, 4, 32, 32, PER>(p, vec, stream);
    if (n <= 64) return launch_scan<8, 8, 32, 32, PER>(p, vec, stream);
    if (n <= 128) return launch_scan<8, 16, 16, 16, PER>(p, vec, stream);
    return launch_scan<16, 16, 16, 16, PER>(p, vec, stream);
}

}  // namespace

int64_t ssm_scan_workspace(int total_tokens, int batch, int num_heads, int head_dim, int dim_state, int seg_units) {
    if (seg_units == 0) return 0;
    const int64_t rows = segment_slots(total_tokens, batch, seg_units) * num_heads * head_dim;
    return rows * padded_states(dim_state) * 4 + (rows * 4 + 127) / 128 * 128;
}

// Units of 128 tokens of a segment, or 0 to leave sequences whole.  Offsets are on the device, so the longest sequence is taken to
// be halfway between the average and all tokens.  In ns, as measured: a token takes `lone` in a block with an SM to itself, and
// `first` and `each` more for each of the blocks that an SM has; cutting does part of the work once more and costs a block the time
// of some tokens (`start`), a segment of the join takes 700 and the two launches 8000.
// 16 states: 5000 tokens of 4096 channels take 216 us so (segments of 256) and 381 whole, 2000 of 2048 channels 60 and 154; 4 x 4096
// of 8192 channels 836 whole and 1150 in segments of 1024.  More states, without a gate: 2000 tokens of 512 channels with 256
// states 161 and 330; 2 x 2048 of 4096 channels with 32 states 235 whole and 525 in segments of 128.
int ssm_scan_segments(int total_tokens, int batch, int num_heads, int num_groups, int head_dim, int dim_state) {
    const char *forced = std::getenv("CCV_SSM_SEGMENT");  // (for testing and tuning)
    if (forced != nullptr) return std::atoi(forced) > 0 && std::atoi(forced) < (1 << 20) ? std::atoi(forced) : 0;
    constexpr double kSms = 152;  // a GB300's: the workspace's size may not depend on the device that is current
    struct Cost {
        double rows, lone, first, each, again, start;
    };
    const Cost t = dim_state <= 16    ? Cost{32, 73, 45, 28, 0.6, 0}
                   : dim_state <= 32  ? Cost{32, 57, 0, 68, 0.4, 100}
                   : dim_state <= 64  ? Cost{32, 82, 0, 82, 0.4, 100}
                   : dim_state <= 128 ? Cost{16, 124, 0, 96, 0.4, 100}
                                      : Cost{16, 165, 0, 193, 0.4, 100};
    const double blocks = num_groups * std::ceil(static_cast<double>(num_heads / num_groups) * head_dim / t.rows);
    const double average = static_cast<double>(total_tokens) / batch, longest = 0.5 * (average + total_tokens);
    const auto token = [&](double n) { return n <= kSms ? t.lone : t.first + t.each * std::ceil(n / kSms); };  // of n blocks
    double best = std::max(average * token(blocks * batch), longest * token(blocks));
    int choice = 0;
    for (int units = 1; units <= 64 && units * kUnit < longest; ++units) {
        const double tokens = units * kUnit, segments = std::ceil(average / tokens) * batch;
        const double cost = (1 + t.again) * (tokens + t.start) * token(blocks * segments) + 700 * longest / tokens + 8000;
        if (cost < best) {
            best = cost;
            choice = units;
        }
    }
    return choice;
}

int ssm_launch_scan(const SsmFwd &call, void *workspace, cudaStream_t stream) {
    SsmFwd p = call;
    const ccv_ssm_args &a = p.a;
    if (p.seg_chunks > 0) {
        const int64_t rows = segment_slots(p.total_tokens, p.batch, p.seg_chunks) * a.num_heads * a.head_dim;
        p.seg_state = static_cast<float *>(workspace);
        p.seg_decay = p.seg_state + rows * padded_states(a.dim_state);
    }
    // A block's rows are contiguous, and start on 16 bytes: one channel a head, or whole heads of contiguous channels.
    const int group_rows = a.num_heads / a.num_groups * a.head_dim;
    auto rows_ok = [&](const ccv_heads_view &v) {
        if (v.data == nullptr || !aligned16(v.data) || v.stride_tok % 8 != 0 || (a.num_groups > 1 && group_rows % 8 != 0)) return false;
        if (a.head_dim == 1) return v.stride_head == 1;
        return v.stride_dim == 1 && v.stride_head % 8 == 0 && a.head_dim % 8 == 0;
    };
    auto states_ok = [&](const ccv_heads_view &v) {
        return (reinterpret_cast<uintptr_t>(v.data) & 7u) == 0 && v.stride_dim == 1 && v.stride_tok % 4 == 0 && (a.num_groups == 1 || v.stride_head % 4 == 0);
    };
    ScanVec vec;
    vec.x = rows_ok(a.x);
    vec.z = rows_ok(a.z);
    vec.out = rows_ok(a.out);
    vec.dt = a.head_dim == 1 && aligned16(a.dt) && a.dt_stride_head == 1 && a.dt_stride_tok % 8 == 0 && (a.num_groups == 1 || group_rows % 8 == 0);
    vec.bc = states_ok(a.B) && states_ok(a.C);
    return a.a_per_state ? launch_states<true>(p, vec, stream) : launch_states<false>(p, vec, stream);
}

}  // namespace ccv
