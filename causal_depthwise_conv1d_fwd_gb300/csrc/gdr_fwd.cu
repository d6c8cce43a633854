// Gated delta rule over varlen sequences (prefill), chunked form on the tensor cores.
//
// A chunk holds C = 64 tokens.  With k and q as normalised, G the running sum of g inside the chunk, and d_j the delta of
// token j, unrolling the recurrence gives
//     (I + A) d = R,   A_ij = b_i (k_i . k_j) e^{G_i - G_j}  (j < i),   R_j = b_j (v_j - e^{G_j} S k_j)
//     o_i = e^{G_i} S q_i + sum_{j <= i} P_ij d_j,   P_ij = (q_i . k_j) e^{G_i - G_j}
//     S  <- e^{G_C} S + sum_j e^{G_C - G_j} d_j k_j^T
// Only the products with S are sequential, so there are two kernels:
//   gdr_prep_kernel   for every chunk and key head at once: the two products, the decays, T = (I + A)^-1, P, and what each
//                     token multiplies by; written to the workspace in the layout the tensor cores read.
//   gdr_chunk_kernel  for every sequence and value head: the chunks in order with S^T kept on chip.
// 4 x 4096 tokens with 32 value heads take 267 us: 95 + 174 and the launches, less what overlaps.
// Where sequences and heads are too few for the card, each sequence is cut into segments of chunks.  A segment takes its
// first state to S M + N; gdr_chunk_kernel first finds N (the segment from a zero state) and M (from the identity, without
// values) of all segments at once, gdr_join_kernel goes through them for each segment's first state, and gdr_chunk_kernel
// then runs all segments from there.  That is three times the work on as many more SMs as there are segments.
//
// Precision.  The state is fp32, so the operands of every product that reaches it keep 24 bits: k and q enter as their own bf16
// values (exact; their norms are factors of a token, applied to sums), and each inexact operand (S, R, T, d) as three bf16
// parts, of whose products the ones above 2^-24 are kept: 3 with an exact operand, 6 without.  T itself is good to 2^-21 of the
// products that it is made of (see multiply_lower), the decays to 2^-22.  The parts' products are added smallest first: the
// tensor cores' sums truncate, each step losing up to 2^-23 of what the sum holds by then.  In the other order the state of
// 500 tokens was 3.2e-7 of itself off instead of 8.6e-8 (the recurrent form: 7.9e-8).  Products that reach the output alone keep
// 16 bits an operand (the output has 8): 0.26% of the outputs are a bf16 step away from the exact result's rounding, and their
// distance from it is that of the rounding itself (0.00166).  bf16 parts span the range of fp32, so nothing needs scaling and
// nothing overflows or vanishes that would not in fp32, however far e^G falls inside a chunk.
//
// What is not finite.  A sum over a chunk takes zeros for the tokens after its own, and 0 * NaN is NaN.  So a token whose key or
// gates are not finite, and a value that is not, are left out of the products; the outputs of the rows that they reach are NaN
// from that token on, and so is the rows' final state, and tokens before it are what they are without it.  A row of the state
// that starts with something not finite is NaN throughout.  (What overflows on the way, from finite inputs, can reach all of
// its chunk.)  The loading warps look at each chunk's values while the one before is worked on, which costs nothing that can
// be measured on 4 x 4096 tokens and 1% on 11027 (the same look by the computing warps cost 2 to 4%).
#include <climits>
#include <cstdlib>
#include <cstring>

#include "ccv_varlen.cuh"
#include "gdr_common.cuh"

namespace ccv {
namespace {

constexpr int C = 64;            // tokens of a chunk
constexpr int kTile = C * 128;   // bytes of 64 rows of 64 bf16 values
constexpr int kScalars = 5;      // vectors of C floats a (chunk, value head) carries
enum { kBeta, kKey, kState, kQuery, kMisc };  // their order; kMisc[0] is e^{G_C}
enum { kT = 0, kP = 3 * kTile, kVec = 5 * kTile };              // T in 3 parts, P in 2, the vectors
constexpr int kHeadBytes = kVec + kScalars * C * 4;

struct FwdArgs {
    ccv_gdr_args a;
    const int32_t *query_start_loc, *cache_indices;
    const uint8_t *has_initial_state;
    int batch, total_tokens, slots;
    uint8_t *heads;  // (slots, num_v_heads) blocks of kHeadBytes
    int *err_count;
    int seg_chunks;  // chunks of a segment; 0: sequences are not cut
    float *seg_state, *seg_step;  // (segment slots, num_v_heads, dim_v or dim_k, 64 panels): first states, and M
};

// Tensor maps (dim, head, token) of q, k and v with boxes of 64 values x 64 tokens; `use` is false where the tensors'
// strides do not allow them.
struct FwdMaps {
    CUtensorMap q, k, v;
    bool use;
};

// Swizzled tiles need shared memory on a 1024-byte boundary.
__device__ __forceinline__ bool misplaced(const void *smem, int *err_count) {
    const bool bad = (smem_u32(smem) & 1023u) != 0;
    if (bad) {
        wait_prior_grid();
        if (threadIdx.x == 0) count_error(err_count);
    }
    return bad;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Copies 64 rows (of which the first n are real) of a head's bf16 vectors into swizzled tiles of 64 values a row, `PANELS`
// tiles `panel_bytes` apart, zeros past n and past dim; by COUNT threads `id`.  VEC: 16-byte asynchronous copies.
template <int PANELS, bool VEC, int COUNT>
__device__ __forceinline__ void stage_rows(uint8_t *tile, int panel_bytes, const ccv_heads_view &view, int64_t tok, int head, int n,
                                           int dim, int id) {
    constexpr int kPieces = 8 * PANELS, kStep = COUNT / kPieces;
    static_assert(C % kStep == 0, "");
    const int piece = id % kPieces, row0 = id / kPieces;
    const uint16_t *src = static_cast<const uint16_t *>(view.data) + (tok + row0) * view.stride_tok + head * view.stride_head;
    const int64_t step = kStep * view.stride_tok;
    uint8_t *dst = tile + (piece >> 3) * panel_bytes + row0 * 128;
    const bool wide = piece * 8 < dim;
    if constexpr (VEC) {
        src += piece * 8;
        const uint32_t to = smem_u32(dst);
#pragma unroll
        for (int i = 0; i < C / kStep; ++i) {
            const int row = row0 + i * kStep;
            const bool real = wide && row < n;
            cp_async16_or_zero(to + i * kStep * 128 + (((piece ^ row) & 7) << 4), real ? src : static_cast<const uint16_t *>(view.data), real);
            src += step;
        }
    } else {
        for (int i = 0; i < C / kStep; ++i) {
            const int row = row0 + i * kStep;
            Raw<8> r;
            r.zero();
            if (row < n) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (piece * 8 + k < dim) r.set_elem(k, src[(piece * 8 + k) * view.stride_dim]);
            }
            *reinterpret_cast<uint4 *>(dst + i * kStep * 128 + (((piece ^ row) & 7) << 4)) = r.v;
            src += step;
        }
    }
}

// ------------------------------------------------------------------ prep ----

constexpr int kPrepThreads = 128;
constexpr int kLd = 68;  // floats of a row of A in shared memory: 16-byte rows, spread over the banks

struct PrepSmem {
    float ghi[2][C], glo[2][C];    // G log2(e) as a float pair
    float beta[2][C];
    float from[2][C / 2];          // e^{G_31 - G_j} times the factor of row j of K, j < 32
    float rk[C], rq[C];            // factors of the rows of K and Q
    uint4 rows[2][2][32 * 8];      // 32 rows of P in two parts, on their way out, a warp each
    int64_t carry[2];
    uint64_t bar;
    uint32_t tmem;
    int seq, start, end, abort;
    int odd;  // a token's key or a strength is not finite
};
constexpr int kMatrixBytes = 2 * C * kLd * 4;  // A, then T, of two value heads; over the rows of K and Q once they are used

// T21 = -T22 (A21 T11) in columns l .. l + 15 of the lower left quarter of the 16 S x 16 S block at d (leading dimension kLd),
// over A21, by a warp on the tensor cores; `sync` comes between the last read and the first write.  Each value goes in as two
// tf32 parts (11 bits each; the second by the unit's own truncation) and three of their products are added, so the result is
// good to 2^-21.  (A21 T11)^T leaves the first product as the second one takes its operand: a lane's accumulators, of two
// rows next to each other, are its two values of an inner step.
template <int S, typename Sync>
__device__ __forceinline__ void multiply_lower(float *d, int l, int lane, Sync sync) {
    const int g = lane >> 2, t = lane & 3;
    const float *t11 = d, *t22 = d + 8 * S * kLd + 8 * S;
    float *a21 = d + 8 * S * kLd;
    auto parts = [](float x, uint32_t &hi, uint32_t &lo) {
        hi = __float_as_uint(x) & 0xffffe000u;
        lo = __float_as_uint(x - __uint_as_float(hi));
    };
    auto mma = [](float (&c)[4], const uint32_t (&x)[4], const uint32_t (&y)[2]) {
        asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(y[0]), "r"(y[1]));
    };
    float x[S][4], y[S / 2][2][4];
#pragma unroll
    for (int n = 0; n < S; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = y[n / 2][n & 1][i] = 0.0f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
        if (8 * k < l) continue;  // T11 has zeros there
        uint32_t ah[4], al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) parts(t11[(8 * k + t + 4 * (i >> 1)) * kLd + l + g + 8 * (i & 1)], ah[i], al[i]);
#pragma unroll
        for (int n = 0; n < S; ++n) {
            uint32_t bh[2], bl[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) parts(a21[(8 * n + g) * kLd + 8 * k + t + 4 * i], bh[i], bl[i]);
            mma(x[n], al, bh);
            mma(x[n], ah, bl);
            mma(x[n], ah, bh);
        }
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
        uint32_t bh[2][2], bl[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) parts(x[k][i], bh[i >> 1][i & 1], bl[i >> 1][i & 1]);
#pragma unroll
        for (int m = k / 2; m < S / 2; ++m) {  // T22 has zeros in the rows before
            uint32_t ah[4], al[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 v = *reinterpret_cast<const float2 *>(t22 + (16 * m + g + 8 * h) * kLd + 8 * k + 2 * t);
                parts(v.x, ah[h], al[h]);
                parts(v.y, ah[h + 2], al[h + 2]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mma(y[m][c], al, bh[c]);
                mma(y[m][c], ah, bl[c]);
                mma(y[m][c], ah, bh[c]);
            }
        }
    }
    sync();
#pragma unroll
    for (int m = 0; m < S / 2; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2 *>(a21 + (16 * m + g + 8 * h) * kLd + l + 8 * c + 2 * t) = make_float2(-y[m][c][2 * h], -y[m][c][2 * h + 1]);
}

// T = (I + A)^-1 for the unit lower triangular 64 x 64 matrices of two heads (strictly lower part A, zeros above), by the
// block's 128 threads: forward substitution of the diagonal 16 x 16 blocks, then twice T21 = -T22 (A21 T11), which doubles
// the blocks.  Substitution and not a power series: its error stays at the rounding of T however alike the keys are.
// Substitution reads a value of A for every column, and a broadcast load fills the shared-memory pipe like any other: done
// for all 64 columns it took 17400 cycles a block (4 blocks an SM), and takes 8000 this way with the products on the tensor
// cores.
__device__ __forceinline__ void invert(float *matrices, int tid) {
    const int warp = tid >> 5, lane = tid & 31;
    if (tid < 64) {  // 8 blocks, two columns a thread, pairs of rows; by the warps that wrote A, while the others are at P
        asm volatile("bar.sync 1, 64;" ::: "memory");
        const int which = tid >> 3, j = (tid & 7) * 2;
        float *d = matrices + (which >> 2) * (C * kLd) + (which & 3) * (16 * kLd + 16);
        f32x2 t[2][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[0][i] = t[1][i] = 0ull;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            f32x2 acc[2][2] = {{0ull, 0ull}, {0ull, 0ull}};
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(d + i * kLd + m);
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    acc[col][0] = fma2(r.x, t[col][m / 2], acc[col][0]);
                    if (m + 2 < i) acc[col][1] = fma2(r.y, t[col][m / 2 + 1], acc[col][1]);
                }
            }
#pragma unroll
            for (int col = 0; col < 2; ++col) {
                float lo, hi;
                unpack2(add2(acc[col][0], acc[col][1]), lo, hi);
                const float x = (i == j + col ? 1.0f : 0.0f) - (lo + hi);
                unpack2(t[col][i / 2], lo, hi);
                t[col][i / 2] = (i & 1) ? pack2(lo, x) : pack2(x, hi);
            }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a0, a1, b0, b1;
            unpack2(t[0][i], a0, a1);
            unpack2(t[1][i], b0, b1);
            *reinterpret_cast<float2 *>(d + (2 * i) * kLd + j) = make_float2(a0, b0);
            *reinterpret_cast<float2 *>(d + (2 * i + 1) * kLd + j) = make_float2(a1, b1);
        }
    }
    __syncthreads();
    float *a = matrices + (warp >> 1) * (C * kLd);
    multiply_lower<2>(a + (warp & 1) * (32 * kLd + 32), 0, lane, [] { __syncwarp(); });  // to 32 x 32, a warp a block
    __syncthreads();
    multiply_lower<4>(a, 16 * (warp & 1), lane, [] { __syncthreads(); });  // to 64 x 64, half of the columns a warp
    __syncthreads();
}

// A block of 4 warps a (chunk, key head), 4 blocks an SM: 4096 of them (4 x 4096 tokens, 16 key and 32 value heads) take 95 us.
// It writes 344 MB, 3.6 TB/s; what bounds it is latency (44% of the issue slots, 50% of the shared-memory pipe): loads that
// wait on the search, 14 barriers, and forward substitution.  3, 5 and 6 blocks an SM and 8 warps a block were slower.
// PANELS: dim_k rounded up to 64 PANELS.  V: rows of q and k allow 16-byte vectors.
template <int PANELS, bool V>
__global__ void __launch_bounds__(kPrepThreads, 4) gdr_prep_kernel(const __grid_constant__ FwdArgs p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ab = smem_raw;  // on a 1024-byte boundary, since the kernel has no static shared memory (checked below)
    float *matrices = reinterpret_cast<float *>(ab);
    PrepSmem &sm = *reinterpret_cast<PrepSmem *>(ab + kMatrixBytes);
    static_assert(kMatrixBytes >= PANELS * 2 * kTile && kMatrixBytes % 16 == 0, "");
    const ccv_gdr_args &a = p.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hk = blockIdx.x % a.num_k_heads, slot = blockIdx.x / a.num_k_heads;
    wait_prior_grid();
    release_next_grid();
    if (misplaced(smem_raw, p.err_count)) return;

    if (warp == 0) {
        int seq, s, e;
        find_sequence(p.query_start_loc, p.batch, slot, C, lane, seq, s, e);
        if (lane == 0) {
            sm.seq = seq;
            sm.start = s;
            sm.end = e;
        }
    }
    if (tid == 32) {
        sm.abort = sm.odd = 0;
        mbar_init(&sm.bar, 1);
        mbar_init_fence();
    }
    __syncthreads();
    const int seq = sm.seq, s = sm.start, e = sm.end;
    if (!sequence_ok(s, e, p.total_tokens)) return;  // counted by the chunk kernel
    const int chunk = slot - first_slot(s, seq, C);
    if (chunk < 0 || chunk * C >= e - s) return;
    if (p.cache_indices != nullptr && p.cache_indices[seq] == a.pad_slot_id) return;
    const int t0 = s + chunk * C, n = min(C, e - t0);

    // The value heads of this key head go two at a time, 64 threads each.
    const int i = tid & (C - 1), side = tid >> 6;
    const int rep = a.num_v_heads / a.num_k_heads;
    GdrGates gates;
    auto load_gates = [&](int r0) {
        const int h = hk * rep + min(r0 + side, rep - 1);
        if (i < n) gates.load(a, (t0 + i) * a.gate_stride_tok + h * a.gate_stride_head, h);
    };
    load_gates(0);  // on their way before the larger copies

    // Panels of 128 rows: the chunk's keys, then its queries.
    stage_rows<PANELS, V, kPrepThreads>(ab, 2 * kTile, a.k, t0, hk, n, a.dim_k, tid);
    stage_rows<PANELS, V, kPrepThreads>(ab + kTile, 2 * kTile, a.q, t0, hk, n, a.dim_k, tid);
    cp_async_commit();
    if (warp == 0) tmem_alloc<2 * C>(&sm.tmem);

    auto block = [&](int w) { return p.heads + (static_cast<int64_t>(slot) * a.num_v_heads + hk * rep + w) * kHeadBytes; };
    // Gates, and G by a scan in 64-bit fixed point: a difference of two sums has to be exact to its own rounding.
    auto scan_gates = [&] {
        float g = 0.0f, beta = 0.0f;
        if (i < n) gates.get(a.a_log != nullptr, g, beta);
        sm.beta[side][i] = g != g ? g : beta;
        // e^-200 is 0 in fp32 and e^1000 infinite: keeps inf - inf out of the differences and the sums in range
        g = g < -200.0f ? -200.0f : g > 1000.0f ? 1000.0f : g == g ? g : 0.0f;
        constexpr float kOne = 1099511627776.0f;  // 2^40
        int64_t sum = __float2ll_rn(g * 1.4426950408889634f * kOne);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(kFullMask, sum, m);
            if (lane >= m) sum += o;
        }
        if ((warp & 1) == 0 && lane == 31) sm.carry[side] = sum;
        __syncthreads();
        if (warp & 1) sum += sm.carry[side];
        const float hi = __ll2float_rn(sum);
        sm.ghi[side][i] = hi / kOne;
        sm.glo[side][i] = __ll2float_rn(sum - __float2ll_rn(hi)) / kOne;
    };
    scan_gates();
    cp_async_wait<0>();
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    if (warp == 0) {  // [K; Q] [K; Q]^T: K K^T, Q K^T, and the rows' squares on the diagonal
        const uint32_t one = elect_lane();
#pragma unroll
        for (int ks = 0; ks < PANELS * 4; ++ks) {
            const uint32_t d = desc_low(smem_u32(ab)) + ((ks / 4) * 2 * kTile + (ks % 4) * 32) / 16;
            mma_ss(tmem, d, d, mma_desc(2 * C, 2 * C, false), ks > 0, one);
        }
        mma_commit(&sm.bar, one);
    }
    const bool done = mbar_wait_warp(&sm.bar, 0, &sm.abort);
    if (!done && lane == 0) count_error(p.err_count);
    tc_fence_after();

    const uint32_t addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    {
        float f[32], square = 0.0f;
        tmem_load(addr + warp * 32, f);
        tmem_wait_load();
#pragma unroll
        for (int j = 0; j < 32; ++j) square = lane == j ? f[j] : square;
        const float r = !done ? NAN : a.qk_l2norm ? rsqrtf(square + kGdrNormEps) : 1.0f;  // NaN from here to the outputs
        (side ? sm.rq : sm.rk)[i] = side ? r * a.scale : square < INFINITY ? r : NAN;
    }
    __syncthreads();  // the rows of K and Q are no longer needed: A takes their place
    for (int r0 = 0; r0 < rep; r0 += 2) {
        const int nh = min(2, rep - r0);
        if (r0 > 0) {
            load_gates(r0);
            scan_gates();
            __syncthreads();
        }
        bool bad = false;  // a key or a strength that is not finite
        if (side < nh) {
            float *vec = reinterpret_cast<float *>(block(r0 + side) + kVec);
            const float ghi = sm.ghi[side][i], glo = sm.glo[side][i], beta = sm.beta[side][i];
            const float decay = ex2(ghi + glo), rk = sm.rk[i];
            bad = !(fabsf(beta * rk) < INFINITY);
            vec[kBeta * C + i] = bad ? NAN : beta;
            vec[kKey * C + i] = bad ? 0.0f : -beta * rk * decay;
            vec[kState * C + i] = ex2((sm.ghi[side][C - 1] - ghi) + (sm.glo[side][C - 1] - glo)) * rk;
            vec[kQuery * C + i] = sm.rq[i] * decay;
            if (i == 0) vec[kMisc * C] = ex2(sm.ghi[side][C - 1] + sm.glo[side][C - 1]);
        }
        if (side < nh && i < C / 2)
            sm.from[side][i] = ex2((sm.ghi[side][31] - sm.ghi[side][i]) + (sm.glo[side][31] - sm.glo[side][i])) * sm.rk[i];
        if (bad) sm.odd = 1;
        __syncthreads();
        // Rows of A (threads of K rows, to shared memory) and of P (threads of Q rows, to the workspace).
        for (int w = 0; w < nh; ++w) {
            const float ghi = sm.ghi[w][i], glo = sm.glo[w][i];
            const float own = side ? sm.rq[i] : sm.beta[w][i] * sm.rk[i];
            float *out_a = matrices + w * (C * kLd) + i * kLd;
            uint4 (&rows)[2][32 * 8] = sm.rows[warp & 1];
            if (side && r0 + w > 0) {
                bulk_wait_read();
                __syncwarp();
            }
#pragma unroll
            for (int j0 = 0; j0 < C; j0 += 32) {
                float f[32];
                if (j0 == 0 && (warp & 1)) {
                    // Rows 32 .. 63, columns 0 .. 31: the decay is a factor of the row times one of the column, both <= 1.
                    const float left = own * ex2((ghi - sm.ghi[w][31]) + (glo - sm.glo[w][31]));
                    tmem_load(addr + j0, f);
                    tmem_wait_load();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 r = *reinterpret_cast<const float4 *>(&sm.from[w][j]);
                        f[j] *= left * r.x;
                        f[j + 1] *= left * r.y;
                        f[j + 2] *= left * r.z;
                        f[j + 3] *= left * r.w;
                    }
                } else if (j0 == 0 || (warp & 1)) {  // on the diagonal
                    tmem_load(addr + j0, f);
                    tmem_wait_load();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 gh = *reinterpret_cast<const float4 *>(&sm.ghi[w][j0 + j]);
                        const float4 gl = *reinterpret_cast<const float4 *>(&sm.glo[w][j0 + j]);
                        const float4 rh = *reinterpret_cast<const float4 *>(&sm.rk[j0 + j]);
                        const float gj[4] = {gh.x, gh.y, gh.z, gh.w}, lj[4] = {gl.x, gl.y, gl.z, gl.w};
                        const float rj[4] = {rh.x, rh.y, rh.z, rh.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const bool in = j0 + j + u < i + side;
                            f[j + u] = in ? f[j + u] * (own * rj[u]) * ex2((ghi - gj[u]) + (glo - lj[u])) : 0.0f;
                        }
                    }
                } else {  // rows 0 .. 31, columns 32 .. 63: nothing, and of A not even read
#pragma unroll
                    for (int j = 0; j < 32; ++j) f[j] = 0.0f;
                    if (!side) continue;
                }
                if (side) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 h, m;
                        split_bf16x2(pack2(f[8 * c], f[8 * c + 1]), h.x, m.x);
                        split_bf16x2(pack2(f[8 * c + 2], f[8 * c + 3]), h.y, m.y);
                        split_bf16x2(pack2(f[8 * c + 4], f[8 * c + 5]), h.z, m.z);
                        split_bf16x2(pack2(f[8 * c + 6], f[8 * c + 7]), h.w, m.w);
                        const int at = lane * 8 + ((j0 / 8 + c) ^ (lane & 7));
                        rows[0][at] = h;
                        rows[1][at] = m;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(out_a + j0 + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                }
            }
            if (!side && sm.odd) {  // T has to be finite in the other tokens' rows
#pragma unroll 1
                for (int j = 0; j < i; ++j)
                    if (!(fabsf(out_a[j]) < INFINITY)) out_a[j] = 0.0f;
            }
            if (side) {
                // Out by bulk copies: a row a thread would touch 32 lines a store.
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    uint8_t *to = block(r0 + w) + kP + (warp & 1) * (kTile / 2);
                    bulk_store(to, rows[0], kTile / 2);
                    bulk_store(to + kTile, rows[1], kTile / 2);
                    bulk_commit();
                }
            }
        }
        invert(matrices, tid);
        if (side < nh) {
            uint8_t *out = block(r0 + side) + kT;
            const int c = i & 7;
#pragma unroll 4
            for (int it = 0; it < 8; ++it) {
                const int row = it * 8 + (i >> 3);
                uint4 hi = make_uint4(0u, 0u, 0u, 0u), mid = hi, lo = hi;
                if (row >= 32 || c < 4) {
                    // 32 bytes apart, 8 lanes would meet in the banks: half of them read their second 16 bytes first
                    const float *x = matrices + side * (C * kLd) + row * kLd + c * 8;
                    const ulonglong2 y0 = *reinterpret_cast<const ulonglong2 *>(x + (c & 4)), y1 = *reinterpret_cast<const ulonglong2 *>(x + 4 - (c & 4));
                    const ulonglong2 x0 = c & 4 ? y1 : y0, x1 = c & 4 ? y0 : y1;
                    split_bf16x3(x0.x, hi.x, mid.x, lo.x);
                    split_bf16x3(x0.y, hi.y, mid.y, lo.y);
                    split_bf16x3(x1.x, hi.z, mid.z, lo.z);
                    split_bf16x3(x1.y, hi.w, mid.w, lo.w);
                }
                const int at = row * 128 + ((c ^ (row & 7)) << 4);
                *reinterpret_cast<uint4 *>(out + at) = hi;
                *reinterpret_cast<uint4 *>(out + kTile + at) = mid;
                *reinterpret_cast<uint4 *>(out + 2 * kTile + at) = lo;
            }
        }
        __syncthreads();
    }
    bulk_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_free<2 * C>(tmem);
}

// ----------------------------------------------------------------- chunks ----

constexpr int kCompute = 512;       // four warpgroups, each a quarter of the columns of every row
constexpr int kChunkThreads = kCompute + 128;
constexpr int kIssueWarp = 16, kStoreWarp = 17, kLoadWarp = 18;
constexpr int kLoaders = 64;
constexpr int kStages = 2;
// Registers a thread: 640 threads launch with 96 each, 61440 in all; the compute warpgroups take 104 and the other 64.
constexpr int kComputeRegs = 104, kOtherRegs = 64;
static_assert(kCompute * kComputeRegs + 128 * kOtherRegs <= kChunkThreads * 96, "register split");

// Columns of tensor memory.  A thread overwrites only columns that it alone reads, or that a barrier says are free.
enum : uint32_t {
    kColS = 0,       // 192: S^T in 3 parts, and in the same columns what the chunk adds to S^T (see s_part)
    kColP = 192,     // 64: S^T k^T
    kColO = 256,     // 64: S^T q^T, then d P^T
    kColR = 320,     // 96: R in 3 parts, then the decayed d in 3 parts
    kColN = 416,     // 64: d; then, 8 of every 16, its second part
    kColD = 480,     // 32: its first part
};
// Warpgroup q holds 16 PANELS keys of every row of S.  They have 24 PANELS columns, 8 PANELS for each part (a column is two
// bf16 values); what is added to them comes in the last 16 PANELS of those where q is even and the first where it is odd, so
// that two warpgroups' are next to each other and one MMA adds to both.
template <int PANELS>
__device__ __forceinline__ constexpr uint32_t s_part(int q, int part) { return kColS + q * 24 * PANELS + part * 8 * PANELS; }
template <int PANELS>
__device__ __forceinline__ constexpr uint32_t s_added(int q) { return s_part<PANELS>(q, 0) + (q & 1 ? 0 : 8 * PANELS); }
// It also holds tokens 8 q .. + 7 and 32 + 8 q .. + 7 of every row of R and d, so that two warpgroups make up the 16 tokens of
// an inner step of the tensor cores, and the steps of tokens 0 .. 31 can run while the others are prepared.
__device__ __forceinline__ constexpr uint32_t r_part(int step, int part) { return kColR + step * 24 + part * 8; }
// The second part of d goes into the middle 8 of the step's 16 columns of d: the upper half of the even warpgroup's own and
// the lower half of the odd one's.
__device__ __forceinline__ constexpr uint32_t d_part(int step, int part) { return part ? kColN + step * 16 + 4 : kColD + step * 8; }

template <int PANELS>
struct Stage {
    static constexpr int kq = PANELS * 2 * kTile;  // per panel: 64 rows of K, 64 of Q
    static constexpr int v = kq;                   // two swizzled tiles of 64 values
    static constexpr int head = v + 2 * kTile;
    static constexpr int bytes = (head + kHeadBytes + 1023) / 1024 * 1024;
};

struct ChunkSmem {
    uint64_t full[kStages], empty[kStages];               // a stage is loaded; its chunk's MMAs, the last to use it, are done
    uint64_t keys_ok[kStages], values_ok[kStages];        // ... and has nothing in its keys, in its values, that is not finite
    uint64_t mma_p, mma_o, mma_n[2], mma_delta[2], mma_out;  // completed by the tensor cores
    uint64_t have_s[2], have_r[2], have_vs[2];            // arrived on by the compute threads, by halves
    uint64_t have_read, have_d;
    uint64_t out_full, out_free;                          // the output tile: written by them, stored by one warp
    uint64_t drain;
    uint32_t tmem;
    int abort;
    int seq, start, end;
    int first, last, line;  // the block's tokens, and the line that it writes its last state to (-1: none)
    int first_bad[128];  // of every row of S: the first token, from the block's first, that is not finite
    int any_bad;         // the least of them
};
__device__ __forceinline__ void note_bad(ChunkSmem &sm, int row, int token) {
    atomicMin(&sm.first_bad[row], token);
    atomicMin(&sm.any_bad, token);
}

// What is not finite of a chunk in shared memory is left out, by the kLoaders threads `id`.  A token whose strength the
// preparation has set to NaN loses its key and its strength, and is noted for all rows ...
template <int PANELS>
__device__ __forceinline__ void leave_out_keys(ChunkSmem &sm, uint8_t *keys, float *strength, int first_token, int id) {
    if (fabsf(strength[id]) < INFINITY) return;
    strength[id] = 0.0f;
    for (int row = 0; row < 128; ++row) note_bad(sm, row, first_token + id);
    for (int i = 0; i < PANELS * 8; ++i)
        *reinterpret_cast<uint4 *>(keys + (i >> 3) * 2 * kTile + id * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_shared();  // for the products, and for the next copy to these places
}
// ... a value is set to 0, and noted for its row.
__device__ __forceinline__ void leave_out_values(ChunkSmem &sm, uint8_t *values, int first_token, int id) {
    constexpr int kPieces = 2 * kTile / 16 / kLoaders;
    uint32_t odd = 0u;  // NaN in a half if one of those added to it is not finite
#pragma unroll 8
    for (int i = 0; i < kPieces; ++i) {
        const uint4 x = *reinterpret_cast<const uint4 *>(values + (i * kLoaders + id) * 16);
        for (uint32_t w : {x.x, x.y, x.z, x.w}) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(odd) : "r"(w), "r"(0u));
    }
    if (odd == 0u) return;
    for (int i = id * 8; i < 2 * kTile / 2; i += kLoaders * 8) {
        uint16_t *v = reinterpret_cast<uint16_t *>(values) + i;
        const int row = (i >> 6) & (C - 1), column = (i >> 12) * 64 + (((i >> 3) ^ row) & 7) * 8;
        for (int k = 0; k < 8; ++k)
            if ((v[k] & 0x7f80u) == 0x7f80u) {
                v[k] = 0;
                note_bad(sm, column + k, first_token + row);
            }
    }
    fence_async_shared();
}

// S^T (128 rows of values on the lanes of tensor memory) stays in registers; its three bf16 parts, R's and d's go to tensor
// memory as the A operands.  16 warps do the arithmetic, one issues MMAs, two load the next chunk and look at its values, and one stores the output.
// The chunks are a chain of product, split into parts, product: S k^T, R, d = T R, decayed d, what is added to S.  Of the
// 2.7 us (5150 cycles) of a chunk the tensor cores work 3200: 24 + 24 products of 32 cycles for S k and d, 16 for S q, 24 for
// the state, 12 for the output.  The rest is splitting (the sixteen warps' integer and conversion pipes: 1200 cycles for S,
// 350 for each half of R and d) and 240 cycles from each commit to the waiting warps; halves of R, d and S overlap the two.
// 4 x 4096 tokens, 32 heads: 128 blocks, 174 us; a block is 640 threads with all registers and all tensor memory of its SM.
//
// FULL: outputs and final states.  Otherwise the first pass over segments: N of all but the last, and M of those between
// (the last block of every group of slices + 1).  V: the state allows 16-byte vectors.  VIO: rows of q, k, v and out do.
template <int PANELS, bool FULL, bool V, bool VIO>
__global__ void __launch_bounds__(kChunkThreads, 1) gdr_chunk_kernel(const __grid_constant__ FwdArgs p,
                                                                     const __grid_constant__ FwdMaps maps, int slices) {
    using St = Stage<PANELS>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = smem_raw;  // on a 1024-byte boundary, since the kernel has no static shared memory (checked below)
    uint16_t *out_tile = reinterpret_cast<uint16_t *>(base + kStages * St::bytes);  // 64 rows of 128 values
    ChunkSmem &sm = *reinterpret_cast<ChunkSmem *>(base + kStages * St::bytes + 2 * kTile);
    const ccv_gdr_args &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFullMask, tid >> 5, 0);
    const int types = FULL ? slices : slices + 1;
    const int slice = blockIdx.x % types;
    const bool step_only = !FULL && slice == slices;  // M
    const int bh = blockIdx.x / types;
    const int h = bh % a.num_v_heads, slot = bh / a.num_v_heads;
    const int hk = h / (a.num_v_heads / a.num_k_heads);
    // The kernels before this one let it start only after their own wait, so the caller's tensors are as they will stay: this
    // one reads them, and waits before it reads what those wrote or writes anything.
    if (misplaced(smem_raw, p.err_count)) return;

    int seq = slot, segment = 0, s, e;
    if (p.seg_chunks > 0) {
        if (warp == 0) {
            find_sequence(p.query_start_loc, p.batch, slot, p.seg_chunks * C, lane, seq, s, e);
            if (lane == 0) {
                sm.seq = seq;
                sm.start = s;
                sm.end = e;
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
    const int line = p.cache_indices != nullptr ? p.cache_indices[seq] : seq;
    const bool good = sequence_ok(s, e, p.total_tokens) && (a.state == nullptr || line == a.pad_slot_id || (line >= 0 && line < a.num_lines));
    if (p.seg_chunks > 0) segment = slot - first_slot(s, seq, p.seg_chunks * C);
    if (!good) {
        wait_prior_grid();
        if (FULL && p.seg_chunks == 0 && tid == 0 && slice == 0 && h == 0) count_error(p.err_count);
        return;
    }
    if (e == s || line == a.pad_slot_id) {
        wait_prior_grid();
        return;
    }
    int chunks = (e - s + C - 1) / C;
    int slot0 = first_slot(s, seq, C);
    bool last = true;  // segment of the sequence
    if (p.seg_chunks > 0) {
        const int segments = (chunks + p.seg_chunks - 1) / p.seg_chunks;
        last = segment == segments - 1;
        if (segment < 0 || segment >= segments || (!FULL && (last || (step_only && segment == 0)))) {
            wait_prior_grid();
            return;
        }
        const int c0 = segment * p.seg_chunks;
        chunks = min(p.seg_chunks, chunks - c0);
        slot0 += c0;
        s += c0 * C;
        if (!last) e = s + chunks * C;
    }

    if (tid == 0) {
        sm.abort = 0;
        sm.first = s;
        sm.last = e;
        sm.line = last && a.state != nullptr ? line : -1;
        for (uint64_t &b : sm.full) mbar_init(&b, kLoaders + 1);
        for (uint64_t *b : {&sm.keys_ok[0], &sm.keys_ok[1], &sm.values_ok[0], &sm.values_ok[1]}) mbar_init(b, kLoaders);
        sm.any_bad = INT_MAX;
        for (uint64_t *b : {&sm.empty[0], &sm.empty[1], &sm.mma_p, &sm.mma_o, &sm.mma_n[0], &sm.mma_n[1], &sm.mma_delta[0],
                            &sm.mma_delta[1], &sm.mma_out, &sm.drain})
            mbar_init(b, 1);
        for (uint64_t *b : {&sm.have_s[0], &sm.have_s[1]}) mbar_init(b, kCompute / 2);
        for (uint64_t *b : {&sm.have_r[0], &sm.have_r[1], &sm.have_vs[0], &sm.have_vs[1], &sm.have_read, &sm.have_d, &sm.out_full})
            mbar_init(b, kCompute);
        mbar_init(&sm.out_free, 32);
        mbar_init_fence();
    }
    if (tid < 128) sm.first_bad[tid] = INT_MAX;
    if (warp == kIssueWarp) tmem_alloc<512>(&sm.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFullMask, sm.tmem, 0);

    if (warp >= kIssueWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kIssueWarp) {
            const uint32_t el = elect_lane();
            const uint32_t smem0 = desc_low(__shfl_sync(kFullMask, smem_u32(base), 0));  // all below in units of 16 bytes
            // keys of warpgroup q from step j on: their place in the rows of K and Q
            auto key_at = [](int q, int j) {
                const int key = q * 16 * PANELS + j * 16;
                return ((key / 64) * 2 * kTile + (key % 64) * 2) / 16;
            };
            constexpr uint32_t kTokens = mma_desc(128, C, false), kLateTokens = mma_desc(128, C / 2, false), kKeys = mma_desc(128, 32 * PANELS, true);
            int c = 0;
            for (; c < chunks; ++c) {
                const uint32_t par = c & 1;
                const uint32_t kq = smem0 + (c % kStages) * (St::bytes / 16);
                const uint32_t head = kq + St::head / 16;
                if (!mbar_wait_warp(&(FULL ? sm.keys_ok : sm.full)[c % kStages], (c / kStages) & 1, &sm.abort)) break;
                bool ok = true;
                // S^T k^T, three parts of S; the keys are exact
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (!(ok = mbar_wait_warp(&sm.have_s[g], par, &sm.abort))) break;
                    tc_fence_after();
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int q = 2 * g; q < 2 * g + 2; ++q)
#pragma unroll
                            for (int j = 0; j < PANELS; ++j)
                                mma_ts(tmem + kColP, tmem + s_part<PANELS>(q, part) + j * 8, kq + key_at(q, j), kTokens,
                                       part < 2 || q + j > 0, el);
                }
                if (!ok) break;
                mma_commit(&sm.mma_p, el);
                // S^T q^T, once the previous chunk's output has left these columns, while R is made
                if constexpr (FULL) {
                    if (!mbar_wait_warp(&sm.have_read, par, &sm.abort)) break;
                    tc_fence_after();
#pragma unroll
                    for (int part = 1; part >= 0; --part)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int j = 0; j < PANELS; ++j)
                                mma_ts(tmem + kColO, tmem + s_part<PANELS>(q, part) + j * 8, kq + kTile / 16 + key_at(q, j), kTokens,
                                       part < 1 || q + j > 0, el);
                    mma_commit(&sm.mma_o, el);
                }
                // d^T = R^T T^T: the six products of parts above 2^-24, for tokens 0 .. 31 of the sum, then the others.  T is lower
                // triangular: these are parts of d's last 32 tokens alone, and the compute threads take up the first 32 meanwhile.
                // (N = 32 costs the tensor cores what N = 64 does.  What had these columns left with the last output.)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = mbar_wait_warp(&sm.have_r[half], par, &sm.abort))) break;
                    tc_fence_after();
#pragma unroll
                    for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                        for (int part = 0; part <= sum; ++part)
#pragma unroll
                            for (int ks = 2 * half; ks < 2 * half + 2; ++ks)
                                mma_ts(tmem + kColN + 32 * half, tmem + r_part(ks, part),
                                       head + (kT + (sum - part) * kTile + ks * 32 + half * (kTile / 2)) / 16, half ? kLateTokens : kTokens,
                                       sum < 2 || part + ks > 0, el);
                    mma_commit(&sm.mma_n[half], el);
                }
                if (!ok) break;
                if (!mbar_wait_warp(&sm.have_vs[0], par, &sm.abort)) break;
                // what the chunk adds to S^T: tokens are the inner axis, so the keys are read MN-major; those of two
                // warpgroups at a time
                auto add = [&](int g, int half) {
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int ks = 2 * half; ks < 2 * half + 2; ++ks)
                            mma_ts(tmem + s_added<PANELS>(2 * g), tmem + r_part(ks, part), kq + key_at(2 * g, 0) + ks * 2048 / 16, kKeys,
                                   part < 2 || ks > 0, el);
                };
                tc_fence_after();
                add(0, 0);
                add(1, 0);
                if (!mbar_wait_warp(&sm.have_vs[1], par, &sm.abort)) break;
                tc_fence_after();
                add(0, 1);
                mma_commit(&sm.mma_delta[0], el);
                add(1, 1);
                mma_commit(&sm.mma_delta[1], el);
                if constexpr (FULL) {
                    if (!mbar_wait_warp(&sm.have_d, par, &sm.abort)) break;
                    tc_fence_after();
                    // d P^T: the three products of parts above 2^-16
#pragma unroll
                    for (int term = 2; term >= 0; --term)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_ts(tmem + kColO, tmem + d_part(ks, term == 1), head + (kP + (term == 2 ? kTile : 0) + ks * 32) / 16, kTokens,
                                   term < 2 || ks > 0, el);
                    mma_commit(&sm.mma_out, el);
                }
                mma_commit(&sm.empty[c % kStages], el);
            }
            if (c < chunks) {  // gave up: let the MMAs end before their memories go
                if (el) count_error(p.err_count);
                int quiet = 0;
                mma_commit(&sm.drain, el);
                mbar_wait_warp(&sm.drain, 0, &quiet);
            }
        } else if (warp == kStoreWarp) {
            wait_prior_grid();
            release_next_grid();
            const int width = min(128, a.dim_v - slice * 128);
            uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + h * a.out.stride_head + slice * 128 * a.out.stride_dim;
            for (int c = 0; FULL && c < chunks; ++c) {
                if (!mbar_wait_warp(&sm.out_full, c & 1, &sm.abort)) break;
                const int t0 = s + c * C, n = min(C, e - t0);
                if (*const_cast<volatile int *>(&sm.any_bad) < (c + 1) * C) {
                    for (int i = lane; i < C * 128; i += 32)
                        if (*const_cast<volatile int *>(&sm.first_bad[i & 127]) <= c * C + (i >> 7)) out_tile[i] = 0x7fffu;
                    __syncwarp();
                }
                if constexpr (VIO) {  // two rows a pass, 16 bytes a lane
                    uint16_t *dst = out + (t0 + (lane >> 4)) * a.out.stride_tok + (lane & 15) * 8;
                    const bool wide = (lane & 15) * 8 < width;
#pragma unroll 8
                    for (int r = lane >> 4; r < C; r += 2) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(out_tile + r * 128 + (lane & 15) * 8);
                        if (wide && r < n) *reinterpret_cast<uint4 *>(dst) = x;
                        dst += 2 * a.out.stride_tok;
                    }
                } else {
                    for (int i = lane; i < n * 128; i += 32)
                        if ((i & 127) < width) out[(t0 + (i >> 7)) * a.out.stride_tok + (i & 127) * a.out.stride_dim] = out_tile[i];
                }
                mbar_arrive(&sm.out_free);
            }
        } else {
            const int id = tid - kLoadWarp * 32;
            const int width = min(128, a.dim_v - slice * 128);
            ccv_heads_view vv = a.v;
            if (!step_only) vv.data = static_cast<const uint16_t *>(a.v.data) + slice * 128 * a.v.stride_dim;
            const uint8_t *heads = p.heads + (static_cast<int64_t>(slot0) * a.num_v_heads + h) * kHeadBytes;
            const int64_t heads_step = static_cast<int64_t>(a.num_v_heads) * kHeadBytes;
            int c = 0, issued = 0;
            for (; c < chunks; ++c) {
                const int t0 = s + c * C, n = min(C, e - t0);
                // Whole chunks come as tensor tiles; a sequence's last rows, which need zeros after them, piece by piece.
                const bool whole = VIO && maps.use && n == C;
                if (id == 0 && c + 1 < chunks) {  // the stage frees up late: let L2 have the next chunk's part by then
                    if (c > 0) bulk_prefetch(heads + (c + 1) * heads_step, kHeadBytes);
                    if (VIO && maps.use) {
                        if (!step_only)
                            for (int i = 0; i < 2; ++i) tensor_prefetch(&maps.v, slice * 128 + i * 64, h, t0 + C);
                        for (int i = 0; i < PANELS; ++i) {
                            tensor_prefetch(&maps.k, i * 64, hk, t0 + C);
                            if (FULL) tensor_prefetch(&maps.q, i * 64, hk, t0 + C);
                        }
                    }
                }
                if (c >= kStages && !mbar_wait_warp(&sm.empty[c % kStages], (c / kStages - 1) & 1, &sm.abort)) break;
                uint8_t *st = base + (c % kStages) * St::bytes;
                uint64_t *bar = &sm.full[c % kStages];
                if (id == 0) {
                    const int tiles = whole ? PANELS * (FULL ? 2 : 1) + (step_only ? 0 : 2) : 0;
                    mbar_expect_tx(bar, (FULL ? kHeadBytes : kHeadBytes - 2 * kTile) + tiles * kTile);
                    if (whole) {
                        for (int i = 0; i < PANELS; ++i) tensor_load(st + i * 2 * kTile, &maps.k, i * 64, hk, t0, bar);
                        if (!step_only)
                            for (int i = 0; i < 2; ++i) tensor_load(st + St::v + i * kTile, &maps.v, slice * 128 + i * 64, h, t0, bar);
                    }
                    const uint8_t *src = heads + c * heads_step;
                    if (FULL && whole)
                        for (int i = 0; i < PANELS; ++i) tensor_load(st + i * 2 * kTile + kTile, &maps.q, i * 64, hk, t0, bar);
                    if (c == 0) {
                        wait_prior_grid();
                        if (chunks > 1) bulk_prefetch(heads + heads_step, kHeadBytes);
                    }
                    if constexpr (FULL) {
                        bulk_load(st + St::head, src, kHeadBytes, bar);
                    } else {  // without P
                        bulk_load(st + St::head + kT, src + kT, kP - kT, bar);
                        bulk_load(st + St::head + kVec, src + kVec, kHeadBytes - kVec, bar);
                    }
                }
                if (!whole) {
                    if (!step_only) stage_rows<2, VIO, kLoaders>(st + St::v, kTile, vv, t0, h, n, width, id);
                    stage_rows<PANELS, VIO, kLoaders>(st, 2 * kTile, a.k, t0, hk, n, a.dim_k, id);
                    if (FULL) stage_rows<PANELS, VIO, kLoaders>(st + kTile, 2 * kTile, a.q, t0, hk, n, a.dim_k, id);
                    cp_async_commit();
                    cp_async_wait<0>();
                    fence_async_shared();
                }
                mbar_arrive(bar);
                issued = c + 1;
                if constexpr (FULL) {  // in the first pass a row that is not finite becomes NaN by itself, and that is all it has to
                    if (!mbar_wait_warp(bar, (c / kStages) & 1, &sm.abort)) break;
                    leave_out_keys<PANELS>(sm, st, reinterpret_cast<float *>(st + St::head + kVec) + kBeta * C, c * C, id);
                    mbar_arrive(&sm.keys_ok[c % kStages]);
                    leave_out_values(sm, st + St::v, c * C, id);
                    mbar_arrive(&sm.values_ok[c % kStages]);
                }
            }
            if (c < chunks) {  // gave up: let the copies land before the shared memory goes
                int quiet = 0;
                for (int i = max(0, issued - kStages); i < issued; ++i) mbar_wait(&sm.full[i % kStages], (i / kStages) & 1, &quiet);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
        constexpr int KH = 16 * PANELS;  // keys of the state a thread holds
        const int q = warp >> 2, d = (warp & 3) * 32 + lane, row = step_only ? d : slice * 128 + d;
        const bool live = row < (step_only ? a.dim_k : a.dim_v);
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t col_s = lanes + s_part<PANELS>(q, 0);
        // Row d of the state this block starts from and ends with: a pool line's, or a segment's in the workspace.
        constexpr int kLdS = 64 * PANELS;
        auto in_segment = [&](float *at, int which, int rows) {
            return at + ((static_cast<int64_t>(which) * a.num_v_heads + h) * rows + row) * kLdS;
        };
        float *pool = a.state != nullptr ? a.state + line * a.s_stride_line + h * a.s_stride_head + row * a.s_stride_v : nullptr;
        const bool init = a.state != nullptr && p.has_initial_state != nullptr && p.has_initial_state[seq] != 0;
        // In the second pass another block may already have written the pool's line when a cut sequence's first segment starts:
        // the first pass keeps the state it read for it.
        const bool kept = FULL && !(segment == 0 && last);
        const float *from = kept ? in_segment(p.seg_state, slot, a.dim_v) : segment == 0 && init ? pool : nullptr;

        if (kept || (!FULL && segment == 0)) wait_prior_grid();  // the join's states; and the first segment's goes to the workspace

        f32x2 st[KH / 2], odd = 0ull;  // this thread's part of row d of S; NaN where it holds a value that is not finite
#pragma unroll
        for (int k = 0; k < KH; k += 4) {
            const int kk = q * KH + k;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (from != nullptr && live) {
                if (V || kept) {
                    if (kk < a.dim_k) x = *reinterpret_cast<const float4 *>(from + kk);
                } else {
                    if (kk < a.dim_k) x.x = from[kk * a.s_stride_k];
                    if (kk + 1 < a.dim_k) x.y = from[(kk + 1) * a.s_stride_k];
                    if (kk + 2 < a.dim_k) x.z = from[(kk + 2) * a.s_stride_k];
                    if (kk + 3 < a.dim_k) x.w = from[(kk + 3) * a.s_stride_k];
                }
            } else if (step_only && live) {
                x = make_float4(kk == row, kk + 1 == row, kk + 2 == row, kk + 3 == row);
            }
            if (!FULL && segment == 0 && live) *reinterpret_cast<float4 *>(in_segment(p.seg_state, slot, a.dim_v) + kk) = x;
            st[k / 2] = pack2(x.x, x.y);
            st[k / 2 + 1] = pack2(x.z, x.w);
            if constexpr (FULL) odd = fma2(st[k / 2], 0ull, fma2(st[k / 2 + 1], 0ull, odd));
        }
        if (odd != 0ull) note_bad(sm, d, 0);
        auto stage = [&](int c) { return base + (c % kStages) * St::bytes; };
        // S^T <- gamma S^T + what the chunk added
        auto add_delta = [&](float gamma) {
            const f32x2 g2 = pack2(gamma, gamma);
#pragma unroll
            for (int k0 = 0; k0 < KH; k0 += 16) {
                float x[16];
                tmem_load(lanes + s_added<PANELS>(q) + k0, x);
                tmem_wait_load();
#pragma unroll
                for (int k = 0; k < 8; ++k) st[k0 / 2 + k] = fma2(g2, st[k0 / 2 + k], pack2(x[2 * k], x[2 * k + 1]));
            }
        };
        // d P^T of chunk c onto oi, into the output tile
        f32x2 oi[8];
        auto finish = [&](int c) {
            float x[2][8];
            tmem_load(lanes + kColO + 8 * q, x[0]);
            tmem_load(lanes + kColO + 32 + 8 * q, x[1]);
            tmem_wait_load();
            tc_fence_before();
            mbar_arrive(&sm.have_read);
            if (c > 0 && !mbar_wait_warp(&sm.out_free, (c - 1) & 1, &sm.abort)) return false;
            uint16_t *o = out_tile + 8 * q * 128 + d;
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = f32x2_to_bf16x2(add2(oi[4 * half + i], pack2(x[half][2 * i], x[half][2 * i + 1])));
                    o[(32 * half + 2 * i) * 128] = static_cast<uint16_t>(w);
                    o[(32 * half + 2 * i + 1) * 128] = static_cast<uint16_t>(w >> 16);
                }
            mbar_arrive(&sm.out_full);
            return true;
        };

        bool ok = true;
        float gamma = 1.0f;
        for (int c = 0; c < chunks; ++c) {
            const uint32_t par = c & 1;
            if (c > 0) {
                if (!(ok = mbar_wait_warp(&sm.mma_delta[q >> 1], par ^ 1, &sm.abort))) break;
                tc_fence_after();
                add_delta(gamma);  // all of it is read before its parts, which are wider, overwrite it
            }
#pragma unroll
            for (int k0 = 0; k0 < KH; k0 += 16) {
                uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) split_bf16x3(st[k0 / 2 + k], hi[k], mid[k], lo[k]);
                tmem_store(col_s + k0 / 2, hi);
                tmem_store(col_s + KH / 2 + k0 / 2, mid);
                tmem_store(col_s + KH + k0 / 2, lo);
            }
            tmem_wait_store();
            tc_fence_before();
            mbar_arrive(&sm.have_s[q >> 1]);

            if constexpr (FULL) {
                if (c > 0) {  // the output of the chunk before, while the tensor cores are at S k
                    if (!(ok = mbar_wait_warp(&sm.mma_out, par ^ 1, &sm.abort))) break;
                    tc_fence_after();
                    if (!(ok = finish(c - 1))) break;
                } else {
                    mbar_arrive(&sm.have_read);
                }
            }

            // b v of this thread's tokens
            if (!(ok = mbar_wait_warp(&(FULL ? sm.values_ok : sm.full)[c % kStages], (c / kStages) & 1, &sm.abort))) break;
            const float *f = reinterpret_cast<const float *>(stage(c) + St::head + kVec) + 8 * q;
            // 4 of a token's factors, as pairs
            auto vec4 = [&](int which, int half, int i) { return *reinterpret_cast<const ulonglong2 *>(f + which * C + 32 * half + 4 * i); };
            f32x2 vb[8];
            if (step_only) {
#pragma unroll
                for (int i = 0; i < 8; ++i) vb[i] = 0ull;
            } else {
                const uint8_t *v = stage(c) + St::v + (d >> 6) * kTile + 8 * q * 128 + (d & 7) * 2;
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const ulonglong2 beta = vec4(kBeta, half, i / 2);
                        auto at = [&](int r) {  // row 8 q + r of the half, whose place within 8 rows is r
                            return bf16_bits(*reinterpret_cast<const uint16_t *>(v + (32 * half + r) * 128 + ((((d & 63) >> 3) ^ r) << 4)));
                        };
                        vb[4 * half + i] = mul2(pack2(at(2 * i), at(2 * i + 1)), (i & 1 ? beta.y : beta.x));
                    }
            }

            // R = b v - b e^G S k
            if (!(ok = mbar_wait_warp(&sm.mma_p, par, &sm.abort))) break;
            tc_fence_after();
            {
                float x[2][8];
                tmem_load(lanes + kColP + 8 * q, x[0]);
                tmem_load(lanes + kColP + 32 + 8 * q, x[1]);
                tmem_wait_load();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const ulonglong2 key = vec4(kKey, half, i / 2);
                        const float *y = &x[half][2 * i];
                        split_bf16x3(fma2(key.x, pack2(y[0], y[1]), vb[4 * half + i]), hi[i], mid[i], lo[i]);
                        split_bf16x3(fma2(key.y, pack2(y[2], y[3]), vb[4 * half + i + 1]), hi[i + 1], mid[i + 1], lo[i + 1]);
                    }
                    const uint32_t at = lanes + r_part(2 * half + (q >> 1), 0) + (q & 1) * 4;
                    tmem_store(at, hi);
                    tmem_store(at + 8, mid);
                    tmem_store(at + 16, lo);
                    tmem_wait_store();
                    tc_fence_before();
                    mbar_arrive(&sm.have_r[half]);
                }
            }

            gamma = f[kMisc * C - 8 * q];  // before the last arrival, after which the stage may be filled again
            // d, decayed for the state (3 parts) and for the output (2)
            {
                float x[2][8];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = mbar_wait_warp(&sm.mma_n[half], par, &sm.abort))) break;
                    tc_fence_after();
                    tmem_load(lanes + kColN + 32 * half + 8 * q, x[half]);
                    tmem_wait_load();
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const ulonglong2 left = vec4(kState, half, i / 2);
                        const float *y = &x[half][2 * i];
                        split_bf16x3(mul2(left.x, pack2(y[0], y[1])), hi[i], mid[i], lo[i]);
                        split_bf16x3(mul2(left.y, pack2(y[2], y[3])), hi[i + 1], mid[i + 1], lo[i + 1]);
                    }
                    const uint32_t at = lanes + r_part(2 * half + (q >> 1), 0) + (q & 1) * 4;
                    tmem_store(at, hi);
                    tmem_store(at + 8, mid);
                    tmem_store(at + 16, lo);
                    tmem_wait_store();
                    tc_fence_before();
                    mbar_arrive(&sm.have_vs[half]);
                }
                if (!ok) break;
                if constexpr (FULL) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t hi[4], mid[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) split_bf16x2(pack2(x[half][2 * i], x[half][2 * i + 1]), hi[i], mid[i]);
                        tmem_store(lanes + d_part(2 * half + (q >> 1), 0) + (q & 1) * 4, hi);
                        tmem_store(lanes + d_part(2 * half + (q >> 1), 1) + (q & 1) * 4, mid);
                    }
                }
            }
            if constexpr (FULL) {
                if (!(ok = mbar_wait_warp(&sm.mma_o, par, &sm.abort))) break;
                tc_fence_after();
                {
                    float x[2][8];
                    tmem_load(lanes + kColO + 8 * q, x[0]);
                    tmem_load(lanes + kColO + 32 + 8 * q, x[1]);
                    tmem_wait_load();
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const ulonglong2 left = vec4(kQuery, half, i / 2);
                            const float *y = &x[half][2 * i];
                            oi[4 * half + i] = mul2(left.x, pack2(y[0], y[1]));
                            oi[4 * half + i + 1] = mul2(left.y, pack2(y[2], y[3]));
                        }
                }
            }
            if constexpr (FULL) {
                tmem_wait_store();
                tc_fence_before();
                mbar_arrive(&sm.have_d);
            }
        }
        // the last chunk's output and the final state
        if (ok && FULL) {
            ok = mbar_wait_warp(&sm.mma_out, (chunks - 1) & 1, &sm.abort);
            if (ok) {
                tc_fence_after();
                finish(chunks - 1);
            }
        }
        if (ok) ok = mbar_wait_warp(&sm.mma_delta[q >> 1], (chunks - 1) & 1, &sm.abort);
        if (ok) {
            tc_fence_after();
            add_delta(gamma);
            float *to = FULL ? (last ? pool : nullptr)
                             : step_only ? in_segment(p.seg_step, slot, a.dim_k) : in_segment(p.seg_state, slot + 1, a.dim_v);
            const bool bad = FULL && *const_cast<volatile int *>(&sm.first_bad[d]) != INT_MAX;
            if (to != nullptr && live) {
#pragma unroll
                for (int k = 0; k < KH; k += 4) {
                    const int kk = q * KH + k;
                    float4 x;
                    unpack2(st[k / 2], x.x, x.y);
                    unpack2(st[k / 2 + 1], x.z, x.w);
                    if (bad) x = make_float4(NAN, NAN, NAN, NAN);
                    if (!FULL) {
                        *reinterpret_cast<float4 *>(to + kk) = x;
                    } else if constexpr (V) {
                        if (kk < a.dim_k) *reinterpret_cast<float4 *>(to + kk) = x;
                    } else {
                        if (kk < a.dim_k) to[kk * a.s_stride_k] = x.x;
                        if (kk + 1 < a.dim_k) to[(kk + 1) * a.s_stride_k] = x.y;
                        if (kk + 2 < a.dim_k) to[(kk + 2) * a.s_stride_k] = x.z;
                        if (kk + 3 < a.dim_k) to[(kk + 3) * a.s_stride_k] = x.w;
                    }
                }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kIssueWarp) tmem_free<512>(tmem);
    if (sm.abort) {  // a wait ran out: nothing that this block should have written may pass for a result
        unsigned block = blockIdx.x;
        asm volatile("" : "+r"(block));  // what follows is worked out again, not kept in registers meanwhile
        const int part = block % types, head = block / types % a.num_v_heads;
        const bool step = !FULL && part == slices;
        const int rows = step ? a.dim_k : min(128, a.dim_v - part * 128), row0 = step ? 0 : part * 128;
        if constexpr (FULL) {
            uint16_t *out = static_cast<uint16_t *>(const_cast<void *>(a.out.data)) + head * a.out.stride_head + row0 * a.out.stride_dim;
            for (int t = sm.first + threadIdx.x / 128; t < sm.last; t += kChunkThreads / 128)
                if (threadIdx.x % 128 < rows) out[t * a.out.stride_tok + threadIdx.x % 128 * a.out.stride_dim] = 0x7fffu;
            float *state = a.state + sm.line * a.s_stride_line + head * a.s_stride_head + row0 * a.s_stride_v;
            for (int i = threadIdx.x; sm.line >= 0 && i < rows * a.dim_k; i += kChunkThreads)
                state[i / a.dim_k * a.s_stride_v + i % a.dim_k * a.s_stride_k] = NAN;
        } else {
            const int64_t at = (static_cast<int64_t>(block / types / a.num_v_heads + (step ? 0 : 1)) * a.num_v_heads + head) * (step ? a.dim_k : a.dim_v) + row0;
            for (int i = threadIdx.x; i < rows * 64 * PANELS; i += kChunkThreads) (step ? p.seg_step : p.seg_state)[at * 64 * PANELS + i] = NAN;
        }
    }
}

// ------------------------------------------------------------------- join ----

// First states of the segments from the third on (the first pass left the first two): S_{j+1} = S_j M_j + N_j, whose N the
// first pass left in S_{j+1}'s place.  In fp32 throughout.  Rows of S are independent: a block takes ROWS of them through a
// whole sequence, with the next M on its way to shared memory.  A thread has 4 columns of up to 8 rows and a part of the
// inner length, so that a value of M serves 8 rows and 16 warps hide one another's loads; the parts are added in order.  Bound
// by latency: 2.4 us a segment with 16 rows a block, 1 us with up to 8 (a warp for 4 whole rows took 6.6).
template <int PANELS, int ROWS>
struct Join {
    static constexpr int kLdS = 64 * PANELS, kColumns = kLdS / 4;  // threads for a row
    static constexpr int threads = 256 * PANELS;
    static constexpr int rows = ROWS < 8 ? ROWS : 8;               // of a thread
    static constexpr int row_groups = ROWS / rows;
    static constexpr int splits = threads / kColumns / row_groups, inner = kLdS / splits;
    static_assert(inner % 4 == 0 && ROWS * kColumns <= threads, "");
    static constexpr int step = 0, sums = step + 2 * kLdS * kLdS, state = sums + splits * ROWS * kLdS;  // floats from the start
    static constexpr size_t smem = 128 + (state + ROWS * kLdS) * 4;
};

template <int PANELS, int ROWS>
__global__ void __launch_bounds__(256 * PANELS) gdr_join_kernel(const __grid_constant__ FwdArgs p) {
    using J = Join<PANELS, ROWS>;
    constexpr int kLdS = J::kLdS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    float *base = reinterpret_cast<float *>(smem_raw);
    float *steps = base + J::step, *sums = base + J::sums, *state = base + J::state;
    __shared__ uint64_t full[2];
    __shared__ int abort;
    const ccv_gdr_args &a = p.a;
    const int tid = threadIdx.x;
    const int groups = (a.dim_v + ROWS - 1) / ROWS;
    const int first = (blockIdx.x % groups) * ROWS;
    const int bh = blockIdx.x / groups;
    const int h = bh % a.num_v_heads, seq = bh / a.num_v_heads;
    wait_prior_grid();
    release_next_grid();
    const int s = p.query_start_loc[seq], e = p.query_start_loc[seq + 1];
    const int line = p.cache_indices != nullptr ? p.cache_indices[seq] : seq;
    if (!sequence_ok(s, e, p.total_tokens) || (a.state != nullptr && line != a.pad_slot_id && (line < 0 || line >= a.num_lines))) {
        if (tid == 0 && first == 0 && h == 0) count_error(p.err_count);  // the passes cannot tell whose block would
        return;
    }
    const int unit = p.seg_chunks * C;
    const int segments = (e - s + unit - 1) / unit, slot0 = first_slot(s, seq, unit);
    if (line == a.pad_slot_id || segments < 3) return;

    if (tid == 0) {
        abort = 0;
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        mbar_init_fence();
    }
    // S is zero past dim_k; M has no rows there.
    for (int i = a.dim_k * kLdS + tid; i < kLdS * kLdS; i += J::threads) steps[i] = steps[kLdS * kLdS + i] = 0.0f;
    const uint32_t bytes = a.dim_k * kLdS * 4;
    auto fetch = [&](int j) {  // M of segment j, by one thread
        mbar_expect_tx(&full[j & 1], bytes);
        bulk_load(steps + (j & 1) * kLdS * kLdS, p.seg_step + (static_cast<int64_t>(slot0 + j) * a.num_v_heads + h) * a.dim_k * kLdS, bytes,
                  &full[j & 1]);
    };
    // As one of the products' threads, and as one that adds up a row's sums.
    const int column = tid % J::kColumns * 4, group = tid / J::kColumns;
    const int row0 = group % J::row_groups * J::rows, split = group / J::row_groups;
    const bool adds = group < ROWS, real = adds && first + group < a.dim_v;
    auto row_at = [&](int j) {
        return reinterpret_cast<float4 *>(p.seg_state + ((static_cast<int64_t>(slot0 + j) * a.num_v_heads + h) * a.dim_v + first + group) * kLdS + column);
    };
    if (adds) *reinterpret_cast<float4 *>(state + group * kLdS + column) = real ? *row_at(1) : make_float4(0.f, 0.f, 0.f, 0.f);
    __syncthreads();
    if (tid == 0) fetch(1);
    for (int j = 1; j + 1 < segments; ++j) {
        if (tid == 0 && j + 2 < segments) fetch(j + 1);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (real) y = *row_at(j + 1);
        const bool ok = mbar_wait_warp(&full[j & 1], ((j - 1) >> 1) & 1, &abort);
        const float *m = steps + ((j & 1) * kLdS + split * J::inner) * kLdS + column;
        const float *x = state + row0 * kLdS + split * J::inner;
        f32x2 acc[J::rows][2];
#pragma unroll
        for (int r = 0; r < J::rows; ++r) acc[r][0] = acc[r][1] = 0ull;
#pragma unroll
        for (int k0 = 0; k0 < J::inner; k0 += 4) {
            ulonglong2 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const ulonglong2 *>(m + (k0 + k) * kLdS);
#pragma unroll
            for (int r = 0; r < J::rows; ++r) {
                const float4 v = *reinterpret_cast<const float4 *>(x + r * kLdS + k0);
                const float s4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x2 both = pack2(s4[k], s4[k]);
                    acc[r][0] = fma2(both, w[k].x, acc[r][0]);
                    acc[r][1] = fma2(both, w[k].y, acc[r][1]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < J::rows; ++r)
            *reinterpret_cast<ulonglong2 *>(sums + (split * ROWS + row0 + r) * kLdS + column) = make_ulonglong2(acc[r][0], acc[r][1]);
        if (!__syncthreads_and(ok)) {  // also: this M may be overwritten
            if (tid == 0) {
                count_error(p.err_count);
                int quiet = 0;
                if (j + 2 < segments) mbar_wait(&full[(j + 1) & 1], (j >> 1) & 1, &quiet);
            }
            for (++j; real && j < segments; ++j) *row_at(j) = make_float4(NAN, NAN, NAN, NAN);
            return;
        }
        if (adds) {
#pragma unroll
            for (int i = 0; i < J::splits; ++i) {
                const float4 v = *reinterpret_cast<const float4 *>(sums + (i * ROWS + group) * kLdS + column);
                y.x += v.x;
                y.y += v.y;
                y.z += v.z;
                y.w += v.w;
            }
            *reinterpret_cast<float4 *>(state + group * kLdS + column) = y;
            if (real) *row_at(j + 1) = y;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host ----

int64_t slot_count(int total_tokens, int batch) { return static_cast<int64_t>(total_tokens / C) + batch; }
int64_t segment_slots(int total_tokens, int batch, int seg_chunks) {
    return static_cast<int64_t>(total_tokens) / (static_cast<int64_t>(seg_chunks) * C) + batch;
}

template <int PANELS>
constexpr size_t prep_smem() { return kMatrixBytes + sizeof(PrepSmem); }
// A chunk block takes all tensor memory of its SM and then waits for the preparation, whose blocks may still be about to take
// theirs: the two must not meet on an SM.  With 64 keys their sizes would let them, so the chunk block asks for the rest.
// (Their registers do not let them either: 61440 and 16384 of 65536.)
constexpr size_t kSmShared = 228 * 1024, kBlockShared = 1024;  // of an SM, and what each block takes beside its own
template <int PANELS>
constexpr size_t chunk_smem() {
    constexpr size_t used = kStages * Stage<PANELS>::bytes + 2 * kTile + sizeof(ChunkSmem);
    constexpr size_t rest = kSmShared - 2 * kBlockShared - prep_smem<PANELS>() + 16;
    constexpr size_t bytes = used > rest ? used : rest;
    static_assert(bytes + prep_smem<PANELS>() + 2 * kBlockShared > kSmShared && bytes + kBlockShared <= kSmShared, "");
    return bytes;
}

template <int PANELS, bool FULL, bool VS, bool VIO>
int launch_chunks(const FwdArgs &p, const FwdMaps &maps, int64_t units, cudaStream_t stream) {
    int dev = 0;
    current_device_sms(&dev);
    cudaError_t err;
    if (resident_blocks<gdr_chunk_kernel<PANELS, FULL, VS, VIO>>(kChunkThreads, chunk_smem<PANELS>(), dev, &err) == 0)
        return static_cast<int>(err);
    const int slices = (p.a.dim_v + 127) / 128;
    const int64_t blocks = units * p.a.num_v_heads * (FULL ? slices : slices + 1);
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    return launch_pdl(gdr_chunk_kernel<PANELS, FULL, VS, VIO>, dim3(static_cast<unsigned>(blocks)), dim3(kChunkThreads),
                      chunk_smem<PANELS>(), stream, p, maps, slices);
}

template <int PANELS, int ROWS>
int launch_join(const FwdArgs &p, cudaStream_t stream) {
    using J = Join<PANELS, ROWS>;
    int dev = 0;
    current_device_sms(&dev);
    cudaError_t err;
    if (resident_blocks<gdr_join_kernel<PANELS, ROWS>>(J::threads, J::smem, dev, &err) == 0) return static_cast<int>(err);
    const int64_t blocks = static_cast<int64_t>(p.batch) * p.a.num_v_heads * ((p.a.dim_v + ROWS - 1) / ROWS);
    if (blocks > 0x7fffffff) return CCV_ERR_SIZE;
    return launch_pdl(gdr_join_kernel<PANELS, ROWS>, dim3(static_cast<unsigned>(blocks)), dim3(J::threads), J::smem, stream, p);
}

template <int PANELS, bool VS, bool VIO>
int launch_chunked(const FwdArgs &p, cudaStream_t stream) {
    int dev = 0;
    current_device_sms(&dev);
    cudaError_t err;
    if (resident_blocks<gdr_prep_kernel<PANELS, VIO>>(kPrepThreads, prep_smem<PANELS>(), dev, &err) == 0) return static_cast<int>(err);
    const int64_t prep = static_cast<int64_t>(p.slots) * p.a.num_k_heads;
    if (prep > 0x7fffffff) return CCV_ERR_SIZE;
    FwdMaps maps;
    maps.use = VIO && encode_heads_map(&maps.q, p.a.q, p.a.dim_k, p.a.num_k_heads, p.total_tokens, C) &&
               encode_heads_map(&maps.k, p.a.k, p.a.dim_k, p.a.num_k_heads, p.total_tokens, C) &&
               encode_heads_map(&maps.v, p.a.v, p.a.dim_v, p.a.num_v_heads, p.total_tokens, C);
    int status = launch_pdl(gdr_prep_kernel<PANELS, VIO>, dim3(static_cast<unsigned>(prep)), dim3(kPrepThreads),
                            prep_smem<PANELS>(), stream, p);
    if (status != CCV_OK) return status;
    if (p.seg_chunks == 0) return launch_chunks<PANELS, true, VS, VIO>(p, maps, p.batch, stream);
    const int64_t segments = segment_slots(p.total_tokens, p.batch, p.seg_chunks);
    status = launch_chunks<PANELS, false, VS, VIO>(p, maps, segments, stream);
    if (status != CCV_OK) return status;
    const int64_t row_sets = static_cast<int64_t>(p.batch) * p.a.num_v_heads;
    const int sms = current_device_sms();
    status = row_sets * ((p.a.dim_v + 3) / 4) <= sms   ? launch_join<PANELS, 4>(p, stream)
             : row_sets * ((p.a.dim_v + 7) / 8) <= sms ? launch_join<PANELS, 8>(p, stream)
                                                       : launch_join<PANELS, 16>(p, stream);
    if (status != CCV_OK) return status;
    return launch_chunks<PANELS, true, VS, VIO>(p, maps, segments, stream);
}

template <int PANELS>
int launch_chunked(const FwdArgs &p, bool vs, bool vio, cudaStream_t stream) {
    if (vio) return vs ? launch_chunked<PANELS, true, true>(p, stream) : launch_chunked<PANELS, false, true>(p, stream);
    return vs ? launch_chunked<PANELS, true, false>(p, stream) : launch_chunked<PANELS, false, false>(p, stream);
}

bool chunked_dims(int dim_k) { return dim_k <= 128; }

// The recurrent form takes 0.85 us a token of the longest sequence, the chunked one 22 us for up to a chunk of each (1
// sequence of 32 heads; 7.6 + 2.2 us a token against 35 us for 8, 45 + 13 us against 215 us for 64): they meet at 12 to 22
// tokens a sequence.  8 on average leaves room for lengths that differ, which only the device knows.  It is an average: with 16
// heads a sequence of 2000 tokens takes 68 us by itself and 1430 in a batch filled up to 256 with empty ones, and one of 1500
// takes 62 by itself and 1220 beside 255 single tokens (which take 69 by themselves).
constexpr int kRecurrentTokens = 8;

// CCV_GDR_PATH=recurrent or =chunked, read at each call, forces one form (for testing and tuning).
bool use_chunked(int batch, int total_tokens, int dim_k) {
    if (!chunked_dims(dim_k)) return false;
    const char *path = std::getenv("CCV_GDR_PATH");
    if (path != nullptr && std::strcmp(path, "recurrent") == 0) return false;
    if (path != nullptr && std::strcmp(path, "chunked") == 0) return true;
    return total_tokens > static_cast<int64_t>(kRecurrentTokens) * batch;
}

// Chunks of a segment, or 0 to leave sequences whole, for sequences of equal lengths (their offsets are on the device; 11027
// tokens and 23 sequences of 1 or 40, which the average leaves whole, take 470 us instead of 200 and 40).  In
// chunk times of a block (2.5 us): the first pass takes 0.95 of one a chunk, a join 0.4 a segment (1 where its blocks take 16
// rows), and the two launches more take 3.5.  Each pass runs in waves of one block an SM.  11027 tokens take 200 us with 16
// heads and 92 with 4, against 457 and 433 whole; 1000 tokens and 4 heads, 48 against 51; 4 x 2000 tokens and 8 heads, 97
// against 102.
int segment_chunks(int total_tokens, int batch, int num_v_heads, int dim_v) {
    constexpr int kSms = 152;  // a GB300's: the workspace's size may not depend on the device that is current
    const int chunks = static_cast<int>((static_cast<int64_t>(total_tokens) + static_cast<int64_t>(batch) * C - 1) / (static_cast<int64_t>(batch) * C));
    const int slices = (dim_v + 127) / 128;
    const int64_t heads = static_cast<int64_t>(batch) * num_v_heads;
    auto waves = [](int64_t blocks) { return static_cast<double>((blocks + kSms - 1) / kSms); };
    const char *forced = std::getenv("CCV_GDR_SEGMENT");  // chunks of a segment (for testing and tuning)
    if (forced != nullptr) return std::atoi(forced) > 0 && std::atoi(forced) < (1 << 20) ? std::atoi(forced) : 0;
    const double join = heads * ((dim_v + 7) / 8) <= kSms ? 0.4 : 1.0;
    double best = waves(heads * slices) * chunks;
    int choice = 0;
    for (int n = 3; n <= 64 && n <= chunks; ++n) {
        const int length = (chunks + n - 1) / n;
        const double cost = 3.5 + waves(heads * ((n - 1) * slices + n - 2)) * length * 0.95 + (n - 2) * join + waves(heads * n * slices) * length;
        if (cost < best) {
            best = cost;
            choice = length;
        }
    }
    return choice;
}

int64_t heads_bytes(int total_tokens, int batch, int num_v_heads) { return slot_count(total_tokens, batch) * num_v_heads * kHeadBytes; }

}  // namespace
}  // namespace ccv

extern "C" int64_t gdr_fwd_workspace(int total_tokens, int batch, int num_k_heads, int num_v_heads, int dim_k, int dim_v) {
    using namespace ccv;
    if (total_tokens <= 0 || batch <= 0 || num_k_heads <= 0 || num_v_heads <= 0 || dim_k <= 0 || dim_v <= 0) return 0;
    if (!use_chunked(batch, total_tokens, dim_k)) return 0;
    int64_t bytes = heads_bytes(total_tokens, batch, num_v_heads);
    if (const int seg = segment_chunks(total_tokens, batch, num_v_heads, dim_v))
        bytes += segment_slots(total_tokens, batch, seg) * num_v_heads * (dim_v + dim_k) * (dim_k <= 64 ? 256 : 512);
    return bytes;
}

extern "C" int gdr_fwd(const ccv_gdr_args *args, const int32_t *query_start_loc, int batch, const int32_t *cache_indices,
                       const uint8_t *has_initial_state, int total_tokens, void *workspace, int64_t workspace_bytes,
                       int *err_count, ccv_stream_t stream) {
    using namespace ccv;
    if (batch < 0 || total_tokens < 0 || total_tokens > (1 << 30)) return CCV_ERR_SIZE;
    const int status = gdr_check(args, 1, total_tokens);
    if (status != CCV_OK) return status;
    if (has_initial_state != nullptr && args->state == nullptr) return CCV_ERR_ARGUMENT;
    if (batch == 0 || total_tokens == 0 || args->num_v_heads == 0 || args->dim_v == 0 || args->dim_k == 0) return CCV_OK;
    if (query_start_loc == nullptr) return CCV_ERR_NULL_POINTER;
    const ccv_gdr_args &a = *args;
    const int64_t need = gdr_fwd_workspace(total_tokens, batch, a.num_k_heads, a.num_v_heads, a.dim_k, a.dim_v);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 127u) != 0))
        return CCV_ERR_WORKSPACE;
    if (!use_chunked(batch, total_tokens, a.dim_k)) {
        const GdrRows rows{query_start_loc, cache_indices, has_initial_state, nullptr, nullptr, 0, 0, 0, batch, 0,
                           total_tokens, err_count};
        return gdr_launch_recurrent(a, rows, stream);
    }
    const int64_t slots = slot_count(total_tokens, batch);
    FwdArgs p{a, query_start_loc, cache_indices, has_initial_state, batch, total_tokens, static_cast<int>(slots),
              static_cast<uint8_t *>(workspace), err_count, segment_chunks(total_tokens, batch, a.num_v_heads, a.dim_v), nullptr, nullptr};
    if (p.seg_chunks > 0) {
        p.seg_state = reinterpret_cast<float *>(p.heads + heads_bytes(total_tokens, batch, a.num_v_heads));
        p.seg_step = p.seg_state + segment_slots(total_tokens, batch, p.seg_chunks) * a.num_v_heads * a.dim_v * (a.dim_k <= 64 ? 64 : 128);
    }
    auto vec = [](const ccv_heads_view &v) {
        return aligned16(v.data) && v.stride_dim == 1 && v.stride_tok % 8 == 0 && v.stride_head % 8 == 0;
    };
    const bool vio = a.dim_k % 8 == 0 && a.dim_v % 8 == 0 && vec(a.q) && vec(a.k) && vec(a.v) && vec(a.out);
    const bool vs = a.state == nullptr || (a.dim_k % 4 == 0 && aligned16(a.state) && a.s_stride_k == 1 && a.s_stride_line % 4 == 0 &&
                                           a.s_stride_head % 4 == 0 && a.s_stride_v % 4 == 0);
    return a.dim_k <= 64 ? launch_chunked<1>(p, vs, vio, stream) : launch_chunked<2>(p, vs, vio, stream);
}
