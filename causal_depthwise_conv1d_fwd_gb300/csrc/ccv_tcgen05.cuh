// Tensor-core and asynchronous-copy primitives for sm_103a: mbarriers with bounded waits, bulk copies, tensor memory,
// and tcgen05.mma on bf16 operands with fp32 accumulators.
#pragma once

#include <cstdint>

#include "ccv_common.cuh"
#include "ccv_math2.cuh"
#include "ccv_pipeline.cuh"

namespace ccv {

// ------------------------------------------------------------ mbarriers ----

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ uint64_t timer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
constexpr uint64_t kMaxWaitNs = 2000000000ull;  // far beyond any wait of a healthy kernel

// Waits until the barrier's phase `parity` is complete.  False when two seconds ran out or another thread of the block
// gave up (`*abort` set): the caller then leaves its loop and goes to the kernel's common end.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t start = timer_ns();
    for (int i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 0) {
            if (*abort) return false;
            if (timer_ns() - start > kMaxWaitNs) {
                *abort = 1;
                return false;
            }
        }
    }
}
// The same for a whole warp, with one answer for all its lanes (tensor-memory accesses are warp-wide).
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// --------------------------------------------------------- bulk copies ----

// Contiguous global -> shared copy, counted in bytes on `bar`; addresses and size are multiples of 16.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// 16-byte asynchronous copy, or 16 zero bytes when `real` is false (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
// Makes this thread's shared-memory writes visible to the asynchronous proxy (bulk copies, tcgen05.mma).
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ------------------------------------------------------- tensor memory ----

// Whole-warp calls.  The column count is a power of two >= 32; every allocation is freed by the kernel.
template <int kColumns>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "n"(kColumns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int kColumns>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "n"(kColumns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// N consecutive columns of this thread's lane (lane base in the address' upper half).  Loads are asynchronous: the values
// are there after tmem_wait_load(), which the caller places before their first use.
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                   "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                   "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
                   "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
                   "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// ----------------------------------------------------------- tcgen05.mma ----

// Shared-memory operand in 128-byte swizzled rows: rows of 64 bf16 values, 16-byte piece c of row r at piece c ^ (r & 7),
// 8 rows (1024 bytes) a group.  K-major: a row is one M/N index, groups are `stride` bytes apart.  MN-major: a row is one
// K index and 64 M/N indices, groups of 8 K indices are `stride` apart, groups of 64 M/N indices `lead` apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>((lead >> 4) & 0x3fffu) << 16) |
           (static_cast<uint64_t>((stride >> 4) & 0x3fffu) << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 x bf16 -> fp32; b_mn: B is MN-major.
constexpr uint32_t mma_desc(int m, int n, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// One lane of a converged warp (the same for every call), as a 0 / 1 flag for the calls below.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// D[tmem] (+)= A B^T, issued by the lane whose `lane` flag is set, with A in tensor memory (lane = row, a 32-bit column = 2
// K indices) ...  Called by the whole warp with uniform operands: from inside a one-lane branch each issue took 52 cycles
// (measured, any N up to 64), this way 16, so that 128 x 64 x 16 takes the tensor cores' own 32.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t lane) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(lane)
        : "memory");
}
// ... or in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t lane) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(lane)
        : "memory");
}
// Arrives on `bar` when every MMA that lane issued so far is complete.
__device__ __forceinline__ void mma_commit(uint64_t *bar, uint32_t lane) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lane)
        : "memory");
}

// ------------------------------------------------------- 8 x 8 transposes ----

// Four 8 x 8 blocks of 16-bit values from shared memory, transposed: lane l gives the address of row l % 8 of block l / 8
// (16-byte aligned) and receives in r[b] the pair (row 2 (l % 4), + 1) of column l / 4 of block b.
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// r[i] of lane j of every four lanes becomes r[j] of lane i.
__device__ __forceinline__ void transpose_quad(uint32_t (&r)[4]) {
    const int lane = threadIdx.x;
#pragma unroll
    for (int m = 1; m < 4; m <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((i & m) == 0) {
                const bool up = (lane & m) != 0;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? r[i] : r[i | m], m);
                if (up) r[i] = got;
                else r[i | m] = got;
            }
}

// Two floats as pairs of bf16 parts, by truncation: each part takes the next 8 bits, so three hold a float exactly and two
// hold 16 bits of it.  (Rounded parts would need conversions at half the rate of these.)
__device__ __forceinline__ uint32_t upper_halves(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ f32x2 below_upper(float a, float b) {  // what upper_halves leaves
    return sub2(pack2(a, b), pack2(__uint_as_float(__float_as_uint(a) & 0xffff0000u), __uint_as_float(__float_as_uint(b) & 0xffff0000u)));
}
__device__ __forceinline__ void split_bf16x2(f32x2 x, uint32_t &hi, uint32_t &mid) {
    float a, b;
    unpack2(x, a, b);
    hi = upper_halves(a, b);
    unpack2(below_upper(a, b), a, b);
    mid = upper_halves(a, b);
}
__device__ __forceinline__ void split_bf16x3(f32x2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float a, b;
    unpack2(x, a, b);
    hi = upper_halves(a, b);
    unpack2(below_upper(a, b), a, b);
    mid = upper_halves(a, b);
    unpack2(below_upper(a, b), a, b);
    lo = upper_halves(a, b);
}

}  // namespace ccv
