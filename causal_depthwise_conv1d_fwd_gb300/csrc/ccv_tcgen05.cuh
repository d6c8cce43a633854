// Tensor-core and asynchronous-copy primitives for sm_103a: mbarriers with bounded waits, bulk copies, tensor memory,
// and tcgen05.mma on bf16 operands with fp32 accumulators.
#pragma once

#include <cstdint>
#include <cuda.h>

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
// Whether the barrier's phase `parity` is complete; the hardware may hold the thread for a while if it is not, which leaves
// the issue slots to the warps that work (polling without it made the chunk kernel of gdr_fwd 4% slower).
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
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
    uint64_t start = 0;
    for (int i = 1; !mbar_try_wait(bar, parity); ++i) {
        if ((i & 63) != 0) continue;
        if (*abort) return false;
        const uint64_t now = timer_ns();
        if (start == 0) start = now;
        if (now - start > kMaxWaitNs) {
            *abort = 1;
            return false;
        }
    }
    return true;
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
// One box of a tensor (coordinates innermost first) into swizzled shared memory, counted in bytes on `bar`.
__device__ __forceinline__ void tensor_load(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                     smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
                 : "memory");
}
// Contiguous shared -> global copy of this thread's (addresses and size as above), and waits for all that it committed:
// until shared memory has been read, or until the values are in global memory.
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Brings a contiguous range, or a tensor's box, into L2.
__device__ __forceinline__ void bulk_prefetch(const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tensor_prefetch(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
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
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
                 "%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(addr));
}
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
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// ----------------------------------------------------------- tcgen05.mma ----

// Shared-memory operand in 128-byte swizzled rows: rows of 64 bf16 values, 16-byte piece c of row r at piece c ^ (r & 7),
// 8 rows (1024 bytes) a group, groups one after the other.  K-major: a row is one M/N index.  MN-major (up to 64 M/N
// indices): a row is one K index.  The upper word of its descriptor is kDescHigh, the lower one the address; addresses and
// descriptors add, byte offsets as offset / 16.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr) { return (addr >> 4) & 0x3fffu; }
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
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t lane) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 bd;\n\tmov.b64 bd, {%2, %6};\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(lane), "n"(kDescHigh)
        : "memory");
}
// ... or in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate, uint32_t lane) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 ad, bd;\n\tmov.b64 ad, {%1, %6};\n\tmov.b64 bd, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(lane), "n"(kDescHigh)
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

// Two floats as pairs of bf16 parts: each part is what the parts before it leave, rounded to 8 bits, so two parts hold 16
// bits of a float and three hold all 24.  The remainder is one mixed-precision FMA (exact) a value: unpacking the parts with
// masks and shifts instead keeps the integer pipe, which has half the rate, busy for twice as long.
__device__ __forceinline__ void take_part(float &a, float &b, uint32_t &part) {
    part = pack_bf16x2(a, b);
    asm("{\n\t.reg .b16 lo, hi, one;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "mov.b16 one, 0xbf80;\n\t"  // -1
        "fma.rn.f32.bf16 %0, lo, one, %0;\n\t"
        "fma.rn.f32.bf16 %1, hi, one, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(part));
}
__device__ __forceinline__ void split_bf16x2(f32x2 x, uint32_t &hi, uint32_t &mid) {
    float a, b;
    unpack2(x, a, b);
    take_part(a, b, hi);
    mid = pack_bf16x2(a, b);
}
__device__ __forceinline__ void split_bf16x3(f32x2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float a, b;
    unpack2(x, a, b);
    take_part(a, b, hi);
    take_part(a, b, mid);
    lo = pack_bf16x2(a, b);
}

}  // namespace ccv
