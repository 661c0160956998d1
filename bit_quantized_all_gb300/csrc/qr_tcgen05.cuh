// qr_tcgen05.cuh -- the tcgen05 instructions the attention kernel uses, as
// inline PTX: tensor memory (TMEM), products of 128 x N x 16 fp16 operands
// with fp32 accumulators in TMEM, and the descriptors of their operands.
//
// Operands in shared memory are stored with the 128-byte swizzle: a tile is
// rows of 128 bytes (64 fp16 values), eight rows a 1024-byte group, the
// 16-byte pieces of row r exchanged by piece ^ (r % 8).  Groups follow one
// another; a tile wider than 64 values is several such slabs.
#pragma once

#include <cstdint>

#include "qr_pipeline.cuh"

namespace qrk {

__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }

// Descriptor of a swizzled operand starting at shared address `addr`:
// `group` bytes between groups of eight rows, `slab` bytes between slabs
// along the rows (read only for operands whose rows run along M or N).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t slab, uint32_t group) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | static_cast<uint64_t>((slab >> 4) & 0x3fff) << 16 |
           static_cast<uint64_t>((group >> 4) & 0x3fff) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: fp16 x fp16 (or bf16 x bf16) -> fp32, M = 128, N = n;
// b_rows_k: the rows of B's tile run along K (else along N).
__host__ __device__ constexpr uint32_t mma_desc(int n, bool b_rows_k, bool bf16 = false) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_rows_k ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}

// One lane of the calling warp, the same at every call.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// D (TMEM) = A (shared) B (shared) [+ D], issued by the lane whose `leader` is
// set.  The whole warp comes here with the same operands: they then stay in
// uniform registers, and eight products are issued in 280 to 390 cycles
// instead of the 560 to 640 that a branch around one thread takes (they run
// for 512).
__device__ __forceinline__ void tc_mma_ss(bool leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
        : "memory");
}
// D (TMEM) = A (TMEM) B (shared) [+ D]; A's row r is lane r, two values a column.
__device__ __forceinline__ void tc_mma_ts(bool leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p, l;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 l, %5, 0;\n\t"
        "@l tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
        : "memory");
}
// One arrival on `bar` when every product issued by this lane is complete.
__device__ __forceinline__ void tc_commit(bool leader, uint64_t *bar) {
    if (leader)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}

__device__ __forceinline__ void tc_alloc(uint32_t *slot, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_free(uint32_t tmem, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;"); }

// Makes this thread's writes to shared memory visible to the tensor cores.
__device__ __forceinline__ void smem_to_tensor_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for a phase, the thread suspended for up to kSuspendNs at a time rather
// than asking again and again: warps that wait beside others that compute leave
// them the issue slots.  After a wait that ran out (counted once a CTA) every
// wait of the CTA fails at its next look.
constexpr uint32_t kSuspendNs = 1000000;
__device__ __forceinline__ bool mbar_try_suspended(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, int *fail, unsigned *timeouts) {
    uint32_t done;  // (asked first without suspension: cheaper when the phase is over)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (done || mbar_try_suspended(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!*static_cast<volatile int *>(fail)) {
        if (mbar_try_suspended(bar, parity)) return true;
        if (global_ns() - t0 > kWaitLimitNs) {
            if (atomicExch(fail, 1) == 0) atomicAdd(timeouts, 1u);
            return false;
        }
    }
    return mbar_try_wait(bar, parity);
}
// ... by a whole warp, whose lanes then go on together.
__device__ __forceinline__ bool tc_wait_warp(uint64_t *bar, uint32_t parity, int *fail, unsigned *timeouts) {
    return __all_sync(~0u, tc_wait(bar, parity, fail, timeouts));
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

#define QR_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define QR_T8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
#define QR_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// 32 columns of this thread's lane (lane l of warp w: lane 32 (w % 4) + l).
// (These keep their order among themselves and the fences and barriers, and
// touch no addressable memory: loads may be moved across them.)
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : QR_R8(v, 0), QR_R8(v, 8), QR_R8(v, 16), QR_R8(v, 24)
        : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : QR_R8(v, 0), QR_R8(v, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), QR_I8(v, 0));
}
// 16 lanes x 32 columns in the order of the m16n8k16 instructions' A fragments:
// lane 4 g + t of the warp holds columns 8 i + 2 t and the next of lane g in
// v[4 i], v[4 i + 1] and of lane g + 8 in v[4 i + 2], v[4 i + 3].
__device__ __forceinline__ void tc_st_fragments(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        QR_I8(v, 0), QR_I8(v, 8));
}
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QR_T8(v, 0), QR_T8(v, 8));
}
// Waits for this thread's loads; the registers pass through, so that nothing
// uses them before.
__device__ __forceinline__ void tc_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : QR_T8(v, 0), QR_T8(v, 8), QR_T8(v, 16), QR_T8(v, 24));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        QR_I8(v, 0), QR_I8(v, 8), QR_I8(v, 16), QR_I8(v, 24));
}
#undef QR_R8
#undef QR_T8
#undef QR_I8

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

}  // namespace qrk
